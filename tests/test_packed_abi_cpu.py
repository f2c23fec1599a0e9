"""mha_packed and residual_rmsnorm on the host: refusals before any device work (no GPU needed).  Addresses are
made up and never dereferenced: every call here is refused by the checks."""
import ctypes

import pytest
import torch

import conv2d_backward_implicit_gb300 as dg
from conv2d_backward_implicit_gb300 import build_ext

A = 4096  # an address with every alignment


@pytest.fixture(scope="module")
def lib():
    if build_ext.is_stale():
        build_ext.build()
    return dg.library()


def packed(**kw):
    base = dict(tokens=100, num_seqs=2, num_heads=8, num_kv_heads=2, head_dim=64, window_size=0, q_stride=0,
                k_stride=0, v_stride=0)
    return dg.MhaPackedParams(**(base | kw))


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), 2), (dict(num_heads=0), 2), (dict(num_kv_heads=0), 2), (dict(head_dim=0), 2),
    (dict(num_kv_heads=3), 2), (dict(q_stride=8 * 64 - 1), 2), (dict(k_stride=64), 2), (dict(v_stride=127), 2),
    (dict(head_dim=257), 4), (dict(tokens=(1 << 30) + 1), 4), (dict(num_seqs=(1 << 30) + 1), 4),
    (dict(tokens=1 << 30, num_heads=128), 4)])
def test_packed_params_are_refused(lib, kw, status):
    p = ctypes.byref(packed(**kw))
    assert lib.mha_packed_forward(A, A, A, A, A, A, p, 1, None) == status
    assert lib.mha_packed_backward(A, A, A, A, A, A, A, A, A, A, A, 1 << 40, p, 1, None) == status
    assert lib.mha_packed_forward_select_kernel(A, A, A, A, p, 1) == -status
    assert lib.mha_packed_workspace_size(p, 1) == 0


def test_packed_arguments_are_refused(lib):
    p = ctypes.byref(packed())
    for i in range(6):
        args = [A] * 6
        args[i] = None
        assert lib.mha_packed_forward(*args, p, 1, None) == 1
    assert lib.mha_packed_forward(A, A, A, A, A, A, None, 1, None) == 1
    assert lib.mha_packed_forward(A, A, A, A, A, A, p, 3, None) == 1
    for i, off in ((0, 1), (1, 1), (2, 1), (3, 2), (4, 1), (5, 2)):
        args = [A] * 6
        args[i] += off
        assert lib.mha_packed_forward(*args, p, 1, None) == 3, i
    size = lib.mha_packed_workspace_size(p, 1)
    assert size >= 100 * 8 * 8
    for i in range(11):
        args = [A] * 11
        args[i] = None
        assert lib.mha_packed_backward(*args, size, p, 1, None) == 1
    assert lib.mha_packed_backward(*[A] * 10, A + 8, size, p, 1, None) == 3
    assert lib.mha_packed_backward(*[A] * 11, size - 1, p, 1, None) == 7


def test_packed_kernel_choice(lib):
    sel = lambda q=A, dtype=1, **kw: lib.mha_packed_forward_select_kernel(  # noqa: E731
        q, A, A, A, ctypes.byref(packed(**kw)), dtype)
    assert sel() == dg.DGRAD_KERNEL_TC and sel(dtype=2) == dg.DGRAD_KERNEL_TC
    assert sel(head_dim=128) == sel(head_dim=8) == sel(head_dim=80) == dg.DGRAD_KERNEL_TC
    assert sel(q_stride=1024, k_stride=1024, v_stride=1024) == dg.DGRAD_KERNEL_TC
    for simt in (sel(dtype=0), sel(head_dim=100), sel(head_dim=136), sel(q=A + 8), sel(q_stride=1021)):
        assert simt == dg.DGRAD_KERNEL_SIMT
    assert dg.mha_packed_set_kernel(7) == 1
    assert dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_TC) == dg.DGRAD_KERNEL_AUTO
    try:
        assert sel(dtype=0) == -4
        assert lib.mha_packed_forward(A, A, A, A, A, A, ctypes.byref(packed()), 0, None) == 4
        dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_SIMT)
        assert sel() == dg.DGRAD_KERNEL_SIMT
    finally:
        dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_AUTO)


def test_packed_binding_refuses_host_and_misshapen_tensors():
    p = packed(tokens=4, num_heads=2, num_kv_heads=1)
    q, kv = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        dg.mha_packed_forward(q, kv, kv, A, A, A, p, 1)
    wide = packed(tokens=4, num_heads=2, num_kv_heads=1, q_stride=256)
    with pytest.raises(ValueError, match="strides"):
        dg.mha_packed_forward(q, kv, kv, A, A, A, wide, 1)
    with pytest.raises(ValueError, match="shape"):
        dg.mha_packed_forward(q.view(4, 128), kv, kv, A, A, A, wide, 1)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        dg.mha_packed_forward(torch.zeros(4, 4, 64, dtype=torch.bfloat16)[:, :2], kv, kv, A, A, A, wide, 1)


def norm(**kw):
    return dg.ResidualRmsnormParams(**(dict(m=3, n=64, gate_kind=1, eps=1e-5, scale=1.0) | kw))


@pytest.mark.parametrize("kw,status", [(dict(m=0), 2), (dict(n=0), 2), (dict(gate_kind=3), 1), (dict(eps=-1.0), 1),
                                       (dict(eps=float("inf")), 1), (dict(scale=float("nan")), 1),
                                       (dict(n=(1 << 20) + 1), 4), (dict(m=1 << 31), 4)])
def test_norm_params_are_refused(lib, kw, status):
    p = ctypes.byref(norm(**kw))
    assert lib.residual_rmsnorm_forward(*[A] * 8, p, 1, None) == status
    assert lib.residual_rmsnorm_backward(*[A] * 14, 1 << 40, p, 1, None) == status
    assert lib.residual_rmsnorm_workspace_size(p, 1) == 0


def test_norm_arguments_are_refused(lib):
    p = ctypes.byref(norm())
    for i in range(7):
        args = [A] * 8
        args[i] = None
        assert lib.residual_rmsnorm_forward(*args, p, 1, None) == 1, i
        args[i] = A + 1
        assert lib.residual_rmsnorm_forward(*args, p, 1, None) == 3, i
    assert lib.residual_rmsnorm_forward(*[A] * 7, A + 2, p, 1, None) == 3
    assert lib.residual_rmsnorm_forward(*[A] * 8, ctypes.byref(norm(gate_kind=0)), 1, None) == 1
    assert lib.residual_rmsnorm_forward(*[A] * 8, p, 5, None) == 1
    size = lib.residual_rmsnorm_workspace_size(p, 1)
    assert size > 0
    for i in range(14):
        if i == 7:
            continue  # dh may be missing
        args = [A] * 14
        args[i] = None
        assert lib.residual_rmsnorm_backward(*args, size, p, 1, None) == 1, i
    assert lib.residual_rmsnorm_backward(*[A] * 14, size - 1, p, 1, None) == 7
    assert lib.residual_rmsnorm_backward(*[A] * 13, A + 4, size, p, 1, None) == 3


def test_norm_binding_refuses_host_tensors():
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="f must be a CUDA tensor"):
        dg.residual_rmsnorm_forward(x, x, None, x[0], x[0], x, x, None, norm(gate_kind=0), 1)
