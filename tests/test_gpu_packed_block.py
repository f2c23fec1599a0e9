"""The training step of examples/packed_block_step.py against float32 autograd of the same block, and its loss going down."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "packed_block_step.py")


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("packed_block_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(block, ex, x, y0, offsets, target):
    """The block in float32 torch, from the bf16 weights, with autograd."""
    w = {k: v.to(torch.bfloat16).float().requires_grad_() for k, v in block.weights.items()}
    x, y0, target = x.float().requires_grad_(), y0.float().requires_grad_(), target.float()
    T, H, G, D = x.shape[0], block.heads, block.kv_heads, block.dim
    q, k, v = (y0 @ w["w_qkv"]).view(T, H + 2 * G, D).split([H, G, G], dim=1)
    rows = []
    ends = offsets.tolist()
    for a, b in zip(ends[:-1], ends[1:]):
        kk, vv = (t[a:b].repeat_interleave(H // G, dim=1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q[a:b], kk) / D ** 0.5
        s = s.masked_fill(torch.ones(b - a, b - a, device=s.device).triu(1).bool(), float("-inf"))
        rows.append(torch.einsum("hqk,khd->qhd", s.softmax(-1), vv))
    rows.append(torch.zeros(T - ends[-1], H, D, device=x.device))
    f = torch.cat(rows).reshape(T, H * D) @ w["w_out"]
    norm = lambda t, g: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + ex.EPS) * g  # noqa: E731
    h = x + block.scale * w["gate"] * norm(f, w["w_post"])
    y = norm(h, w["w_pre"])
    loss = (y - target).square().mean()
    loss.backward()
    return loss, {k: v.grad for k, v in w.items()}, x.grad, y0.grad


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (4, 4, 128)])
def test_step_matches_autograd(ex, heads, kv_heads, dim):
    """Tolerance: the step holds activations and gradients in bf16 (2^-8 each) over a chain of eight rounded tensors, in
    random directions: sqrt(8) 2^-8 = 1.1e-2 of a gradient's norm; twice that is the bar."""
    block = ex.Block(width=256, heads=heads, kv_heads=kv_heads, dim=dim, seed=3)
    batch = ex.documents([150, 1, 77, 300], 9, 256, 4)
    loss, grads, dx, dy0 = block.step(*batch)
    ref_loss, ref, ref_dx, ref_dy0 = reference(block, ex, *batch)
    assert abs(float(loss) - float(ref_loss)) <= 1e-2 * float(ref_loss)
    for name, got, want in [(k, grads[k], ref[k]) for k in ref] + [("x", dx, ref_dx), ("y0", dy0, ref_dy0)]:
        rel = float((got.float() - want).norm() / want.norm())
        assert rel <= 2.2e-2, f"{name}: {rel:.3g}"


def test_loss_goes_down(ex):
    block = ex.Block(width=256, seed=1)
    batch = ex.documents([200, 56], 0, 256, 2)
    losses = []
    for _ in range(8):
        loss, grads, _, _ = block.step(*batch)
        block.update(grads, 30.0)
        losses.append(float(loss))
    assert losses[-1] < 0.98 * losses[0]
