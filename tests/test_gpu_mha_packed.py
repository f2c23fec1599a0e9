"""GPU parity of causal attention over packed sequences (include/mha_packed.h) with the float64 oracle
(oracle/mha_packed.py), through the C ABI.

Inputs are drawn in float32 and rounded to the input type; the oracle gets exactly those values.  The bars are the
oracle module's element-wise bounds (first-order float32 error terms of the data at hand, the rounding of P and dS to
the input type in the tensor-core kernels, the rounding of the outputs), derived there; an output passes when no
element is off by more.  Buffers carry guard bands of NaN, checked after each call.
"""
import numpy as np
import pytest
import torch

from oracle import mha_packed as om

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}          # rounding of P and dS (tensor cores)
OUT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # rounding of the results
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}          # half the smallest step
GUARD = 64


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import conv2d_backward_implicit_gb300 as mod
    mod.library()
    yield mod
    mod.mha_packed_set_kernel(mod.DGRAD_KERNEL_AUTO)


class Problem:
    def __init__(self, lens, H, G, d, window=0, head=0, tail=0, dtype="bf16", fused=False, seed=0, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.offsets = [head + sum(lens[:i]) for i in range(len(lens) + 1)]
        self.T = T = self.offsets[-1] + tail
        self.H, self.G, self.d, self.window, self.dtype, self.fused = H, G, d, window, dtype, fused
        t = TORCH[dtype]
        x = torch.randn(T, H + 2 * G, d, generator=g).to(t)
        if fused:
            self.q, self.k, self.v = x.split([H, G, G], dim=1)
        else:
            self.q, self.k, self.v = (y.contiguous() for y in x.split([H, G, G], dim=1))
        self.go = (torch.randn(T, H, d, generator=g) * scale).to(t)

    def params(self, dg):
        return dg.MhaPackedParams(self.T, len(self.offsets) - 1, self.H, self.G, self.d, self.window,
                                  *((x.stride(0) if self.fused else 0) for x in (self.q, self.k, self.v)))

    def f64(self, *names):
        return [getattr(self, n).double().numpy() for n in names]


def guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), float("nan"), device="cuda", dtype=dtype)
    return buf, buf[GUARD:GUARD + n].view(shape)


def intact(buf):
    return bool(torch.isnan(buf[:GUARD].float()).all() and torch.isnan(buf[-GUARD:].float()).all())


def to_gpu(p):
    """q, k, v on the GPU, strided as the problem's are."""
    if not p.fused:
        return p.q.cuda(), p.k.cuda(), p.v.cuda()
    base = torch.cat([p.q, p.k, p.v], dim=1).cuda()
    return base.split([p.H, p.G, p.G], dim=1)


def run_forward(dg, p, stream=None):
    q, k, v = to_gpu(p)
    t = TORCH[p.dtype]
    off = torch.tensor(p.offsets, dtype=torch.int32, device="cuda")
    ob, o = guarded((p.T, p.H, p.d), t)
    lb, lse = guarded((p.T, p.H, 2), torch.float32)
    dg.mha_packed_forward(q, k, v, off, o, lse, p.params(dg), dg.DTYPE_CODE[p.dtype], stream)
    rc = dg.mha_packed_check_errors(stream)
    assert rc == 0, dg.STATUS.get(rc, rc)
    assert intact(ob) and intact(lb)
    return o, lse


def run_backward(dg, p, o, lse, stream=None):
    """o and lse: CPU tensors in the types the call takes."""
    q, k, v = to_gpu(p)
    t, code, params = TORCH[p.dtype], dg.DTYPE_CODE[p.dtype], p.params(dg)
    off = torch.tensor(p.offsets, dtype=torch.int32, device="cuda")
    outs = [guarded((p.T, h, p.d), t) for h in (p.H, p.G, p.G)]
    size = dg.mha_packed_workspace_size(params, code)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, and a guard band behind it
    dg.mha_packed_backward(q, k, v, o.cuda(), p.go.cuda(), lse.cuda(), off, *(x[1] for x in outs), ws, size, params,
                           code, stream)
    rc = dg.mha_packed_check_errors(stream)
    assert rc == 0, dg.STATUS.get(rc, rc)
    assert all(intact(b) for b, _ in outs) and bool((ws[size:] == 0xFF).all())
    return [x[1] for x in outs]


def within(got, ref, bound, what):
    got = got.double().cpu().numpy()
    same = np.isfinite(ref) == np.isfinite(got)
    assert same.all(), f"{what}: {np.count_nonzero(~same)} elements finite on one side only"
    assert (np.isposinf(ref) == np.isposinf(got)).all() or np.isnan(got[~np.isfinite(got)]).all()
    fine = np.isfinite(ref)
    worst = float(np.max((np.abs(got - ref) - bound)[fine], initial=-np.inf))
    assert worst <= 0, f"{what}: error above the bound by {worst:.3g}"
    return float(np.abs(got - ref)[fine].max(initial=0) / max(np.abs(ref[fine]).max(initial=0), 1e-30))


def check_forward(dg, p, kernel, parity_log, name):
    u = U[p.dtype] if kernel == dg.DGRAD_KERNEL_TC else 0.0
    o, lse = run_forward(dg, p)
    qkv = p.f64("q", "k", "v")
    ref_o, ref_l = om.forward(*qkv, p.offsets, p.window)
    bo, bl = om.forward_bounds(*qkv, p.offsets, p.window, u, OUT[p.dtype], TINY[p.dtype])
    err = within(o, ref_o, bo, "O")
    within(lse, ref_l, bl, "LSE")
    assert (np.isposinf(ref_l) == np.isposinf(lse.cpu().numpy())).all()
    parity_log(f"mha_packed_forward {name}", err, u + OUT[p.dtype])


def check_backward(dg, p, kernel, parity_log, name):
    u = U[p.dtype] if kernel == dg.DGRAD_KERNEL_TC else 0.0
    qkv = p.f64("q", "k", "v")
    ref_o, ref_l = om.forward(*qkv, p.offsets, p.window)
    o, lse = torch.from_numpy(ref_o).to(TORCH[p.dtype]), torch.from_numpy(ref_l).float()
    args = (*qkv, o.double().numpy(), p.f64("go")[0], lse.double().numpy(), p.offsets, p.window)
    refs, bounds = om.backward(*args), om.backward_bounds(*args, u, OUT[p.dtype], TINY[p.dtype])
    for what, got, ref, bound in zip(("dQ", "dK", "dV"), run_backward(dg, p, o, lse), refs, bounds):
        err = within(got, ref, bound, what)
        parity_log(f"mha_packed_backward {what} {name}", err, u + OUT[p.dtype])


# lens, heads, KV heads, head_dim, window, rows before, rows after, fused
CASES = {
    "one token": ([1], 2, 1, 64),
    "tile": ([128], 2, 2, 128),
    "one past a tile": ([129], 4, 2, 64),
    "ragged": ([5, 0, 130, 1, 64, 300], 8, 2, 64, 0, 3, 70),
    "ragged fused": ([257, 31, 2], 4, 2, 128, 0, 0, 9, True),
    "odd group": ([200, 150], 6, 2, 128),
    "one group": ([190], 8, 1, 64),
    "three heads": ([260, 3], 3, 3, 64, 0, 1, 0, True),
    "window": ([300, 40], 4, 2, 128, 50),
    "window of one": ([140], 2, 1, 64, 1),
    "window of a tile": ([515], 2, 2, 64, 128, 7, 7),
    "head 80": ([150, 10], 4, 2, 80, 0, 0, 0, True),
    "head 8": ([70], 2, 1, 8),
    "head 40": ([333], 2, 2, 40, 33),
    "nothing but padding": ([0, 0], 2, 1, 64, 0, 5, 140),
    "no sequence": ([], 2, 2, 64, 0, 3, 70),
}


def problem(case, dtype, seed=1):
    lens, H, G, d, *rest = (CASES | LONG)[case]
    names = ("window", "head", "tail", "fused")
    return Problem(lens, H, G, d, dtype=dtype, seed=seed + sum(lens) + d, **dict(zip(names, rest)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", list(CASES))
def test_cuda_core_kernels(dg, case, dtype, parity_log):
    p = problem(case, dtype)
    dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_SIMT)
    try:
        check_forward(dg, p, dg.DGRAD_KERNEL_SIMT, parity_log, f"simt {dtype} {case}")
        check_backward(dg, p, dg.DGRAD_KERNEL_SIMT, parity_log, f"simt {dtype} {case}")
    finally:
        dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_AUTO)


# Few KV heads and many tokens: the heads of a group are dealt to several blocks, and a third launch adds their sums.
SHARED = {
    "shared keys": ([2000], 8, 1, 64),
    "shared keys padded": ([1500, 40], 12, 1, 128, 0, 5, 130),
    "shared keys window": ([1700], 8, 1, 80, 900),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", list(SHARED))
def test_blocks_that_share_keys(dg, case, dtype, parity_log):
    lens, H, G, d, *rest = SHARED[case]
    p = Problem(lens, H, G, d, dtype=dtype, seed=5, **dict(zip(("window", "head", "tail"), rest)))
    plain = 256 + (p.T * H * 8 + 255) // 256 * 256
    assert dg.mha_packed_workspace_size(p.params(dg), dg.DTYPE_CODE[dtype]) > plain  # room for the partial sums
    check_backward(dg, p, dg.DGRAD_KERNEL_TC, parity_log, f"tc {dtype} {case}")


def test_shared_keys_recompute_what_is_not_finite(dg):
    """A query row that is not finite early in the sequence: later keys' gradients stay finite and right."""
    p = Problem([1600], 8, 1, 64, dtype="bf16", seed=6)
    p.q[1, :, 2] = float("nan")
    with np.errstate(all="ignore"):
        qkv = p.f64("q", "k", "v")
        ref_o, ref_l = om.forward(*qkv, p.offsets, 0)
        o_in, l_in = torch.from_numpy(ref_o).to(torch.bfloat16), torch.from_numpy(ref_l).float()
        refs = om.backward(*qkv, o_in.double().numpy(), p.f64("go")[0], l_in.double().numpy(), p.offsets, 0)
    for name, got, ref in zip(("dQ", "dK", "dV"), run_backward(dg, p, o_in, l_in), refs):
        within(got, ref, 8 * 2.0 ** -7 * np.abs(ref[np.isfinite(ref)]).max(), name)


# More key blocks than ring stages, tiles and blocks that end inside a sequence, windows that skip blocks.
LONG = {
    "long": ([1000], 4, 2, 128),
    "long 64": ([1111, 640], 4, 1, 64),
    "long odd group": ([900, 259], 3, 1, 128),
    "long window": ([1300], 4, 2, 64, 300),
    "long window odd": ([1200], 1, 1, 128, 129, 0, 0, True),
    "long head 96": ([700], 2, 1, 96),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", list(CASES) + list(LONG))
def test_tensor_core_kernels(dg, case, dtype, parity_log):
    p = problem(case, dtype)
    dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_TC)
    try:
        check_forward(dg, p, dg.DGRAD_KERNEL_TC, parity_log, f"tc {dtype} {case}")
        check_backward(dg, p, dg.DGRAD_KERNEL_TC, parity_log, f"tc {dtype} {case}")
    finally:
        dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_AUTO)


@pytest.mark.parametrize("dtype,lens,H,G,d", [("f32", [70, 9], 2, 1, 100), ("bf16", [90], 2, 2, 33),
                                               ("f32", [100, 1], 2, 1, 256), ("f16", [75], 2, 1, 192),
                                               ("bf16", [65], 3, 1, 132)])
def test_head_sizes_off_the_tensor_cores(dg, dtype, lens, H, G, d, parity_log):
    p = Problem(lens, H, G, d, dtype=dtype, seed=d)
    check_forward(dg, p, dg.DGRAD_KERNEL_SIMT, parity_log, f"{dtype} d={d}")
    check_backward(dg, p, dg.DGRAD_KERNEL_SIMT, parity_log, f"{dtype} d={d}")


def plant(p, what):
    """Infinities and NaN where some queries must not see them: a key and a value late in a sequence, whole rows
    of padding, and a query and dO row early in a sequence (which later keys' gradients must not see)."""
    a, b = p.offsets[0], p.offsets[1]
    if what == "late keys":
        p.v[b - 2, :, 3], p.k[b - 2, :, 1] = float("inf"), float("nan")
    elif what == "early queries":
        p.q[a + 1, :, 2], p.go[a + 1, :, 0] = float("nan"), float("inf")
    else:
        for x in (p.q, p.k, p.v, p.go):
            x[:a], x[p.offsets[-1]:], x[b:p.offsets[2]] = float("nan"), float("inf"), float("nan")


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["late keys", "early queries", "padding"])
def test_what_is_not_attended_never_shows(dg, what, d, dtype, kernel, parity_log):
    p = Problem([150, 20, 133], 4, 2, d, head=4, tail=30, dtype=dtype, seed=8)
    plant(p, what)
    run = dg.DGRAD_KERNEL_SIMT if kernel == "simt" else dg.DGRAD_KERNEL_AUTO
    u = U[dtype]
    dg.mha_packed_set_kernel(run)
    try:
        o, lse = run_forward(dg, p)
        qkv = p.f64("q", "k", "v")
        with np.errstate(all="ignore"):
            ref_o, ref_l = om.forward(*qkv, p.offsets, 0)
            clean = [np.nan_to_num(x, nan=0, posinf=0, neginf=0) for x in qkv]
            bo, _ = om.forward_bounds(*clean, p.offsets, 0, u, OUT[dtype], TINY[dtype])
            within(o, ref_o, 2 * bo + 1e-6, "O")
            o_in, l_in = torch.from_numpy(ref_o).to(TORCH[dtype]), torch.from_numpy(ref_l).float()
            args = (*qkv, o_in.double().numpy(), p.f64("go")[0], l_in.double().numpy(), p.offsets, 0)
            refs = om.backward(*args)
        for name, got, ref in zip(("dQ", "dK", "dV"), run_backward(dg, p, o_in, l_in), refs):
            size = np.abs(ref[np.isfinite(ref)]).max()
            within(got, ref, 8 * (u + OUT[dtype]) * size, name)
    finally:
        dg.mha_packed_set_kernel(dg.DGRAD_KERNEL_AUTO)


def test_large_scores_keep_the_statistics(dg, parity_log):
    """Scores in the hundreds: the running maximum moves by far more than one exponent between key tiles."""
    for dtype in ("bf16", "f32"):
        p = Problem([400], 2, 1, 64, dtype=dtype, seed=4)
        p.k *= torch.linspace(0.5, 12, 400).view(400, 1, 1).to(p.k.dtype)
        kernel = dg.DGRAD_KERNEL_TC if dtype == "bf16" else dg.DGRAD_KERNEL_SIMT
        check_forward(dg, p, kernel, parity_log, f"{dtype} large scores")


def test_many_short_sequences(dg, parity_log):
    """More sequences than a thread block has threads, many of them empty."""
    lens = [(7 * i) % 4 for i in range(1200)]
    p = Problem(lens, 2, 1, 64, dtype="bf16", seed=3)
    check_forward(dg, p, dg.DGRAD_KERNEL_TC, parity_log, "1200 sequences")
    check_backward(dg, p, dg.DGRAD_KERNEL_TC, parity_log, "1200 sequences")


@pytest.mark.parametrize("H,G,window", [(8, 2, 0), (3, 3, 70)])
def test_more_tiles_than_blocks_run_at_once(dg, H, G, window, parity_log):
    """Each block takes one tile after another, of all lengths, with padding among them; fp16's tiles are whole again after
    one with values that are not finite."""
    lens = [(53 * i) % 260 for i in range(200)]
    p = Problem(lens, H, G, 128, dtype="f16", seed=12, window=window, head=300, tail=200, fused=True)
    assert sum(-(-n // 256) for n in lens) * H > 3 * 152
    check_forward(dg, p, dg.DGRAD_KERNEL_TC, parity_log, f"tiles in a row {H}/{G}")
    for name in ("k", "v"):
        x = getattr(p, name)
        x[p.offsets[7::9][:8], 0, 3] = float("inf")   # the first position of some sequences: every query attends it
        x[[p.offsets[i + 1] - 1 for i in range(4, 200, 11) if lens[i] > 1], -1, 5] = float("nan")  # their last alone does
    o, _ = run_forward(dg, p)
    qkv = p.f64("q", "k", "v")
    with np.errstate(all="ignore"):
        ref, _ = om.forward(*qkv, p.offsets, window)
    clean = [np.nan_to_num(x, nan=0, posinf=0, neginf=0) for x in qkv]
    bound, _ = om.forward_bounds(*clean, p.offsets, window, U["f16"], OUT["f16"], TINY["f16"])
    got, rows = o.double().cpu().numpy(), np.isfinite(ref).all(axis=2)  # what attends no such value
    assert (np.abs(got - ref)[rows] <= 2 * bound[rows] + 1e-6).all()
    assert (np.isnan(got) | np.isinf(got))[~np.isfinite(ref)].all()


def test_two_streams_at_once(dg):
    """Two forwards in flight together, each taking tiles of its own grid alone."""
    p = [Problem([(31 * i) % 400 for i in range(90)], 8, 2, 64, dtype="bf16", seed=21 + j) for j in range(2)]
    alone = [run_forward(dg, x) for x in p]
    code = dg.DTYPE_CODE["bf16"]
    streams = [torch.cuda.Stream() for _ in p]
    sets = [(to_gpu(x), torch.tensor(x.offsets, dtype=torch.int32, device="cuda"), torch.empty_like(o), torch.empty_like(l))
            for x, (o, l) in zip(p, alone)]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s, (qkv, off, o, l) in zip(p, streams, sets):
            dg.mha_packed_forward(*qkv, off, o, l, x.params(dg), code, s)
    torch.cuda.synchronize()
    assert dg.mha_packed_check_errors() == 0
    for (a, b), (_, _, o, l) in zip(alone, sets):
        assert torch.equal(a, o) and torch.equal(b, l)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_results_repeat_and_follow_the_stream(dg, dtype):
    p = problem("ragged", dtype)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = run_forward(dg, p)
    with torch.cuda.stream(s):
        b = run_forward(dg, p, s)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    o, lse = a[0].cpu(), a[1].cpu()
    c = run_backward(dg, p, o, lse)
    with torch.cuda.stream(s):
        d = run_backward(dg, p, o, lse, s)
    assert all(torch.equal(x, y) for x, y in zip(c, d))


def test_forward_statistics_serve_the_dv_operator(dg):
    """One sequence: mha_grad_v takes the forward's LSE, and its dV is the packed backward's."""
    p = Problem([300], 8, 2, 64, dtype="bf16", seed=6)
    o, lse = run_forward(dg, p)
    dv = torch.empty(300, 2, 64, device="cuda")
    dg.mha_grad_v(p.q.cuda(), p.k.cuda(), p.go.cuda(), lse, dv, dg.MhaParams(300, 0, 8, 2, 64, 0), dg.DGRAD_BF16)
    assert dg.mha_grad_v_check_errors() == 0
    got = run_backward(dg, p, o.cpu(), lse.cpu())[2].float()
    qkv = p.f64("q", "k", "v")
    args = (*qkv, o.double().cpu().numpy(), p.f64("go")[0], lse.double().cpu().numpy(), [0, 300], 0)
    bound = om.backward_bounds(*args, U["bf16"], OUT["bf16"], TINY["bf16"])[2]
    assert (np.abs((got - dv).cpu().numpy()) <= 2 * bound).all()


def test_gradients_against_differences(dg):
    """Central differences of the float32 forward itself, in a few directions: with step h and results of size 1, the
    differences are off by about eps / h + h^2 (float32 outputs summed in float64)."""
    p = Problem([70, 33], 4, 2, 64, dtype="f32", seed=12)
    o, lse = run_forward(dg, p)
    grads = run_backward(dg, p, o.cpu(), lse.cpu())
    g = torch.Generator().manual_seed(1)
    h = 1e-2
    for name, grad in zip("qkv", grads):
        x = getattr(p, name)
        direction = torch.randn(x.shape, generator=g)
        keep = x.clone()
        loss = []
        for sign in (1, -1):
            setattr(p, name, keep + sign * h * direction)
            loss.append(float((run_forward(dg, p)[0].double().cpu() * p.go.double()).sum()))
        setattr(p, name, keep)
        want = (loss[0] - loss[1]) / (2 * h)
        terms = (grad.double().cpu() * direction.double())
        assert abs(float(terms.sum()) - want) <= 1e-2 * float(terms.square().sum().sqrt()) + 1e-3


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128), ("f32", 64)])
def test_captured_in_a_graph(dg, dtype, d):
    """Both directions replayed from a CUDA graph on new inputs give what calls give."""
    p = Problem([200, 75], 4, 1, d, tail=5, dtype=dtype, seed=1)
    other = Problem([200, 75], 4, 1, d, tail=5, dtype=dtype, seed=2)
    t, code, params = TORCH[dtype], dg.DTYPE_CODE[dtype], p.params(dg)
    q, k, v, go = p.q.cuda(), p.k.cuda(), p.v.cuda(), p.go.cuda()
    off = torch.tensor(p.offsets, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(p.T, 4, 2, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    size = dg.mha_packed_workspace_size(params, code)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def both():
        s = torch.cuda.current_stream()
        dg.mha_packed_forward(q, k, v, off, o, lse, params, code, s)
        dg.mha_packed_backward(q, k, v, o, go, lse, off, dq, dk, dv, ws, size, params, code, s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for buf, new in ((q, other.q), (k, other.k), (v, other.v), (go, other.go)):
        buf.copy_(new.cuda())
    for out in (o, lse, dq, dk, dv):
        out.zero_()
    for _ in range(3):  # replays one after another, each waiting for the last
        graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (o, lse, dq, dk, dv)]
    both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (o, lse, dq, dk, dv)))
    assert dg.mha_packed_check_errors() == 0


def test_calls_in_a_row_read_what_the_last_one_wrote(dg):
    """Forward and backward over and over on the same buffers with new inputs, nothing waiting between: the launches
    overlap at their edges, and each must see its predecessor's results."""
    a, b = (Problem([300, 128, 41], 4, 2, 64, dtype="bf16", seed=s) for s in (1, 2))
    want = []
    for p in (a, b):
        o, lse = run_forward(dg, p)
        want.append([o.cpu(), lse.cpu()] + [x.cpu() for x in run_backward(dg, p, o.cpu(), lse.cpu())])
    params, code = a.params(dg), dg.DGRAD_BF16
    q, k, v, go = (torch.empty_like(x, device="cuda") for x in (a.q, a.k, a.v, a.go))
    off = torch.tensor(a.offsets, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(a.T, 4, 2, device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]
    size = dg.mha_packed_workspace_size(params, code)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    inputs = [[x.cuda() for x in (p.q, p.k, p.v, p.go)] for p in (a, b)]
    got, s = [], torch.cuda.current_stream()
    for i in range(20):
        for buf, new in zip((q, k, v, go), inputs[i % 2]):
            buf.copy_(new)
        for _ in range(2):
            dg.mha_packed_forward(q, k, v, off, o, lse, params, code, s)
            dg.mha_packed_backward(q, k, v, o, go, lse, off, *grads, ws, size, params, code, s)
        got.append([x.clone() for x in (o, lse, *grads)])
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(x.cpu(), y) for x, y in zip(out, want[i % 2])), i


@pytest.mark.parametrize("offsets", [[0, 50, 40, 90], [-3, 50, 60, 90], [0, 50, 60, 1000]])
def test_malformed_offsets_are_reported_and_stay_in_bounds(dg, offsets):
    p = Problem([50, 10, 30], 2, 1, 64, dtype="bf16", seed=2)
    q, k, v = to_gpu(p)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ob, o = guarded((p.T, 2, 64), torch.bfloat16)
    lb, lse = guarded((p.T, 2, 2), torch.float32)
    dg.mha_packed_forward(q, k, v, off, o, lse, p.params(dg), dg.DGRAD_BF16)
    assert dg.mha_packed_check_errors() == 1  # DGRAD_ERR_INVALID_ARG
    assert intact(ob) and intact(lb)
    assert dg.mha_packed_check_errors() == 0  # reported once


def test_refusals_leave_the_outputs_alone(dg):
    p = Problem([40], 4, 2, 64, dtype="bf16", seed=2)
    q, k, v = to_gpu(p)
    off = torch.tensor(p.offsets, dtype=torch.int32, device="cuda")
    o = torch.full((40, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((40, 4, 2), 7.0, device="cuda")
    code = dg.DGRAD_BF16
    with pytest.raises(dg.DgradError):
        dg.mha_packed_forward(q, k, v, off, o, lse, dg.MhaPackedParams(40, 1, 4, 2, 64, 0, 0, 0, 0), 9)
    for bad in ((q.float(), k, v, off, o, lse), (q, k.cpu(), v, off, o, lse), (q, k, v, off.long(), o, lse),
                (q, k, v[:39], off, o, lse), (q, k, v, off, o, lse[:, :, :1]), (q.transpose(0, 1), k, v, off, o, lse)):
        with pytest.raises(ValueError):
            dg.mha_packed_forward(*bad, p.params(dg), code)
    torch.cuda.synchronize()
    assert bool((o == 7).all()) and bool((lse == 7).all())
