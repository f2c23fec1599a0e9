"""GPU parity of the residual RMSNorm step (include/residual_rmsnorm.h) with the float64 oracle
(oracle/residual_rmsnorm.py), whose module derives the element-wise bounds used here."""
import numpy as np
import pytest
import torch

from oracle import residual_rmsnorm as rr

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
OUT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}
EPS = 1e-5
GUARD = 64
KIND = {"none": 0, "channel": 1, "element": 2}


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import conv2d_backward_implicit_gb300 as mod
    mod.library()
    return mod


def inputs(m, n, gate, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + m + 3 * n)
    t = TORCH[dtype]
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = {"f": r(m, n) * torch.exp(r(m, 1)), "x": r(m, n), "dy": r(m, n), "dh": r(m, n), "w_post": 1 + 0.2 * r(n),
         "w_pre": 1 + 0.2 * r(n)}
    d["gate"] = {"none": None, "channel": r(n), "element": r(m, n)}[gate]
    return {k: None if v is None else v.to(t) for k, v in d.items()}


def f64(x):
    return None if x is None else x.double().cpu().numpy()


def guarded(shape, dtype, offset=0):
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD + offset,), float("nan"), device="cuda", dtype=dtype)
    return buf, buf[GUARD + offset:GUARD + offset + n].view(shape)


def placed(x, offset):
    """x on the GPU, its first element `offset` elements past an aligned address."""
    if x is None:
        return None
    buf = torch.empty(x.numel() + offset, dtype=x.dtype, device="cuda")
    buf[offset:] = x.reshape(-1).cuda()
    return buf[offset:].view(x.shape)


def intact(buf, offset=0):
    return bool(torch.isnan(buf[:GUARD + offset].float()).all() and torch.isnan(buf[-GUARD:].float()).all())


def within(got, ref, bound, what):
    err = np.abs(f64(got) - ref)
    assert np.isfinite(err).all(), what
    worst = float((err - bound).max())
    assert worst <= 0, f"{what}: error above the bound by {worst:.3g}"
    return float(err.max() / max(np.abs(ref).max(), 1e-30))


def check(dg, m, n, gate, dtype, scale=0.7, offset=0, in_place=False, with_dh=True, seed=0, vectors=None):
    d = inputs(m, n, gate, dtype, seed)
    t, code = TORCH[dtype], dg.DTYPE_CODE[dtype]
    p = dg.ResidualRmsnormParams(m, n, KIND[gate], EPS, scale)
    c = {k: placed(v, vectors if vectors is not None and v is not None and v.dim() == 1 else offset)
         for k, v in d.items()}
    yb, y = guarded((m, n), t, offset)
    hb, h = guarded((m, n), t, offset)
    rb, rstd = guarded((m, 2), torch.float32)
    if in_place:
        h = c["x"]
    dg.residual_rmsnorm_forward(c["f"], c["x"], c["gate"], c["w_post"], c["w_pre"], h, y, rstd, p, code)
    torch.cuda.synchronize()
    assert intact(yb, offset) and intact(hb, offset) and intact(rb)
    a = [f64(d[k]) for k in ("f", "x", "gate", "w_post", "w_pre")] + [EPS, scale]
    errs = [within(g, r, b, w) for g, r, b, w in zip((h, y, rstd), rr.forward(*a),
                                                     rr.forward_bounds(*a, OUT[dtype], TINY[dtype]), ("H", "Y", "rstd"))]
    h_in, rstd_in = h.clone(), rstd.clone()
    outs = {k: guarded((m, n), t, offset) for k in ("df", "dx")}
    outs |= {k: guarded((n,), torch.float32) for k in ("dw_post", "dw_pre")}
    outs["dgate"] = {"none": (None, None), "channel": guarded((n,), torch.float32),
                     "element": guarded((m, n), t, offset)}[gate]
    dh = c["dh"] if with_dh else None
    dx = dh if in_place and with_dh else outs["dx"][1]
    size = dg.residual_rmsnorm_workspace_size(p, code)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    dg.residual_rmsnorm_backward(c["f"], placed(h_in.cpu(), offset), c["gate"], c["w_post"], c["w_pre"], rstd_in, c["dy"],
                                 dh, outs["df"][1], dx, outs["dgate"][1], outs["dw_post"][1], outs["dw_pre"][1], ws,
                                 size, p, code)
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xFF).all())
    for k, (b, _) in outs.items():
        assert b is None or intact(b, b.numel() - 2 * GUARD - outs[k][1].numel()), k
    a = [f64(d["f"]), f64(h_in), f64(d["gate"]), f64(d["w_post"]), f64(d["w_pre"]), f64(rstd_in), f64(d["dy"]),
         f64(d["dh"]) if with_dh else None, scale]
    df, g, dgate, dw_post, dw_pre = rr.backward(*a)
    bound = rr.backward_bounds(*a, OUT[dtype], TINY[dtype])
    errs.append(within(outs["df"][1], df, bound["df"], "dF"))
    errs.append(within(dx, g, bound["dx"], "dX"))
    within(outs["dw_post"][1], dw_post, bound["dw_post"], "dW_post")
    within(outs["dw_pre"][1], dw_pre, bound["dw_pre"], "dW_pre")
    if gate == "channel":
        within(outs["dgate"][1], dgate.sum(0), bound["dgate_sum"], "dgate")
    if gate == "element":
        within(outs["dgate"][1], dgate, bound["dgate"], "dgate")
    return max(errs)


# One row; widths below, at and above vectors, warps and blocks; more rows than blocks; a wide row.
# Widths that are no multiple of a 16-byte piece have rows that begin inside one, with one row per team and with many.
SIZES = [(1200, 577), (650, 2050), (333, 4090), (2500, 9), (153, 130), (9, 6883), (1, 1), (1, 1024), (3, 7), (700, 64), (5, 96), (33, 1001), (650, 256), (17, 2048), (9, 4096), (4, 5000),
         (3, 8192), (2, 20000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gate", ["none", "channel", "element"])
@pytest.mark.parametrize("m,n", SIZES)
def test_both_directions(dg, m, n, gate, dtype, parity_log):
    parity_log(f"residual_rmsnorm {dtype} {m}x{n} {gate}", check(dg, m, n, gate, dtype), OUT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["channel", "element"])
def test_off_alignment(dg, gate, dtype):
    check(dg, 20, 1024, gate, dtype, offset=1)
    check(dg, 20, 512, gate, dtype, offset=4 if dtype == "bf16" else 2)


@pytest.mark.parametrize("gate", ["channel", "element"])
@pytest.mark.parametrize("m,n", [(700, 577), (650, 1024), (2, 1001)])
def test_vectors_off_alignment(dg, m, n, gate):
    """The weights (and a channel's gate) lie anywhere; the [m, n] tensors are aligned."""
    check(dg, m, n, gate, "bf16", vectors=3)


@pytest.mark.parametrize("n", [512, 333])
def test_in_place(dg, n):
    check(dg, 400, n, "channel", "bf16", in_place=True)


def test_without_the_other_gradient(dg):
    check(dg, 50, 768, "element", "bf16", with_dh=False)
    check(dg, 50, 70, "none", "f32", with_dh=False, scale=-2.0)


def test_zero_rows_and_large_values(dg):
    """A row of zeros has rstd 1 / sqrt(eps) and no NaN; float32 rows of 1e18 overflow nothing (squares to 1e36)."""
    m, n = 4, 256
    f = torch.zeros(m, n)
    f[2] = 1e18 * torch.randn(n, generator=torch.Generator().manual_seed(0)).clamp(-2, 2)
    x = torch.zeros(m, n)
    w = torch.ones(n).cuda()
    h, y, rstd = (torch.empty(m, k, device="cuda") for k in (n, n, 2))
    p = dg.ResidualRmsnormParams(m, n, 0, EPS, 1.0)
    dg.residual_rmsnorm_forward(f.cuda(), x.cuda(), None, w, w, h, y, rstd, p, dg.DGRAD_F32)
    ref = rr.forward(f64(f), f64(x), None, np.ones(n), np.ones(n), EPS, 1.0)
    for got, want in zip((h, y, rstd), ref):
        assert np.allclose(f64(got), want, rtol=1e-5, atol=1e-6)


def test_results_repeat_on_another_stream(dg):
    m, n = 900, 512
    d = {k: None if v is None else v.cuda() for k, v in inputs(m, n, "channel", "bf16").items()}
    p = dg.ResidualRmsnormParams(m, n, 1, EPS, 0.5)
    rstd = torch.rand(m, 2, device="cuda") + 0.5
    size = dg.residual_rmsnorm_workspace_size(p, 1)
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            out = [torch.empty_like(d["f"]), torch.empty_like(d["f"])] + [torch.empty(n, device="cuda") for _ in range(3)]
            ws = torch.empty(size, dtype=torch.uint8, device="cuda")
            dg.residual_rmsnorm_backward(d["f"], d["x"], d["gate"], d["w_post"], d["w_pre"], rstd, d["dy"], d["dh"],
                                         out[0], out[1], out[2], out[3], out[4], ws, size, p, 1, s)
            s.synchronize()
            got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_gradients_against_differences(dg):
    """Central differences of the float32 forward, in random directions (step 1e-2: truncation about 1e-4 relative)."""
    m, n, scale = 6, 40, 0.8
    d = inputs(m, n, "element", "f32", seed=5)
    p = dg.ResidualRmsnormParams(m, n, 2, 1e-3, scale)

    def forward():
        h, y, rstd = (torch.empty(m, k, device="cuda") for k in (n, n, 2))
        c = {k: v.cuda() for k, v in d.items()}
        dg.residual_rmsnorm_forward(c["f"], c["x"], c["gate"], c["w_post"], c["w_pre"], h, y, rstd, p, 0)
        return h, y, rstd

    def loss():
        h, y, _ = forward()
        return float((y.cpu().double() * d["dy"].double()).sum() + (h.cpu().double() * d["dh"].double()).sum())

    h, _, rstd = forward()
    c = {k: v.cuda() for k, v in d.items()}
    grads = {k: torch.empty_like(c[a]) for k, a in (("f", "f"), ("x", "x"), ("gate", "f"), ("w_post", "w_post"),
                                                    ("w_pre", "w_pre"))}
    size = dg.residual_rmsnorm_workspace_size(p, 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dg.residual_rmsnorm_backward(c["f"], h, c["gate"], c["w_post"], c["w_pre"], rstd, c["dy"], c["dh"], grads["f"],
                                 grads["x"], grads["gate"], grads["w_post"], grads["w_pre"], ws, size, p, 0)
    g = torch.Generator().manual_seed(3)
    for name, grad in grads.items():
        direction, keep, step = torch.randn(d[name].shape, generator=g), d[name].clone(), 1e-2
        values = []
        for sign in (1, -1):
            d[name] = keep + sign * step * direction
            values.append(loss())
        d[name] = keep
        terms = grad.cpu().double() * direction.double()
        assert abs(float(terms.sum()) - (values[0] - values[1]) / (2 * step)) <= 1e-2 * float(terms.norm()) + 2e-3, name


def test_refusals(dg):
    d = {k: v.cuda() for k, v in inputs(4, 64, "channel", "bf16").items()}
    h, y = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    args = (d["f"], d["x"], d["gate"], d["w_post"], d["w_pre"], h, y, None)
    dg.residual_rmsnorm_forward(*args, dg.ResidualRmsnormParams(4, 64, 1, EPS, 1.0), 1)  # rstd may be None
    h.zero_(), y.zero_()
    for p, status in ((dg.ResidualRmsnormParams(4, 64, 1, float("nan"), 1.0), 1),
                      (dg.ResidualRmsnormParams(4, 64, 1, EPS, float("inf")), 1)):
        with pytest.raises(dg.DgradError) as e:
            dg.residual_rmsnorm_forward(*args, p, 1)
        assert e.value.status == status
    with pytest.raises(ValueError):
        dg.residual_rmsnorm_forward(*args, dg.ResidualRmsnormParams(4, 63, 1, EPS, 1.0), 1)
    with pytest.raises(ValueError):
        dg.residual_rmsnorm_forward(d["f"].float(), *args[1:], dg.ResidualRmsnormParams(4, 64, 1, EPS, 1.0), 1)
    torch.cuda.synchronize()
    assert not h.any() and not y.any()
