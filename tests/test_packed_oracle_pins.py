"""The float64 oracles of packed attention and the residual RMSNorm, pinned: against the C oracle of the
attention dV, closed forms, and central differences of their own forward passes."""
import numpy as np
import pytest

from oracle import mha, mha_packed, residual_rmsnorm as rr


def attention_inputs(T, H, G, d, seed):
    g = np.random.default_rng(seed)
    return [g.standard_normal(s) for s in ((T, H, d), (T, G, d), (T, G, d), (T, H, d))]


@pytest.mark.parametrize("n,H,G,d,window", [(1, 2, 1, 8, 0), (37, 4, 2, 16, 0), (50, 3, 1, 8, 7), (20, 2, 2, 8, 1)])
def test_single_sequence_against_the_dv_oracle(n, H, G, d, window):
    q, k, v, go = attention_inputs(n, H, G, d, n + d)
    o, lse = mha_packed.forward(q, k, v, [0, n], window)
    assert np.allclose(lse, mha.forward_lse(q, k, 0, window), rtol=1e-12, atol=1e-12)
    dv = mha_packed.backward(q, k, v, o, go, lse, [0, n], window)[2]
    assert np.allclose(dv, mha.grad_v(q, k, go, lse, 0, window), rtol=1e-11, atol=1e-12)


def test_sequences_do_not_see_each_other():
    T, offsets = 60, [3, 3, 20, 21, 50]
    q, k, v, go = attention_inputs(T, 4, 2, 8, 5)
    o, lse = mha_packed.forward(q, k, v, offsets, 0)
    grads = mha_packed.backward(q, k, v, o, go, lse, offsets, 0)
    for a, b in ((3, 20), (20, 21), (21, 50)):
        alone, l1 = mha_packed.forward(q[a:b], k[a:b], v[a:b], [0, b - a], 0)
        assert np.array_equal(alone, o[a:b]) and np.array_equal(l1, lse[a:b])
    outside = np.r_[0:3, 50:60]
    assert (o[outside] == 0).all() and (lse[outside, :, 0] == 0).all() and np.isposinf(lse[outside, :, 1]).all()
    assert all((x[outside] == 0).all() for x in grads)


def test_window_of_one_copies_v():
    q, k, v, _ = attention_inputs(9, 4, 2, 8, 1)
    o, lse = mha_packed.forward(q, k, v, [0, 9], 1)
    assert np.allclose(o, np.repeat(v, 2, axis=1)) and np.allclose(lse[..., 1], 0)


def test_what_is_not_attended_stays_out():
    q, k, v, go = attention_inputs(12, 2, 1, 8, 2)
    o, lse = mha_packed.forward(q, k, v, [0, 6, 12], 0)
    v2, k2 = v.copy(), k.copy()
    v2[5], k2[5], v2[7:] = np.inf, np.nan, np.nan
    o2, _ = mha_packed.forward(q, k2, v2, [0, 6, 12], 0)
    # Another order of summation (only the attended terms): a few float64 roundings.
    assert np.allclose(o2[:5], o[:5], rtol=1e-12, atol=1e-14) and np.allclose(o2[6], o[6], rtol=1e-12, atol=1e-14)
    assert np.isnan(o2[5]).all()


def central(fn, x, step=1e-5):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + step
        up = fn()
        x[i] = old - step
        g[i] = (up - fn()) / (2 * step)
        x[i] = old
    return g


@pytest.mark.parametrize("window", [0, 3])
def test_attention_gradients_against_differences(window):
    offsets = [1, 5, 5, 12]
    q, k, v, go = attention_inputs(13, 4, 2, 4, 9)

    def loss():
        return float((mha_packed.forward(q, k, v, offsets, window)[0] * go).sum())

    o, lse = mha_packed.forward(q, k, v, offsets, window)
    for got, x in zip(mha_packed.backward(q, k, v, o, go, lse, offsets, window), (q, k, v)):
        assert np.allclose(got, central(loss, x), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("kind", ["none", "channel", "element"])
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_gradients_against_differences(kind, with_dh):
    g = np.random.default_rng(3)
    m, n, eps, scale = 4, 7, 1e-3, 0.7
    f, x, dy, dh = (g.standard_normal((m, n)) for _ in range(4))
    w_post, w_pre = 1 + 0.3 * g.standard_normal((2, n))
    gate = {"none": None, "channel": g.standard_normal(n), "element": g.standard_normal((m, n))}[kind]

    def loss():
        h, y, _ = rr.forward(f, x, gate, w_post, w_pre, eps, scale)
        return float((y * dy).sum() + ((h * dh).sum() if with_dh else 0.0))

    h, _, rstd = rr.forward(f, x, gate, w_post, w_pre, eps, scale)
    df, dx, dgate, dw_post, dw_pre = rr.backward(f, h, gate, w_post, w_pre, rstd, dy, dh if with_dh else None, scale)
    pairs = [(df, f), (dx, x), (dw_post, w_post), (dw_pre, w_pre)]
    if gate is not None:
        pairs.append((dgate.sum(0) if kind == "channel" else dgate, gate))
    for got, arg in pairs:
        assert np.allclose(got, central(loss, arg), rtol=1e-6, atol=1e-8)


def test_norm_closed_form():
    """A constant row has rms |c|: with eps 0 the normalised row is sign(c), so H = X + scale gate w."""
    f, x = np.full((2, 5), -3.0), np.zeros((2, 5))
    h, y, rstd = rr.forward(f, x, np.full(5, 0.5), np.full(5, 2.0), np.full(5, 4.0), 0.0, 3.0)
    assert np.allclose(h, -3.0) and np.allclose(y, -4.0) and np.allclose(rstd, 1 / 3)
