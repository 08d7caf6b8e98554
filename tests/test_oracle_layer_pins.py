"""Pins of oracle/layer.py (CPU): closed forms, the quadratic form of linear attention,
continuation of a stream, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import layer

RNG = np.random.default_rng


def _la(seed, B=2, T=7, H=3, K=4, V=5):
    r = RNG(seed)
    return (r.standard_normal((B, T, H, K)), r.standard_normal((B, T, H, K)), r.standard_normal((B, T, H, V)),
            -r.uniform(0.0, 1.0, H), r.standard_normal((B, H, V, K)))


def _difference(f, x, e=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += e
        lo[i] -= e
        g[i] = (f(hi) - f(lo)) / (2 * e)
    return g


def test_la_equals_the_quadratic_form():
    q, k, v, g, s0 = _la(0)
    o, final, _ = layer.la_fwd(q, k, v, g, s0)
    T = q.shape[1]
    t = np.arange(T)
    w = np.where(t[:, None] >= t[None, :], np.exp(g[:, None, None] * (t[:, None] - t[None, :])), 0.0)
    ref = np.einsum("bthk,bshk,hts,bshv->bthv", q, k, w, v)
    ref += np.exp(g[None, None, :, None] * (t[None, :, None, None] + 1)) * np.einsum("bhvk,bthk->bthv", s0, q)
    np.testing.assert_allclose(o, ref, rtol=1e-12, atol=1e-12)
    fade = np.exp(g[:, None] * (T - 1 - t))
    ref = np.exp(g * T)[None, :, None, None] * s0 + np.einsum("hs,bshv,bshk->bhvk", fade, v, k)
    np.testing.assert_allclose(final, ref, rtol=1e-12, atol=1e-12)


def test_la_no_decay_sums_and_full_decay_forgets():
    q, k, v, _, s0 = _la(1)
    _, final, _ = layer.la_fwd(q, k, v, np.zeros(3), s0)
    np.testing.assert_allclose(final, s0 + np.einsum("bthv,bthk->bhvk", v, k), rtol=1e-12, atol=1e-12)
    o, final, _ = layer.la_fwd(q, k, v, np.full(3, -np.inf), s0)
    np.testing.assert_allclose(final, np.einsum("bhv,bhk->bhvk", v[:, -1], k[:, -1]), atol=1e-14)
    np.testing.assert_allclose(o, v * (q * k).sum(-1, keepdims=True), atol=1e-13)


def test_la_stream_continues():
    q, k, v, g, s0 = _la(2)
    o, final, _ = layer.la_fwd(q, k, v, g, s0)
    o1, mid, _ = layer.la_fwd(q[:, :3], k[:, :3], v[:, :3], g, s0)
    o2, end, _ = layer.la_fwd(q[:, 3:], k[:, 3:], v[:, 3:], g, mid)
    np.testing.assert_array_equal(np.concatenate([o1, o2], 1), o)
    np.testing.assert_array_equal(end, final)


def test_la_gradients_by_differences():
    q, k, v, g, s0 = _la(3, B=1, T=4, H=2, K=3, V=2)
    r = RNG(4)
    d_o, dS = r.standard_normal(v.shape), r.standard_normal(s0.shape)

    def loss(q_, k_, v_, s_):
        o, final, _ = layer.la_fwd(q_, k_, v_, g, s_)
        return (o * d_o).sum() + (final * dS).sum()

    got = layer.la_bwd(q, k, v, g, s0, d_o, dS)
    ref = (_difference(lambda x: loss(x, k, v, s0), q), _difference(lambda x: loss(q, x, v, s0), k),
           _difference(lambda x: loss(q, k, x, s0), v), _difference(lambda x: loss(q, k, v, x), s0))
    for a, b in zip(got, ref):
        np.testing.assert_allclose(a, b, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(interleaved):
    r = RNG(5)
    B, T, H, D, R = 2, 3, 2, 8, 4
    x, w, dy = r.standard_normal((B, T, H, D)), r.uniform(0.5, 1.5, D), r.standard_normal((B, T, H, D))
    a = r.uniform(-3, 3, (B, T, R // 2))
    c, s = np.cos(a), np.sin(a)
    y = layer.norm_rope_fwd(x, np.ones(D), c, s, 0.0, interleaved)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)  # rotations keep the length
    np.testing.assert_array_equal(layer.rotate(x, c * 0 + 1, s * 0, interleaved), x)
    np.testing.assert_allclose(layer.rotate(layer.rotate(x, c, s, interleaved), c, s, interleaved, -1.0), x, atol=1e-13)
    # a pair is a complex number times e^(i angle)
    p, n = layer._pairs(R, interleaved)
    z = (x[..., p] + 1j * x[..., n]) * np.exp(1j * a)[:, :, None]
    turned = layer.rotate(x, c, s, interleaved)
    np.testing.assert_allclose(turned[..., p] + 1j * turned[..., n], z, atol=1e-13)
    np.testing.assert_array_equal(turned[..., R:], x[..., R:])
    dx, dw = layer.norm_rope_bwd(x, w, c, s, 1e-3, interleaved, dy)
    loss = lambda x_, w_: (layer.norm_rope_fwd(x_, w_, c, s, 1e-3, interleaved) * dy).sum()  # noqa: E731
    np.testing.assert_allclose(dx, _difference(lambda t: loss(t, w), x), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(dw, _difference(lambda t: loss(x, t), w), rtol=1e-6, atol=1e-7)


def test_gated_norm():
    r = RNG(6)
    x, z, dy = (r.standard_normal((2, 2, 2, 6)) for _ in range(3))
    w = r.uniform(0.5, 1.5, 6)
    assert not layer.gated_norm_fwd(x, z * 0, w, 1e-6).any()  # a closed gate
    big = layer.gated_norm_fwd(x, z * 0 + 50.0, np.ones(6), 0.0) / 50.0
    np.testing.assert_allclose((big * big).mean(-1), 1.0, rtol=1e-12)
    dx, dz, dw = layer.gated_norm_bwd(x, z, w, 1e-3, dy)
    loss = lambda x_, z_, w_: (layer.gated_norm_fwd(x_, z_, w_, 1e-3) * dy).sum()  # noqa: E731
    np.testing.assert_allclose(dx, _difference(lambda t: loss(t, z, w), x), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(dz, _difference(lambda t: loss(x, t, w), z), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(dw, _difference(lambda t: loss(x, z, t), w), rtol=1e-6, atol=1e-7)
