"""Pins of oracle/block.py (CPU): closed forms, worked numbers, and gradients against central
differences."""
import numpy as np
import pytest

from oracle import block

RNG = np.random.default_rng


def _difference(f, x, e=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += e
        lo[i] -= e
        g[i] = (f(hi) - f(lo)) / (2 * e)
    return g


def test_add_norm_closed_forms():
    r = RNG(0)
    x, s, w = r.standard_normal((3, 5, 8)), r.standard_normal((3, 5, 8)), r.standard_normal(8)
    y, h = block.add_norm_fwd(x, s, w, 0.0)
    np.testing.assert_array_equal(h, x + s)
    np.testing.assert_allclose(((y / w) ** 2).mean(-1), 1.0, rtol=1e-12)  # a row of length sqrt(D)
    np.testing.assert_allclose(block.add_norm_fwd(7 * h, None, w, 0.0)[0], y, rtol=1e-12)  # whatever its size
    np.testing.assert_allclose(block.add_norm_fwd(np.full((1, 4), 3.0), None, np.ones(4), 7.0)[0], 0.75)  # 3 / sqrt(9 + 7)


@pytest.mark.parametrize("eps", [0.0, 0.3])
def test_add_norm_gradients_by_differences(eps):
    r = RNG(1)
    x, s, dy, dh = (r.standard_normal((2, 3, 4)) for _ in range(4))
    w = r.standard_normal(4)

    def loss(x, s, w):
        y, h = block.add_norm_fwd(x, s, w, eps)
        return (y * dy).sum() + (h * dh).sum()

    d, dw = block.add_norm_bwd(x + s, w, eps, dy, dh)
    np.testing.assert_allclose(d, _difference(lambda t: loss(t, s, w), x), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(d, _difference(lambda t: loss(x, t, w), s), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, _difference(lambda t: loss(x, s, t), w), rtol=1e-6, atol=1e-8)
    size, _ = block.add_norm_bwd_sizes(x + s, w, eps, dy, dh)
    assert (np.abs(d) <= size * (1 + 1e-12)).all()


def test_e4m3_numbers():
    t = block.e4m3_numbers()
    assert len(t) == 127 and t[0] == 0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[-1] == 448 and t[-2] == 416
    np.testing.assert_array_equal(block.e4m3(np.concatenate([t, -t])), np.concatenate([t, -t]))
    # ties to even: 17 between 16 and 18, 19 between 18 and 20; half of the least number; past the largest
    np.testing.assert_array_equal(block.e4m3(np.array([17.0, 19.0, 2.0 ** -10, -3 * 2.0 ** -10, 500.0, -431.9])),
                                  [16.0, 20.0, 0.0, -2.0 ** -8, 448.0, -416.0])


def test_quantise():
    y = np.array([[100.0, -200.0, 51.0, 448.0, 0.0, 0.0, 0.0, 0.0]]) / 64
    q, s = block.quantise(y, 4)
    np.testing.assert_array_equal(s, [[1 / 64, block.LEAST]])
    np.testing.assert_array_equal(q[0], [96.0, -192.0, 52.0, 448.0, 0, 0, 0, 0])  # 100 and 200 are ties
    r = RNG(2).standard_normal((5, 64))
    for group in (0, 32):
        q, s = block.quantise(r, group)
        back = (q.reshape(5, -1, group or 64) * s[..., None]).reshape(r.shape)
        assert (np.abs(back - r) <= np.abs(r) / 16 + np.repeat(s, group or 64, -1) * 2.0 ** -10).all()


def test_axes():
    np.testing.assert_array_equal(block.axis_of_pair((2, 1, 3), False), [0, 0, 1, 2, 2, 2])
    np.testing.assert_array_equal(block.axis_of_pair((3, 1, 2), True), [0, 1, 2, 0, 0, 2])
    cos, sin = np.arange(12.0).reshape(4, 3), -np.arange(12.0).reshape(4, 3)
    c, s = block.angles(cos, sin, np.array([[[0, 3]], [[1, 1]]]), (2, 1), False)
    np.testing.assert_array_equal(c, [[[0, 1, 5], [9, 10, 5]]])
    np.testing.assert_array_equal(s, -c)


def test_clip():
    norm, out = block.clip([np.array([3.0, 0.0]), np.array([[4.0]])], 1.0)
    assert norm == 5.0
    np.testing.assert_allclose(np.concatenate([o.ravel() for o in out]), [0.6, 0.0, 0.8])
    assert block.clip([np.array([3.0, 4.0])], 5.0)[1][0].tolist() == [3.0, 4.0]
    assert block.clip([np.array([np.inf, 4.0])], 5.0)[1][0].tolist() == [np.inf, 4.0]
    assert block.clip([np.array([3.0, 4.0])], 0.0)[1][0].tolist() == [0.0, 0.0]


def test_park():
    x = np.array([[127.0, 2.5, -3.5, 0.49], [0.0, 0.0, 0.0, 0.0], [-254.0, 1.0, 3.0, 5.0]])
    codes, s = block.park(x)
    np.testing.assert_array_equal(s, [1.0, block.LEAST, 2.0])
    np.testing.assert_array_equal(codes, [[127, 2, -4, 0], [0, 0, 0, 0], [-127, 0, 2, 2]])
    x = RNG(3).standard_normal((50, 128)).astype(np.float32)
    codes, s = block.park(x)
    assert np.abs(codes).max() == 127
    assert (np.abs(codes * s[:, None] - x) <= s[:, None] * (0.5 + 1e-6)).all()
