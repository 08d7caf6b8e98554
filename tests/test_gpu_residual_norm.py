"""GPU tests of the residual's addition with the RMS norm (gdn_add_norm_fwd, _quant, _bwd)
against float64.

Tolerances, for every element.  A rounding to type t is off by at most half a step, u =
eps(t)/2 of the value: bf16 2^-8, float32 2^-24, e4m3 2^-4 (2^-10 below its normal numbers).
The float32 arithmetic before it: sums of squares of up to 8192 terms, at most 16 a lane one
after another and ten more levels, each off by 2^-24: 26 * 6e-8 = 1.6e-6, of which the root
takes half; 1 / sqrt and three products 5 * 6e-8 = 3e-7: within F = 2e-6 of the value (y and
the scales), or of the sizes of the terms where terms cancel (gradients: two sums, 4 F).  A
weight's gradient adds rows: with the sizes here at most 60 float32 additions one after
another, 60 * 6e-8 = 4e-6 of the sum of the terms' sizes, besides the terms' own F."""
import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F = 2e-6
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _np(t):
    return t.detach().double().cpu().numpy()


def _within(name, got, ref, size=None, f=F):
    x, u = _np(got), U[got.dtype]
    assert x.shape == ref.shape and np.isfinite(x).all(), name
    off = np.abs(x - ref) - (u * np.abs(ref) + f * (1 + u) * (np.abs(ref) if size is None else size))
    assert x.size == 0 or off.max() <= 0, f"{name}: {off.max():.2e} past its bound at {np.unravel_index(off.argmax(), off.shape)}"


def _nan(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _inputs(rows, D, dtype, stream, slices, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * D + rows)
    dt, rt = DT[dtype], DT[stream]

    def n(t, cut, std=1.0):
        if cut:
            return (torch.randn(rows, 2 * D + 64, generator=g, device="cuda") * std).to(t)[:, 64:64 + D]
        return (torch.randn(rows, D, generator=g, device="cuda") * std).to(t)

    x, r = n(dt, slices), n(rt, slices, 3.0)
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    return x, r, w, n(dt, False), n(rt, False)


CASES = [
    # rows, D, dtype, stream's type, slices of wider rows
    (1, 8, "bf16", "bf16", False),
    (3, 4, "f32", "f32", False),
    (1, 2048, "bf16", "bf16", False),
    (8, 128, "bf16", "f32", True),
    (17, 256, "bf16", "bf16", True),
    (9, 264, "f32", "f32", True),
    (100, 768, "bf16", "bf16", False),
    (33, 1000, "bf16", "f32", True),
    (7, 1024, "f32", "f32", False),
    (5, 1032, "bf16", "bf16", False),
    (12, 1540, "f32", "f32", True),
    (6, 2056, "bf16", "f32", False),
    (11, 4096, "bf16", "bf16", True),
    (4, 4100, "f32", "f32", False),
    (3, 4104, "bf16", "f32", False),
    (5, 5000, "bf16", "bf16", False),
    (3, 8192, "bf16", "bf16", False),
    (2, 8192, "bf16", "f32", True),
    (3, 8192, "f32", "f32", False),
    (3000, 96, "bf16", "bf16", False),
    (2500, 512, "f32", "f32", False),
    (1900, 1536, "bf16", "f32", False),
    # a backward of one cluster of 2, 11, 15 and 16 blocks of eight rows, and one block more; of
    # 16 blocks of a row
    (9, 512, "bf16", "bf16", False), (88, 256, "bf16", "bf16", False), (115, 1000, "bf16", "bf16", False),
    (128, 512, "f32", "f32", False), (129, 768, "bf16", "bf16", False),
    (1000, 24, "bf16", "bf16", False), (777, 40, "f32", "f32", False), (500, 200, "bf16", "f32", False),
    (16, 8192, "f32", "f32", False), (15, 8192, "bf16", "bf16", False), (17, 8192, "bf16", "f32", False),
]


@pytest.mark.parametrize("rows,D,dtype,stream,slices", CASES)
def test_forward_and_backward(rows, D, dtype, stream, slices):
    x, r, w, dy, dh = _inputs(rows, D, dtype, stream, slices)
    dt, rt = x.dtype, r.dtype
    y, h = gdn.gdn_add_norm_fwd(x, r, w, eps=EPS, y=_nan(rows, D, dtype=dt), h=_nan(rows, D, dtype=rt))
    grads = [_nan(rows, D, dtype=dt), _nan(rows, D, dtype=rt) if rt != dt else None, _nan(D, dtype=dt)]
    dx, dr, dw = gdn.gdn_add_norm_bwd(h, w, dy, dh, eps=EPS, grads=grads)
    again = gdn.gdn_add_norm_bwd(h, w, dy, dh, eps=EPS)
    torch.cuda.synchronize()
    ry, rh = block.add_norm_fwd(_np(x), _np(r), _np(w), EPS)
    _within("y", y, ry)
    _within("h", h, rh, f=2.0 ** -23)
    rd, rdw = block.add_norm_bwd(_np(h), _np(w), EPS, _np(dy), _np(dh))  # of the h that was kept
    sd, sdw = block.add_norm_bwd_sizes(_np(h), _np(w), EPS, _np(dy), _np(dh))
    _within("dx", dx, rd, sd, 4 * F)
    _within("d_residual", dr, rd, sd, 4 * F)
    _within("dw", dw, rdw, sdw, 4 * F)
    assert (dr is dx) == (rt == dt) or torch.equal(dr, dx)
    assert all(torch.equal(a, b) for a, b in zip((dx, dr, dw), again))


@pytest.mark.parametrize("rows,D,dtype,stream,slices", CASES[:1] + CASES[4:7] + CASES[11:15])
def test_without_residual_or_its_gradient(rows, D, dtype, stream, slices):
    x, r, w, dy, dh = _inputs(rows, D, dtype, stream, slices)
    y, h = gdn.gdn_add_norm_fwd(x, None, w, eps=EPS)
    assert h is None
    ry, _ = block.add_norm_fwd(_np(x), None, _np(w), EPS)
    _within("y", y, ry)
    dx, dr, dw = gdn.gdn_add_norm_bwd(x, w, dy, eps=EPS)  # a slice, where the case has one
    kept = (x.to(r.dtype) + r).contiguous()
    d2 = gdn.gdn_add_norm_bwd(kept, w, dy, None, eps=EPS)
    torch.cuda.synchronize()
    for h, got in ((x, (dx, dr, dw)), (kept, d2)):
        rd, rdw = block.add_norm_bwd(_np(h), _np(w), EPS, _np(dy))
        sd, sdw = block.add_norm_bwd_sizes(_np(h), _np(w), EPS, _np(dy))
        _within("dx", got[0], rd, sd, 4 * F)
        _within("d_residual", got[1], rd, sd, 4 * F)
        _within("dw", got[2], rdw, sdw, 4 * F)


@pytest.mark.parametrize("rows,D,dtype,stream,slices,group", [
    (1, 8, "bf16", "bf16", False, 0), (3, 32, "f32", "f32", False, 32), (5, 128, "bf16", "bf16", False, 128),
    (17, 256, "bf16", "bf16", True, 64), (9, 260, "f32", "f32", True, 0), (100, 768, "bf16", "bf16", False, 128),
    (33, 1000, "bf16", "f32", True, 0), (31, 992, "bf16", "f32", False, 32), (8, 2048, "f32", "f32", False, 128),
    (6, 2176, "bf16", "f32", False, 64), (7, 4096, "bf16", "bf16", False, 0), (3, 4224, "f32", "f32", True, 32),
    (3, 8192, "bf16", "bf16", False, 128), (2, 8192, "bf16", "f32", False, 0), (3000, 96, "bf16", "bf16", False, 32),
    (70, 256, "f32", "f32", False, 128), (70, 256, "f32", "f32", False, 32), (129, 256, "bf16", "bf16", False, 128),
    (129, 512, "bf16", "f32", False, 0), (333, 64, "bf16", "bf16", False, 0), (333, 128, "bf16", "f32", False, 32), (5, 24, "bf16", "bf16", False, 0)])
def test_quant(rows, D, dtype, stream, slices, group):
    x, r, w, _, _ = _inputs(rows, D, dtype, stream, slices)
    out = torch.full((rows, D), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # NaN
    parts = D // group if group else 1
    y, s, h = gdn.gdn_add_norm_quant(x, r, w, eps=EPS, group=group, y=out, scales=_nan(rows, parts, dtype=torch.float32))
    torch.cuda.synchronize()
    ry, rh = block.add_norm_fwd(_np(x), _np(r), _np(w), EPS)
    _, rs = block.quantise(ry, group)
    _within("h", h, rh, f=2.0 ** -23)
    _within("scales", s, rs)
    step = np.repeat(_np(s), D // parts, -1)
    q = _np(y.float())
    off = np.abs(q * step - ry) - (np.abs(ry) * (2.0 ** -4 + 4 * F) + step * 2.0 ** -10)
    assert np.isfinite(q).all() and off.max() <= 0, off.max()
    # the group's largest number is e4m3's
    assert (np.abs(q).reshape(rows, parts, -1).max(-1) == 448).all()
    plain, h2 = gdn.gdn_add_norm_fwd(x, r, w, eps=EPS)
    assert torch.equal(h, h2)


@pytest.mark.parametrize("rows,D,dtype,stream,group", [
    (4000, 768, "bf16", "bf16", 128), (4000, 768, "bf16", "f32", 128), (4000, 768, "f32", "f32", 64), (900, 4096, "bf16", "bf16", 0),
    (900, 4096, "f32", "f32", 0), (900, 4096, "bf16", "f32", 0), (3000, 1000, "f32", "f32", 0), (3000, 992, "bf16", "bf16", 32),
    (20000, 128, "f32", "f32", 0), (20000, 192, "bf16", "f32", 64), (700, 4960, "f32", "f32", 32)])
def test_quant_gives_the_nearest_number(rows, D, dtype, stream, group):
    """Every 8-bit number is the one nearest to the exact quotient 448 t / max|t| of the group
    (t = (x + residual) w; the row's norm divides out): of 3 million elements not one is on the
    wrong side of a middle.  Below 2^-6 a middle may be decided by float32's error: within 2^-20
    of it either side is taken.  (In bf16 the largest t is a float32, off by up to 2^-24: these
    cases have no quotient that close to a middle but exact ties.)"""
    x, r, w, _, _ = _inputs(rows, D, dtype, stream, False, seed=9)
    y, _, _ = gdn.gdn_add_norm_quant(x, r, w, eps=EPS, group=group)
    torch.cuda.synchronize()
    t = ((_np(x) + _np(r)) * _np(w)).reshape(rows, -1, group or D)
    exact = t * 448.0 / np.abs(t).max(-1, keepdims=True)
    want, got = block.e4m3(exact), _np(y.float()).reshape(t.shape)
    wrong = want != got
    low = np.abs(exact) < 2.0 ** -6
    assert not (wrong & ~low).any()
    middle = (want + got) / 2
    assert (np.abs(exact - middle) <= 2.0 ** -20 * np.abs(middle))[wrong].all()


def test_quant_of_no_residual_and_of_the_least_numbers():
    """Rows of zeros and of numbers so small that their scale would be subnormal."""
    x = torch.zeros(4, 256, device="cuda")
    x[1] = 1e-38
    x[2, :128] = 3.0
    x[3] = -2.0
    w = torch.ones(256, device="cuda")
    y, s, h = gdn.gdn_add_norm_quant(x, None, w, eps=1.0, group=128)
    torch.cuda.synchronize()
    assert h is None
    ry, _ = block.add_norm_fwd(_np(x), None, _np(w), 1.0)
    q, rs = block.quantise(ry, 128)
    _within("scales", s, rs)
    assert torch.equal(s[0], torch.full((2,), 2.0 ** -126, device="cuda")) and s[2, 1] == 2.0 ** -126
    assert not y[0].float().any() and not y[2, 128:].float().any()
    np.testing.assert_array_equal(_np(y.float())[2:], q[2:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_row(bad):
    x, r, w, dy, dh = _inputs(40, 768, "bf16", "bf16", False)
    y, h = gdn.gdn_add_norm_fwd(x, r, w)
    q, s, _ = gdn.gdn_add_norm_quant(x, r, w, group=128)
    g = gdn.gdn_add_norm_bwd(h, w, dy, dh)
    x2 = x.clone()
    x2[13, 300] = bad
    y2, h2 = gdn.gdn_add_norm_fwd(x2, r, w)
    q2, s2, _ = gdn.gdn_add_norm_quant(x2, r, w, group=128)
    row, _, _ = gdn.gdn_add_norm_quant(x2, r, w)
    g2 = gdn.gdn_add_norm_bwd(h2, w, dy, dh)
    torch.cuda.synchronize()
    other = torch.arange(40, device="cuda") != 13
    for a, b in ((y, y2), (q.float(), q2.float()), (s, s2), (g[0], g2[0])):
        assert torch.equal(a[other], b[other])
    assert y2[13, 300].isnan() and (q2.float() * s2.repeat_interleave(128, -1))[13, 256:384].isnan().all()
    assert row.float()[13].isnan().all() or bad == float("inf")
    assert torch.equal(h2[13, :300], h[13, :300]) and not h2[13, 300].isfinite()


def test_sum_is_normalised_before_it_is_rounded():
    """x and the residual cancel to a small rest that bf16 does not keep beside them in one
    type: the norm is that of the rest as float32 has it, and of nothing else."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = torch.randn(20, 512, generator=g, device="cuda") * 1e3
    x = (-r + torch.randn(20, 512, generator=g, device="cuda")).to(torch.bfloat16)
    w = torch.ones(512, device="cuda", dtype=torch.bfloat16)
    y, h = gdn.gdn_add_norm_fwd(x, r, w)
    rb = r.to(torch.bfloat16)
    y2, h2 = gdn.gdn_add_norm_fwd(x, rb, w)
    torch.cuda.synchronize()
    for got, kept, res in ((y, h, r), (y2, h2, rb)):
        ry, rh = block.add_norm_fwd(_np(x), _np(res), _np(w), 1e-6)
        _within("y", got, ry)
        _within("h", kept, rh, f=2.0 ** -23)


def test_without_eps():
    """eps = 0 is accepted; the places of a block without a row add nothing to the sums."""
    for rows, D in ((1, 64), (5, 768), (9, 4096)):
        x, r, w, dy, dh = _inputs(rows, D, "f32", "f32", False)
        y, h = gdn.gdn_add_norm_fwd(x, r, w, eps=0.0)
        dx, _, dw = gdn.gdn_add_norm_bwd(h, w, dy, dh, eps=0.0)
        torch.cuda.synchronize()
        _within("y", y, block.add_norm_fwd(_np(x), _np(r), _np(w), 0.0)[0])
        rd, rdw = block.add_norm_bwd(_np(h), _np(w), 0.0, _np(dy), _np(dh))
        sd, sdw = block.add_norm_bwd_sizes(_np(h), _np(w), 0.0, _np(dy), _np(dh))
        _within("dx", dx, rd, sd, 4 * F)
        _within("dw", dw, rdw, sdw, 4 * F)


def test_gradient_by_differences():
    """Central differences of the forward in float32: with a step of 2^-5 the third
    derivative's part is 2^-10 / 6 of numbers of order 1 (rows of a length of 8 and more:
    1e-4 of the gradient's size), a rounding of the loss 6e-8 * 64 terms / 2^-5 = 1e-4."""
    x, r, w, dy, dh = (t[:1] if t.dim() == 2 else t for t in _inputs(2, 64, "f32", "f32", False))
    d, _, dw = gdn.gdn_add_norm_bwd((x + r).contiguous(), w, dy, dh)
    e = 2.0 ** -5
    step = torch.eye(64, device="cuda") * e

    def loss(x, w):
        y, h = gdn.gdn_add_norm_fwd(x.contiguous(), r.expand(len(x), 64).contiguous(), w)
        return (y.double() * dy + h.double() * dh).sum(-1)

    by_x = (loss(x + step, w) - loss(x - step, w)) / (2 * e)
    by_w = torch.stack([(loss(x, w + s) - loss(x, w - s))[0] / (2 * e) for s in step])
    torch.cuda.synchronize()
    assert (by_x - d[0]).abs().max() < 3e-3 and (by_w - dw).abs().max() < 3e-3
    assert d.abs().max() > 0.3 and dw.abs().max() > 0.3


@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_residual_stream_in_place(dtype, stream):
    x, r, w, _, _ = _inputs(700, 768, dtype, stream, False)
    y, h = gdn.gdn_add_norm_fwd(x, r, w)
    q, s, _ = gdn.gdn_add_norm_quant(x, r, w, group=128)
    for call in (lambda k: gdn.gdn_add_norm_fwd(x, k, w, h=k)[0], lambda k: gdn.gdn_add_norm_quant(x, k, w, group=128, h=k)[0]):
        kept = r.clone()
        before = kept._version
        got = call(kept)
        torch.cuda.synchronize()
        assert torch.equal(kept, h) and kept._version > before
        assert torch.equal(got.view(torch.uint8), (y if got.dtype == y.dtype else q).view(torch.uint8))


def test_nothing_is_written_past_the_rows():
    for rows, D, dtype in ((5, 264, "bf16"), (3, 4100, "f32"), (9, 40, "bf16")):
        x, r, w, dy, dh = _inputs(rows, D, dtype, dtype, False)
        n = rows * D
        keep = {}

        def room(k, count, t, byte=0x5a):
            pad = 1024
            full = torch.full((count * t.itemsize + 2 * pad,), byte, dtype=torch.uint8, device="cuda")
            keep[k] = (full, pad, count * t.itemsize)
            return full[pad:pad + count * t.itemsize].view(t)

        dt = x.dtype
        gdn.gdn_add_norm_fwd(x, r, w, y=room("y", n, dt).view(rows, D), h=room("h", n, dt).view(rows, D))
        gdn.gdn_add_norm_bwd(x + r, w, dy, dh, grads=(room("dx", n, dt).view(rows, D), None, room("dw", D, dt)))
        gdn.gdn_add_norm_quant(x, r, w, y=room("q", n, torch.float8_e4m3fn).view(rows, D),
                               scales=room("s", rows, torch.float32).view(rows, 1))
        torch.cuda.synchronize()
        for k, (full, pad, count) in keep.items():
            assert (full[:pad] == 0x5a).all() and (full[pad + count:] == 0x5a).all(), k


def test_no_rows_and_shapes():
    w = torch.ones(64, device="cuda")
    x = torch.zeros(2, 0, 64, device="cuda")
    y, h = gdn.gdn_add_norm_fwd(x, x, w)
    dx, _, dw = gdn.gdn_add_norm_bwd(x, w, x, x)
    q, s, _ = gdn.gdn_add_norm_quant(x, x, w, group=32)
    assert y.shape == h.shape == dx.shape == x.shape and s.shape == (2, 0, 2) and not dw.any()
    x = torch.randn(3, 2, 5, 64, device="cuda")
    y, h = gdn.gdn_add_norm_fwd(x, x, w)
    flat, _ = gdn.gdn_add_norm_fwd(x.view(-1, 64), x.view(-1, 64), w)
    one, _ = gdn.gdn_add_norm_fwd(x[0, 0, 0], None, w)
    q, s, _ = gdn.gdn_add_norm_quant(x, x, w, group=64)
    torch.cuda.synchronize()
    assert torch.equal(y.view(-1, 64), flat) and one.shape == (64,) and s.shape == (3, 2, 5, 1)
    ry, _ = block.add_norm_fwd(_np(x[0, 0, 0]), None, _np(w), 1e-6)
    _within("y", one, ry)


def test_rows_that_are_not_a_stride_apart_are_refused():
    x = torch.randn(3, 4, 5, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (x[:, :2], x.transpose(0, 1), x[..., ::2], x.expand(3, 4, 5, 64)[:, :, :1].expand(3, 4, 5, 64)):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_add_norm_fwd(bad, None, w[:bad.shape[-1]])
    ok = x[:, :, 2]  # every fifth row
    y, _ = gdn.gdn_add_norm_fwd(ok, None, w)
    ref, _ = gdn.gdn_add_norm_fwd(ok.contiguous(), None, w)
    torch.cuda.synchronize()
    assert torch.equal(y, ref)


def test_other_stream_and_graph():
    x, r, w, dy, dh = _inputs(900, 768, "bf16", "bf16", True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def run(**kw):
        y, h = gdn.gdn_add_norm_fwd(x, r, w, **kw)
        q, s, _ = gdn.gdn_add_norm_quant(x, r, w, group=128, **kw)
        dx, _, dw = gdn.gdn_add_norm_bwd(h, w, dy, dh, **kw)
        return y, h, q.view(torch.uint8), s, dx, dw

    got = run(stream=side)
    ref = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = run()
    x.copy_(x.flip(0))
    graph.replay()
    now = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert all(torch.equal(a, b) for a, b in zip(caught, now))
    assert not torch.equal(caught[0], ref[0])


def test_more_than_2_31_elements():
    rows, D = 270001, 8192  # 4.4 GB a tensor in bf16
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").fill_(0.25)
    x[-1] = torch.linspace(-3, 3, D, device="cuda")
    w = torch.full((D,), 0.5, dtype=torch.bfloat16, device="cuda")
    y, h = gdn.gdn_add_norm_fwd(x, x, w)
    dx, _, dw = gdn.gdn_add_norm_bwd(h, w, x)
    q, s, _ = gdn.gdn_add_norm_quant(x, x, w, group=128)
    torch.cuda.synchronize()
    last = slice(rows - 2, rows)
    _within("y", y[last], block.add_norm_fwd(_np(x[last]), _np(x[last]), _np(w), 1e-6)[0])
    rd, _ = block.add_norm_bwd(_np(h[last]), _np(w), 1e-6, _np(x[last]))
    sd, _ = block.add_norm_bwd_sizes(_np(h[last]), _np(w), 1e-6, _np(x[last]))
    _within("dx", dx[last], rd, sd, 4 * F)
    small, ss, _ = gdn.gdn_add_norm_quant(x[last], x[last], w, group=128)
    assert torch.equal(q[last].view(torch.uint8), small.view(torch.uint8)) and torch.equal(s[last], ss)
    assert (y[:-1] == y[0, 0]).all() and (dx[:-1] == dx[0, 0]).all()


def test_refusals():
    x, r, w, dy, dh = _inputs(20, 512, "bf16", "bf16", False)
    bad = [dict(x=x.half()), dict(x=x.cpu()), dict(x=None), dict(residual=r[:5]), dict(residual=r.half()), dict(weight=w[:8]),
           dict(weight=w.float()), dict(weight=None), dict(eps=-1.0), dict(h=x), dict(y=r), dict(h=r[:5]), dict(h=r.float()),
           dict(x=x.float(), weight=w.float()), dict(x=x[:, :500], residual=r[:, :500], weight=w[:500]),
           dict(residual=None, h=torch.empty_like(x)), dict(x=x[0, 0], residual=None)]
    for over in bad:
        with pytest.raises(gdn.GdnError):
            gdn.gdn_add_norm_fwd(**{**dict(x=x, residual=r, weight=w), **over})
    for over in bad[:10] + [dict(group=48), dict(group=-1), dict(group=1 << 20), dict(y=torch.empty_like(x)),
                            dict(scales=torch.empty(20, 4, device="cuda"))]:
        with pytest.raises(gdn.GdnError):
            gdn.gdn_add_norm_quant(**{**dict(x=x, residual=r, weight=w), **over})
    ok = dict(h=r, weight=w, dy=dy, dh=dh)
    for over in (dict(h=r[:5]), dict(dy=None), dict(dy=dy.float()), dict(dh=dh.float()), dict(dh=dh[:, :8]), dict(weight=None),
                 dict(dy=_inputs(20, 512, "bf16", "bf16", True)[0]), dict(h=r.half()), dict(grads=(r, None, None)),
                 dict(grads=(None, torch.empty_like(r), None))):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_add_norm_bwd(**{**ok, **over})
    many = torch.zeros(3000, 512, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(gdn.GdnError, match="workspace"):
        gdn.gdn_add_norm_bwd(many, w, many, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        gdn.gdn_add_norm_fwd(1, r, w)
    gdn.gdn_add_norm_bwd(**ok)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,D,dtype,stream,group,ones", [
    (1700, 2304, "bf16", "bf16", 128, False), (1700, 1152, "f32", "f32", 32, False), (1601, 1280, "bf16", "f32", 128, True),
    (803, 3000, "bf16", "bf16", 0, False), (1000, 2560, "f32", "f32", 0, True), (931, 5120, "bf16", "bf16", 128, True),
    (1403, 1032, "bf16", "f32", 0, False), (400, 2052, "f32", "f32", 0, False)])
def test_rows_of_three_or_five_warps(rows, D, dtype, stream, group, ones):
    """Rows that neither one, two, four nor more powers of two of warps hold well, some turns a
    block: 8-bit numbers to the last one, also where exact ties are frequent (a weight of ones),
    and the norm without a residual."""
    x, r, w, _, _ = _inputs(rows, D, dtype, stream, True, seed=4)
    if ones:
        w = torch.ones_like(w)
    y, s, h = gdn.gdn_add_norm_quant(x, r, w, eps=EPS, group=group)
    plain, _ = gdn.gdn_add_norm_fwd(x, None, w, eps=EPS)
    torch.cuda.synchronize()
    rh = _np(x) + _np(r)
    _within("h", h, rh, f=2.0 ** -23)
    ry, _ = block.add_norm_fwd(_np(x), _np(r), _np(w), EPS)
    _within("scales", s, block.quantise(ry, group)[1])
    t = (rh * _np(w)).reshape(rows, -1, group or D)
    exact = t * 448.0 / np.abs(t).max(-1, keepdims=True)
    want, got = block.e4m3(exact), _np(y.float()).reshape(t.shape)
    wrong = want != got
    middle = (want + got) / 2
    # bf16: the largest t is rounded to float32, by up to 2^-24 (and 2^-53 of float64's own)
    near = np.where(np.abs(exact) < 2.0 ** -6, 2.0 ** -20, 1.01 * 2.0 ** -24 if stream == "bf16" else 0.0)
    assert (np.abs(exact - middle) <= near * np.abs(middle))[wrong].all()
    _within("y", plain, block.add_norm_fwd(_np(x), None, _np(w), EPS)[0])
