"""GPU tests of the gradients' global norm and clipping (gdn_grad_norm, gdn_clip_grads) against
float64.

Tolerances.  The norm: a thread's 32 squares of a tile are added in float32, 16 after one
another in each of two halves (17 roundings of 2^-24 each, all of one sign at worst: 1e-6,
half of it after the root; the exact order of the rest is in 64 bits): 6e-7 with its own
rounding.  A clipped value: the factor carries the norm's error and two roundings, its product
one more: 6e-7 + 3 * 6e-8 = 8e-7, and a rounding to its type, half a step u (bf16 2^-8,
float32 in the above)."""
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NORM = 6e-7
OFF = {torch.float32: 8e-7, torch.bfloat16: 2.0 ** -8 + 8e-7}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _np(t):
    return t.detach().double().cpu().numpy()


def _tensors(shapes, dtypes, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * std).to(DT[t]) for s, t in zip(shapes, dtypes)]


def _expect(grads, max_norm, norm, outs):
    ref, clipped = block.clip([_np(g) for g in grads], max_norm)
    assert abs(float(norm) - ref) <= NORM * ref, (float(norm), ref)
    for i, (o, r) in enumerate(zip(outs, clipped)):
        x = _np(o)
        assert x.shape == r.shape
        assert (np.abs(x - r) <= OFF[o.dtype] * np.abs(r) + 2.0 ** -140).all(), f"output {i}"


LISTS = {
    "one": ([(1,)], "f"),
    "odd": ([(3,), (7, 11), (1,), (8191,), (8193,), (5,)], "bfbfbf"),
    "tiles": ([(8192,), (16384,), (8200,), (100001,)], "bbff"),
    "layer": ([(512, 64), (64, 128), (32,), (32,), (32,), (64,)], "bbbbbb"),
    "empty": ([(0,), (5,), (0, 3), (0,), (70000,), (0,)], "bffbbf"),
    "many": ([(1 + 37 * i % 301,) for i in range(64)] + [(40000,)], "bf" * 32 + "b"),
    "cluster": ([(250000,), (300, 1000), (500000,), (1 << 19,)], "bfbf"),
    "past the cluster": ([(250000,), (300, 1000), (500000,), (1 << 19,), (8192,)], "bfbfb"),
    "thousands": ([(1 + 7 * i % 13,) for i in range(2500)] + [(9000, 3)], "fb" * 1250 + "f"),
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("factor", [0.3, 1.7])
def test_clip(name, factor):
    shapes, kinds = LISTS[name]
    types = ["bf16" if k == "b" else "f32" for k in kinds]
    grads = _tensors(shapes, types, seed=len(shapes))
    most = factor * math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    before = [g.clone() for g in grads]
    norm = gdn.gdn_grad_norm(grads)
    ref_norm = norm.clone()
    for turn in range(2):  # in place, and into outputs of the other type
        g = [b.clone() for b in before]
        if turn == 0:
            outs, n = g, gdn.gdn_clip_grads(g, most)
        else:
            outs = [torch.full(b.shape, float("nan"), device="cuda", dtype=DT["f32" if t == "bf16" else "bf16"]) for b, t in zip(before, types)]
            n = gdn.gdn_clip_grads(g, most, out=outs)
            assert all(torch.equal(a, b) for a, b in zip(g, before))
        torch.cuda.synchronize()
        assert torch.equal(n, ref_norm) and n.shape == () and n.dtype == torch.float32
        _expect(before, most, n, outs)
        if factor > 1 and turn == 0:
            assert all(torch.equal(a, b) for a, b in zip(outs, before))


def test_same_call_same_bits_and_generators():
    grads = _tensors([(1000, 1001), (77,)], ["bf16", "f32"])
    a = gdn.gdn_grad_norm(grads)
    b = gdn.gdn_grad_norm(g for g in grads)
    c = gdn.gdn_grad_norm((None, grads[0], None, grads[1]))
    o = [torch.empty_like(g) for g in grads]
    d = gdn.gdn_clip_grads([None, *grads], 1.0, out=[None, *o])
    gdn.gdn_clip_grads(tuple(grads), 1.0)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
    assert all(torch.equal(x, y) for x, y in zip(grads, o))
    # the same tensor twice has twice the squares
    twice = gdn.gdn_grad_norm([grads[0], grads[0]])
    one = gdn.gdn_grad_norm([grads[0]])
    assert abs(float(twice) / float(one) - math.sqrt(2)) < 1e-6


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("first,behind", [(0, 0), (1, 0), (0, 1), (3, 3), (2, 5), (5, 2), (4, 8), (7, 7), (0, 3), (6, 1), (1, 6), (4, 5), (0, 6), (7, 0)])
def test_parts_of_one_buffer(dtype, out, first, behind):
    """Tensors that begin anywhere in a buffer, outputs anywhere in another; what lies between
    stays."""
    sizes = [1, 9000, 6, 8192, 33, 20000, 8191, 16390, 0, 24571]
    flat, = _tensors([(sum(sizes) + 64,)], [dtype], seed=first)
    to = torch.full((sum(sizes) + 64,), 7.0, device="cuda", dtype=DT[out])
    grads, outs, at = [], [], 0
    for n in sizes:
        grads.append(flat[first + at:first + at + n])
        outs.append(to[behind + at:behind + at + n])
        at += n + 3
    norm = gdn.gdn_clip_grads(grads, 2.0, out=outs)
    torch.cuda.synchronize()
    _expect(grads, 2.0, norm, outs)
    used = torch.zeros(to.shape, dtype=torch.bool, device="cuda")
    at = 0
    for n in sizes:
        used[behind + at:behind + at + n] = True
        at += n + 3
    assert (to[~used] == 7.0).all()
    keep = flat.clone()
    norm2 = gdn.gdn_clip_grads(grads, 2.0)
    torch.cuda.synchronize()
    assert torch.equal(norm, norm2)
    at, mine = 0, torch.zeros(flat.shape, dtype=torch.bool, device="cuda")
    for n in sizes:
        mine[first + at:first + at + n] = True
        at += n + 3
    assert torch.equal(flat[~mine], keep[~mine]) and not torch.equal(flat[mine], keep[mine])


def test_any_order_of_dimensions():
    a, = _tensors([(30, 40, 50)], ["f32"])
    p = a.permute(2, 0, 1)
    o = torch.empty_like(p)
    assert o.stride() == p.stride()
    n = gdn.gdn_clip_grads([p], 1.0, out=[o])
    torch.cuda.synchronize()
    _expect([p], 1.0, n, [o])
    for g, to in ((a[:, ::2], None), (a.expand(2, 30, 40, 50), None), (p, torch.empty(p.shape, device="cuda"))):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_clip_grads([g], 1.0, out=None if to is None else [to])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-22, 1e-19, 1e18, 1e20, 1e30, 1e36])
def test_sizes_whose_squares_leave_float32(dtype, size):
    grads = _tensors([(5000,), (17,), (9000,)], [dtype, "f32", dtype], std=1.0)
    grads = [(g.double() * size).to(g.dtype) for g in grads]
    most = 0.25 * size
    outs = [torch.empty_like(g) for g in grads]
    norm = gdn.gdn_clip_grads(grads, most, out=outs)
    torch.cuda.synchronize()
    ref, clipped = block.clip([_np(g) for g in grads], float(np.float32(most)))
    assert abs(float(norm) - ref) <= NORM * ref + 2.0 ** -149
    for o, r in zip(outs, clipped):
        assert (np.abs(_np(o) - r) <= OFF[o.dtype] * np.abs(r) + 2.0 ** -133).all()  # a subnormal's half step in bf16: 2^-134


def test_one_large_number_among_small_ones():
    g, = _tensors([(100000,)], ["f32"], std=1e-3)
    for x in (3e38, 1e-3, 2.0 ** -80):
        g[77777] = x
        n = gdn.gdn_grad_norm([g])
        torch.cuda.synchronize()
        ref = math.sqrt(float(g.double().square().sum()))
        assert abs(float(n) - ref) <= NORM * ref
    z = torch.zeros(50000, device="cuda")
    z[40000] = 2.0 ** -80
    assert float(gdn.gdn_grad_norm([z])) == 2.0 ** -80
    z[3] = 2.0 ** -149
    assert float(gdn.gdn_grad_norm([z])) == 2.0 ** -80
    z.zero_()
    assert float(gdn.gdn_clip_grads([z], 0.0)) == 0.0 and not z.any()


def test_norm_past_float32_still_clips():
    g = torch.full((9000,), 3e38, device="cuda")
    n = gdn.gdn_clip_grads([g], 1.0)
    torch.cuda.synchronize()
    assert float(n) == math.inf
    assert (g - 1 / math.sqrt(9000)).abs().max() < 1e-7


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norm_that_is_not_finite_leaves_the_gradients(bad):
    grads = _tensors([(9000,), (100,)], ["bf16", "f32"])
    grads[1][50] = bad
    before = [g.clone() for g in grads]
    outs = [torch.empty(g.shape, device="cuda") for g in grads]
    n = gdn.gdn_clip_grads(grads, 1e-3, out=outs)
    m = gdn.gdn_clip_grads(grads, 1e-3)
    torch.cuda.synchronize()
    assert float(n) == math.inf if math.isinf(bad) else math.isnan(float(n))
    assert torch.equal(n.view(torch.int32), m.view(torch.int32))
    assert all(torch.equal(a.nan_to_num(nan=9.0), b.nan_to_num(nan=9.0)) for a, b in zip(grads, before))
    assert all(torch.equal(a.nan_to_num(nan=9.0), b.float().nan_to_num(nan=9.0)) for a, b in zip(outs, before))


def test_limits():
    g, = _tensors([(1000,)], ["f32"])
    before = g.clone()
    gdn.gdn_clip_grads([g], math.inf)
    assert torch.equal(g, before)
    gdn.gdn_clip_grads([g], 1e39)  # an infinite float32
    assert torch.equal(g, before)
    exact = torch.tensor([3.0, 4.0], device="cuda")
    assert float(gdn.gdn_clip_grads([exact], 5.0)) == 5.0 and exact.tolist() == [3.0, 4.0]
    gdn.gdn_clip_grads([g], 0.0)
    assert not g.any()


def test_no_gradients():
    n = torch.full((), 9.0, device="cuda")
    assert gdn.gdn_grad_norm([], norm=n) is not None and float(n) == 0.0
    e = torch.empty(0, device="cuda")
    assert float(gdn.gdn_grad_norm([e])) == 0.0 and float(gdn.gdn_clip_grads([e, None], 1.0)) == 0.0
    for empty in ([], [None]):
        with pytest.raises(gdn.GdnError, match="no gradients"):
            gdn.gdn_grad_norm(empty)


def test_more_than_2_31_elements():
    g = torch.zeros(2 ** 31 + 12345, dtype=torch.bfloat16, device="cuda")
    g[-1], g[5], g[2 ** 31 + 3] = 3.0, 4.0, 12.0
    n = gdn.gdn_clip_grads([g], 6.5)
    torch.cuda.synchronize()
    assert float(n) == 13.0 and g[[-1, 5, 2 ** 31 + 3]].tolist() == [1.5, 2.0, 6.0] and int(g.count_nonzero()) == 3


def test_streams_and_graphs():
    """Calls side by side each have memory of their own; a captured call reads the gradients
    of its replay."""
    a, b = _tensors([(300000,), (300,)], ["f32", "f32"]), _tensors([(700000,), (1,)], ["bf16", "bf16"], seed=1)
    want = [float(gdn.gdn_grad_norm(x)) for x in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norms = []
    for _ in range(20):
        norms += [gdn.gdn_grad_norm(a), gdn.gdn_grad_norm(b, stream=side)]
    torch.cuda.synchronize()
    assert [float(n) for n in norms] == want * 20
    graphs, caught = [], []
    for x in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            caught.append(gdn.gdn_clip_grads(x, 1.0))
        graphs.append(gr)
    keep = [[t.clone() for t in x] for x in (a, b)]
    for turn in range(2):
        for x, k in zip((a, b), keep):
            for t, s in zip(x, k):
                t.copy_(s * (turn + 1))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for x, k, n, w in zip((a, b), keep, caught, want):
            assert abs(float(n) / (w * (turn + 1)) - 1) < 1e-6
            _expect([s * (turn + 1) for s in k], 1.0, n, x)


def test_written_gradients_count_as_changed():
    x = torch.randn(100, device="cuda", requires_grad=True)
    y = x * 2
    loss = (y * y).sum()
    with torch.no_grad():
        gdn.gdn_clip_grads([y], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    g = torch.randn(100, device="cuda")
    o = torch.empty_like(g)
    gdn.gdn_clip_grads([g], 1.0, out=[o])
    gdn.gdn_grad_norm([g])
    assert g._version == 0 and o._version > 0
    with pytest.raises(gdn.GdnError):
        gdn.gdn_clip_grads([g], -1.0)
    assert g._version == 0
    torch.cuda.synchronize()


def test_refusals():
    g, h = _tensors([(100,), (50,)], ["f32", "bf16"])
    for call in (lambda: gdn.gdn_clip_grads([g, g], 1.0), lambda: gdn.gdn_clip_grads([g, g[10:]], 1.0),
                 lambda: gdn.gdn_clip_grads([g, h], 1.0, out=[h.float(), g[:50]]), lambda: gdn.gdn_clip_grads([g], 1.0, out=[g[:50]]),
                 lambda: gdn.gdn_clip_grads([g], 1.0, out=[]), lambda: gdn.gdn_clip_grads([g], 1.0, out=[None]),
                 lambda: gdn.gdn_clip_grads([g], 1.0, out=[g.half()]), lambda: gdn.gdn_clip_grads([g.half()], 1.0),
                 lambda: gdn.gdn_clip_grads([g.cpu()], 1.0), lambda: gdn.gdn_clip_grads([g.double()], 1.0), lambda: gdn.gdn_clip_grads(g, 1.0),
                 lambda: gdn.gdn_clip_grads([g], 1.0, out=g), lambda: gdn.gdn_clip_grads([g], float("nan")), lambda: gdn.gdn_grad_norm(g),
                 lambda: gdn.gdn_grad_norm([g], norm=torch.empty(2, device="cuda")), lambda: gdn.gdn_grad_norm([g], norm=torch.empty(1)),
                 lambda: gdn.gdn_grad_norm([g], norm=h[:1]), lambda: gdn.gdn_grad_norm([g], norm=g[5]),
                 lambda: gdn.gdn_grad_norm([torch.zeros(1 << 21, device="cuda")], workspace=torch.empty(8, device="cuda")),
                 lambda: gdn.gdn_grad_norm([g.to_sparse()]), lambda: gdn.gdn_grad_norm([g, g.cpu()])):
        with pytest.raises(gdn.GdnError):
            call()
    for call in (lambda: gdn.gdn_grad_norm(3), lambda: gdn.gdn_grad_norm([g, 3]), lambda: gdn.gdn_clip_grads([g], "a"),
                 lambda: gdn.gdn_clip_grads([g], None)):
        with pytest.raises(TypeError):
            call()
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    out = torch.empty(1, device="cuda")
    assert gdn.gdn_grad_norm([g], norm=out, workspace=ws).data_ptr() == out.data_ptr()
    torch.cuda.synchronize()
    assert abs(float(out) - float(g.double().norm())) < 1e-5
