"""GPU tests of the calls that are one cluster where they are small (the backward of the residual
norm and of the rotation by axes, the gradients' norm and clipping): every largest cluster, down
to the two launches; lists of tiles at the bound between the two; another stream, a captured
and replayed call, two at once."""
import ctypes
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # a rounding to the type
# the norm and a clipped value, as derived for the gradients' other tests: ten roundings of
# 2^-24 in a thread's 32 squares, halved by the root, and three more
NORM, CLIPPED = 6e-7, 8e-7


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture
def limit():
    yield gdn.gdn_test_set_cluster_limit
    gdn.gdn_test_set_cluster_limit(0)


def _randn(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _norm_inputs(rows, D, dtype, stream):
    a, b = DT[dtype], DT[stream]
    return _randn(rows, D, seed=1, dtype=b), (1 + 0.1 * _randn(D, seed=2)).to(a), _randn(rows, D, seed=3, dtype=a), _randn(rows, D, seed=4, dtype=b)


def _axes_inputs(B, T, H, Hk, D, dtype):
    a = DT[dtype]
    ang = torch.rand(64, D // 2, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)) * 6
    pos = torch.randint(0, 64, (3, B, T), device="cuda", dtype=torch.int32, generator=torch.Generator(device="cuda").manual_seed(8))
    n = D // 2
    return (_randn(B, T, H, D, seed=1, dtype=a), _randn(B, T, Hk, D, seed=2, dtype=a), (1 + 0.1 * _randn(D, seed=3)).to(a),
            (1 + 0.1 * _randn(D, seed=4)).to(a), ang.cos(), ang.sin(), pos, (n - 2 * (n // 3), n // 3, n // 3),
            _randn(B, T, H, D, seed=5, dtype=a), _randn(B, T, Hk, D, seed=6, dtype=a))


@pytest.mark.parametrize("dtype,stream,D", [("bf16", "bf16", 512), ("bf16", "f32", 1000), ("f32", "f32", 4096), ("bf16", "f32", 8192)])
def test_norm_backward_in_every_cluster(limit, dtype, stream, D):
    """The same bits whatever the cluster: up to 16 blocks' sums for the weight are added in their
    order in either form.  Against float64, relative to the sum of the terms' sizes: two roundings a
    row, and those of the row's norm (up to 64 squares a lane and its exchanges, halved by the root)."""
    for rows in (1, 7, 16):
        args = _norm_inputs(rows, D, dtype, stream)
        ref = None
        for most in (0, 16, 8, 4, 2, 1):
            limit(most)
            grads = gdn.gdn_add_norm_bwd(*args)
            torch.cuda.synchronize()
            ref = ref or grads
            for a, b in zip(grads, ref):
                assert torch.equal(a, b), (rows, most)
        h, w, dy, dh = (t.double() for t in args)
        r = (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        terms = dy * h * r
        off = (ref[2].double() - terms.sum(0)).abs()
        assert (off <= (2 * rows + 64) * 2.0 ** -24 * terms.abs().sum(0) + HALF[DT[dtype]] * terms.sum(0).abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_axes_backward_in_every_cluster(limit, dtype):
    for B, T, H, Hk in ((1, 1, 2, 1), (3, 5, 4, 2), (1, 16, 16, 16), (2, 31, 4, 1)):
        args = _axes_inputs(B, T, H, Hk, 128, dtype)
        ref = None
        for most in (0, 16, 8, 4, 2, 1):
            limit(most)
            grads = gdn.gdn_qk_norm_rope_axes_bwd(*args)
            torch.cuda.synchronize()
            ref = ref or grads
            for a, b in zip(grads, ref):
                assert torch.equal(a, b), (B, T, H, most)


def _bytes(grads, outs=None):
    lib = gdn.load_library()
    code = {torch.float32: 0, torch.bfloat16: 1}
    rows = (gdn.gdn_grad * len(grads))(*[gdn.gdn_grad(g.data_ptr(), (o if outs else g).data_ptr(), g.numel(), code[g.dtype],
                                                      code[(o if outs else g).dtype]) for g, o in zip(grads, outs or grads)])
    return lib.gdn_grad_workspace_bytes(rows, len(grads))


def _check(before, most, norm, outs):
    ref, clipped = block.clip([g.double().cpu().numpy() for g in before], most)
    assert abs(float(norm) - ref) <= NORM * ref
    for o, r in zip(outs, clipped):
        x = o.double().cpu().numpy()
        assert (np.abs(x - r) <= (CLIPPED + (HALF[torch.bfloat16] if o.dtype == torch.bfloat16 else 0)) * np.abs(r) + 2.0 ** -133).all()


TILE = 8192
BOUND = {
    "48 tiles": ([48 * TILE], True), "48 tiles in four": ([TILE, 30 * TILE, 16 * TILE, TILE], True), "49 tiles": ([48 * TILE, 1], False),
    "49 tiles in one": ([48 * TILE + 1], False), "120 tensors": ([3000] * 48 + [0] * 72, True), "121 tensors": ([3000] * 48 + [0] * 73, False),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", BOUND)
def test_gradients_at_the_bound_of_one_cluster(name, dtype):
    sizes, one = BOUND[name]
    grads = [_randn(n, seed=i, dtype=DT[dtype]) for i, n in enumerate(sizes)]
    assert (_bytes(grads) == 0) == one
    most = 0.5 * math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    before = [g.clone() for g in grads]
    outs = [torch.full(g.shape, float("nan"), device="cuda", dtype=DT["f32" if dtype == "bf16" else "bf16"]) for g in grads]
    a = gdn.gdn_grad_norm(grads)
    b = gdn.gdn_clip_grads(grads, most, out=outs)
    c = gdn.gdn_clip_grads(grads, most)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    _check(before, most, a, outs)
    _check(before, most, a, grads)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tiles_that_begin_before_their_tensors(limit, dtype):
    """48 tensors of a tile each that begin behind a 16-byte boundary: two tiles each, more than the
    cluster's workers, so that some take several."""
    flat = _randn(48 * (TILE + 16) + 8, seed=3, dtype=DT[dtype])
    to = torch.full((flat.numel() + 3,), 7.0, device="cuda", dtype=DT[dtype])
    at = [i * (TILE + 16) + 1 + i % 3 for i in range(48)]
    before = [flat[a:a + TILE].clone() for a in at]
    keep = flat.clone()
    inside = torch.zeros(flat.shape, dtype=torch.bool, device="cuda")
    for a in at:
        inside[a:a + TILE] = True
    most = 0.4 * math.sqrt(sum(float(g.double().square().sum()) for g in before))
    for blocks in (0, 1):
        limit(blocks)
        flat.copy_(keep)
        to.fill_(7.0)
        grads, outs = [flat[a:a + TILE] for a in at], [to[a + 2:a + 2 + TILE] for a in at]
        assert (_bytes(grads) == 0) == (blocks == 0)
        n = gdn.gdn_clip_grads(grads, most, out=outs)
        m = gdn.gdn_clip_grads(grads, most)
        torch.cuda.synchronize()
        assert torch.equal(n, m)
        _check(before, most, n, outs)
        _check(before, most, n, grads)
        assert torch.equal(flat[~inside], keep[~inside]) and (to[2:-1][~inside] == 7.0).all() and (to[:2] == 7.0).all()


def test_gradients_in_every_cluster(limit):
    for sizes in ([1], [5, 9000], [40000, 3, 100001], [47 * TILE]):
        grads = [_randn(n, seed=n, dtype=torch.bfloat16 if i % 2 else torch.float32) for i, n in enumerate(sizes)]
        before = [g.clone() for g in grads]
        for most in (0, 16, 8, 4, 2, 1):
            limit(most)
            for g, b in zip(grads, before):
                g.copy_(b)
            outs = [torch.full_like(g, float("nan")) for g in grads]
            a, b, c = gdn.gdn_grad_norm(grads), gdn.gdn_clip_grads(grads, 0.25, out=outs), gdn.gdn_clip_grads(grads, 0.25)
            torch.cuda.synchronize()
            assert torch.equal(a, b) and torch.equal(a, c)
            _check(before, 0.25, a, outs)
            _check(before, 0.25, a, grads)


def _small_calls():
    """Calls that are one cluster each: a backward of the norm, one of the rotation, a clipping, and
    a clipping in place of a copy that the call makes."""
    norm, axes = _norm_inputs(12, 1000, "bf16", "f32"), _axes_inputs(2, 9, 6, 2, 64, "bf16")
    g = [_randn(30000, seed=5), _randn(7777, seed=6, dtype=torch.bfloat16)]
    assert _bytes(g) == 0

    def clip(stream=None):
        outs = [torch.full_like(x, float("nan")) for x in g]
        return (gdn.gdn_clip_grads(g, 1.0, out=outs, stream=stream), *outs)

    calls = [lambda stream=None: gdn.gdn_add_norm_bwd(*norm, stream=stream),
             lambda stream=None: gdn.gdn_qk_norm_rope_axes_bwd(*axes, stream=stream), clip]
    return calls, (*norm, *axes[:2], *axes[-2:], *g)


def test_small_calls_on_another_stream():
    calls, _ = _small_calls()
    want = [c() for c in calls]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):  # on two streams at once, by the argument and by the current one
        for i, c in enumerate(calls):
            with torch.cuda.stream(side[0]):
                got.append((i, c()))
            if i < 2:
                got.append((i, c(stream=side[1])))
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[i])), i


def test_small_calls_in_a_graph():
    """Two graphs that share a memory pool, replayed in turn with inputs that change."""
    calls, inputs = _small_calls()
    for c in calls:
        c()
    torch.cuda.synchronize()
    pool, graphs, caught = None, [], []
    for order in (calls, calls[::-1]):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, pool=pool):
            caught.append([c() for c in order])
        pool = gr.pool()
        graphs.append(gr)
    keep = [t.clone() for t in inputs]
    for turn in (1, 2):
        for t, k in zip(inputs, keep):
            t.copy_(k * turn)
        want = [c() for c in calls]
        for gr, got, ref in zip(graphs, caught, (want, want[::-1])):
            gr.replay()
            torch.cuda.synchronize()
            for g, r in zip(got, ref):
                assert all(torch.equal(a, b) for a, b in zip(g, r)), turn


def test_more_than_a_thousand_tensors_in_a_graph():
    grads = [_randn(1 + 37 * i % 301, seed=i, dtype=torch.bfloat16 if i % 3 else torch.float32) for i in range(2345)]
    grads.append(_randn(300001, seed=1))
    keep = [g.clone() for g in grads]
    outs = [torch.empty_like(g) for g in grads]
    gdn.gdn_clip_grads(grads, 1.0, out=outs)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        into = gdn.gdn_clip_grads(grads, 1.0, out=outs)
        place = gdn.gdn_clip_grads(grads, 1.0)
    for turn in (1, 3):
        now = [k * turn for k in keep]
        for g, k, o in zip(grads, now, outs):
            g.copy_(k)
            o.fill_(float("nan"))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(into, place)
        _check(now, 1.0, into, outs)
        _check(now, 1.0, into, grads)


def test_what_the_context_places_is_what_the_queries_say():
    lib = gdn.load_library()
    for rows, few in ((128, True), (129, False)):  # 8 rows of 512 bf16 a block, 16 blocks: this GPU places them
        p = gdn.gdn_add_norm_problem(rows, 512, 0, 0, 1e-6, 1, 1)
        assert (lib.gdn_add_norm_bwd_workspace_bytes(ctypes.byref(p)) == 0) == few
