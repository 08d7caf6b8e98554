"""GPU tests of the q, k norm with a rotation by several positions
(gdn_qk_norm_rope_axes_fwd/bwd) against float64.

Tolerances, relative L2 over a tensor and, twice as wide, over each row: everything is computed
in float32, so float32 results are within 1e-5 (a few dozen roundings of 6e-8 each, sums of
256 terms or, for the weights' gradients, of all rows), and bf16 results carry one rounding, at
most 2^-8 of each element and so of any norm: 4e-3."""
import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import block, layer

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {torch.float32: 1e-5, torch.bfloat16: 4e-3}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _np(t):
    return t.double().cpu().numpy()


def _check(name, got, ref):
    tol = TOL[got.dtype]
    x, r = _np(got), np.asarray(ref)
    assert x.shape == r.shape and np.isfinite(x).all(), name
    err = np.linalg.norm(x - r) / max(np.linalg.norm(r), 1e-30)
    assert err <= tol, f"{name}: {err:.2e}"
    if x.ndim == 4:
        rows = np.linalg.norm(x - r, axis=-1) / np.maximum(np.linalg.norm(r, axis=-1), 1e-30)
        assert rows.size == 0 or rows.max() <= 2 * tol, f"{name}: a row {rows.max():.2e}"


CASES = [
    # B, T, Hq, Hk, D, R, dtype, interleaved, slices, sections, alternating
    (1, 1, 1, 1, 16, 16, "bf16", False, False, (8,), False),
    (1, 1, 6, 6, 128, 128, "bf16", False, False, (16, 24, 24), False),
    (2, 37, 6, 2, 128, 128, "bf16", False, True, (16, 24, 24), False),
    (2, 37, 6, 2, 128, 128, "bf16", True, True, (16, 24, 24), False),
    (2, 19, 5, 1, 128, 128, "bf16", False, False, (22, 21, 21), False),
    (2, 19, 5, 5, 128, 128, "bf16", True, False, (21, 22, 21), False),
    (1, 70, 4, 4, 128, 128, "bf16", False, False, (28, 18, 18), True),
    (1, 70, 4, 4, 128, 128, "bf16", True, True, (24, 20, 20), True),
    (3, 33, 3, 1, 96, 96, "f32", False, False, (12, 16, 20), False),
    (3, 33, 3, 1, 96, 96, "f32", True, True, (17, 15, 16), False),
    (1, 129, 4, 2, 96, 32, "f32", False, True, (6, 5, 5), True),
    (1, 40, 3, 3, 64, 64, "bf16", True, False, (0, 16, 16), False),
    (2, 21, 2, 2, 64, 32, "bf16", False, False, (4, 0, 4, 8), False),
    (2, 21, 2, 2, 64, 64, "f32", True, False, (8, 8, 8, 8), True),
    (2, 5, 16, 4, 256, 256, "bf16", False, False, (32, 48, 48), False),
    (1, 9, 2, 2, 256, 256, "f32", True, False, (43, 43, 42), True),
    (1, 9, 3, 1, 256, 128, "bf16", False, True, (1, 62, 1), False),
    (2, 11, 3, 2, 8, 8, "f32", False, False, (1, 1, 1, 1), True),
    (2, 11, 3, 2, 16, 8, "f32", True, False, (3, 1), False),
    (1, 2000, 6, 6, 128, 128, "bf16", False, True, (16, 24, 24), False),
    (2, 700, 7, 7, 128, 128, "f32", False, False, (23, 20, 21), False),
    (2, 50, 4, 3, 64, 0, "bf16", False, False, (0,), False),
    # as many rows as have their angles gathered in front
    (1, 3001, 6, 6, 128, 128, "bf16", False, True, (23, 20, 21), False),
    (2, 1111, 12, 4, 128, 128, "f32", True, False, (24, 20, 20), True),
    (3, 2749, 3, 1, 96, 32, "bf16", True, False, (5, 4, 3, 4), False),
    (1, 4100, 8, 8, 64, 64, "f32", False, True, (14, 9, 9), True),
    # a backward of one cluster, of 1, 2, 15 and 16 blocks, and one block more
    (1, 16, 1, 1, 128, 128, "bf16", False, False, (16, 24, 24), False),
    (1, 17, 1, 1, 128, 128, "f32", False, False, (16, 24, 24), False),
    (1, 240, 1, 1, 64, 64, "bf16", False, False, (8, 12, 12), False),
    (1, 64, 4, 4, 256, 256, "f32", False, False, (32, 48, 48), False),
    (1, 257, 1, 1, 128, 128, "bf16", False, False, (16, 24, 24), False),
]


def _inputs(B, T, Hq, Hk, D, R, dtype, slices, axes, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + D + T)
    dt = DT[dtype]

    def rows(H, std=1.0):
        if slices:
            return (torch.randn(B, T, 2 * H * D + 64, generator=g, device="cuda") * std).to(dt)[..., 64:64 + H * D].unflatten(-1, (H, D))
        return (torch.randn(B, T, H, D, generator=g, device="cuda") * std).to(dt)

    q, k = rows(Hq, 3.0), rows(Hk, 0.2)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2))
    n = T + 60
    a = torch.randn(n, R // 2, generator=g, device="cuda") * 3
    pos = torch.randint(0, n, (axes, B, T), generator=g, device="cuda", dtype=torch.int32)
    dq, dk = (torch.randn(B, T, H, D, generator=g, device="cuda").to(dt) for H in (Hq, Hk))
    return q, k, wq, wk, a.cos(), a.sin(), pos, dq, dk


@pytest.mark.parametrize("B,T,Hq,Hk,D,R,dtype,interleaved,slices,sections,alternating", CASES)
def test_axes(B, T, Hq, Hk, D, R, dtype, interleaved, slices, sections, alternating):
    q, k, wq, wk, cos, sin, pos, dqo, dko = _inputs(B, T, Hq, Hk, D, R, dtype, slices, len(sections))
    how = dict(eps=1e-5, interleaved=interleaved, alternating=alternating)
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda")  # noqa: E731
    args = (q, k, wq, wk, cos, sin, pos, sections)
    yq, yk = gdn.gdn_qk_norm_rope_axes_fwd(*args, **how, q_out=nan(q), k_out=nan(k))
    grads = gdn.gdn_qk_norm_rope_axes_bwd(*args, dqo, dko, **how, grads=(nan(q), nan(k), nan(wq), nan(wk)))
    again = gdn.gdn_qk_norm_rope_axes_bwd(*args, dqo, dko, **how)
    torch.cuda.synchronize()
    c, s = block.angles(_np(cos), _np(sin), pos.cpu().numpy(), sections, alternating) if R else (np.zeros((B, T, 0)),) * 2
    for name, y, x, w, dy, dx, dw in (("q", yq, q, wq, dqo, grads[0], grads[2]), ("k", yk, k, wk, dko, grads[1], grads[3])):
        _check(name, y, layer.norm_rope_fwd(_np(x), _np(w), c, s, 1e-5, interleaved))
        rx, rw = layer.norm_rope_bwd(_np(x), _np(w), c, s, 1e-5, interleaved, _np(dy))
        _check("d" + name, dx, rx)
        _check("dw" + name, dw, rw)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections,alternating", [((16, 24, 24), False), ((23, 20, 21), False), ((24, 20, 20), True), ((64,), False)])
@pytest.mark.parametrize("T", [7, 45, 1900])
def test_equal_positions_are_one(dtype, interleaved, sections, alternating, T):
    """Text among images has the same position on every axis: the call of one position, bit
    for bit."""
    q, k, wq, wk, cos, sin, pos, dqo, dko = _inputs(2, T, 6, 3, 128, 128, dtype, True, 1)
    many = pos.expand(len(sections), 2, T).contiguous()
    one = (q, k, wq, wk, cos, sin, pos[0])
    all_ = (q, k, wq, wk, cos, sin, many, sections)
    how = dict(interleaved=interleaved)
    ref = gdn.gdn_qk_norm_rope_fwd(*one, **how) + gdn.gdn_qk_norm_rope_bwd(*one, dqo, dko, **how)
    how["alternating"] = alternating
    got = gdn.gdn_qk_norm_rope_axes_fwd(*all_, **how) + gdn.gdn_qk_norm_rope_axes_bwd(*all_, dqo, dko, **how)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("sections,alternating", [((8, 4, 4), False), ((7, 5, 4), False), ((6, 5, 5), True)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [4, 4100])
def test_positions_outside_the_tables(interleaved, sections, alternating, T):
    """They show in their own axis's pairs of their own token."""
    q, k, wq, wk, cos, sin, pos, dqo, dko = _inputs(2, T, 3, 1, 64, 32, "bf16", False, 3)
    pos[0, 0, 1], pos[2, 1, 2], pos[1, 0, 3] = -1, cos.shape[0], -2 ** 31
    yq, yk = gdn.gdn_qk_norm_rope_axes_fwd(q, k, wq, wk, cos, sin, pos, sections, interleaved=interleaved, alternating=alternating)
    g = gdn.gdn_qk_norm_rope_axes_bwd(q, k, wq, wk, cos, sin, pos, sections, dqo, dko, interleaved=interleaved, alternating=alternating)
    torch.cuda.synchronize()
    axis = torch.from_numpy(block.axis_of_pair(sections, alternating))
    first, second = layer._pairs(32, interleaved)
    bad = torch.zeros(2, T, 64, dtype=torch.bool)
    for a, b, t in ((0, 0, 1), (2, 1, 2), (1, 0, 3)):
        on = (axis == a).nonzero().flatten().numpy()
        bad[b, t, first[on]] = bad[b, t, second[on]] = True
    for y in (yq, yk):
        assert torch.equal(y.isnan().cpu(), bad[:, :, None].expand(y.shape))
    assert torch.equal(g[0].isnan().all(-1).all(-1).cpu(), bad.any(-1)) and torch.equal(g[0].isnan().any(-1).any(-1).cpu(), bad.any(-1))


def test_no_tokens_other_stream_and_graph():
    w = torch.ones(64, device="cuda")
    e = torch.zeros(2, 0, 3, 64, device="cuda")
    t = torch.zeros(5, 32, device="cuda")
    p = torch.zeros(2, 2, 0, dtype=torch.int32, device="cuda")
    yq, _ = gdn.gdn_qk_norm_rope_axes_fwd(e, e, w, w, t, t, p, (16, 16))
    g = gdn.gdn_qk_norm_rope_axes_bwd(e, e, w, w, t, t, p, (16, 16), e, e)
    assert yq.shape == e.shape and not g[2].any() and not g[3].any()
    q, k, wq, wk, cos, sin, pos, dqo, dko = _inputs(1, 300, 6, 6, 128, 128, "bf16", True, 3)
    args = (q, k, wq, wk, cos, sin, pos, (16, 24, 24))
    run = lambda **kw: gdn.gdn_qk_norm_rope_axes_fwd(*args, **kw) + gdn.gdn_qk_norm_rope_axes_bwd(*args, dqo, dko, **kw)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, ref = run(stream=side), run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = run()
    pos.copy_(pos.flip(-1))
    graph.replay()
    now = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and all(torch.equal(a, b) for a, b in zip(caught, now))
    assert not torch.equal(caught[0], ref[0])


def test_refusals():
    q, k, wq, wk, cos, sin, pos, dqo, dko = _inputs(2, 20, 4, 2, 64, 32, "bf16", False, 3)
    ok = dict(q=q, k=k, q_weight=wq, k_weight=wk, cos=cos, sin=sin, positions=pos, sections=(6, 5, 5))
    bad = [dict(q=q.float()), dict(k=k[:, :5]), dict(q_weight=None), dict(k_weight=wk[:32]), dict(cos=None), dict(sin=sin[:5]),
           dict(positions=None), dict(positions=pos[0]), dict(positions=pos[:2]), dict(positions=pos.long()), dict(sections=(8, 8)),
           dict(sections=(6, 5, 4)), dict(sections=(6, 5, 6)), dict(sections=(18, -1, -1)), dict(sections=()),
           dict(sections=(4, 4, 4, 2, 2)), dict(sections=(1, 7, 8), alternating=True), dict(sections=(2 ** 40, 5, 5)), dict(eps=-1.0),
           dict(q_out=q), dict(positions=pos.transpose(1, 2).contiguous())]
    for over in bad:
        with pytest.raises(gdn.GdnError):
            gdn.gdn_qk_norm_rope_axes_fwd(**{**ok, **over})
        if "q_out" not in over:
            with pytest.raises(gdn.GdnError):
                gdn.gdn_qk_norm_rope_axes_bwd(**{**ok, **over}, dq_out=dqo, dk_out=dko)
    for s in (7, ("a", 1, 2), (6.5, 5, 4.5), (2 ** 70, 1, 1)):
        with pytest.raises((TypeError, OverflowError)):
            gdn.gdn_qk_norm_rope_axes_fwd(**{**ok, "sections": s})
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm_rope_axes_bwd(**ok, dq_out=dqo, dk_out=None)
    with pytest.raises(gdn.GdnError):
        many = dict(zip(("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "dq_out", "dk_out"),
                        _inputs(2, 500, 4, 2, 64, 32, "bf16", False, 3)))
        gdn.gdn_qk_norm_rope_axes_bwd(**many, sections=(6, 5, 5), workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    gdn.gdn_qk_norm_rope_axes_fwd(**ok)
    torch.cuda.synchronize()
