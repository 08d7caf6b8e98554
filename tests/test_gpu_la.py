"""GPU tests of linear attention with a decay per head (gdn_la_fwd, gdn_la_bwd,
gdn_la_decode) against the float64 token loop.

Tolerances, relative L2 over a tensor and, twice as wide, over every (b, 64-token
block, h) of it: float32 results 1e-5 (the sums run over at most a few thousand
products of 24-bit numbers; states of bf16 inputs keep 16 bits of every decayed
product).  bf16 results 5e-3: rounding to bf16 has an rms error of 2^-8 / sqrt(12) *
1.4 = 1.6e-3 per value, and an output goes through three of them (the scores or the
state that feed a product, and the result), so at most sqrt(3) * 1.6e-3 = 2.8e-3
together where they are independent."""
import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import layer

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {torch.float32: 1e-5, torch.bfloat16: 5e-3}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(name, got, ref):
    tol = TOL[got.dtype]
    x, r = _np(got), np.asarray(ref)
    assert x.shape == r.shape and np.isfinite(x).all(), name
    rel = lambda a, b: np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-30)  # noqa: E731
    assert rel(x, r) <= tol, f"{name}: {rel(x, r):.2e}"
    if "state" in name:
        blocks = [(i, x[i], r[i]) for i in np.ndindex(x.shape[:2])]
    else:
        blocks = [((b, t, h), x[b, t:t + 64, h], r[b, t:t + 64, h]) for b in range(x.shape[0])
                  for t in range(0, x.shape[1], 64) for h in range(x.shape[2])]
    for at, a, c in blocks:
        assert rel(a, c) <= 2 * tol, f"{name} {at}: {rel(a, c):.2e}"


def _inputs(B, T, H, K, V, dtype, decay, seed, fused=False, state=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = DT[dtype]
    if fused:  # slices of one projection's rows
        row = n(B, T, H * (2 * K + V) + 32)
        row[..., :H * K] *= K ** -0.5
        row = row.to(dt)
        q = row[..., :H * K].unflatten(-1, (H, K))
        k = row[..., H * K:2 * H * K].unflatten(-1, (H, K))
        v = row[..., 2 * H * K:H * (2 * K + V)].unflatten(-1, (H, V))
    else:
        q, k, v = (n(B, T, H, K) * K ** -0.5).to(dt), n(B, T, H, K).to(dt), n(B, T, H, V).to(dt)
    h = torch.arange(1, H + 1, device="cuda", dtype=torch.float32)
    ld = {"slopes": -torch.exp2(-8 * h / H), "slow": torch.log1p(-torch.exp2(-7 - 5 * h / H)), "none": h * 0,
          "strong": -3.0 * h, "inf": torch.full_like(h, float("-inf"))}[decay]
    s0 = n(B, H, V, K) * 0.5 if state else None
    return q, k, v, ld, s0, n(B, T, H, V).to(dt), (n(B, H, V, K) * 0.1 if state else None)


CASES = [
    # B, T, H, K, V, dtype, decay, fused, state
    (1, 1, 1, 16, 16, "f32", "slopes", False, True),
    (2, 1, 3, 128, 128, "bf16", "slopes", False, True),
    (1, 2, 2, 64, 128, "bf16", "none", True, False),
    (1, 63, 2, 128, 64, "bf16", "slow", False, True),
    (2, 64, 2, 32, 16, "bf16", "slopes", False, True),
    (1, 65, 3, 16, 128, "f32", "slopes", True, True),
    (1, 127, 1, 128, 128, "bf16", "strong", False, True),
    (3, 128, 2, 128, 128, "bf16", "slopes", True, False),
    (2, 129, 2, 64, 64, "f32", "strong", False, True),
    (1, 129, 5, 128, 128, "bf16", "slopes", False, True),
    (2, 300, 3, 128, 32, "bf16", "inf", False, True),
    (1, 300, 2, 32, 128, "f32", "inf", False, True),
    (2, 777, 4, 128, 128, "bf16", "slow", False, True),
    (1, 777, 4, 128, 128, "f32", "slow", False, True),
    (1, 1000, 16, 64, 64, "bf16", "none", True, True),
    (1, 2049, 1, 128, 128, "bf16", "slow", False, True),
    (1, 2049, 2, 16, 64, "f32", "none", False, False),
    (7, 200, 23, 32, 32, "bf16", "slopes", False, True),  # more streams than SMs
    (5, 150, 40, 16, 16, "f32", "slopes", False, True),
    (1, 1100, 160, 128, 16, "bf16", "slopes", False, True),  # nine tiles a segment
    (1, 1100, 160, 16, 128, "bf16", "slow", True, True),
]


@pytest.mark.parametrize("B,T,H,K,V,dtype,decay,fused,state", CASES)
def test_forward_and_gradients(B, T, H, K, V, dtype, decay, fused, state):
    q, k, v, ld, s0, d_o, dS = _inputs(B, T, H, K, V, dtype, decay, 100 + T, fused, state)
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda")  # noqa: E731
    o, final, saved = gdn.gdn_la_fwd(q, k, v, ld, s0, o=nan(d_o), saved=True)
    grads = (nan(q), nan(k), nan(v))
    dq, dk, dv, ds0 = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS, saved=saved, grads=grads)
    again = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS)
    torch.cuda.synchronize()
    args = (_np(q), _np(k), _np(v), _np(ld), _np(s0))
    ro, rs, _ = layer.la_fwd(*args)
    rg = layer.la_bwd(*args, _np(d_o), _np(dS))
    _check("o", o, ro)
    _check("final_state", final, rs)
    for name, t, r in zip(("dq", "dk", "dv", "d_initial_state"), (dq, dk, dv, ds0), rg):
        _check(name, t, r)
    for a, b in zip((dq, dk, dv, ds0), again):  # with what the forward saved, or without
        assert torch.equal(a, b)


def test_equal_calls_give_equal_bits():
    q, k, v, ld, s0, d_o, dS = _inputs(2, 700, 3, 128, 128, "bf16", "slopes", 7)
    runs = [gdn.gdn_la_fwd(q, k, v, ld, s0)[:2] + gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS) for _ in range(3)]
    torch.cuda.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("dtype,H", [("bf16", 2), ("f32", 160)])
def test_states_updated_in_place(dtype, H):
    """final_state = initial_state and d_initial_state = d_final_state give the bits of
    separate buffers, with one segment and with several."""
    q, k, v, ld, s0, d_o, dS = _inputs(1, 600, H, 32, 64, dtype, "slow", 8)
    _, final, _ = gdn.gdn_la_fwd(q, k, v, ld, s0)
    o1 = gdn.gdn_la_fwd(q, k, v, ld, s0)[0]
    ref = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS)
    got = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS, d_initial_state=dS)
    o2, same, _ = gdn.gdn_la_fwd(q, k, v, ld, s0, final_state=s0)
    torch.cuda.synchronize()
    assert same is s0 and torch.equal(s0, final) and torch.equal(o1, o2)
    assert got[3] is dS and all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_optional_states_left_out(dtype):
    q, k, v, ld, s0, d_o, _ = _inputs(1, 500, 2, 64, 32, dtype, "slow", 9)
    o, final, saved = gdn.gdn_la_fwd(q, k, v, ld, None, final_state=False)
    zero = torch.zeros_like(s0)
    o0, f0, _ = gdn.gdn_la_fwd(q, k, v, ld, zero)
    g = gdn.gdn_la_bwd(q, k, v, ld, None, d_o, None, d_initial_state=False)
    g0 = gdn.gdn_la_bwd(q, k, v, ld, zero, d_o, zero)
    torch.cuda.synchronize()
    assert final is None and saved is None and g[3] is None
    assert torch.equal(o, o0) and all(torch.equal(a, b) for a, b in zip(g[:3], g0[:3]))


def test_long_sequence_in_calls():
    """A stream cut into calls that pass the state on agrees with one call."""
    q, k, v, ld, s0, _, _ = _inputs(1, 5000, 3, 128, 128, "bf16", "slow", 10)
    o, final, _ = gdn.gdn_la_fwd(q, k, v, ld, s0)
    state, outs = s0, []
    for lo, hi in ((0, 1), (1, 130), (130, 2048), (2048, 5000)):
        x, state, _ = gdn.gdn_la_fwd(q[:, lo:hi], k[:, lo:hi], v[:, lo:hi], ld, state)
        outs.append(x)
    torch.cuda.synchronize()
    _check("o", torch.cat(outs, 1), _np(o))
    _check("final_state", state, _np(final))


def test_sampled_heads_of_a_long_training_shape():
    """B8 T4096 H6 K=V=128 forward and backward, three streams against the token loop."""
    q, k, v, ld, s0, d_o, dS = _inputs(8, 4096, 6, 128, 128, "bf16", "slow", 11)
    o, final, saved = gdn.gdn_la_fwd(q, k, v, ld, s0, saved=True)
    grads = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS, saved=saved)
    torch.cuda.synchronize()
    for b, h in ((0, 0), (3, 5), (7, 2)):
        pick = lambda t: _np(t[b:b + 1, :, h:h + 1])  # noqa: E731
        st = lambda t: _np(t[b:b + 1, h:h + 1])  # noqa: E731
        args = (pick(q), pick(k), pick(v), _np(ld[h:h + 1]), st(s0))
        ro, rs, _ = layer.la_fwd(*args)
        rg = layer.la_bwd(*args, pick(d_o), st(dS))
        _check("o", o[b:b + 1, :, h:h + 1], ro)
        _check("final_state", final[b:b + 1, h:h + 1], rs)
        for n, t, r in zip(("dq", "dk", "dv"), grads, rg):
            _check(n, t[b:b + 1, :, h:h + 1], r)
        _check("d_initial_state", grads[3][b:b + 1, h:h + 1], rg[3])


def test_rows_past_2_31_elements():
    """Offsets beyond 32 bits: the last batch rows of a tensor of 2^31 + elements."""
    B, T, H, K = 1030, 128, 128, 128  # 2.16e9 elements a tensor
    q = torch.empty(B, T, H, K, device="cuda", dtype=torch.bfloat16)
    small = _inputs(2, T, H, K, K, "bf16", "slopes", 12)
    q[:2] = small[0]
    q[-2:] = small[0]
    q[2:-2] = 0
    v = torch.zeros_like(q)
    v[:2] = small[2]
    v[-2:] = small[2]
    o, _, _ = gdn.gdn_la_fwd(q, q, v, small[3], final_state=False)
    dq, dk, dv, _ = gdn.gdn_la_bwd(q, q, v, small[3], None, v, d_initial_state=False)
    torch.cuda.synchronize()
    for t in (o, dq, dk, dv):
        assert torch.equal(t[:2], t[-2:]) and float(t[:2].float().abs().max()) > 0


@pytest.mark.parametrize("B,T,H,K,V,dtype,decay", [
    (1, 1, 6, 128, 128, "bf16", "slopes"), (3, 1, 5, 64, 16, "f32", "slow"), (2, 5, 3, 16, 32, "bf16", "none"),
    (1, 9, 2, 32, 128, "f32", "inf"), (64, 2, 16, 128, 64, "bf16", "strong"), (300, 1, 7, 16, 16, "bf16", "slopes"),
])
def test_decode(B, T, H, K, V, dtype, decay):
    q, k, v, ld, s0, _, _ = _inputs(B, T, H, K, V, dtype, decay, 200 + K, fused=T > 1)
    ro, rs, _ = layer.la_fwd(_np(q), _np(k), _np(v), _np(ld), _np(s0))
    state = s0.clone()
    o, st = gdn.gdn_la_decode(q, k, v, ld, state)
    torch.cuda.synchronize()
    assert st is state
    _check("o", o, ro)
    _check("state", state, rs)
    one = s0.clone()
    outs = [gdn.gdn_la_decode(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], ld, one)[0] for t in range(T)]
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(outs, 1), o) and torch.equal(one, state)


def test_empty_calls():
    q = torch.zeros(2, 0, 3, 32, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(2, 0, 3, 16, device="cuda", dtype=torch.bfloat16)
    ld = torch.zeros(3, device="cuda")
    s = torch.randn(2, 3, 16, 32, device="cuda")
    o, f, _ = gdn.gdn_la_fwd(q, q, v, ld, s)
    _, f0, _ = gdn.gdn_la_fwd(q, q, v, ld, None)
    g = gdn.gdn_la_bwd(q, q, v, ld, s, v, s)
    kept = s.clone()
    od, _ = gdn.gdn_la_decode(q, q, v, ld, kept)
    torch.cuda.synchronize()
    assert o.shape == v.shape and torch.equal(f, s) and not f0.any()
    assert g[0].shape == q.shape and torch.equal(g[3], s) and od.shape == v.shape and torch.equal(kept, s)
    e = torch.zeros(0, 5, 3, 32, device="cuda")
    assert gdn.gdn_la_fwd(e, e, e, ld)[0].shape == e.shape


def test_other_stream_and_its_own_workspace():
    q, k, v, ld, s0, d_o, dS = _inputs(1, 900, 4, 128, 64, "bf16", "slow", 13)
    ref = gdn.gdn_la_fwd(q, k, v, ld, s0)[:2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.gdn_la_fwd(q, k, v, ld, s0, stream=side)[:2]
    with torch.cuda.stream(side):
        g1 = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS)
    g2 = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref + g2, got + g1))


def test_graph_capture_replays():
    q, k, v, ld, s0, _, _ = _inputs(2, 300, 3, 64, 64, "bf16", "slow", 14)
    gdn.gdn_la_fwd(q, k, v, ld, s0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, f, _ = gdn.gdn_la_fwd(q, k, v, ld, s0)
    q.copy_(-q)
    graph.replay()
    ref = gdn.gdn_la_fwd(q, k, v, ld, s0)[:2]
    torch.cuda.synchronize()
    assert torch.equal(o, ref[0]) and torch.equal(f, ref[1])


def test_refusals():
    q, k, v, ld, s0, d_o, dS = _inputs(2, 20, 3, 32, 16, "bf16", "slopes", 15)
    bad = [
        dict(q=q.float()), dict(k=k[:, :10]), dict(v=v.transpose(1, 2)), dict(log_decay=ld.double()),
        dict(log_decay=ld[:2]), dict(log_decay=None), dict(initial_state=s0.bfloat16()), dict(q=q.cpu()),
        dict(k=k.flip(-1)[..., ::2]), dict(o=d_o[..., :8]), dict(final_state=s0[:1]),
        dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda")), dict(q=q[..., :24], k=k[..., :24]),
    ]
    for over in bad:
        args = dict(q=q, k=k, v=v, log_decay=ld, initial_state=s0)
        args.update(over)
        with pytest.raises(gdn.GdnError):
            gdn.gdn_la_fwd(**args)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_la_fwd(q, k, v, ld, s0, o=d_o, final_state=s0[:, :, :, :16].contiguous())
    with pytest.raises(gdn.GdnError):
        gdn.gdn_la_bwd(q, k, v, ld, s0, None)
    with pytest.raises(gdn.GdnError, match="overlaps"):
        gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS, grads=(q, torch.empty_like(k), torch.empty_like(v)))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_la_decode(q, k, v, ld, None)
    # the context is as it was
    gdn.gdn_la_fwd(q, k, v, ld, s0)
    torch.cuda.synchronize()


def test_new_tensors_belong_to_the_given_stream():
    """Memory that a call makes is the given stream's, so that what it gives back (its
    workspace) is not handed to the current stream while the given one still runs."""
    q, k, v, ld, s0, d_o, dS = _inputs(1, 2500, 2, 128, 128, "bf16", "slow", 15)
    ref = gdn.gdn_la_fwd(q, k, v, ld, s0)[:2] + gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = {s["stream"]: s["active_size"] for s in torch.cuda.memory_snapshot()}
    got = gdn.gdn_la_fwd(q, k, v, ld, s0, stream=side)[:2] + gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS, stream=side)
    torch.cuda.synchronize()
    assert side.cuda_stream not in held
    mine = [s for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream]
    for t in got:
        assert any(s["address"] <= t.data_ptr() < s["address"] + s["total_size"] for s in mine)
    # more than the outputs: the workspaces came and went here too
    assert sum(s["total_size"] for s in mine) > sum(t.numel() * t.element_size() for t in got)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
