"""GPU tests of the linear-attention layer's operators at the edges of what they accept,
against the float64 forms.

Tolerances, relative L2: float32 results 1e-5 (a few dozen roundings of 6e-8 each, sums of
at most a few thousand terms); bf16 results of the norms 3e-3 (one rounding: 2^-8 / sqrt(12)
* 1.4 = 1.6e-3 rms, 2^-9 = 2e-3 for a row of one size)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import layer

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {torch.float32: 1e-5, torch.bfloat16: 3e-3}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(name, got, ref, tol=None):
    x, r = _np(got), np.asarray(ref)
    assert x.shape == r.shape and np.isfinite(x).all(), name
    err = np.linalg.norm(x - r) / max(np.linalg.norm(r), 1e-30)
    assert err <= (tol or TOL[got.dtype]), f"{name}: {err:.2e}"


def _normal(seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,D", [(1, 1, 1, 128), (2, 5, 3, 96), (1, 37, 5, 256), (3, 700, 7, 128)])
def test_gated_norm_without_eps(B, T, H, D, dtype):
    """eps = 0 is accepted, and every row here has a length: the places of a block that
    have no row add nothing to the weight's gradient."""
    n = _normal(B * T + D, dtype)
    x, z, dy, w = n(B, T, H, D), n(B, T, H, D), n(B, T, H, D), 1 + 0.2 * n(D)
    y = gdn.gdn_gated_norm_fwd(x, z, w, eps=0.0)
    grads = gdn.gdn_gated_norm_bwd(x, z, w, dy, eps=0.0)
    torch.cuda.synchronize()
    _close("y", y, layer.gated_norm_fwd(_np(x), _np(z), _np(w), 0.0))
    for name, t, r in zip(("dx", "dgate", "dw"), grads, layer.gated_norm_bwd(_np(x), _np(z), _np(w), 0.0, _np(dy))):
        _close(name, t, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", [(1, 1, 1, 1, 128, 128), (2, 5, 3, 1, 96, 32), (1, 37, 5, 2, 256, 0),
                                           (3, 500, 7, 3, 128, 64)])
def test_norm_rope_without_eps(B, T, Hq, Hk, D, R, dtype):
    """As above for the q, k norm: also the second head of an item of an odd count."""
    n = _normal(B * T + D, dtype)
    q, k, dq, dk, wq, wk = n(B, T, Hq, D), n(B, T, Hk, D), n(B, T, Hq, D), n(B, T, Hk, D), 1 + 0.2 * n(D), 1 + 0.2 * n(D)
    a = torch.linspace(-3, 3, T * (R // 2), device="cuda").view(T, R // 2)
    cos, sin = (a.cos(), a.sin()) if R else (None, None)
    c, s = (np.broadcast_to(_np(t), (B, T, R // 2)) for t in (a.cos(), a.sin()))
    grads = gdn.gdn_qk_norm_rope_bwd(q, k, wq, wk, cos, sin, None, dq, dk, eps=0.0)
    torch.cuda.synchronize()
    for x, w, dy, dx, dw in ((q, wq, dq, grads[0], grads[2]), (k, wk, dk, grads[1], grads[3])):
        rx, rw = layer.norm_rope_bwd(_np(x), _np(w), c, s, 0.0, False, _np(dy))
        _close("dx", dx, rx)
        _close("dw", dw, rw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_norm_gates_past_2_24(dtype):
    """The slope of silu is 1 for a large gate of any size, and 0 for a large negative one."""
    gates = [3e3, 2.0 ** 22 + 2 ** 20, 2.0 ** 24 + 2, 2.0 ** 24 + 2 ** 18, 2.0 ** 26, 1e8, 1e30, -1e8, -1e30]
    n = _normal(1, dtype)
    shape = (1, len(gates), 1, 64)
    z = torch.tensor(gates, device="cuda").view(1, -1, 1, 1).expand(shape).to(DT[dtype]).contiguous()
    x, dy, w = n(*shape), n(*shape), 1 + 0.2 * n(64)
    _, dz, _ = gdn.gdn_gated_norm_bwd(x, z, w, dy)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        ref = layer.gated_norm_bwd(_np(x), _np(z), _np(w), 1e-6, _np(dy))[1]
    for t, gate in enumerate(gates):
        _close(f"dgate of {gate}", dz[:, t], ref[:, t])


def test_memory_that_runs_out_is_torchs_error():
    """An allocation that fails raises what torch's own do, and leaves calls usable.  In a
    process of its own: memory that other tests left cached would serve the call."""
    import os
    import subprocess
    import sys

    run = """
import torch
from gated_delta_rule_19_gb300 import gdn
q = torch.zeros(1, 32768, 16, 128, device="cuda", dtype=torch.bfloat16)  # outputs of 128 MB
ld = torch.zeros(16, device="cuda")
torch.cuda.set_per_process_memory_fraction(1e-6)
for call in (lambda: gdn.gdn_la_fwd(q, q, q, ld), lambda: gdn.gdn_gated_norm_fwd(q, q, q[0, 0, 0])):
    try:
        call()
        raise SystemExit("no error")
    except torch.OutOfMemoryError:
        pass
torch.cuda.set_per_process_memory_fraction(1.0)
o, _, _ = gdn.gdn_la_fwd(q, q, q, ld)
torch.cuda.synchronize()
assert o.shape == q.shape and not o.any()
print("done")
"""
    r = subprocess.run([sys.executable, "-c", run], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr


def test_autograd_sees_a_state_that_was_overwritten():
    B, T, H, K, V = 2, 3, 3, 32, 16
    n = _normal(3, "f32")
    q, v, state, ld, w = n(B, T, H, K), n(B, T, H, V), n(B, H, V, K), torch.zeros(H, device="cuda"), n(K)
    for call in (lambda s: gdn.gdn_la_decode(q, q, v, ld, s), lambda s: gdn.gdn_la_fwd(q, q, v, ld, s, final_state=s),
                 lambda s: gdn.gdn_la_bwd(q, q, v, ld, None, v, s, d_initial_state=s)):
        x = state.clone().requires_grad_()
        s = x * 2
        loss = (s * s).sum()  # saves s
        with torch.no_grad():
            call(s)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    y, out = n(B, T, H, V), n(B, T, H, K)
    before = y._version, out._version
    gdn.gdn_la_fwd(q, q, v, ld, o=y)
    gdn.gdn_gated_norm_fwd(q, q, w, y=out)
    assert y._version > before[0] and out._version > before[1] and q._version == v._version == 0
    with torch.inference_mode():
        kept = state.clone()
    gdn.gdn_la_decode(q, q, v, ld, kept)  # a state of inference mode has no version
    before = state._version
    with pytest.raises(gdn.GdnError):
        gdn.gdn_la_decode(q, q, v, None, state)
    assert state._version == before  # nothing was written
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H,K,V", [(150, 2, 16, 16), (1000, 2, 64, 64), (150, 160, 128, 128), (1000, 2, 128, 32)])
def test_float32_values_next_to_the_largest(T, H, K, V):
    """Inputs and states up to the largest float32 give finite results where the definition
    does; with one segment and with several."""
    n = _normal(K + T, "f32")
    q, k, v, d_o = n(1, T, H, K) * 1e-6, n(1, T, H, K) * 1e-3, n(1, T, H, V), n(1, T, H, V) * 1e-3
    ld = torch.full((H,), -0.05, device="cuda")
    most = torch.finfo(torch.float32).max
    v[0, 70, 0, 3], v[0, 71, 1, 5] = most, -3.4025e38
    k[0, 140, 1, 0], v[0, 140, 1, 2] = 1.0, most  # the state's element itself next to the largest
    s0 = torch.zeros(1, H, V, K, device="cuda")
    s0[0, 0, 1, 2] = most
    o, final, saved = gdn.gdn_la_fwd(q, k, v, ld, s0, saved=True)
    grads = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, saved=saved)
    torch.cuda.synchronize()
    args = [_np(t[:, :, :2]) for t in (q, k, v)] + [_np(ld[:2]), _np(s0[:, :2])]
    ro, rs, _ = layer.la_fwd(*args)
    ref = layer.la_bwd(*args, _np(d_o[:, :, :2]))
    for name, t, r in zip(("o", "dq", "dk", "dv"), (o, *grads[:3]), (ro, *ref[:3])):
        _close(name, t[:, :, :2], r)
    _close("final_state", final[:, :2], rs)
    _close("d_initial_state", grads[3][:, :2], ref[3])
    gdn.gdn_la_fwd(q, k, v, ld, s0, final_state=s0)  # a state that is overwritten is read first
    torch.cuda.synchronize()
    assert torch.equal(s0, final)


@pytest.mark.parametrize("D", [32, 128])
def test_float32_values_that_are_not_finite_stay_in_their_stream(D):
    """A NaN or an infinity reaches its own stream from its 64-token chunk on, no other stream
    and no earlier chunk, and an infinite result stays one; and its gradients likewise."""
    n = _normal(5, "f32")
    B, T, H = 2, 700, 3
    q, k, v, d_o = n(B, T, H, D), n(B, T, H, D), n(B, T, H, D), n(B, T, H, D)
    ld = torch.full((H,), -0.01, device="cuda")
    o, final, _ = gdn.gdn_la_fwd(q, k, v, ld)
    grads = gdn.gdn_la_bwd(q, k, v, ld, None, d_o)
    bad = v.clone()
    bad[1, 300, 2, 5] = float("nan")
    bad[0, 400, 1, 7] = float("inf")
    o2, final2, _ = gdn.gdn_la_fwd(q, k, bad, ld)
    grads2 = gdn.gdn_la_bwd(q, k, bad, ld, None, d_o)
    torch.cuda.synchronize()
    for a, b in [(o, o2)] + list(zip(grads[:3], grads2[:3])):
        same = (a == b).all(-1)
        assert same[0, :, 0].all() and same[0, :, 2].all() and same[1, :, :2].all()
    assert torch.equal(o[1, :256, 2], o2[1, :256, 2]) and torch.equal(o[0, :384, 1], o2[0, :384, 1])
    assert o2[1, 300:, 2, 5].isnan().all() and final2[1, 2, 5].isnan().all()
    assert not o2[0, 400:, 1, 7].isfinite().any() and torch.equal(final[0, 0], final2[0, 0])
    # the state's row is v k^T: infinities of k's signs
    assert torch.equal(final2[0, 1, 7], float("inf") * k[0, 400, 1])
    assert torch.equal(grads[1][1, 320:, 2], grads2[1][1, 320:, 2])


def test_example_refuses_second_derivatives():
    """The operators have first derivatives; a second one through the example's functions is
    an error, not a gradient that takes the first for a constant."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "linear_attention_layer.py")
    spec = importlib.util.spec_from_file_location("linear_attention_layer_edges", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    n = _normal(9, "f32")
    x, w, ld, s0 = n(1, 4, 2, 32).requires_grad_(), n(32), torch.zeros(2, device="cuda"), n(1, 2, 32, 32)
    for y in (ex.GatedNorm.apply(x, x, w), ex.NormRope.apply(x, x, w, w, None, None, None)[0],
              ex.LinearAttention.apply(x, x, x, ld, s0)[0]):
        (d,) = torch.autograd.grad((y * y).sum() + (x ** 3).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiate twice"):
            d.sum().backward()


def _bf16(x):
    """Rounded to bf16 (float64 in and out)."""
    return torch.from_numpy(np.ascontiguousarray(x)).float().bfloat16().double().numpy()


@pytest.mark.parametrize("B,T,H,K,V,dtype", [
    (1, 100, 200, 128, 128, "bf16"), (1, 1500, 2, 128, 128, "bf16"), (2, 700, 3, 64, 32, "bf16"),
    (1, 1500, 160, 16, 16, "bf16"), (1, 100, 200, 128, 128, "f32"), (1, 1500, 2, 128, 128, "f32"),
    (2, 700, 3, 64, 32, "f32"),
])
def test_returned_states_and_float32_results_are_as_exact_as_float32_sums(B, T, H, K, V, dtype):
    """Decays of 100 to 4000 tokens, one segment and several.  Tolerance 1.5e-6: bf16 inputs'
    states are sums of 24-bit products in float32, 24 partial sums a tile, each cut to 24
    bits: 24 * 2^-24 = 1.4e-6 if all went one way.  float32 products are exact to 2 * 2^-23
    and their sums of 8 tokens or columns at a time go the same way.  With decayed rows of 16
    bits (two bf16 numbers) a state is about 2.5e-6 off, which this tells apart."""
    n = _normal(T + K, "f32")
    cast = lambda t: t.to(DT[dtype])  # noqa: E731
    q, k, v, d_o = cast(n(B, T, H, K) * K ** -0.5), cast(n(B, T, H, K)), cast(n(B, T, H, V)), cast(n(B, T, H, V))
    h = torch.arange(1, H + 1, device="cuda", dtype=torch.float32)
    ld = torch.log1p(-torch.exp2(-7 - 5 * h / H))
    s0, dS = n(B, H, V, K) * 0.5, n(B, H, V, K) * 0.1
    o, final, saved = gdn.gdn_la_fwd(q, k, v, ld, s0, saved=True)
    grads = gdn.gdn_la_bwd(q, k, v, ld, s0, d_o, dS, saved=saved)
    torch.cuda.synchronize()
    at = sorted({0, H // 2, H - 1})
    rows = lambda t: t[:1, :, at]  # noqa: E731
    args = [_np(rows(t)) for t in (q, k, v)] + [_np(ld[at]), _np(s0[:1, at])]
    ro, rs, _ = layer.la_fwd(*args)
    ref = layer.la_bwd(*args, _np(rows(d_o)), _np(dS[:1, at]))
    _close("final_state", final[:1, at], rs, 1.5e-6)
    _close("d_initial_state", grads[3][:1, at], ref[3], 1.5e-6)
    if dtype == "f32":
        for name, t, r in zip(("o", "dq", "dk", "dv"), (o, *grads[:3]), (ro, *ref[:3])):
            _close(name, rows(t), r, 1.5e-6)
    else:  # the state that decayed rows of 16 bits would give
        fade = np.exp(args[3][None, None, :, None] * (T - 1 - np.arange(T))[None, :, None, None])
        c = args[2] * fade
        short = np.einsum("bthv,bthk->bhvk", _bf16(c) + _bf16(c - _bf16(c)) - c, args[1])
        with pytest.raises(AssertionError):
            _close("final_state", final[:1, at], rs + short, 1.5e-6)
