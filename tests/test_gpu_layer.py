"""GPU tests of the linear-attention layer's operators together: the example's layer
(training, a prompt, single tokens), its gradients against the float64 forms chained by
hand, and the tensor-core kernels' bounded waits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import layer as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("linear_attention_layer",
                                                  os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_trains_and_serves(example):
    losses, o_off, s_off = example.main(width=128, heads=3, dim=64, batch=2, tokens=333, steps=12, new_tokens=5)
    assert losses[-1] < 0.9 * losses[0]
    # the outputs pass through five roundings to bf16 each way; states differ by the 16
    # bits that the chunked form keeps of a decayed value
    assert o_off < 2e-2 and s_off < 1e-4


def _np(t):
    return t.detach().double().cpu().numpy()


def test_example_gradients(example):
    """Every input gradient of norm + rotation -> attention -> gated norm in float32,
    from slices of one projection, against the float64 forms."""
    B, T, H, D = 2, 150, 3, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = n(B, T, 4, H, D).requires_grad_()
    wq, wk, wo = ((1 + 0.2 * n(D)).requires_grad_() for _ in range(3))
    state = n(B, H, D, D).requires_grad_()
    a = n(T, D // 2)
    cos, sin, pos = a.cos(), a.sin(), torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    ld = -torch.rand(H, generator=g, device="cuda")
    dy, dS = n(B, T, H, D), n(B, H, D, D)
    q, k, v, gate = rows.unbind(2)
    qn, kn = example.NormRope.apply(q, k, wq, wk, cos, sin, pos)
    o, final = example.LinearAttention.apply(qn, kn, v, ld, state)
    y = example.GatedNorm.apply(o, gate, wo)
    got = torch.autograd.grad((y, final), (rows, wq, wk, wo, state), (dy, dS))
    c, s = (_np(t)[None].repeat(B, 0) for t in (cos, sin))
    Q, K, V, G = (_np(t) for t in (q, k, v, gate))
    rq = ref.norm_rope_fwd(Q, _np(wq), c, s, 1e-6, False)
    rk = ref.norm_rope_fwd(K, _np(wk), c, s, 1e-6, False)
    ro, rS, _ = ref.la_fwd(rq, rk, V, _np(ld), _np(state))
    d_o, d_gate, d_wo = ref.gated_norm_bwd(ro, G, _np(wo), 1e-6, _np(dy))
    dq, dk, dv, ds0 = ref.la_bwd(rq, rk, V, _np(ld), _np(state), d_o, _np(dS))
    dQ, d_wq = ref.norm_rope_bwd(Q, _np(wq), c, s, 1e-6, False, dq)
    dK, d_wk = ref.norm_rope_bwd(K, _np(wk), c, s, 1e-6, False, dk)
    want = (np.stack([dQ, dK, dv, d_gate], 2), d_wq, d_wk, d_wo, ds0)
    for t, r in zip((y, final), (ref.gated_norm_fwd(ro, G, _np(wo), 1e-6), rS)):
        assert np.linalg.norm(_np(t) - r) <= 1e-5 * np.linalg.norm(r)
    for t, r in zip(got, want):  # each passes through three operators of 1e-5
        assert np.linalg.norm(_np(t) - r) <= 3e-5 * np.linalg.norm(r)


def test_values_that_are_not_finite_stay_in_their_stream(example):
    """A NaN or an infinity reaches its own stream from its 128-token tile on, no other
    stream and no earlier tile; and its gradients likewise."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    B, T, H, D = 2, 700, 3, 64
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
    assert o2[1, 300:, 2, 5].isnan().all() and not o2[0, 400:, 1, 7].isfinite().any()
    assert final2[1, 2, 5].isnan().all() and torch.equal(final[0, 0], final2[0, 0])
    # dk goes against the order of time: tiles behind the value's are not reached
    assert torch.equal(grads[1][1, 384:, 2], grads2[1][1, 384:, 2])


def test_wait_limit_ends_the_kernels(example):
    """With a limit of a few nanoseconds the first wait that does not succeed at once gives
    up: a bit in the workspace's error word, a context that still works, and the bits of
    an undisturbed call afterwards."""
    g = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    for T, H in ((1000, 2), (300, 200)):  # several segments (sums, link, scan), and one
        q, k, v, d_o = n(1, T, H, 128), n(1, T, H, 128), n(1, T, H, 128), n(1, T, H, 128)
        ld = torch.full((H,), -0.02, device="cuda")
        ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
        run = lambda: (gdn.gdn_la_fwd(q, k, v, ld, workspace=ws)[:2] +  # noqa: E731
                       gdn.gdn_la_bwd(q, k, v, ld, None, d_o, workspace=ws))
        word = lambda: int(ws[:4].view(torch.int32).item())  # noqa: E731
        want = run()
        torch.cuda.synchronize()
        assert word() == 0
        try:
            gdn.gdn_test_set_wait_limit(2)
            run()
            torch.cuda.synchronize()
            assert word() != 0
        finally:
            gdn.gdn_test_set_wait_limit(0)
        ws[:4].zero_()
        got = run()
        torch.cuda.synchronize()
        assert word() == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 50, 400])
def test_calls_behind_one_another(dtype, T):
    """A chain of calls, each on the one before's outputs and over what an earlier one
    still reads, gives the bits of the same chain with a wait after every call."""
    B, H, D = 2, 6, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, k0, gate, w = n(B, T, H, D), n(B, T, H, D), n(B, T, H, D), 1 + 0.1 * n(D)
    a = torch.randn(T, D // 2, generator=g, device="cuda")
    cos, sin, ld = a.cos(), a.sin(), torch.full((H,), -0.05, device="cuda")
    state0 = torch.randn(B, H, D, D, generator=g, device="cuda")

    def chain(wait):
        q, state, bufs = x.clone(), state0.clone(), (torch.empty_like(x), torch.empty_like(x), torch.empty_like(x))
        qn, kn, y = bufs
        out = []
        for _ in range(30):
            gdn.gdn_qk_norm_rope_fwd(q, k0, w, w, cos, sin, q_out=qn, k_out=kn)
            wait()
            if T == 1:
                o, _ = gdn.gdn_la_decode(qn, kn, q, ld, state)
            else:
                o, _, saved = gdn.gdn_la_fwd(qn, kn, q, ld, state, final_state=state, saved=True)
            wait()
            gdn.gdn_gated_norm_fwd(o, gate, w, y=y)
            wait()
            dx, dz, dw = gdn.gdn_gated_norm_bwd(o, gate, w, y)
            wait()
            dq, dk, dv, ds = gdn.gdn_la_bwd(qn, kn, q, ld, state, dx, state)
            wait()
            gdn.gdn_qk_norm_rope_bwd(q, k0, w, w, cos, sin, None, dq, dk, grads=None)
            wait()
            q.copy_(y)
            wait()
        return q, state, dx, dz, dw, dq, dk, dv, ds

    apart = chain(torch.cuda.synchronize)
    for _ in range(3):
        together = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(apart, together))
