"""GPU tests of what surrounds the layer, run together: the example's block and model
(training, waiting sequences, single tokens), and its gradients against the float64 forms
chained by hand."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import block as ref
from oracle import layer

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("linear_attention_block", os.path.join(ROOT, "examples", "linear_attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_trains_and_serves(example):
    norms, o_off, s_off = example.main(depth=2, width=256, heads=3, dim=64, batch=3, text=20, side=7, new_tokens=5, steps=4)
    assert len(norms) == 4 and all(np.isfinite(norms)) and min(norms) > 0
    # a state's row of 64 is off by at most 1/254 of its largest element in each (under 1% of
    # the row), an 8-bit norm by 2^-4 of each element at most (2.6% rms) in every projection
    assert 0 < o_off < 0.1 and 0 < s_off < 0.1


def _np(t):
    return t.detach().double().cpu().numpy()


def test_block_gradients(example):
    """Every gradient of residual norm -> norm and rotation by axes -> attention -> gated norm
    in float32 with the projections as plain products, against the float64 forms; then the
    norm of all of them and their clipped values."""
    B, T, H, D = 2, 70, 3, 32
    W = H * D
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    m = example.Block(W, H, D, T, dtype=torch.float32)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(0.2 * n(*p.shape))
    x, res, state = n(B, T, W).requires_grad_(), n(B, T, W).requires_grad_(), n(B, H, D, D).requires_grad_()
    pos = torch.randint(0, T, (3, B, T), generator=g, device="cuda", dtype=torch.int32)
    dy, dh, dS = n(B, T, W), n(B, T, W), n(B, H, D, D)
    allow = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        y, h, end = m(x, res, state, pos)
        names = ["norm", "project.weight", "out.weight", "wq", "wk", "wo"]
        params = dict(m.named_parameters())
        got = torch.autograd.grad((y, h, end), [x, res, state] + [params[k] for k in names], (dy, dh, dS))
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allow
    P = {k: _np(params[k]) for k in names}
    c, s = ref.angles(_np(m.cos), _np(m.sin), pos.cpu().numpy(), m.sections, False)
    ry, rh = ref.add_norm_fwd(_np(x), _np(res), P["norm"], 1e-6)
    rows = (ry @ P["project.weight"].T).reshape(B, T, 4, H, D)
    Q, K, V, G = (rows[:, :, i] for i in range(4))
    rq = layer.norm_rope_fwd(Q, P["wq"], c, s, 1e-6, False)
    rk = layer.norm_rope_fwd(K, P["wk"], c, s, 1e-6, False)
    ro, rS, _ = layer.la_fwd(rq, rk, V, _np(m.log_decay), _np(state))
    rg = layer.gated_norm_fwd(ro, G, P["wo"], 1e-6).reshape(B, T, W)
    d_out = np.einsum("btw,bti->wi", _np(dy), rg)
    d_o, d_gate, d_wo = layer.gated_norm_bwd(ro, G, P["wo"], 1e-6, (_np(dy) @ P["out.weight"]).reshape(B, T, H, D))
    dq, dk, dv, ds0 = layer.la_bwd(rq, rk, V, _np(m.log_decay), _np(state), d_o, _np(dS))
    dQ, d_wq = layer.norm_rope_bwd(Q, P["wq"], c, s, 1e-6, False, dq)
    dK, d_wk = layer.norm_rope_bwd(K, P["wk"], c, s, 1e-6, False, dk)
    d_rows = np.stack([dQ, dK, dv, d_gate], 2).reshape(B, T, -1)
    d_project = np.einsum("bti,btw->iw", d_rows, ry)
    dx, d_norm = ref.add_norm_bwd(rh, P["norm"], 1e-6, d_rows @ P["project.weight"], _np(dh))
    want = (dx, dx, ds0, d_norm, d_project, d_out, d_wq, d_wk, d_wo)
    for t, r in ((y, rg @ P["out.weight"].T), (h, rh), (end, rS)):
        assert np.linalg.norm(_np(t) - r) <= 2e-5 * np.linalg.norm(r)
    # float32 throughout: a few hundred roundings of 6e-8 along the chain
    for name, t, r in zip(["x", "residual", "state"] + names, got, want, strict=True):
        assert np.linalg.norm(_np(t) - r) <= 1e-4 * np.linalg.norm(r), name
    norm = gdn.gdn_clip_grads(got[3:], 1.0)
    total = np.sqrt(sum((r * r).sum() for r in want[3:]))
    assert total > 1 and abs(float(norm) / total - 1) <= 1e-4
    for name, t, r in zip(names, got[3:], want[3:], strict=True):
        assert np.linalg.norm(_np(t) * total - r) <= 2e-4 * np.linalg.norm(r), name


def test_step_in_a_graph(example):
    """A serving step of the model, captured with its parking and resuming, equals the calls one
    by one, bit for bit."""
    torch.manual_seed(1)
    model = example.Model(2, 256, 2, 64, 64)
    x = torch.randn(4, 1, 256, device="cuda", dtype=torch.bfloat16)
    states = [torch.randn(4, 2, 64, 64, device="cuda") for _ in range(2)]
    cache, scales = torch.zeros(6, 2, 64, 64, dtype=torch.int8, device="cuda"), torch.zeros(6, 2, 64, device="cuda")
    slots = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device="cuda")
    pos = torch.full((3, 4, 1), 9, dtype=torch.int32, device="cuda")

    def run(states):
        y = model.step(x, states, pos)
        gdn.gdn_state_store(states[0], slots, cache, scales)
        return y, gdn.gdn_state_load(cache, scales, slots)

    start = [s.clone() for s in states]
    ref_y, ref_back = run([s.clone() for s in start])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, back = run(states)
    for s, k in zip(states, start):
        s.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref_y) and torch.equal(back, ref_back)
