"""GPU tests of the q, k norm with the rotation (gdn_qk_norm_rope_fwd/bwd) and of the
gated norm (gdn_gated_norm_fwd/bwd) against float64.

Tolerances, relative L2 over a tensor and, twice as wide, over each row: everything
is computed in float32, so float32 results are within 1e-5 (a few dozen roundings of
6e-8 each, sums of 256 terms or, for the weights' gradients, of all rows), and bf16
results carry one rounding: 2^-8 / sqrt(12) * 1.4 = 1.6e-3 rms, 2^-9 = 2e-3 for a row
of one size, 3e-3 taken."""
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


def _rows(g, B, T, H, D, dt, fused, std=1.0):
    if fused:
        x = (torch.randn(B, T, 2 * H * D + 64, generator=g, device="cuda") * std).to(dt)
        return x[..., 64:64 + H * D].unflatten(-1, (H, D))
    return (torch.randn(B, T, H, D, generator=g, device="cuda") * std).to(dt)


ROPE = [
    # B, T, Hq, Hk, D, R, dtype, interleaved, fused, positions
    (1, 1, 1, 1, 16, 16, "bf16", False, False, "own"),
    (1, 1, 6, 6, 128, 128, "bf16", False, False, "own"),
    (2, 3, 5, 1, 128, 64, "bf16", True, True, "own"),
    (2, 17, 6, 2, 128, 128, "f32", False, True, None),
    (1, 70, 3, 3, 8, 8, "f32", True, False, "own"),
    (3, 33, 4, 4, 96, 96, "bf16", False, False, None),
    (1, 129, 9, 3, 96, 32, "f32", False, True, "own"),
    (2, 5, 16, 4, 256, 256, "bf16", True, False, "own"),
    (1, 40, 2, 2, 256, 128, "f32", False, False, "own"),
    (2, 50, 7, 7, 64, 0, "bf16", False, False, None),
    (2, 600, 12, 4, 32, 32, "bf16", False, True, "own"),
    (1, 2000, 6, 6, 128, 128, "bf16", False, True, "own"),
]


def _rope(B, T, Hq, Hk, D, R, dtype, interleaved, fused, positions, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + D + T)
    dt = DT[dtype]
    q, k = _rows(g, B, T, Hq, D, dt, fused, 3.0), _rows(g, B, T, Hk, D, dt, fused, 0.2)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2))
    cos = sin = pos = None
    n = T + 50
    if R:
        a = torch.randn(n, R // 2, generator=g, device="cuda") * 3
        cos, sin = a.cos(), a.sin()
    if positions == "own":
        pos = torch.randint(0, n, (B, T), generator=g, device="cuda", dtype=torch.int32)
    at = (pos if pos is not None else torch.arange(T, device="cuda").expand(B, T)).long()
    c = _np(cos[at]) if R else np.zeros((B, T, 0))
    s = _np(sin[at]) if R else np.zeros((B, T, 0))
    dq, dk = _rows(g, B, T, Hq, D, dt, False), _rows(g, B, T, Hk, D, dt, False)
    return q, k, wq, wk, cos, sin, pos, c, s, dq, dk


@pytest.mark.parametrize("B,T,Hq,Hk,D,R,dtype,interleaved,fused,positions", ROPE)
def test_norm_rope(B, T, Hq, Hk, D, R, dtype, interleaved, fused, positions):
    q, k, wq, wk, cos, sin, pos, c, s, dqo, dko = _rope(B, T, Hq, Hk, D, R, dtype, interleaved, fused, positions)
    eps = 1e-5
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda")  # noqa: E731
    yq, yk = gdn.gdn_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos, eps=eps, interleaved=interleaved, q_out=nan(q),
                                      k_out=nan(k))
    bwd = lambda **kw: gdn.gdn_qk_norm_rope_bwd(q, k, wq, wk, cos, sin, pos, dqo, dko, eps=eps,  # noqa: E731
                                                interleaved=interleaved, **kw)
    grads = bwd(grads=(nan(q), nan(k), nan(wq), nan(wk)))
    again = bwd()
    torch.cuda.synchronize()
    for name, y, x, w, dy, dx, dw in (("q", yq, q, wq, dqo, grads[0], grads[2]), ("k", yk, k, wk, dko, grads[1], grads[3])):
        _check(name, y, layer.norm_rope_fwd(_np(x), _np(w), c, s, eps, interleaved))
        rx, rw = layer.norm_rope_bwd(_np(x), _np(w), c, s, eps, interleaved, _np(dy))
        _check("d" + name, dx, rx)
        _check("dw" + name, dw, rw)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_norm_rope_positions_outside_the_tables():
    q, k, wq, wk, cos, sin, pos, *_ = _rope(2, 4, 3, 1, 64, 32, "bf16", False, False, "own")
    pos[0, 1], pos[1, 2] = -1, cos.shape[0]
    yq, yk = gdn.gdn_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos)
    torch.cuda.synchronize()
    bad = torch.zeros(2, 4, dtype=torch.bool)
    bad[0, 1] = bad[1, 2] = True
    for y in (yq, yk):
        assert torch.equal(y[..., :32].float().isnan().all(-1).all(-1).cpu(), bad)
        assert not y[..., 32:].float().isnan().any()  # the part that is not rotated


def test_norm_rope_zero_rows_stay_finite():
    q = torch.zeros(1, 5, 2, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    yq, _ = gdn.gdn_qk_norm_rope_fwd(q, q, w, w)
    dq, dk, dw, _ = gdn.gdn_qk_norm_rope_bwd(q, q, w, w, None, None, None, q + 1, q + 1)
    torch.cuda.synchronize()
    assert not yq.any() and dq.isfinite().all() and dk.isfinite().all() and not dw.any()


GATED = [
    # B, T, H, D, dtype, fused
    (1, 1, 1, 16, "bf16", False),
    (256, 1, 16, 128, "bf16", False),
    (2, 3, 5, 128, "bf16", True),
    (2, 17, 3, 8, "f32", True),
    (3, 33, 4, 96, "bf16", False),
    (1, 129, 9, 96, "f32", True),
    (2, 5, 16, 256, "bf16", False),
    (1, 40, 2, 256, "f32", False),
    (2, 700, 6, 64, "bf16", True),
    (1, 3000, 6, 128, "bf16", False),
]


@pytest.mark.parametrize("B,T,H,D,dtype,fused", GATED)
def test_gated_norm(B, T, H, D, dtype, fused):
    g = torch.Generator(device="cuda").manual_seed(D + T)
    dt, eps = DT[dtype], 1e-5
    x, z, dy = _rows(g, B, T, H, D, dt, fused, 2.0), _rows(g, B, T, H, D, dt, fused, 2.0), _rows(g, B, T, H, D, dt, False)
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda")  # noqa: E731
    y = gdn.gdn_gated_norm_fwd(x, z, w, eps=eps, y=nan(x))
    grads = gdn.gdn_gated_norm_bwd(x, z, w, dy, eps=eps, grads=(nan(x), nan(x), nan(w)))
    again = gdn.gdn_gated_norm_bwd(x, z, w, dy, eps=eps)
    torch.cuda.synchronize()
    _check("y", y, layer.gated_norm_fwd(_np(x), _np(z), _np(w), eps))
    for name, t, r in zip(("dx", "dgate", "dw"), grads, layer.gated_norm_bwd(_np(x), _np(z), _np(w), eps, _np(dy))):
        _check(name, t, r)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_gated_norm_gates_far_out():
    """Gates of large size: silu is the gate itself or 0, its slope 1 or 0."""
    x = torch.randn(1, 4, 1, 64, device="cuda")
    z = torch.tensor([200.0, -200.0, 88.0, -88.0], device="cuda").view(1, 4, 1, 1).expand(1, 4, 1, 64).contiguous()
    w = torch.ones(64, device="cuda")
    y = gdn.gdn_gated_norm_fwd(x, z, w)
    dx, dz, _ = gdn.gdn_gated_norm_bwd(x, z, w, torch.ones_like(x))
    torch.cuda.synchronize()
    assert all(t.isfinite().all() for t in (y, dx, dz))
    assert not y[0, 1].any() and not dx[0, 1].any() and not dz[0, 1].any()
    assert torch.allclose(y[0, 0], 200 * dz[0, 0], rtol=1e-5)


def test_no_rows():
    q = torch.zeros(2, 0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    yq, yk = gdn.gdn_qk_norm_rope_fwd(q, q, w, w)
    g = gdn.gdn_qk_norm_rope_bwd(q, q, w, w, None, None, None, q, q)
    y = gdn.gdn_gated_norm_fwd(q, q, w)
    h = gdn.gdn_gated_norm_bwd(q, q, w, q)
    torch.cuda.synchronize()
    assert yq.shape == yk.shape == y.shape == q.shape
    assert not g[2].any() and not g[3].any() and not h[2].any()  # sums over no rows


def test_other_stream():
    q, k, wq, wk, cos, sin, pos, _, _, dqo, dko = _rope(1, 300, 6, 6, 128, 128, "bf16", False, True, "own")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = (q, k, wq, wk, cos, sin, pos)
    got = gdn.gdn_qk_norm_rope_fwd(*args, stream=side)
    with torch.cuda.stream(side):
        got += gdn.gdn_qk_norm_rope_bwd(*args, dqo, dko)
    ref = gdn.gdn_qk_norm_rope_fwd(*args) + gdn.gdn_qk_norm_rope_bwd(*args, dqo, dko)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_refusals():
    q, k, wq, wk, cos, sin, pos, _, _, dqo, dko = _rope(2, 20, 4, 2, 64, 32, "bf16", False, False, "own")
    ok = dict(q=q, k=k, q_weight=wq, k_weight=wk, cos=cos, sin=sin, positions=pos)
    bad = [dict(q=q.float()), dict(k=k[:, :5]), dict(q=q.transpose(1, 2)), dict(q_weight=None), dict(k_weight=wk[:32]),
           dict(q_weight=wq.float()), dict(cos=cos.double()), dict(sin=None), dict(sin=sin[:5]), dict(positions=pos.long()),
           dict(positions=pos[:1]), dict(cos=cos[:, :3], sin=sin[:, :3]), dict(q=q.cpu()), dict(eps=-1.0),
           dict(cos=cos.repeat(1, 3), sin=sin.repeat(1, 3)), dict(positions=None, cos=cos[:10], sin=sin[:10]),
           dict(q=q[..., :40], k=k[..., :40], q_weight=wq[:40], k_weight=wk[:40]), dict(q_out=q), dict(k_out=wk)]
    for over in bad:
        with pytest.raises(gdn.GdnError):
            gdn.gdn_qk_norm_rope_fwd(**{**ok, **over})
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm_rope_bwd(*ok.values(), None, dko)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm_rope_bwd(*ok.values(), dqo, dko, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    x, z, w = q, q + 1, wq
    for args in ((x, z[:, :5], w), (x, z.float(), w), (x, z, None), (x, z, w[:8]), (x.half(), z.half(), w.half()),
                 (x[0], z[0], w)):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_gated_norm_fwd(*args)
    with pytest.raises(gdn.GdnError, match="overlaps"):
        gdn.gdn_gated_norm_fwd(x, z, w, y=x)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_gated_norm_bwd(x, z, w, None)
    gdn.gdn_gated_norm_fwd(x, z, w)
    torch.cuda.synchronize()
