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
