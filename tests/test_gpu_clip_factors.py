"""GPU tests of clipping by factors that leave float32's normal range (gdn_clip_grads): large
gradients, also ones whose norm is past float32's range, and small limits, each value against
float64.

Tolerance, relative to each value: the norm's error (a thread's 32 squares of a tile: ten
roundings of 2^-24, half of them after the root, and the root's own: 3.6e-7; 6e-7 is
documented), the factor's rounding and the product's, 1.2e-7: 8e-7, and the output type's
rounding (bf16 2^-8).  What is below a value's own precision: a factor below 2^-252 is held as a
subnormal times 2^-126, off by 2^-150 * 2^-126, times the largest gradient 2^128: 2^-148, and a
result below 2^-126 is rounded to a multiple of 2^-149 (bf16 2^-133)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
REL = {torch.float32: 8e-7, torch.bfloat16: 2.0 ** -8 + 8e-7}
ABS = {torch.float32: 2.0 ** -148 + 2.0 ** -150, torch.bfloat16: 2.0 ** -134 + 2.0 ** -148}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _gradients(dtype, size, shapes, at=0, seed=0):
    """Numbers of 0.1 to 1 times `size`, of both signs; `at`: where in a buffer each begins."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n in shapes:
        u = torch.rand(n + at, generator=g, device="cuda", dtype=torch.float64) * 0.9 + 0.1
        sign = torch.randint(0, 2, (n + at,), generator=g, device="cuda") * 2 - 1
        out.append((u * sign * size).to(DT[dtype])[at:])
    return out


# one cluster; two launches; and outputs whose boundaries are not the input's
FORMS = {"cluster": ([9000, 33, 8193], 0), "two launches": ([500000, 77], 0), "apart": ([9000, 33, 24571], 3),
         "apart, two launches": ([500001, 9], 5)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("size,limits", [(3e38, (1e38, 1e30, 20.0, 1.0, 1e-3, 1e-5, 1e-20, 1e-30, 1e-38, 2.0 ** -149)),
                                         (1e36, (1.0, 1e-3, 1e-10)), (1e18, (1.0, 1e-18, 3e-20, 1e-21, 1e-30)),
                                         (1e12, (1e-23, 1e-26, 1e-30)), (1.0, (1e-36, 1e-38, 1e-40))])
def test_factors_below_the_normal_range(form, dtype, out, size, limits):
    shapes, at = FORMS[form]
    grads = _gradients(dtype, size, shapes)
    before = [g.clone() for g in grads]
    for limit in limits:
        limit = float(np.float32(limit))
        ref_norm, ref = block.clip([g.double().cpu().numpy() for g in before], limit)
        outs = [torch.full((g.numel() + at,), float("nan"), device="cuda", dtype=DT[out])[at:] for g in grads]
        norm = gdn.gdn_clip_grads(grads, limit, out=outs)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        if ref_norm > torch.finfo(torch.float32).max:
            assert float(norm) == float("inf")
        else:
            assert abs(float(norm) - ref_norm) <= 6e-7 * ref_norm
        results = [outs]
        if dtype == out:
            mine = [b.clone() for b in before]
            gdn.gdn_clip_grads(mine, limit)
            torch.cuda.synchronize()
            results.append(mine)
        for got in results:
            for o, r in zip(got, ref):
                x = o.double().cpu().numpy()
                off = np.abs(x - r)
                assert (off <= REL[o.dtype] * np.abs(r) + ABS[o.dtype]).all(), (limit, float((off / np.abs(r)).max()))


def test_a_limit_of_zero():
    for size in (1.0, 3e38):
        grads = _gradients("f32", size, [9000])
        gdn.gdn_clip_grads(grads, 0.0)
        torch.cuda.synchronize()
        assert not grads[0].any()
