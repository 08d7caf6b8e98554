"""GPU test of the 8-bit norm's numbers (gdn_add_norm_quant) against the exact quotient 448 t / max|t|,
t = (x + residual) weight, of every element: the nearest e4m3 number, ties to even.

Of these bf16 inputs 448 t has at most 46 bits (8 + 26 of a sum whose numbers lie between 2^-24 and
2^4, 8 of the weight, 3 of 448), and a middle between two e4m3 numbers (5 bits) times max|t| as
many, so that float64 compares them exactly.  Where float32 does not hold max|t| itself (which is
documented for bf16) a quotient within 2^-24 of a middle may fall on either side, and so may one
below 2^-6, where e4m3's steps are coarse, within 8 of float32's last bits, 2^-20."""
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _grid():
    """e4m3's numbers from 0 to 448 by their codes."""
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().cuda()


@pytest.mark.parametrize("rows,D,group", [(256, 2048, 0), (999, 4096, 128), (400, 768, 64), (801, 2304, 32), (7, 264, 0), (1, 8192, 128)])
@pytest.mark.parametrize("ones", [False, True])
def test_every_number_is_the_nearest(rows, D, group, ones):
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    x = torch.randn(rows, D, generator=g, device="cuda").bfloat16()
    res = (torch.randn(rows, D, generator=g, device="cuda") * 3).bfloat16()
    x, res = (torch.where(t.abs() < 2.0 ** -16, 0, t) for t in (x, res))
    w = torch.ones(D, device="cuda").bfloat16() if ones else (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    y, scales, _ = gdn.gdn_add_norm_quant(x, res, w, group=group)
    torch.cuda.synchronize()
    t = (x.double() + res.double()) * w.double()
    most = t.unflatten(-1, (-1, group or D)).abs().amax(-1, keepdim=True).expand(rows, -1, group or D).flatten(-2)
    a = 448 * t.abs()
    code = y.view(torch.uint8)
    assert ((code >> 7 == 1) == (t < 0))[t != 0].all()
    code = (code & 127).long()
    assert int(code.max()) == 126  # every group's largest is 448
    grid = _grid()
    even = code % 2 == 0
    rounded = most.float().double() != most
    below = torch.where(code > 0, (grid[code] + grid[(code - 1).clamp(min=0)]) / 2, -1.0)
    above = torch.where(code < 126, (grid[code] + grid[(code + 1).clamp(max=126)]) / 2, 1e9)
    for middle, side in ((below, 1.0), (above, -1.0)):
        d, b = side * (a - middle * most), middle.abs() * most
        slack = torch.where(middle < 2.0 ** -6, 2.0 ** -20, torch.where(rounded, 2.0 ** -24, 0.0)) * b
        assert ((d > 0) | ((d == 0) & even) | (d >= -slack) & (slack > 0)).all()
    if not group:
        r = ((x.double() + res.double()).square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        ref = most[:, :1] * r / 448
        assert ((scales.double() - ref).abs() <= 1e-6 * ref).all()
