"""Host-side tests of overlaps that the calls around the layer refuse (no GPU needed): outputs over
the positions, and a sum over a residual that x lies over too.  Without a GPU a call that passes
the checks fails at its launch, with another status."""
import ctypes

import pytest
import torch
from test_block_host import FAKE, FWD, GAP, INVALID, QUANT, ROPE_BWD, ROPE_FWD, _axes, _call, lib  # noqa: F401

# on a GPU a call that the checks let through would run on addresses that are not memory
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not memory")


def test_outputs_over_the_positions(lib):  # noqa: F811
    p = _axes(lib, B=2, T=1000)
    at = FAKE + ROPE_FWD.index("positions") * GAP
    span = 3 * 2 * 1000 * 4
    for fn, names, outs in (("gdn_qk_norm_rope_axes_fwd", ROPE_FWD, ("q_out", "k_out")),
                            ("gdn_qk_norm_rope_axes_bwd", ROPE_BWD, ("dq", "dk", "dq_weight", "dk_weight", "workspace"))):
        for out in outs:
            for on in (at, at + span - 16):
                assert _call(lib, fn, p, names, sized=1 << 30, **{out: on}) == INVALID, (fn, out)
                assert "overlaps input positions" in lib.gdn_last_error(), lib.gdn_last_error()
            assert _call(lib, fn, p, names, sized=1 << 30, **{out: at + span + 64}) not in (0, INVALID), (fn, out)
    # the gathered angles' memory
    turns = _axes(lib, sections=(12, 10, 10), alternating=1, T=10000)
    assert _call(lib, "gdn_qk_norm_rope_axes_fwd", turns, ROPE_FWD, sized=1 << 40, workspace=at) == INVALID
    # no pairs: no positions are read
    none = _axes(lib, sections=(0, 0), R=0)
    assert _call(lib, "gdn_qk_norm_rope_axes_fwd", none, ROPE_FWD, sized=1 << 30, q_out=at) != INVALID


def test_outputs_over_one_axis_positions(lib):  # noqa: F811
    p = lib.gdn_rope_problem(2, 1000, 4, 2, 128, 64, 1000, 0, 0, 1e-6, 0, 1)
    names = ROPE_FWD[:-1]
    at = FAKE + names.index("positions") * GAP
    for on in (at, at + 2 * 1000 * 4 - 16):
        assert _call(lib, "gdn_qk_norm_rope_fwd", p, names, q_out=on) == INVALID
        assert _call(lib, "gdn_qk_norm_rope_bwd", p, ROPE_BWD, sized=1 << 30, dk=on) == INVALID
        assert "overlaps input positions" in lib.gdn_last_error()
    assert _call(lib, "gdn_qk_norm_rope_fwd", p, names, q_out=at + 2 * 1000 * 4) not in (0, INVALID)
    assert _call(lib, "gdn_qk_norm_rope_fwd", p, names, positions=None) not in (0, INVALID)
