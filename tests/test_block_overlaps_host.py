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


def test_a_sum_over_a_residual_that_x_lies_over(lib):  # noqa: F811
    """h may be the residual; x at the same address is only the same rows where it has the residual's
    type and stride.  Else rows of h lie over rows of x that are still to be read."""
    at = FAKE + FWD.index("residual") * GAP

    def norm(**kw):
        d = dict(rows=10, D=512, sx=0, ss=0, dtype=1, stream=1)
        d.update(kw)
        return lib.gdn_add_norm_problem(d["rows"], d["D"], d["sx"], d["ss"], 1e-6, d["dtype"], d["stream"])

    def both(p, **over):
        return [_call(lib, "gdn_add_norm_fwd", p, FWD, **over), _call(lib, "gdn_add_norm_quant", p, QUANT, first=(0,), **over)]

    for p in (norm(sx=1024), norm(stream=0), norm(rows=2, sx=1536, stream=0), norm(rows=1, stream=0), norm(rows=2, sx=520)):
        assert both(p, x=at, h=at) == [INVALID] * 2
        assert "overlaps input x" in lib.gdn_last_error(), lib.gdn_last_error()
    # the same rows: each is read before it is written
    for p in (norm(), norm(dtype=0, stream=0), norm(rows=1, sx=1024)):
        assert not set(both(p, x=at, h=at)) & {0, INVALID}
    # the weight there
    assert both(norm(), weight=at, h=at) == [INVALID] * 2
    assert "overlaps input weight" in lib.gdn_last_error()
    # x elsewhere, and a part of the residual
    assert not set(both(norm(), h=at)) & {0, INVALID}
    assert both(norm(), x=at + 512, h=at) == [INVALID] * 2
    # no address is not an address that agrees
    assert both(norm(), x=None, residual=None, h=None) == [INVALID] * 2
    assert both(norm(), x=None, h=at) == [INVALID] * 2


def test_linear_attention_states_over_other_inputs(lib):  # noqa: F811
    """The final state may be the initial one, the initial state's gradient the final state's: that
    allows no other input at their address."""
    p = lib.gdn_la_problem(1, 65536, 4, 128, 128, 0, 0, 0, 1)  # with saved sums
    fwd = ("q", "k", "v", "log_decay", "initial_state", "o", "final_state", "saved", "workspace")
    bwd = ("q", "k", "v", "log_decay", "initial_state", "saved", "d_o", "d_final_state", "dq", "dk", "dv", "d_initial_state", "workspace")
    at = FAKE + 50 * GAP
    for fn, names, pair, others in (("gdn_la_fwd", fwd, ("initial_state", "final_state"), ("q", "k", "v")),
                                    ("gdn_la_bwd", bwd, ("d_final_state", "d_initial_state"), ("q", "v", "d_o", "initial_state", "saved"))):
        same = dict.fromkeys(pair, at)
        assert _call(lib, fn, p, names, sized=1 << 40, **same) not in (0, INVALID), fn
        for n in others:
            assert _call(lib, fn, p, names, sized=1 << 40, **same, **{n: at}) == INVALID, (fn, n)
            assert f"overlaps input {n}" in lib.gdn_last_error(), lib.gdn_last_error()
