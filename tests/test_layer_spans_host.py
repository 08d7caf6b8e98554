"""Host-side test (no GPU needed): rows whose span in bytes does not fit 64 bits are refused
before their overlaps are looked at."""
import ctypes

import pytest

UNSUP = 2


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_19_gb300 import _build, gdn

    _build.build()
    return gdn


def _call(gdn, fn, p, pointers, sized):
    vp = ctypes.c_void_p  # aligned, 2^46 bytes apart, never read
    args = [vp((1 << 40) + i * (1 << 46)) for i in range(pointers)] + ([1 << 40] if sized else []) + [vp(None)]
    return getattr(gdn.load_library(), fn)(ctypes.byref(p), *args)


def test_spans_past_64_bits_refused(lib):
    big = 1 << 40  # a stride that is accepted by itself
    la = lambda **s: lib.gdn_la_problem(2, 1 << 30, 3, 64, 32, s.get("q", 0), s.get("k", 0), s.get("v", 0), 1)  # noqa: E731
    for name in ("q", "k", "v"):
        p = la(**{name: big})
        for fn, pointers, sized in (("gdn_la_fwd", 9, True), ("gdn_la_bwd", 13, True), ("gdn_la_decode", 6, False)):
            assert _call(lib, fn, p, pointers, sized) == UNSUP
            assert f"{name}_stride" in lib.gdn_last_error() and "2^58" in lib.gdn_last_error()
        h = lib.load_library()
        for fn in ("gdn_la_fwd_workspace_bytes", "gdn_la_bwd_workspace_bytes", "gdn_la_saved_bytes"):
            assert getattr(h, fn)(ctypes.byref(p)) == 0
    for sq, sk in ((big, 0), (0, big)):
        p = lib.gdn_rope_problem(2, 1 << 25, 3, 3, 64, 0, 0, sq, sk, 1e-6, 0, 1)
        assert _call(lib, "gdn_qk_norm_rope_fwd", p, 9, False) == UNSUP
        assert _call(lib, "gdn_qk_norm_rope_bwd", p, 14, True) == UNSUP
        assert "2^58" in lib.gdn_last_error()
    for sx, sg in ((big, 0), (0, big)):
        p = lib.gdn_gated_norm_problem(2, 1 << 25, 3, 64, sx, sg, 1e-6, 1)
        assert _call(lib, "gdn_gated_norm_fwd", p, 4, False) == UNSUP
        assert _call(lib, "gdn_gated_norm_bwd", p, 8, True) == UNSUP
        assert "2^58" in lib.gdn_last_error()
