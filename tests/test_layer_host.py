"""Host-side tests of the linear-attention layer's entry points (no GPU needed): sizes,
and the refusal of bad arguments with the right status before any launch."""
import ctypes

import pytest

FAKE = 1 << 40  # a 16-byte aligned address that is never dereferenced
INVALID, UNSUP, WS = 1, 2, 3
GAP = 1 << 32


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_19_gb300 import _build, gdn

    _build.build()
    return gdn


def _call(lib, fn, p, names, nulls=(), sized=None, **over):
    args = {n: None if n in nulls else FAKE + i * GAP for i, n in enumerate(names)}
    args.update(over)
    vp = ctypes.c_void_p
    extra = [sized] if sized is not None else []
    return getattr(lib.load_library(), fn)(ctypes.byref(p), *[vp(args[n]) for n in names], *extra, vp(None))


LA_FWD = ("q", "k", "v", "log_decay", "initial_state", "o", "final_state", "saved", "workspace")
LA_BWD = ("q", "k", "v", "log_decay", "initial_state", "saved", "d_o", "d_final_state", "dq", "dk", "dv",
          "d_initial_state", "workspace")
LA_DEC = ("q", "k", "v", "log_decay", "state", "o")


def _la(lib, B=2, T=100, H=3, K=64, V=32, sq=0, sk=0, sv=0, dtype=1):
    return lib.gdn_la_problem(B, T, H, K, V, sq, sk, sv, dtype)


def _la_calls(lib, p, size=1 << 40, **over):
    out = [_call(lib, "gdn_la_fwd", p, LA_FWD, sized=size, **{k: v for k, v in over.items() if k in LA_FWD}),
           _call(lib, "gdn_la_bwd", p, LA_BWD, sized=size, **{k: v for k, v in over.items() if k in LA_BWD}),
           _call(lib, "gdn_la_decode", p, LA_DEC, **{k: v for k, v in over.items() if k in LA_DEC})]
    return out


def test_la_problems_refused(lib):
    for kw, status, word in ((dict(K=24), UNSUP, "K=24"), (dict(V=256), UNSUP, "V=256"), (dict(dtype=2), UNSUP, "dtype"),
                             (dict(B=-1), INVALID, "negative"), (dict(T=-5), INVALID, "negative"),
                             (dict(B=70000), UNSUP, "B=70000"), (dict(B=5000, H=5000), UNSUP, "2^24"),
                             (dict(T=(1 << 30) + 1), UNSUP, "2^30"), (dict(sq=100), INVALID, "q_stride"),
                             (dict(sk=3 * 64 + 4), INVALID, "k_stride"), (dict(sv=-96), INVALID, "v_stride")):
        p = _la(lib, **kw)
        for st in _la_calls(lib, p):
            assert st == status, kw
            assert word in lib.gdn_last_error()
        h = lib.load_library()
        for fn in ("gdn_la_fwd_workspace_bytes", "gdn_la_bwd_workspace_bytes", "gdn_la_saved_bytes"):
            assert getattr(h, fn)(ctypes.byref(p)) == 0
    for st in (_call(lib, "gdn_la_fwd", _la(lib), LA_FWD, sized=0), _call(lib, "gdn_la_bwd", _la(lib), LA_BWD, sized=8)):
        assert st == WS
    assert lib.load_library().gdn_la_fwd(None, *[None] * 9, 0, None) == INVALID


def test_la_pointers_refused(lib):
    p = _la(lib)
    for n in ("q", "k", "v", "log_decay"):
        assert _la_calls(lib, p, **{n: None}) == [INVALID] * 3, n
        assert n in lib.gdn_last_error()
        assert _la_calls(lib, p, **{n: FAKE + 40 * GAP + 2}) == [INVALID] * 3, n
    for fn, names, out in (("gdn_la_fwd", LA_FWD, "o"), ("gdn_la_bwd", LA_BWD, "dk"), ("gdn_la_decode", LA_DEC, "state")):
        size = None if fn == "gdn_la_decode" else 1 << 40
        assert _call(lib, fn, p, names, sized=size, **{out: None}) == INVALID
        assert _call(lib, fn, p, names, sized=size, **{out: FAKE + 64}) == INVALID  # on q
        assert "overlaps" in lib.gdn_last_error()
    # an output behind the dense end of a strided q, but inside its rows
    wide = _la(lib, sq=4096)
    assert _call(lib, "gdn_la_fwd", wide, LA_FWD, sized=1 << 40, o=FAKE + 100 * 4096) == INVALID
    # the final state may be the initial state itself, not a part of it
    assert _call(lib, "gdn_la_fwd", p, LA_FWD, sized=1 << 40, final_state=FAKE + 4 * GAP + 16) == INVALID


def test_la_sizes(lib):
    h = lib.load_library()
    one = _la(lib, T=128)
    assert h.gdn_la_saved_bytes(ctypes.byref(one)) == 0  # one tile: nothing to pass between segments
    long = _la(lib, B=1, T=1 << 20, H=1, K=128, V=128)
    saved = h.gdn_la_saved_bytes(ctypes.byref(long))
    assert saved > 0 and saved % (128 * 128 * 4) == 0
    assert h.gdn_la_bwd_workspace_bytes(ctypes.byref(long)) > h.gdn_la_fwd_workspace_bytes(ctypes.byref(long)) > saved
    many = _la(lib, B=1000, T=1 << 20, H=8, K=128, V=128)  # more streams than the GPU has SMs
    assert h.gdn_la_saved_bytes(ctypes.byref(many)) == 0


ROPE_FWD = ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "q_out", "k_out")
ROPE_BWD = ROPE_FWD[:7] + ("dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight", "workspace")
GATED_FWD = ("x", "gate", "weight", "y")
GATED_BWD = ("x", "gate", "weight", "dy", "dx", "dgate", "dweight", "workspace")


def _rope(lib, B=2, T=10, Hq=4, Hk=2, D=128, R=64, rows=10, sq=0, sk=0, eps=1e-6, inter=0, dtype=1):
    return lib.gdn_rope_problem(B, T, Hq, Hk, D, R, rows, sq, sk, eps, inter, dtype)


def _gated(lib, B=2, T=10, H=4, D=128, sx=0, sg=0, eps=1e-6, dtype=1):
    return lib.gdn_gated_norm_problem(B, T, H, D, sx, sg, eps, dtype)


def test_row_problems_refused(lib):
    both = lambda p: (_call(lib, "gdn_qk_norm_rope_fwd", p, ROPE_FWD),  # noqa: E731
                      _call(lib, "gdn_qk_norm_rope_bwd", p, ROPE_BWD, sized=1 << 40))
    for kw, status in ((dict(D=24), UNSUP), (dict(D=272), UNSUP), (dict(D=0, R=0), UNSUP), (dict(R=24), UNSUP),
                       (dict(D=64, R=128), INVALID), (dict(rows=-1), INVALID), (dict(eps=float("nan")), INVALID),
                       (dict(sq=256), INVALID), (dict(sk=257), INVALID), (dict(Hk=-1), INVALID), (dict(dtype=7), UNSUP),
                       (dict(B=60000, T=1 << 20), UNSUP)):
        assert set(both(_rope(lib, **kw))) == {status}, kw
    for fn, names, extra in (("gdn_gated_norm_fwd", GATED_FWD, None), ("gdn_gated_norm_bwd", GATED_BWD, 1 << 40)):
        for kw, status in ((dict(D=8), UNSUP), (dict(D=512), UNSUP), (dict(eps=-1.0), INVALID), (dict(sx=8), INVALID),
                           (dict(sg=4 * 128 + 4), INVALID), (dict(H=-1), INVALID), (dict(dtype=-1), UNSUP)):
            assert _call(lib, fn, _gated(lib, **kw), names, sized=extra) == status, kw
        for n in names[:3]:
            assert _call(lib, fn, _gated(lib), names, sized=extra, **{n: None}) == INVALID
            assert _call(lib, fn, _gated(lib), names, sized=extra, **{n: FAKE + 50 * GAP + 8}) == INVALID
        assert _call(lib, fn, _gated(lib), names, sized=extra, **{"y" if extra is None else "dgate": FAKE + GAP}) == INVALID
        assert "overlaps" in lib.gdn_last_error()


def test_row_pointers_refused(lib):
    for fn, names, extra, out in (("gdn_qk_norm_rope_fwd", ROPE_FWD, None, "k_out"),
                                  ("gdn_qk_norm_rope_bwd", ROPE_BWD, 1 << 40, "dk")):
        for n in ("q", "k", "q_weight", "k_weight", "cos", "sin", out):
            assert _call(lib, fn, _rope(lib), names, sized=extra, **{n: None}) == INVALID, n
            assert n in lib.gdn_last_error()
        assert _call(lib, fn, _rope(lib), names, sized=extra, **{out: FAKE}) == INVALID
        assert "overlaps" in lib.gdn_last_error()
        # without positions every token needs a row of the tables
        assert _call(lib, fn, _rope(lib, rows=9), names, nulls=("positions",), sized=extra) == INVALID
        assert "table_rows" in lib.gdn_last_error()
    assert _call(lib, "gdn_qk_norm_rope_bwd", _rope(lib), ROPE_BWD, sized=16) == WS
    assert _call(lib, "gdn_gated_norm_bwd", _gated(lib), GATED_BWD, sized=16) == WS
    h = lib.load_library()
    assert h.gdn_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(_rope(lib))) > 0
    assert h.gdn_gated_norm_bwd_workspace_bytes(ctypes.byref(_gated(lib, D=8))) == 0


def test_empty_problems_need_nothing(lib):
    p = _la(lib, B=0)
    assert _call(lib, "gdn_la_fwd", p, LA_FWD, nulls=LA_FWD[:-1], sized=1 << 20) == 0
    assert _call(lib, "gdn_la_decode", p, LA_DEC, nulls=LA_DEC) == 0
    assert _call(lib, "gdn_qk_norm_rope_fwd", _rope(lib, T=0), ROPE_FWD, nulls=ROPE_FWD[:2] + ROPE_FWD[4:]) == 0
    assert _call(lib, "gdn_gated_norm_fwd", _gated(lib, H=0), GATED_FWD, nulls=("x", "gate", "y")) == 0
