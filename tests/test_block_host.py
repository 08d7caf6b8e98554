"""Host-side tests of the entry points around the layer (no GPU needed): sizes, and the refusal
of bad arguments with the right status before any launch.  No call here is valid but the
empty ones: the addresses are not memory."""
import ctypes

import pytest

FAKE = 1 << 40  # a 16-byte aligned address that is never dereferenced
INVALID, UNSUP, WS = 1, 2, 3
GAP = 1 << 34


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_19_gb300 import _build, gdn

    _build.build()
    return gdn


def _call(lib, fn, p, names, sized=None, first=(), **over):
    args = {n: FAKE + i * GAP for i, n in enumerate(names)}
    args.update(over)
    vp = ctypes.c_void_p
    extra = [sized] if sized is not None else []
    return getattr(lib.load_library(), fn)(ctypes.byref(p), *first, *[vp(args[n]) for n in names], *extra, vp(None))


# ------------------------------------------------------------ rotation by axes

ROPE_FWD = ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "q_out", "k_out", "workspace")
ROPE_BWD = ROPE_FWD[:7] + ("dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight", "workspace")


def _axes(lib, sections=(8, 12, 12), alternating=0, axes=None, B=2, T=1000, D=128, R=64, rows=1000, dtype=1):
    rope = lib.gdn_rope_problem(B, T, 4, 2, D, R, rows, 0, 0, 1e-6, 0, dtype)
    return lib.gdn_rope_axes_problem(rope, len(sections) if axes is None else axes, alternating,
                                     (ctypes.c_int32 * 4)(*sections[:4]))


def test_axes_refused(lib):
    both = lambda p, **o: {_call(lib, "gdn_qk_norm_rope_axes_fwd", p, ROPE_FWD, sized=1 << 40, **o),  # noqa: E731
                           _call(lib, "gdn_qk_norm_rope_axes_bwd", p, ROPE_BWD, sized=1 << 40, **o)}
    for kw, status, word in ((dict(axes=0), UNSUP, "axes=0"), (dict(axes=5), UNSUP, "axes=5"),
                             (dict(sections=(8, 12, 11)), INVALID, "sum"), (dict(sections=(40, -4, -4)), INVALID, "sections[0]"),
                             (dict(sections=(33, -1)), INVALID, "sections[0]"), (dict(sections=(32, -1, 1)), INVALID, "sections[1]"),
                             (dict(sections=(8, 12, 12), axes=2), INVALID, "sum"),
                             (dict(sections=(2, 15, 15), alternating=1), INVALID, "alternating"),
                             (dict(sections=(16, 16), R=96, D=64), INVALID, "sum"), (dict(sections=(48,), R=96, D=64), INVALID, "exceeds"),
                             (dict(sections=(12,), R=24), UNSUP, "R=24"), (dict(sections=(150,), R=300), UNSUP, "R=300"),
                             (dict(dtype=3), UNSUP, "dtype")):
        p = _axes(lib, **kw)
        assert both(p) == {status}, kw
        assert word in lib.gdn_last_error(), (kw, lib.gdn_last_error())
    ok = _axes(lib)
    for n in ("q", "k_weight", "cos", "sin", "positions"):
        assert both(ok, **{n: None}) == {INVALID}, n
        assert n in lib.gdn_last_error()
    assert both(ok, positions=FAKE + 2) == {INVALID}
    assert _call(lib, "gdn_qk_norm_rope_axes_fwd", ok, ROPE_FWD, sized=0, k_out=FAKE + 16) == INVALID
    # pairs that are copied one by one, of many tokens: their angles are gathered first
    turns = _axes(lib, sections=(12, 10, 10), alternating=1, T=10000)
    need = lib.load_library().gdn_qk_norm_rope_axes_fwd_workspace_bytes
    assert need(ctypes.byref(ok)) == 0 and need(ctypes.byref(_axes(lib, sections=(12, 10, 10), alternating=1, T=10))) == 0
    assert need(ctypes.byref(turns)) == 2 * 10000 * 64 * 4
    assert _call(lib, "gdn_qk_norm_rope_axes_fwd", turns, ROPE_FWD, sized=1000) == WS
    assert _call(lib, "gdn_qk_norm_rope_axes_fwd", turns, ROPE_FWD, sized=1 << 40, workspace=None) == INVALID
    assert _call(lib, "gdn_qk_norm_rope_axes_fwd", turns, ROPE_FWD, sized=1 << 40, workspace=FAKE + GAP) == INVALID
    assert _call(lib, "gdn_qk_norm_rope_axes_bwd", ok, ROPE_BWD, sized=16) == WS
    need = lib.load_library().gdn_qk_norm_rope_axes_bwd_workspace_bytes
    assert need(ctypes.byref(ok)) > 0 and need(ctypes.byref(_axes(lib, T=10))) == 0  # few tokens: one cluster
    assert need(ctypes.byref(_axes(lib, axes=5))) == 0
    assert lib.load_library().gdn_qk_norm_rope_axes_fwd(None, *[None] * 10, 0, None) == INVALID
    # nothing to do: nothing is needed
    assert _call(lib, "gdn_qk_norm_rope_axes_fwd", _axes(lib, T=0), ROPE_FWD, sized=0, q=None, k=None, positions=None, q_out=None,
                 k_out=None) == 0


# ------------------------------------------------------------- residual norm

FWD = ("x", "residual", "weight", "h", "y")
QUANT = ("x", "residual", "weight", "h", "y", "scales")
BWD = ("h", "weight", "dy", "dh", "dx", "d_residual", "dweight", "workspace")


def _norm(lib, rows=10000, D=512, sx=0, ss=0, eps=1e-6, dtype=1, stream=1):
    return lib.gdn_add_norm_problem(rows, D, sx, ss, eps, dtype, stream)


def _fwd(lib, p, **over):
    return _call(lib, "gdn_add_norm_fwd", p, FWD, **over)


def _quant(lib, p, group=0, **over):
    return _call(lib, "gdn_add_norm_quant", p, QUANT, first=(group,), **over)


def _bwd(lib, p, sized=1 << 40, **over):
    return _call(lib, "gdn_add_norm_bwd", p, BWD, sized=sized, **{**({} if p.dtype != p.stream_dtype else dict(d_residual=None)), **over})


def test_add_norm_problems_refused(lib):
    for kw, status, word in ((dict(rows=-1), INVALID, "negative"), (dict(rows=(1 << 33) + 1), UNSUP, "2^33"),
                             (dict(D=0), UNSUP, "D=0"), (dict(D=12), UNSUP, "multiple of 8"), (dict(D=8200), UNSUP, "8192"),
                             (dict(D=6, dtype=0, stream=0), UNSUP, "multiple of 4"), (dict(D=12, dtype=1, stream=0), UNSUP, "of 8"),
                             (dict(dtype=2), UNSUP, "dtype 2"), (dict(stream=-1), UNSUP, "dtype -1"),
                             (dict(dtype=0, stream=1), UNSUP, "bf16 residual stream"), (dict(eps=-1.0), INVALID, "eps"),
                             (dict(eps=float("nan")), INVALID, "eps"), (dict(sx=504), INVALID, "x_stride"),
                             (dict(sx=516), INVALID, "16 bytes"), (dict(ss=-512), INVALID, "stream_stride"),
                             (dict(rows=1 << 30, sx=1 << 40), UNSUP, "2^58")):
        p = _norm(lib, **kw)
        for call in (_fwd, _quant, _bwd):
            assert call(lib, p) == status, kw
            assert word in lib.gdn_last_error(), (kw, lib.gdn_last_error())
        assert lib.load_library().gdn_add_norm_bwd_workspace_bytes(ctypes.byref(p)) == 0
    for group in (-1, 1, 16, 96, 256):
        assert _quant(lib, _norm(lib, D=768), group) == UNSUP
        assert "group" in lib.gdn_last_error()
    assert _quant(lib, _norm(lib, D=1000), 64) == UNSUP  # does not divide
    assert _bwd(lib, _norm(lib), sized=64) == WS
    need = lib.load_library().gdn_add_norm_bwd_workspace_bytes
    assert need(ctypes.byref(_norm(lib))) > 0 and need(ctypes.byref(_norm(lib, rows=40))) == 0  # few rows: one cluster


def test_add_norm_pointers_refused(lib):
    p = _norm(lib)
    for call, names in ((_fwd, ("x", "weight", "y")), (_quant, ("x", "weight", "y", "scales")),
                        (_bwd, ("h", "weight", "dy", "dx", "dweight", "workspace"))):
        for n in names:
            assert call(lib, p, **{n: None}) == INVALID, n
            assert n in lib.gdn_last_error()
            assert call(lib, p, **{n: FAKE + 20 * GAP + 8}) == INVALID, n
            assert "aligned" in lib.gdn_last_error()
    for call, out, on in ((_fwd, "y", FAKE), (_fwd, "h", FAKE + 64), (_quant, "y", FAKE + 3 * GAP), (_quant, "scales", FAKE + 2 * GAP),
                          (_fwd, "h", FAKE + GAP + 16),  # a part of the residual, not the residual
                          (_bwd, "dx", FAKE + 2 * GAP), (_bwd, "dx", FAKE + 3 * GAP), (_bwd, "dweight", FAKE + GAP)):
        assert call(lib, p, **{out: on}) == INVALID, (call, out)
        assert "overlap" in lib.gdn_last_error()
    # h over a residual that is not dense
    assert _fwd(lib, _norm(lib, ss=1024), h=FAKE + GAP) == INVALID
    assert "dense" in lib.gdn_last_error()
    # without a residual there is no sum to keep, and no type of one
    assert _fwd(lib, p, residual=None) == INVALID
    assert _fwd(lib, _norm(lib, stream=0), residual=None, h=None) == INVALID
    # one gradient where the types agree, two where they do not
    assert _bwd(lib, p, d_residual=FAKE + 9 * GAP) == INVALID
    assert "both" in lib.gdn_last_error()
    assert _bwd(lib, _norm(lib, stream=0), d_residual=None) == INVALID
    assert _fwd(lib, _norm(lib, rows=0), x=None, residual=None, h=None, y=None) == 0
    assert lib.load_library().gdn_add_norm_fwd(None, *[None] * 6) == INVALID


# --------------------------------------------------------------- gradients

def _grads(lib, *rows):
    return (lib.gdn_grad * max(1, len(rows)))(*[lib.gdn_grad(*r) for r in rows])


def _clip(lib, rows, count=None, max_norm=1.0, norm=FAKE + 90 * GAP, ws=FAKE + 91 * GAP, size=1 << 30):
    vp = ctypes.c_void_p
    return lib.load_library().gdn_clip_grads(_grads(lib, *rows), len(rows) if count is None else count, max_norm, vp(norm),
                                             vp(ws), size, vp(None))


def _length(lib, rows, count=None, norm=FAKE + 90 * GAP, ws=FAKE + 91 * GAP, size=1 << 30):
    vp = ctypes.c_void_p
    return lib.load_library().gdn_grad_norm(_grads(lib, *rows), len(rows) if count is None else count, vp(norm), vp(ws), size,
                                            vp(None))


def test_grads_refused(lib):
    A, B, C = FAKE, FAKE + GAP, FAKE + 2 * GAP
    ok = (A, A, 1 << 22, 0, 0)  # more than one cluster takes: with a workspace
    for call in (_clip, _length):
        for row, status, word in (((A, A, -1, 0, 0), INVALID, "negative"), ((A, A, (1 << 43) + 1, 0, 0), UNSUP, "2^43"),
                                  ((A, A, 8, 2, 0), UNSUP, "dtype 2"), ((None, None, 8, 0, 0), INVALID, "NULL"),
                                  ((A + 2, A + 2, 8, 0, 0), INVALID, "aligned"), ((A + 1, A + 1, 8, 1, 1), INVALID, "aligned")):
            assert call(lib, [row]) == status, row
            assert word in lib.gdn_last_error()
            assert call(lib, [(B, B, 5, 0, 0), row]) == status, row
        for kw, status in ((dict(norm=A + 8), INVALID), (dict(ws=A + 16), INVALID), (dict(norm=A + 6 + GAP), INVALID),
                           (dict(ws=None), INVALID), (dict(ws=C + 8), INVALID), (dict(size=8), WS), (dict(count=-1), INVALID),
                           (dict(count=(1 << 20) + 1), UNSUP), (dict(norm=FAKE + 91 * GAP), INVALID)):
            assert call(lib, [ok], **kw) == status, kw
        # more elements together than tiles can be counted
        big = [(FAKE + (i << 45), FAKE + (i << 45), 1 << 42, 1, 1) for i in range(5)]
        assert call(lib, big) == UNSUP
    assert _length(lib, [ok], norm=None) == INVALID
    for row in ((A, None, 8, 0, 0), (A, B + 2, 8, 0, 0), (A, A, 8, 0, 1)):
        assert _clip(lib, [row]) == INVALID, row
    assert _clip(lib, [(A, B, 8, 0, 5)]) == UNSUP
    # outputs on one another, on another gradient, or on a part of their own
    for rows in ([ok, ok], [(A, C, 1000, 0, 0), (B, C + 3996, 1000, 0, 0)], [(A, B, 1000, 0, 0), (B, C, 1000, 0, 0)],
                 [(A, A + 16, 1 << 22, 0, 0)], [(A, C, 1000, 0, 1), (B, C + 1998, 1000, 0, 1)],
                 [(A, B, 1 << 20, 1, 1), (C, C, 9, 0, 0), (B + 1024, B + 1024, 4, 1, 1)]):
        assert _clip(lib, rows) == INVALID, rows
        assert "overlaps" in lib.gdn_last_error()
    for m in (-1.0, float("nan"), -float("inf")):
        assert _clip(lib, [ok], max_norm=m) == INVALID
        assert "max_norm" in lib.gdn_last_error()
    h = lib.load_library()
    assert h.gdn_clip_grads(None, 3, 1.0, None, None, 0, None) == INVALID
    size = lambda *rows, **kw: h.gdn_grad_workspace_bytes(_grads(lib, *rows), kw.get("count", len(rows)))  # noqa: E731
    assert size(ok, count=-1) == 0 and size() == 0 and h.gdn_grad_workspace_bytes(None, 3) == 0
    assert size((A, A, 1000, 0, 0)) == 0 and 0 < size(ok) == size(ok, ok) < size(*[ok] * 5000)


# -------------------------------------------------------------- state cache

STORE = ("states", "slot", "cache", "scales")
LOAD = ("cache", "scales", "slot", "states")


def _cache(lib, B=4, H=3, K=64, V=32, slots=9):
    return lib.gdn_state_cache_problem(B, H, K, V, slots)


def test_state_cache_refused(lib):
    calls = lambda p, **o: [_call(lib, "gdn_state_store", p, STORE, **o), _call(lib, "gdn_state_load", p, LOAD, **o)]  # noqa: E731
    for kw, status, word in ((dict(B=-1), INVALID, "negative"), (dict(H=-1), INVALID, "negative"), (dict(K=24), UNSUP, "K=24"),
                             (dict(V=256), UNSUP, "V=256"), (dict(slots=-1), INVALID, "slots"), (dict(slots=1 << 31), UNSUP, "slots"),
                             (dict(B=70000), UNSUP, "B=70000"), (dict(B=5000, H=5000), UNSUP, "2^24")):
        assert calls(_cache(lib, **kw)) == [status] * 2, kw
        assert word in lib.gdn_last_error()
    p = _cache(lib)
    for n in STORE:
        assert calls(p, **{n: None}) == [INVALID] * 2, n
        assert n in lib.gdn_last_error()
        assert calls(p, **{n: FAKE + 30 * GAP + 2}) == [INVALID] * 2, n
    for fn, names, out, on in (("gdn_state_store", STORE, "cache", FAKE + 64), ("gdn_state_store", STORE, "scales", FAKE + 2 * GAP),
                               ("gdn_state_store", STORE, "slot", FAKE + 3 * GAP + 4), ("gdn_state_load", LOAD, "states", FAKE + 16),
                               ("gdn_state_load", LOAD, "states", FAKE + GAP), ("gdn_state_load", LOAD, "slot", FAKE + 3 * GAP)):
        assert _call(lib, fn, p, names, **{out: on}) == INVALID, (fn, out)
        assert "overlap" in lib.gdn_last_error()
    assert calls(_cache(lib, B=0), states=None, slot=None) == [0, 0]
    h = lib.load_library()
    assert h.gdn_state_store(None, *[None] * 5) == INVALID and h.gdn_state_load(None, *[None] * 5) == INVALID
