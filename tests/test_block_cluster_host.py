"""Host-side tests of the choice between one cluster and two launches (no GPU needed): what a
context cannot place as a cluster takes the two launches, which need a workspace."""
import ctypes

import pytest
from test_block_host import FAKE, GAP, INVALID, ROPE_BWD, WS, _axes, _call, _grads, _norm, lib  # noqa: F401


@pytest.fixture
def limit(lib):  # noqa: F811
    yield lib.gdn_test_set_cluster_limit
    lib.gdn_test_set_cluster_limit(0)


def _needs(lib):  # noqa: F811
    h, ref = lib.load_library(), ctypes.byref
    grads = [(FAKE, FAKE, n * 8192, 0, 0) for n in (3, 24, 48)]
    return {"norm": [h.gdn_add_norm_bwd_workspace_bytes(ref(_norm(lib, rows=r))) for r in (1, 17, 65, 128)],
            "axes": [h.gdn_qk_norm_rope_axes_bwd_workspace_bytes(ref(_axes(lib, B=1, T=t))) for t in (1, 8, 33, 64)],
            "grads": [h.gdn_grad_workspace_bytes(_grads(lib, g), 1) for g in grads]}


def test_what_fits_no_cluster_takes_two_launches(lib, limit):  # noqa: F811
    # 8 rows of 512 bf16 a block; 4 tokens of 4 heads; 3 tiles, of a power of two blocks
    limit(16)
    assert _needs(lib) == {"norm": [0] * 4, "axes": [0] * 4, "grads": [0] * 3}
    for most in (8, 4, 2, 1):
        limit(most)
        need = _needs(lib)
        for what, blocks in (("norm", (1, 3, 9, 16)), ("axes", (1, 2, 9, 16)), ("grads", (1, 8, 16))):
            assert [n == 0 for n in need[what]] == [b <= most for b in blocks], (what, most, need[what])
    # and the call asks for what the query says
    limit(4)
    vp = ctypes.c_void_p
    row = _grads(lib, (FAKE, FAKE, 48 * 8192, 0, 0))
    for call in (lambda size: lib.load_library().gdn_clip_grads(row, 1, 1.0, vp(FAKE + 90 * GAP), vp(FAKE + 91 * GAP), size, None),
                 lambda size: _call(lib, "gdn_qk_norm_rope_axes_bwd", _axes(lib, B=1, T=64), ROPE_BWD, sized=size),
                 lambda size: _call(lib, "gdn_add_norm_bwd", _norm(lib, rows=128), ("h", "weight", "dy", "dh", "dx", "d_residual",
                                                                                 "dweight", "workspace"), sized=size, d_residual=None)):
        assert call(8) == WS, lib.gdn_last_error()


def test_limits_refused(lib, limit):  # noqa: F811
    for bad in (-1, 17):
        with pytest.raises(lib.GdnError):
            limit(bad)
    assert lib.load_library().gdn_test_set_cluster_limit(99) == INVALID
