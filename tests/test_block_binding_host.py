"""Host-side tests of the C++ binding of the calls around the layer (no GPU needed): the device
they run on, and what they say where the library is older."""
import os
import subprocess
import sys

import pytest
from test_layer_binding_host import FAKE, ROOT, RUN

MORE = r"""
extern "C" {
SIZE(gdn_add_norm_bwd_workspace_bytes) SIZE(gdn_grad_workspace_bytes) SIZE(gdn_qk_norm_rope_axes_bwd_workspace_bytes)
SIZE(gdn_qk_norm_rope_axes_fwd_workspace_bytes)
CALL(gdn_qk_norm_rope_axes_fwd) CALL(gdn_qk_norm_rope_axes_bwd) CALL(gdn_add_norm_fwd) CALL(gdn_add_norm_quant)
CALL(gdn_add_norm_bwd) CALL(gdn_grad_norm) CALL(gdn_clip_grads) CALL(gdn_state_store) CALL(gdn_state_load)
}
"""
CALLS = r"""
pos = tensor(2, B, T, code=0)
y8, scales = tensor(B, T, H, K, code=1, bits=8).view(torch.float8_e4m3fn), tensor(B, T, H, 1)
cache, steps, slots = tensor(9, H, V, K, code=0, bits=8), tensor(9, H, V), tensor(B, code=0)
one = tensor(1)
calls = {
    "rope_axes_fwd": lambda: gdn.gdn_qk_norm_rope_axes_fwd(q, q, w, w, cos, cos, pos, (8, 8), q_out=q, k_out=q),
    "rope_axes_bwd": lambda: gdn.gdn_qk_norm_rope_axes_bwd(q, q, w, w, cos, cos, pos, [8, 8], q, q, grads=(q, q, w, w), workspace=ws),
    "add_norm_fwd": lambda: gdn.gdn_add_norm_fwd(q, q, w, h=q, y=q),
    "add_norm_quant": lambda: gdn.gdn_add_norm_quant(q, q, w, h=q, y=y8, scales=scales),
    "add_norm_bwd": lambda: gdn.gdn_add_norm_bwd(q, w, q, q, grads=(q, None, w), workspace=ws),
    "grad_norm": lambda: gdn.gdn_grad_norm([q, None, w], norm=one, workspace=ws),
    "clip_grads": lambda: gdn.gdn_clip_grads([q, w], 1.0, norm=one, workspace=ws),
    "state_store": lambda: gdn.gdn_state_store(state, slots, cache, steps),
    "state_load": lambda: gdn.gdn_state_load(cache, steps, slots, states=state),
}
"""


@pytest.fixture(scope="module")
def built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()


def _compile(text, path):
    import torch
    from torch.utils import cpp_extension

    src = path.with_suffix(".cpp")
    src.write_text(text)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", *(f for d in cpp_extension.include_paths() + [cuda]
                                                                    for f in ("-isystem", d)),
                    str(src), "-o", str(path), "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10"], check=True)


def test_calls_run_on_their_tensors_device(built, tmp_path):
    lib = tmp_path / "fake.so"
    _compile(FAKE + MORE, lib)
    head, tail = RUN.split("calls = {", 1)
    run = head + CALLS + tail[tail.index("\n}\n") + 3:]
    # an integer tensor's type in DLPack is code 0, an unsigned one's 1
    r = subprocess.run([sys.executable, "-c", run, str(lib)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr


def test_an_older_library_says_so(built, tmp_path):
    lib = tmp_path / "fake.so"
    _compile(FAKE, lib)
    run = r"""
import sys
from gated_delta_rule_19_gb300 import _layer, gdn
_layer.load(sys.argv[1], gdn.GdnError)
gdn._layer = _layer
for call in (lambda: gdn.gdn_add_norm_fwd(None, None, None), lambda: gdn.gdn_clip_grads([], 1.0), lambda: gdn.gdn_grad_norm([]),
             lambda: gdn.gdn_state_load(None, None, None), lambda: gdn.gdn_qk_norm_rope_axes_fwd(*[None] * 8)):
    try:
        call()
        raise SystemExit("no error")
    except RuntimeError as e:
        assert "build it again" in str(e), e
print("done")
"""
    r = subprocess.run([sys.executable, "-c", run, str(lib)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr
