"""Host-side tests of the linear-attention layer's C++ binding (no GPU needed): the
device its calls run on, and when it is built."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Stands in for the library and for torch's CUDA device functions, with eight devices: every
# call notes the device that is current.
FAKE = r"""
#include <c10/core/impl/FakeGuardImpl.h>
using Fake = c10::impl::FakeGuardImpl<c10::DeviceType::CUDA>;
static Fake fake;
static int noted = -1, status = 0;
extern "C" {
void use_fake() { c10::impl::device_guard_impl_registry[(size_t)c10::DeviceType::CUDA].store(&fake); }
void set_device(int d) { Fake::setDeviceIndex((c10::DeviceIndex)d); }
int get_device() { return Fake::getDeviceIndex(); }
void set_status(int s) { status = s; }
int take_noted() { const int n = noted; noted = -1; return n; }
const char* gdn_last_error() { return "refused by the test"; }
#define SIZE(name) size_t name() { return 0; }
SIZE(gdn_la_fwd_workspace_bytes) SIZE(gdn_la_saved_bytes) SIZE(gdn_la_bwd_workspace_bytes)
SIZE(gdn_qk_norm_rope_bwd_workspace_bytes) SIZE(gdn_gated_norm_bwd_workspace_bytes)
#define CALL(name) int name() { noted = Fake::getDeviceIndex(); return status; }
CALL(gdn_la_fwd) CALL(gdn_la_bwd) CALL(gdn_la_decode) CALL(gdn_qk_norm_rope_fwd) CALL(gdn_qk_norm_rope_bwd)
CALL(gdn_gated_norm_fwd) CALL(gdn_gated_norm_bwd)
}
"""

RUN = textwrap.dedent(r"""
    import ctypes, sys
    import torch
    from gated_delta_rule_19_gb300 import _layer, gdn

    fake = ctypes.CDLL(sys.argv[1])
    _layer.load(sys.argv[1], gdn.GdnError)
    gdn._layer = _layer
    fake.use_fake()
    torch.cuda.init = torch.cuda._lazy_init = lambda: None

    class Device(ctypes.Structure):
        _fields_ = [("type", ctypes.c_int), ("id", ctypes.c_int)]
    class Type(ctypes.Structure):
        _fields_ = [("code", ctypes.c_uint8), ("bits", ctypes.c_uint8), ("lanes", ctypes.c_uint16)]
    class Managed(ctypes.Structure):  # a DLPack tensor
        _fields_ = [("data", ctypes.c_void_p), ("device", Device), ("ndim", ctypes.c_int), ("dtype", Type),
                    ("shape", ctypes.POINTER(ctypes.c_int64)), ("strides", ctypes.c_void_p),
                    ("offset", ctypes.c_uint64), ("ctx", ctypes.c_void_p), ("deleter", ctypes.c_void_p)]
    capsule = ctypes.pythonapi.PyCapsule_New
    capsule.restype, capsule.argtypes = ctypes.py_object, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p]
    keep = []

    def tensor(*shape, code=2, bits=32):  # float32 on cuda:3, at an address that nothing reads
        sizes = (ctypes.c_int64 * len(shape))(*shape)
        m = Managed(1 << 40, Device(2, 3), len(shape), Type(code, bits, 1), sizes, None, 0, None, None)
        keep.extend((sizes, m))
        return torch.utils.dlpack.from_dlpack(capsule(ctypes.addressof(m), b"dltensor", None))

    B, T, H, K, V = 2, 5, 3, 32, 16
    q, v, ld, state, ws = tensor(B, T, H, K), tensor(B, T, H, V), tensor(H), tensor(B, H, V, K), tensor(8)
    w, cos = tensor(K), tensor(T, K // 2)
    assert q.device == torch.device("cuda:3")
    calls = {
        "la_fwd": lambda: gdn.gdn_la_fwd(q, q, v, ld, state, o=v, final_state=False, workspace=ws),
        "la_bwd": lambda: gdn.gdn_la_bwd(q, q, v, ld, None, v, grads=(q, q, v), d_initial_state=False, workspace=ws),
        "la_decode": lambda: gdn.gdn_la_decode(q, q, v, ld, state, o=v),
        "rope_fwd": lambda: gdn.gdn_qk_norm_rope_fwd(q, q, w, w, cos, cos, q_out=q, k_out=q),
        "rope_bwd": lambda: gdn.gdn_qk_norm_rope_bwd(q, q, w, w, cos, cos, None, q, q, grads=(q, q, w, w), workspace=ws),
        "gated_fwd": lambda: gdn.gdn_gated_norm_fwd(q, q, w, y=q),
        "gated_bwd": lambda: gdn.gdn_gated_norm_bwd(q, q, w, q, grads=(q, q, w), workspace=ws),
    }
    for current in (0, 3):
        for name, call in calls.items():
            fake.set_device(current)
            call()
            noted = fake.take_noted()
            assert noted == 3, f"{name}: ran on device {noted}, its tensors are on 3"
            assert fake.get_device() == current, name
            fake.set_status(1)  # and where the library refuses the call
            try:
                call()
                raise SystemExit("no error")
            except gdn.GdnError:
                pass
            fake.set_status(0)
            assert fake.take_noted() == 3 and fake.get_device() == current, name
    print("done")
""")


@pytest.fixture(scope="module")
def built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()


def test_calls_run_on_their_tensors_device(built, tmp_path):
    import torch
    from torch.utils import cpp_extension

    src, lib = tmp_path / "fake.cpp", tmp_path / "fake.so"
    src.write_text(FAKE)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", *(f for d in cpp_extension.include_paths() + [cuda]
                                                                    for f in ("-isystem", d)),
                    str(src), "-o", str(lib), "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10"],
                   check=True)
    r = subprocess.run([sys.executable, "-c", RUN, str(lib)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr


def test_binding_of_another_torch_or_python_is_rebuilt(built, monkeypatch):
    """Sources that are older do not make a binding current: it belongs to the torch and
    the Python that it was compiled against."""
    from importlib import metadata

    from gated_delta_rule_19_gb300 import _build

    made = []
    monkeypatch.setattr(_build, "build_binding", lambda verbose=False: made.append(1))
    monkeypatch.setattr(_build, "is_stale", lambda: False)
    _build.build()
    assert not made  # as it is, it is current
    version = metadata.version
    with monkeypatch.context() as m:
        m.setattr(metadata, "version", lambda name: "99.0" if name == "torch" else version(name))
        _build.build()
        assert len(made) == 1
    with monkeypatch.context() as m:
        m.setattr(sys, "version", "3.99.0 (another)")
        _build.build()
        assert len(made) == 2
    monkeypatch.setattr(_build, "BINDING_FOR", _build.BINDING_FOR + ".gone")
    _build.build()
    assert len(made) == 3


def test_library_builds_without_the_bindings_headers(built, monkeypatch, tmp_path):
    """A caller of the C ABI needs neither torch's nor Python's C++ headers; the layer's calls
    through gdn.py say what is missing."""
    import sysconfig

    from gated_delta_rule_19_gb300 import _build, gdn

    old = tmp_path / "_layer.so"
    old.write_bytes(b"of another torch")
    monkeypatch.setattr(_build, "BINDING", str(old))
    monkeypatch.setattr(_build, "BINDING_FOR", str(tmp_path / "none.txt"))
    monkeypatch.setattr(_build, "is_stale", lambda: False)
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    with pytest.warns(UserWarning, match="Python.h"):
        assert _build.build() == _build.LIB
    assert not old.exists()
    monkeypatch.setattr(gdn, "_PKG", str(tmp_path))
    monkeypatch.setattr(gdn, "_layer", None)
    with pytest.raises(RuntimeError, match="_layer.so is missing"):
        gdn.gdn_la_decode(None, None, None, None, None)
