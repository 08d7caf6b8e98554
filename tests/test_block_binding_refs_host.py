"""Host-side test of the C++ binding of the gradients' calls (no GPU needed): a refused call keeps
no reference to what it was given."""
import subprocess
import sys

from test_block_binding_host import MORE, _compile
from test_layer_binding_host import FAKE, ROOT, RUN

CALLS = r"""
one = tensor(1)
half = tensor(B, T, bits=16)
cpu = torch.zeros(5)
lists = {
    "dtype": ([q, half], None), "cpu": ([q, cpu], None), "device": ([cpu], None), "not a tensor": ([q, 3], None),
    "out's length": ([q, w], [q]), "out's entry": ([q, w], [q, 3]), "out's shape": ([q, w], [q, q]), "out's dtype": ([q], [half]),
    "out a tensor": ([q], q), "out no sequence": ([q], 3), "no tensors": ([None], None),
}
kept = []
for name, (grads, out) in lists.items():
    for what, call in (("clip", lambda: gdn.gdn_clip_grads(grads, 1.0, out=out, workspace=ws)),
                       ("norm", lambda: gdn.gdn_grad_norm(grads, workspace=ws))):
        if what == "norm" and out is not None:
            continue
        seen = [x for x in (grads, out) if isinstance(x, list)]
        before = [sys.getrefcount(x) for x in seen]
        for _ in range(5):
            try:
                call()
            except (gdn.GdnError, TypeError):
                continue
            raise SystemExit(f"{name}: no error")
        if [sys.getrefcount(x) for x in seen] != before:
            kept.append(f"{what}, {name}")
if kept:
    raise SystemExit("references kept: " + "; ".join(kept))
fake.set_status(1)  # refused by the library itself
grads, out = [q, w], [q, w]
before = sys.getrefcount(grads), sys.getrefcount(out)
for _ in range(5):
    try:
        gdn.gdn_clip_grads(grads, 1.0, out=out, norm=one, workspace=ws)
    except gdn.GdnError:
        continue
    raise SystemExit("no error")
if (sys.getrefcount(grads), sys.getrefcount(out)) != before:
    raise SystemExit("references kept: the library's refusal")
print("done")
"""


def test_refused_gradients_are_not_kept(tmp_path):
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    lib = tmp_path / "fake.so"
    _compile(FAKE + MORE, lib)
    run = RUN.split("calls = {", 1)[0] + CALLS
    r = subprocess.run([sys.executable, "-c", run, str(lib)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr
