"""Without the extension module of the losses over rows of logits, or with one
that does not load (built against another torch, say), the package imports and
everything else in it works; the losses say what is missing when called."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "fp32_reductions_amd")

CHILD = r"""
import sys
sys.path.insert(0, {root!r})
import fp32_reductions_amd as red
assert red.__file__.startswith({root!r}), red.__file__
assert red.abi_version() == 3 and red.status_str(0)
import torch
x = torch.zeros(4)
try:
    red.sum_f32(x, x[:1])  # its own check of the tensors
except ValueError as e:
    assert "device" in str(e)
for name in ("token_logprob", "token_logprob_grad", "distill_topk", "policy_loss",
             "preference_loss"):
    for t in ("f32", "f16", "bf16"):
        called = "%s_%s" % (name, t)
        f = getattr(red, called)
        assert f.__name__ == called
        for call in (f, lambda *a, **k: red.plan(called, *a, **k)):
            try:
                call(x, x, scale=1.0)
            except ImportError as e:
                assert "_rowloss.so" in str(e) and "build.py" in str(e) and called in str(e), e
            else:
                raise AssertionError(called)
print("imported")
"""


@pytest.mark.parametrize("extension", ["absent", "broken"])
def test_import(tmp_path, extension):
    if not os.path.exists(os.path.join(PACKAGE, "libreduce.so")):
        pytest.skip("libreduce.so is not built")
    copy = tmp_path / "fp32_reductions_amd"
    copy.mkdir()
    for name in ("__init__.py", "build.py", "libreduce.so"):
        shutil.copy(os.path.join(PACKAGE, name), str(copy / name))
    if extension == "broken":
        (copy / "_rowloss.so").write_bytes(b"not a library")
    p = subprocess.run([sys.executable, "-c", CHILD.format(root=str(tmp_path))],
                       capture_output=True, text=True, timeout=300, cwd=str(tmp_path))
    assert p.returncode == 0, p.stderr[-2000:]
    assert p.stdout.strip() == "imported"


def test_the_built_package_has_the_losses():
    red = pytest.importorskip("fp32_reductions_amd")
    if os.path.exists(os.path.join(PACKAGE, "_rowloss.so")):
        import torch

        with pytest.raises(TypeError, match="missing"):
            red.token_logprob_f32(torch.zeros(1, 1))
