"""The package without its native binding (built against one version of torch): every entry point that goes through
ctypes works, the full-precision operators say what is missing."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
import bit_linear_layers_b200 as bl
assert bl.status_string(0) and bl.lib.bl_abi_version() >= 1
assert bl.workspace_bytes(bl.BL_OP_GRAD_CLIP, 5, 0, 0) > 0
try:
    bl.bin_linear_w1a16(torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4))
except ValueError as e:
    assert "CUDA" in str(e)
x = torch.zeros(2, 8)
for call in (lambda: bl.layer_norm(x), lambda: bl.layer_norm_backward(x, None, x[0], x[0], x),
             lambda: bl.embedding(torch.zeros(2, dtype=torch.int64), x),
             lambda: bl.embedding_backward(torch.zeros(2, dtype=torch.int64), x, 2), lambda: bl.grad_clip([x], 1.0),
             lambda: bl.grad_norm([x])):
    for _ in range(2):
        try:
            call()
        except ImportError as e:
            assert "_native.so" in str(e), e
        else:
            raise AssertionError("no ImportError")
print("fine")
"""


@pytest.mark.parametrize("binding", [None, b"not a library"], ids=["missing", "broken"])
def test_import_without_the_native_binding(tmp_path, binding):
    pkg, src = tmp_path / "bit_linear_layers_b200", os.path.join(ROOT, "bit_linear_layers_b200")
    pkg.mkdir()
    for f in ("__init__.py", "libbitlinear.so"):
        os.symlink(os.path.realpath(os.path.join(src, f)), pkg / f)
    if binding is not None:
        (pkg / "_native.so").write_bytes(binding)
    p = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "fine", p.stdout + p.stderr


def test_refusals_come_through_the_native_binding():
    """Loaded by the first call; its refusals are Python's."""
    import torch

    import bit_linear_layers_b200 as bl
    for _ in range(2):
        with pytest.raises(ValueError, match="x must be a CUDA tensor"):
            bl.layer_norm(torch.zeros(2, 8))
