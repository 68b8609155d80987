"""The package without the module that the attention block's operators go through (no GPU): it imports, the recurrent
block's entry points are there, and the attention block's say what is missing."""
import os
import shutil
import subprocess
import sys

import gated_linear_recurrence_conv1d_amd as rg

PKG = os.path.dirname(os.path.abspath(rg.__file__))

SCRIPT = """
import torch
import gated_linear_recurrence_conv1d_amd as rg
assert rg.__file__.startswith({root!r}), rg.__file__
assert rg.rglru_forward_workspace_size(2, 300, 256, 1, torch.bfloat16) > 0
x = torch.zeros(1, 5, 64)
try:
    rg.prefill_state(x)
except ValueError as e:
    assert "device" in str(e)
q = torch.zeros(1, 5, 2, 64, dtype=torch.bfloat16)
i32 = torch.int32
for call in (lambda: rg.local_attention(q, q, q, 4),
             lambda: rg.rglru_local_attention(q, q, q, q, 4),
             lambda: rg.qk_norm_rope(q, q, torch.zeros(1, 5, dtype=i32), torch.zeros(16)),
             lambda: rg.paged_attention(q[0], q, q, torch.zeros(5, 1, dtype=i32), torch.zeros(5, dtype=i32), 4)):
    try:
        call()
    except ImportError as e:
        assert "_rglru_torch.so" in str(e) and "build" in str(e), e
        assert isinstance(e.__cause__, ImportError)
    else:
        raise AssertionError("nothing was raised")
print("as expected")
"""


def test_package_without_the_module(tmp_path):
    here = tmp_path / "gated_linear_recurrence_conv1d_amd"
    here.mkdir()
    for f in ("__init__.py", "librglru.so"):
        shutil.copy(os.path.join(PKG, f), here / f)
    out = subprocess.run([sys.executable, "-c", SCRIPT.format(root=str(tmp_path))], cwd=tmp_path, text=True,
                         capture_output=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert out.returncode == 0 and "as expected" in out.stdout, out.stderr
