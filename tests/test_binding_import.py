"""The package under a torch built without CUDA: it imports, and what needs no GPU answers."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda")]:
    delattr(torch._C, name)
import mxfp8_mxfp4_moe_gb300 as K
p = K.make_params(16, 128, 128, 8, 2)
assert K.kmoe_workspace_size(p) == K.kmoe_workspace_layout(p).total > 0
assert K.kmoe_rmsnorm_workspace_size(4, 128) > 0 and K.kmoe_status_string(1)
for call in (lambda: K.kmoe_rmsnorm(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)),
             lambda: K.kmoe_rmsnorm_backward(*[torch.zeros(4, 64, dtype=torch.bfloat16)] * 2, torch.zeros(64)),
             lambda: K.kmoe_route(torch.zeros(4, 8), torch.zeros(8), 2)):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
print("imported")
"""


def test_import_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
