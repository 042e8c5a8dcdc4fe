"""The package imports on a torch that was built without GPU support (no GPU)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import gated_deltanet_chunked_delta_amd as gdn
x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
for call in (lambda: gdn.causal_conv1d(x, w), lambda: gdn.fused_add_rms_norm(x, x, w[:, 0]),
             lambda: gdn.fused_gated_rms_norm(x, x, w[:, 0])):
    try:
        call()
    except ValueError as e:
        assert "GPU" in str(e), e
    else:
        raise AssertionError("no error")
print("imported")
"""


def test_import_without_gpu_support():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("imported"), r.stderr[-2000:]
