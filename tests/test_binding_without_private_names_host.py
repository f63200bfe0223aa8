"""Host-only: the binding imports and works with a torch that lacks its private shortcuts."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import compressed_sparse_long_csa_b200 as csa
from compressed_sparse_long_csa_b200 import _native as N
assert N._device_now is torch.cuda.current_device
class Now:
    cuda_stream = 77
torch.cuda.current_stream = lambda device=None: Now
torch.cuda.current_device = lambda: 0
assert N._stream_now(0) == 77 and N._stream(None) == 77 and N._stream(5) == 5 and N._stream(Now) == 77
try:
    csa.latent_append_paged(torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(4, 16, 64), torch.zeros(2, 2, dtype=torch.int32))
except csa.CsaError as e:
    assert "current CUDA device" in str(e)
    print("refused")
"""


def test_public_calls_serve():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]
