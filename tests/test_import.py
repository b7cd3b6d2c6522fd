"""The binding imports, and answers what needs no GPU, on a torch without the
private symbols that a GPU build has."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from microscaling_fp4_block_fp4q_amd import fp4q
assert fp4q._raw_stream is None
assert fp4q.nvfp4().block == 16 and fp4q.mxfp4().block == 32
assert "fp4q_linear" in fp4q.declared_entry_points()

class Stream:
    cuda_stream = 7
torch.cuda.current_stream = lambda: Stream
assert fp4q._stream(None) == 7 and fp4q._stream(Stream) == 7
print("imported")
"""


def test_import_without_the_gpu_symbols_of_torch():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr
