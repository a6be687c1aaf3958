"""The package imports, and refuses as it should, on a torch build that lacks the
private CUDA functions the cache's binding takes for speed (builds without CUDA)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import causal_gqa_attention_online_gb300 as attn
from causal_gqa_attention_online_gb300 import cache
for name in attn.__all__:
    assert hasattr(attn, name), name
pages = torch.zeros((2, 16, 1, 64), dtype=torch.int8)
scale = torch.ones((2, 1, 1))
table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
try:
    attn.attn_fwd_paged_q8(torch.zeros((1, 1, 2, 64)), pages, pages, scale, scale, table, lens)
    raise SystemExit("no refusal")
except ValueError as e:
    assert "CUDA devices only" in str(e), e
# the public functions stand in
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda device=None: Stream() if device == 3 else None
torch.cuda.current_device = lambda: 5
assert cache._raw_stream(3) == 77 and cache._current_device() == 5
print("imported")
"""


def test_import_without_torchs_private_cuda_functions():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stdout + r.stderr
