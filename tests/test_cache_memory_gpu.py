"""First calls of the 8-bit decode leave the device's free memory alone: a kernel's stack is
reserved for every thread the device can hold (152 SMs x 2048), so one of 2 KB above what
a context has takes 600 MB."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
import causal_gqa_attention_online_gb300 as attn
calls = []
for D in (64, 128, 256):
    for Q in (1, 4, 12):
        for dtype in (torch.int8, torch.float8_e4m3fn):
            pages = [torch.zeros((5, 64, 2, D), dtype=torch.int8, device="cuda").view(dtype) for _ in "kv"]
            scales = [torch.ones((5, 1, 2), device="cuda") for _ in "kv"]
            table = torch.arange(5, dtype=torch.int32, device="cuda")[None]
            lens = torch.tensor([300], dtype=torch.int32, device="cuda")
            q = torch.zeros((1, Q, 8, D), dtype=torch.bfloat16, device="cuda")
            calls.append((q, *pages, *scales, table, lens, torch.empty_like(q),
                          torch.empty((1, Q, 8), device="cuda")))
torch.cuda.synchronize()
free = torch.cuda.mem_get_info()[0]
for c in calls:
    attn.attn_fwd_paged_q8(*c, algo="decode")
torch.cuda.synchronize()
print("taken", free - torch.cuda.mem_get_info()[0])
"""


def test_first_calls_take_no_memory_to_speak_of():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    taken = int(r.stdout.split("taken")[1])
    # (the library's pool grows by 32 MB; 100 bytes of stack are 31 MB)
    assert taken <= 128 << 20, f"{taken / 2 ** 20:.0f} MB"
