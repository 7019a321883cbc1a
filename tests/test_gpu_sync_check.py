"""What pa_sync_check costs a process that makes none of the calls around decode."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import time
import torch
import paged_kv_cache_335_b200 as pa

def cost():
    best = 1e9
    for _ in range(300):
        t = time.perf_counter()
        pa.pa_sync_check()
        best = min(best, time.perf_counter() - t)
    return best * 1e6

x = lambda *s: torch.zeros(s, device="cuda", dtype=torch.bfloat16)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
kc, vc = x(4, 1, 16, 64), x(4, 1, 16, 64)
pa.pa_decode(x(1, 1, 64), x(1, 1, 64), kc, vc, i32([[0]]), i32([5]), 0.1)
before = cost()
pa.pa_rope_append(x(1, 1, 64), x(1, 1, 64), x(1, 1, 64), x(1, 1, 64), i32([[3]]), i32([0]).long(), kc, vc, pa.rope_desc(64))
for t in (torch.bfloat16, torch.float32):
    pa.pa_prefill(x(8, 1, 64).to(t), *(x(8, 1, 64).to(t) for _ in range(3)), i32([0, 8]), 0.1)
w = torch.zeros((1, 1, 16), device="cuda")
pa.pa_evict(kc, vc, i32([[0]]), i32([5]), w, w, i32([0]), i32([[[0] * 3]]), 3, 1)
after = cost()
print(before, after)
"""


def test_status_words_of_calls_not_made_are_not_read():
    out = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    before, after = map(float, out.stdout.split())
    assert before < 0.85 * after, f"{before:.1f} us before and {after:.1f} us after the four calls"
