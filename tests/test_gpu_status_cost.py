"""attn_fwd_last_error asks for the status words of what has run: a process that uses attention alone does not
wait for those of the norms, the paged cache and its eviction."""
import os
import subprocess
import sys

import pytest
import torch

from bf16_forward_attention_gb300 import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import time
import torch
import bf16_forward_attention_gb300 as attn

def best():
    torch.cuda.synchronize()
    t = []
    for _ in range(20):
        t0 = time.perf_counter()
        for _ in range(50):
            assert attn.attn_fwd_last_error() == attn.ATTN_OK
        t.append(time.perf_counter() - t0)
    return min(t)

q = torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
attn.attn_fwd(q, q, q)
best()
before = best()
w, table = q[0, 0, 0].contiguous(), torch.zeros(4, 64, device="cuda")
zero = torch.zeros(1, dtype=torch.int32, device="cuda")
one = zero + 1
x = q[0, :, :1].contiguous()
attn.attn_qk_norm_rope(x, x, w, w, table, table, zero)
out, lse = attn.attn_fwd_paged(q[:, :, :1].contiguous(), q, q, zero[None], one)
attn.attn_cache_evict(q, q.clone(), zero[None], one, torch.zeros(1, 1, 16, device="cuda"), 4)
best()
print(before, best())
"""


def test_words_of_what_never_ran_are_not_read():
    """Three words before, six after: half the time, of which a fifth is asked."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    out = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    before, after = map(float, out.stdout.split()[-2:])
    assert before < 0.8 * after, (before, after)
