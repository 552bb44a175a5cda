"""Threads of one process that make their first calls at once, each on a stream of its own (the binding lets go of the
interpreter's lock during a call)."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

PROGRAM = """
import threading, torch
import structured_causal_attention_b200 as hd
B, n, T, Hq, Hkv, D = 2, 4, 900, 8, 2, 64
hd.lib()
seqlen = torch.full((B,), T, dtype=torch.int32, device="cuda")
g = torch.Generator(device="cuda").manual_seed(1)
k, v = (torch.randn(B, T * n, Hkv, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
q = torch.randn(B, n, Hq, D, device="cuda", generator=g).to(torch.bfloat16)
torch.cuda.synchronize()
start, got = threading.Barrier(8), [None] * 8

def work(i):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        cache = hd.kv_cache_q8(B, T, n, Hkv, D, (torch.int8, torch.float8_e4m3fn)[i % 2])
        start.wait()
        hd.kv_write_q8(k, v, cache)
        got[i] = hd.decode_attn_q8(q, cache, seqlen, hd.CROSS_FULL)
        s.synchronize()

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
for t in threads: t.start()
for t in threads: t.join()
assert hd.hd_device_status() == hd.HD_OK
for i in range(2, 8):
    assert torch.equal(got[i][0], got[i % 2][0]) and torch.equal(got[i][1], got[i % 2][1])
print("same")
"""


def test_first_calls_of_threads_at_once():
    need_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
