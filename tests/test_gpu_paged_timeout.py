"""What an abandoned fa_prefill_paged call leaves in its workspace (the call's tag, in the word behind the
publication flags) against a replay of the same captured call.  No wait runs out here: the word is
written by the test."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# in a process of its own, where the calls' tags are known: call number 0 is the eager one
SCRIPT = r"""
import sys
sys.path.insert(0, "tests")
import torch
import quantized_kv_cache_sm_gb300 as fa
from paged_common import make_ragged
from test_gpu_prefill_paged import make_q

def tag(call):
    m = (1 << 64) - 1
    z = (call + 0x9E3779B97F4A7C15) & m
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
    t = (z ^ (z >> 31)) >> 32
    return t - (1 << 32) if t >> 31 else t

r = make_ragged([1, 300], [9000, 5000], 2, 128, 64, "f16", "dense", "q4_0", seed=201)
q = make_q(301, 8, 128, "f16", seed=202).cuda()
k, v, batch = r.pool(fa, "k"), r.pool(fa, "v"), r.batch()
ws = torch.zeros(fa.fa_prefill_paged_workspace_bytes(8, 2, 128), dtype=torch.uint8, device="cuda")
word = ws[:4 * (ws.numel() // 4)].view(torch.int32)
behind = 2 * torch.cuda.get_device_properties(0).multi_processor_count
want = fa.fa_prefill_paged(q, k, v, *batch, workspace=ws)
o = torch.zeros_like(want)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fa.fa_prefill_paged(q, k, v, *batch, o, workspace=ws)

def replay():
    o.fill_(7.0)
    g.replay()
    return fa.fa_get_status()

assert replay() == fa.FA_OK and torch.equal(o, want)
word[behind] = tag(0)  # another call's: nothing to this one
assert replay() == fa.FA_OK and torch.equal(o, want)
word[behind] = tag(1)
for _ in range(2):
    assert replay() == fa.FA_ERR_TIMEOUT
eager = fa.fa_prefill_paged(q, k, v, *batch, workspace=ws)
assert fa.fa_get_status() == fa.FA_OK and torch.equal(eager, want)
word[:behind] = tag(1)  # and its flags, as if published
assert replay() == fa.FA_ERR_TIMEOUT
ws.zero_()
assert replay() == fa.FA_OK and torch.equal(o, want)
"""


def test_replay_over_an_abandoned_calls_workspace_is_reported(fa):
    p = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr[-2000:]
