"""The first attention call of a process may be a captured one: what the library prepares then leaves the capture
alone."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import math, sys
import torch
from quantized_decoder_decode_gb300 import fq
from tests.prompt_ops_util import D, DEV, assert_within, attend, causal, gen, normal
L, K, hq, hkv = {shape}
g = gen(1)
q, k, v = normal(g, L, hq, D), normal(g, hkv, K, D), normal(g, hkv, K, D)
view = fq.fq_kv_view(k.data_ptr(), v.data_ptr(), K, D, K * D)
ws = torch.empty(max(1, fq.fq_attn_prompt_workspace([L], [K], hq, hkv)), dtype=torch.uint8, device=DEV)
out = torch.zeros_like(q)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    fq.fq_attn_prompt(q.data_ptr(), view, [L], [K], hq, hkv, 1 / math.sqrt(D), out.data_ptr(), ws.data_ptr(), ws.numel(),
                      torch.cuda.current_stream().cuda_stream)
for _ in range(2):
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    fq.fq_attn_check()
    for h in range(hq):
        ref, bound = attend(q[:, h], k[h // (hq // hkv)], v[h // (hq // hkv)], causal(L, K), 1 / math.sqrt(D))
        assert_within(out[:, h], ref, bound, True)
print("captured")
"""


@pytest.mark.parametrize("shape", [(300, 300, 8, 2), (1, 5000, 8, 2), (40, 9000, 8, 2)])   # tiles, few rows, split and joined
def test_first_call_is_captured(shape):
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(shape=shape)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
