"""Pools in the layouts that programs have: rows appended and attended to there, against the same in a pool of its own for K and
for V, bit for bit; what is nobody's stays."""
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, SCALE, junk, stream
from tests.prompt_ops_util import gen, normal
from tests.test_gpu_window_paged import rope_table

pytestmark = pytest.mark.gpu

N, R, H = 40, 16, 2   # pages, rows, heads
# dims of the storage in their order; 0, 1 of "kv": K, V
LAYOUTS = ["kv page head row", "page kv head row", "page row kv head", "page row head kv", "head page kv row", "page layer kv row head", "row head kv page"]


def pool(order, fill):
    size = {"kv": 2, "page": N, "row": R, "head": H, "layer": 3}
    dims = order.split()
    store = torch.full([size[d] for d in dims] + [D], fill, dtype=torch.bfloat16, device=DEV)
    stride = dict(zip(dims, store.stride()))
    first = stride["layer"] if "layer" in stride else 0
    base = store.data_ptr() + 2 * first
    pages = fq.fq_kv_pages(base, base + 2 * stride["kv"], N, R, stride["page"], stride["row"], stride["head"])
    kv = [store.as_strided((N, H, R, D), (stride["page"], stride["head"], stride["row"], 1), first + i * stride["kv"]) for i in range(2)]
    return store, pages, kv


@pytest.mark.parametrize("order", LAYOUTS)
@pytest.mark.parametrize("lens,row0", [([1, 1, 1], [5, 100, 47]), ([150, 33], [0, 61])])
def test_append_and_attend(order, lens, row0):
    g, hq = gen(401), 8
    n_seq, k_len = len(lens), [a + b for a, b in zip(lens, row0)]
    ids, stride = torch.randperm(N, generator=g, device=DEV).int(), 12
    table = torch.full((n_seq, stride), -1, dtype=torch.int32, device=DEV)
    used = 0
    for s, K in enumerate(k_len):
        need = -(-K // R)
        table[s, :need] = ids[used:used + need]
        used += need
    old = normal(g, 2, N, H, R, D)
    qkv = torch.randn(sum(lens), (hq + 2 * H) * D, generator=g, device=DEV)
    gains = 1 + 0.1 * torch.randn(2, D, generator=g, device=DEV)
    rope = rope_table(max(k_len))
    ws = junk(fq.fq_attn_window_workspace(lens, k_len, hq, H, 90, 3))
    results = []
    for o in ("kv page head row", order):
        store, pages, kv = pool(o, 3.0)
        for t, x in zip(kv, old):
            t.copy_(x)
        q = torch.empty(sum(lens), hq, D, dtype=torch.bfloat16, device=DEV)
        out, lse = torch.empty_like(q), torch.empty(sum(lens), hq, device=DEV)
        fq.fq_qk_norm_rope_paged(qkv.data_ptr(), lens, row0, pages, table.data_ptr(), stride, row0, hq, H, gains[0].data_ptr(), gains[1].data_ptr(),
                                 1e-6, rope.data_ptr(), rope.shape[0], q.data_ptr(), stream())
        fq.fq_attn_paged(q.data_ptr(), pages, table.data_ptr(), stride, lens, k_len, hq, H, 90, 3, SCALE, out.data_ptr(), ws.data_ptr(),
                         ws.numel() * 4, stream(), lse_ptr=lse.data_ptr())
        fq.fq_attn_check(stream())
        results.append((q, out, lse, kv[0].clone(), kv[1].clone()))
        if "layer" in o:   # the other layers' rows
            for t in kv:
                t.fill_(3.0)
            assert bool((store == 3).all())
    assert not bool((results[0][3] == old[0]).all())
    for a, b in zip(*results):
        assert bool((a == b).all())
