"""The operators on windows, pages and caches made shorter as programs use them: as the first call of a process and that a
captured one, from two threads on two streams, at offsets that pass 32 bits, again and again with the same bits."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, SCALE, Pool, assert_lse, junk, log_sum, reference, visible
from tests.prompt_ops_util import assert_within, gen, normal

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import sys, torch
from quantized_decoder_decode_gb300 import fq
D, DEV, hq, hkv, L, K = 128, torch.device("cuda:0"), 8, 2, {L}, 2000
g = torch.Generator(device=DEV); g.manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
q, k, v, lse = r(L, hq, D), r(hkv, K, D), r(hkv, K, D), torch.full((L, hq), 9.0, device=DEV)
w, tk, tv = torch.zeros(hkv, K, device=DEV), torch.empty(hkv, 100, D, device=DEV).bfloat16(), torch.empty(hkv, 100, D, device=DEV).bfloat16()
kept, out = torch.zeros(hkv * 100, dtype=torch.int32, device=DEV), torch.zeros(L, hq, D, device=DEV).bfloat16()
qkv, one, rope = torch.randn(L, (hq + 2 * hkv) * D, device=DEV), torch.ones(D, device=DEV), torch.ones(K, 64, 2, device=DEV)
view = fq.fq_kv_view(k.data_ptr(), v.data_ptr(), K, D, K * D)
pk, pv = (t.reshape(hkv, K // 16, 16, D).transpose(0, 1).contiguous() for t in (k, v))
pages = fq.fq_kv_pages(pk.data_ptr(), pv.data_ptr(), K // 16, 16, hkv * 16 * D, D, 16 * D)
table = torch.arange(K // 16, dtype=torch.int32, device=DEV)
need = max(fq.fq_attn_window_workspace([L], [K], hq, hkv, 0, 0), fq.fq_attn_key_weights_workspace([L], [K], hq, hkv, 0, 0), 1)
ws = torch.empty(need, dtype=torch.uint8, device=DEV)
calls = dict(
    window=lambda s: fq.fq_attn_window(q.data_ptr(), view, [L], [K], hq, hkv, 0, 0, .088, out.data_ptr(), ws.data_ptr(), need, s),
    paged=lambda s: fq.fq_attn_paged(q.data_ptr(), pages, table.data_ptr(), K // 16, [L], [K], hq, hkv, 0, 0, .088, out.data_ptr(), ws.data_ptr(), need, s),
    append=lambda s: fq.fq_qk_norm_rope_paged(qkv.data_ptr(), [L], [0], pages, table.data_ptr(), K // 16, [5], hq, hkv, one.data_ptr(),
                                              one.data_ptr(), 1e-6, rope.data_ptr(), K, out.data_ptr(), s),
    weights=lambda s: fq.fq_attn_key_weights(q.data_ptr(), lse.data_ptr(), view, [L], [K], hq, hkv, 0, 0, .088, None,
                                             fq.fq_key_weights(w.data_ptr(), K), ws.data_ptr(), need, s),
    evict=lambda s: fq.fq_kv_evict(view, fq.fq_key_weights(w.data_ptr(), K), None, [K], [100], 4, 32, hkv,
                                   fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), 100, D, 100 * D), None, None, kept.data_ptr(), s))
call = calls["{op}"]
result = lambda: torch.cat([t.float().flatten() for t in (out, w, tk, tv, kept, pk, pv)])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call(torch.cuda.current_stream().cuda_stream)
graph.replay()
torch.cuda.synchronize()
a = result()
fq.fq_attn_check()
for t in (out, w, tk, tv, kept): t.zero_()
call(torch.cuda.current_stream().cuda_stream)
torch.cuda.synchronize()
b = result()
assert torch.equal(a, b) and float(a.abs().sum()) > 0
print("captured")
"""


@pytest.mark.parametrize("op", ["window", "paged", "append", "weights", "evict"])
@pytest.mark.parametrize("L", [1, 300])
def test_first_call_is_captured(op, L):
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(op=op, L=L)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def whole_run(seed, stream_):
    """A prompt into pages, attention, weights and an eviction on a stream; everything that comes out."""
    with torch.cuda.stream(stream_):
        g, hq, hkv, q_len, k_len = gen(seed), 8, 2, [200, 1, 3], [1200, 3000, 40]
        q = normal(g, sum(q_len), hq, D)
        pool = Pool(g, k_len, hkv, 32, fill=0.0)
        s = stream_.cuda_stream
        rows = sum(k_len)
        k, v = normal(g, hkv, rows, D), normal(g, hkv, rows, D)
        view = fq.fq_kv_view(k.data_ptr(), v.data_ptr(), rows, D, rows * D)
        n = max(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, 0, 0), fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, 500, 4),
                fq.fq_attn_key_weights_workspace(q_len, k_len, hq, hkv, 500, 4))
        ws = junk(n)
        paged, window = torch.empty(sum(q_len), hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(sum(q_len), hq, D, dtype=torch.bfloat16, device=DEV)
        lse, w = torch.empty(sum(q_len), hq, device=DEV), torch.empty(hkv, rows, device=DEV)
        keep = [min(K, 100) for K in k_len]
        tk, tv = (torch.empty(hkv, sum(keep), D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kept = torch.empty(hkv * sum(keep), dtype=torch.int32, device=DEV)
        fq.fq_attn_paged(q.data_ptr(), pool.pages(), pool.table.data_ptr(), pool.stride, q_len, k_len, hq, hkv, 0, 0, SCALE, paged.data_ptr(),
                         ws.data_ptr(), ws.numel() * 4, s)
        fq.fq_attn_window(q.data_ptr(), view, q_len, k_len, hq, hkv, 500, 4, SCALE, window.data_ptr(), ws.data_ptr(), ws.numel() * 4, s,
                          lse_ptr=lse.data_ptr())
        fq.fq_attn_key_weights(q.data_ptr(), lse.data_ptr(), view, q_len, k_len, hq, hkv, 500, 4, SCALE, None, fq.fq_key_weights(w.data_ptr(), rows),
                               ws.data_ptr(), ws.numel() * 4, s)
        fq.fq_kv_evict(view, fq.fq_key_weights(w.data_ptr(), rows), None, k_len, keep, 4, 20, hkv,
                       fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), sum(keep), D, sum(keep) * D), None, None, kept.data_ptr(), s)
        out = torch.cat([t.float().flatten() for t in (paged, window, lse, w, tk, tv, kept)])
        stream_.synchronize()
        fq.fq_attn_check(s)
        return out


def test_two_threads_on_two_streams_get_what_one_gets():
    want = [whole_run(seed, torch.cuda.Stream(DEV)) for seed in (3, 4)]
    got, errors = [[], []], []

    def work(i):
        try:
            s = torch.cuda.Stream(DEV)
            for _ in range(15):
                got[i].append(whole_run(3 + i, s))
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])   # and each time the same bits


@pytest.mark.parametrize("q_len,k_len", [([1], [300]), ([150], [300])])
def test_pages_beyond_32_bits(q_len, k_len):
    """A pool whose last pages begin beyond 2^32 elements: read and written there."""
    g, hq, hkv, page, n_pages = gen(61), 4, 2, 32, 20
    page_stride = (1 << 32) // 17 // 8 * 8
    store = [torch.empty((n_pages - 1) * page_stride + hkv * page * D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    k, v = (t.as_strided((n_pages, hkv, page, D), (page_stride, page * D, D, 1)) for t in store)
    for t in (k, v):
        t.copy_(normal(g, n_pages, hkv, page, D))
    table = torch.arange(n_pages - 1, n_pages - 11, -1, dtype=torch.int32, device=DEV)
    assert (n_pages - 1) * page_stride > 1 << 32
    pages = fq.fq_kv_pages(store[0].data_ptr(), store[1].data_ptr(), n_pages, page, page_stride, D, page * D)
    q = normal(g, sum(q_len), hq, D)
    rows = lambda s, h: tuple(t[table.long()][:, h].reshape(-1, D)[:k_len[0]] for t in (k, v))  # noqa: E731
    for window, sinks in ((0, 0), (100, 4)):
        ws = junk(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, window, sinks))
        out = torch.empty(sum(q_len), hq, D, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(sum(q_len), hq, device=DEV)
        s = torch.cuda.current_stream(DEV).cuda_stream
        fq.fq_attn_paged(q.data_ptr(), pages, table.data_ptr(), 10, q_len, k_len, hq, hkv, window, sinks, SCALE, out.data_ptr(), ws.data_ptr(),
                         ws.numel() * 4, s, lse_ptr=lse.data_ptr())
        fq.fq_attn_check(s)
        ref, bound, e, eb = reference(q, rows, q_len, k_len, hq, hkv, window, sinks)
        assert_within(out, ref, bound, True)
        assert_lse(lse, e, eb)
    n = 40
    qkv = torch.randn(n, (hq + 2 * hkv) * D, generator=g, device=DEV)
    one, rope = torch.ones(D, device=DEV), torch.tensor([1.0, 0.0], device=DEV).repeat(n, 64, 1).contiguous()
    qo = torch.empty(n, hq, D, dtype=torch.bfloat16, device=DEV)
    fq.fq_qk_norm_rope_paged(qkv.data_ptr(), [n], [0], pages, table.data_ptr(), 10, [7], hq, hkv, one.data_ptr(), one.data_ptr(), 1e-6,
                             rope.data_ptr(), n, qo.data_ptr(), s)
    fq.fq_attn_check(s)
    want = qkv.reshape(n, -1, D)[:, hq + hkv:].to(torch.bfloat16)
    for h in range(hkv):
        assert bool((v[table.long()][:, h].reshape(-1, D)[7:7 + n] == want[:, h]).all())


def test_rows_beyond_32_bits():
    """Views whose rows in use lie beyond 2^32 elements: window attention, weights and eviction."""
    g, hq, hkv, L, K, keep = gen(67), 4, 2, 120, 900, 200
    rows = (1 << 25) + 1000                      # of 128 elements: more than 2^32 in each head
    row0 = (1 << 25) + 50
    big = [torch.empty(rows, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    # both heads in one array, their rows 1 << 25 apart in turn: head stride below the rows' extent
    k, v = (t.as_strided((hkv, K, D), (K * D, D, 1), (row0 - (hkv - 1) * K - 100) * D) for t in big)
    for t in (k, v):
        t.copy_(normal(g, hkv, K, D))
    first = row0 - (hkv - 1) * K - 100
    view = fq.fq_kv_view(big[0].data_ptr(), big[1].data_ptr(), first + K, D, K * D)
    q = normal(g, L, hq, D)
    s = torch.cuda.current_stream(DEV).cuda_stream
    ws = junk(max(fq.fq_attn_window_workspace([L], [K], hq, hkv, 300, 4), fq.fq_attn_key_weights_workspace([L], [K], hq, hkv, 300, 4)))
    out, lse = torch.empty(L, hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(L, hq, device=DEV)
    fq.fq_attn_window(q.data_ptr(), view, [L], [K], hq, hkv, 300, 4, SCALE, out.data_ptr(), ws.data_ptr(), ws.numel() * 4, s, kv_row0=[first],
                      lse_ptr=lse.data_ptr())
    ref, bound, e, eb = reference(q, lambda _, h: (k[h], v[h]), [L], [K], hq, hkv, 300, 4)
    assert_within(out, ref, bound, True)
    assert_lse(lse, e, eb)
    # gathered weights of so many rows, one head stride of floats apart
    w = torch.zeros(hkv * (first + K), device=DEV)
    weights = fq.fq_key_weights(w.data_ptr(), first + K)
    fq.fq_attn_key_weights(q.data_ptr(), lse.data_ptr(), view, [L], [K], hq, hkv, 300, 4, SCALE, weights, weights, ws.data_ptr(), ws.numel() * 4, s,
                           kv_row0=[first])
    got = w.reshape(hkv, first + K)
    assert float(got[:, :first].abs().max()) == 0
    for h in range(hkv):
        total = torch.zeros(K, dtype=torch.float64, device=DEV)
        for x in range(hq // hkv):
            qq = q[:, h * 2 + x].double()
            total += torch.where(visible(L, K, 300, 4), torch.exp(qq @ k[h].double().T * SCALE - log_sum(q[:, h * 2 + x], k[h], visible(L, K, 300, 4), SCALE)[0][:, None]), 0.0).sum(dim=0)
        # (scores and log-sums in f32: some 1e-5 of a weight)
        assert float((got[h, first:].double() - total).abs().max()) < 1e-4 * float(total.max())
    tk, tv = (torch.empty(hkv, keep, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kept = torch.empty(hkv * keep, dtype=torch.int32, device=DEV)
    fq.fq_kv_evict(view, weights, [first], [K], [keep], 4, 32, hkv, fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), keep, D, keep * D), None, None,
                   kept.data_ptr(), s)
    fq.fq_attn_check(s)
    for h in range(hkv):
        idx = kept[h * keep:(h + 1) * keep].long()
        assert bool((tk[h] == k[h, idx]).all()) and bool((tv[h] == v[h, idx]).all())
        x = got[h, first:].clone()
        x[:4] = x[K - 32:] = float("inf")
        assert idx.tolist() == torch.sort(torch.sort(x, descending=True, stable=True).indices[:keep]).values.tolist()
