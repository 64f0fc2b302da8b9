"""A step of a program in one graph: rows into pages, attention over them, attention of a window with its log-sums, the weights of the
keys, a cache made shorter and attention over that, all with one workspace.  Replayed again and again, two such graphs at once on two streams, with the bits of calls one by one."""
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, NAN, SCALE, Pool, junk
from tests.prompt_ops_util import gen, normal
from tests.test_gpu_window_paged import rope_table

pytestmark = pytest.mark.gpu

HQ, HKV, KEEP = 8, 2, 120
# single tokens, a chunk beside tokens, a chunk over keys that are split
LENGTHS = [([1, 1, 1], [300, 2000, 900]), ([1, 333, 2], [3000, 1333, 40]), ([64], [9000])]


class Step:
    def __init__(self, seed, q_len, k_len):
        g = gen(seed)
        self.q_len, self.k_len, T, rows = q_len, k_len, sum(q_len), sum(k_len)
        self.pool = Pool(g, k_len, HKV, 32, fill=0.0)
        self.qkv = torch.randn(T, (HQ + 2 * HKV) * D, generator=g, device=DEV)
        self.gain, self.rope = torch.ones(D, device=DEV), rope_table(max(k_len))
        self.k, self.v = normal(g, HKV, rows, D), normal(g, HKV, rows, D)
        self.keep = [min(K, KEEP) for K in k_len]
        n = sum(self.keep)
        self.q = torch.empty(T, HQ, D, dtype=torch.bfloat16, device=DEV)
        self.out = [torch.empty_like(self.q) for _ in range(3)]
        self.lse, self.w, self.tw = torch.empty(T, HQ, device=DEV), torch.empty(HKV, rows, device=DEV), torch.empty(HKV, n, device=DEV)
        self.tk, self.tv = (torch.empty(HKV, n, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.kept = torch.empty(HKV * n, dtype=torch.int32, device=DEV)
        sizes = [fq.fq_attn_window_workspace(q_len, K, HQ, HKV, *m) for K in (k_len, self.keep) for m in ((0, 0), (700, 4))]
        self.ws = junk(max(sizes + [fq.fq_attn_key_weights_workspace(q_len, k_len, HQ, HKV, 700, 4)]))

    def run(self, s):
        q_len, k_len, pool, ws, n, rows = self.q_len, self.k_len, self.pool, self.ws.data_ptr(), self.ws.numel() * 4, sum(self.k_len)
        row0 = [K - L for L, K in zip(q_len, k_len)]
        view = fq.fq_kv_view(self.k.data_ptr(), self.v.data_ptr(), rows, D, rows * D)
        short = fq.fq_kv_view(self.tk.data_ptr(), self.tv.data_ptr(), sum(self.keep), D, sum(self.keep) * D)
        w, tw = fq.fq_key_weights(self.w.data_ptr(), rows), fq.fq_key_weights(self.tw.data_ptr(), sum(self.keep))
        fq.fq_qk_norm_rope_paged(self.qkv.data_ptr(), q_len, row0, pool.pages(), pool.table.data_ptr(), pool.stride, row0, HQ, HKV, self.gain.data_ptr(),
                                 self.gain.data_ptr(), 1e-6, self.rope.data_ptr(), self.rope.shape[0], self.q.data_ptr(), s)
        fq.fq_attn_paged(self.q.data_ptr(), pool.pages(), pool.table.data_ptr(), pool.stride, q_len, k_len, HQ, HKV, 0, 0, SCALE,
                         self.out[0].data_ptr(), ws, n, s)
        fq.fq_attn_window(self.out[0].data_ptr(), view, q_len, k_len, HQ, HKV, 700, 4, SCALE, self.out[1].data_ptr(), ws, n, s, lse_ptr=self.lse.data_ptr())
        fq.fq_attn_key_weights(self.out[0].data_ptr(), self.lse.data_ptr(), view, q_len, k_len, HQ, HKV, 700, 4, SCALE, None, w, ws, n, s)
        fq.fq_kv_evict(view, w, None, k_len, self.keep, 4, 20, HKV, short, tw, None, self.kept.data_ptr(), s)
        fq.fq_attn_window(self.out[1].data_ptr(), short, q_len, self.keep, HQ, HKV, 0, 0, SCALE, self.out[2].data_ptr(), ws, n, s)

    def result(self):
        return torch.cat([t.float().flatten() for t in (self.q, *self.out, self.lse, self.w, self.tw, self.tk, self.tv, self.kept, *self.pool.store)])

    def clear(self):
        for t in (self.q, *self.out, self.lse, self.w, self.tw, self.tk, self.tv, self.ws):
            t.fill_(NAN)
        self.kept.fill_(-1)


@pytest.mark.parametrize("lengths", LENGTHS)
def test_steps_in_graphs(lengths):
    steps = [Step(701, *lengths), Step(702, *LENGTHS[1])]
    want = []
    for x in steps:
        x.clear()
        x.run(torch.cuda.current_stream(DEV).cuda_stream)
        torch.cuda.synchronize()
        want.append(x.result())
        assert bool(torch.isfinite(want[-1]).all())
    streams, graphs = [torch.cuda.Stream(DEV) for _ in steps], []
    for x, side in zip(steps, streams):
        x.clear()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            x.run(torch.cuda.current_stream(DEV).cuda_stream)
    for _ in range(5):
        for x in steps:
            x.clear()
        torch.cuda.synchronize()
        for _ in range(4):
            for graph, side in zip(graphs, streams):
                with torch.cuda.stream(side):
                    graph.replay()
        torch.cuda.synchronize()
        fq.fq_attn_check()
        for x, w in zip(steps, want):
            assert bool((x.result() == w).all())
