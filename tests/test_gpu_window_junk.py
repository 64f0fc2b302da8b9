"""Rows that no query row of a call sees may hold anything: they change neither the outputs nor, to speak of, the time."""
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, NAN, SCALE, Pool, stream
from tests.prompt_ops_util import gen, normal

pytestmark = pytest.mark.gpu


def timed(call):
    """Microseconds of a call as part of a replayed graph, the least of five turns."""
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    call(stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(5):
            call(torch.cuda.current_stream(DEV).cuda_stream)
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 200)
    return min(times)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("q_len,k_len,window,sinks", [([333], [1333], 0, 0), ([17], [1017], 256, 4), ([500], [3000], 1000, 300), ([1, 150, 40], [50, 1700, 330], 64, 5)])
def test_rows_that_nobody_sees(paged, q_len, k_len, window, sinks):
    """NaN behind the last keys, and between the sinks and the window, in place of zeros."""
    hq, hkv = 16, 8
    n = fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, window, sinks)
    ws = torch.zeros(n + 32, dtype=torch.uint8, device=DEV)
    outs, times = [], []
    for fill in (0.0, NAN):
        g = gen(501)
        pool = Pool(g, k_len, hkv, 64, fill=fill)
        k, v = (torch.full((hkv, sum(k_len) + 60 * len(k_len), D), fill, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        row0 = [sum(k_len[:s]) + 60 * s for s in range(len(k_len))]   # (rows of nobody behind each sequence)
        for s, (L, K) in enumerate(zip(q_len, k_len)):
            for t, p in ((k, 0), (v, 1)):
                t[:, row0[s]:row0[s] + K] = torch.stack([pool.rows(s, h)[p] for h in range(hkv)])
            first = max(0, K - L + 1 - window) if window else 0
            if first > sinks:   # keys between the sinks and the first row's window
                k[:, row0[s] + sinks:row0[s] + first], v[:, row0[s] + sinks:row0[s] + first] = fill, fill
                for t in (pool.k, pool.v):
                    pool.put(t, s, sinks, torch.full((hkv, first - sinks, D), fill, dtype=torch.bfloat16, device=DEV))
        q = normal(g, sum(q_len), hq, D)
        out, lse = torch.full_like(q, NAN), torch.full((sum(q_len), hq), NAN, device=DEV)
        view = fq.fq_kv_view(k.data_ptr(), v.data_ptr(), k.shape[1], D, k.shape[1] * D)
        if paged:
            call = lambda s: fq.fq_attn_paged(q.data_ptr(), pool.pages(), pool.table.data_ptr(), pool.stride, q_len, k_len, hq, hkv, window,  # noqa: E731
                                              sinks, SCALE, out.data_ptr(), ws.data_ptr(), n, s, lse_ptr=lse.data_ptr())
        else:
            call = lambda s: fq.fq_attn_window(q.data_ptr(), view, q_len, k_len, hq, hkv, window, sinks, SCALE, out.data_ptr(),  # noqa: E731
                                               ws.data_ptr(), n, s, kv_row0=row0, lse_ptr=lse.data_ptr())
        times.append(timed(call))
        fq.fq_attn_check(stream())
        outs.append((out, lse))
    for a, b in zip(*outs):
        assert bool((a == b).all())
    # (tiles with such values are gone through row by row, some 11 us)
    assert times[1] < 3 * times[0] + 20, times
