"""Caches made shorter, on the GPU against a plain selection by sorting: rows beyond what the thread blocks of a cluster hold at a time,
ragged calls of which one sequence is that long, with first and recent rows and with weights that move along."""
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, stream
from tests.prompt_ops_util import gen, normal
from tests.test_gpu_key_weights_evict import kinds, plain_evict, weights

pytestmark = pytest.mark.gpu

KINDS = ["wide", "ties", "same", "odd"]


def bits(t):
    return t.contiguous().view(torch.int32)


def chosen(w, n, sinks, recent):
    """The rows of one head that stay: NaN counts above infinity, equal ones from the first on."""
    K = w.shape[0]
    if n == K:
        return torch.arange(K, device=DEV)
    x = torch.where(torch.isinf(w), torch.sign(w).double() * 1e300, w.double())
    x[torch.isnan(w)] = float("inf")
    best = torch.sort(x[sinks:K - recent], descending=True, stable=True).indices[:n - sinks - recent] + sinks
    fixed = torch.cat((torch.arange(sinks, device=DEV), torch.arange(K - recent, K, device=DEV)))
    return torch.sort(torch.cat((best, fixed))).values


@pytest.mark.parametrize("kind", KINDS)
def test_two_plain_forms(kind):
    g = gen(201)
    for K, n, sinks, recent in ((1, 0, 0, 0), (300, 100, 0, 0), (301, 100, 3, 40), (300, 299, 100, 100), (300, 300, 4, 4)):
        w = kinds(g, kind, 1, K)[0]
        assert bool((chosen(w, n, sinks, recent) == plain_evict(w, n, sinks, recent)).all())


# 8 thread blocks of 8192 rows at a time: up to 65536 at once, then two and three chunks of each block
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K,keep,sinks,recent", [(65536, 20001, 4, 32), (65537, 65536, 0, 0), (140001, 9000, 100, 4000),
                                                 (140001, 139000, 0, 1), (140001, 1, 0, 0), (140001, 70000, 0, 70000), (200000, 123456, 50000, 20000)])
def test_long_sequences(kind, K, keep, sinks, recent):
    g, hkv = gen(211 + KINDS.index(kind)), 2
    k, v = normal(g, hkv, K, D), normal(g, hkv, K, D)
    w = kinds(g, kind, hkv, K)
    tk, tv = (torch.full((hkv, keep + 3, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tw = torch.full((hkv, keep + 3), 7.0, device=DEV)
    kept = torch.full((hkv * keep + 4,), -5, dtype=torch.int32, device=DEV)
    fq.fq_kv_evict(fq.fq_kv_view(k.data_ptr(), v.data_ptr(), K, D, K * D), weights(w), None, [K], [keep], sinks, recent, hkv,
                   fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), keep + 3, D, (keep + 3) * D), weights(tw), None, kept.data_ptr(), stream())
    for h in range(hkv):
        want = chosen(w[h], keep, sinks, recent)
        assert bool((kept[h * keep:(h + 1) * keep] == want).all())
        assert bool((tk[h, :keep] == k[h, want]).all()) and bool((tv[h, :keep] == v[h, want]).all())
        assert bool((bits(tw[h, :keep]) == bits(w[h, want])).all())
        for t in (tk[h, keep:], tv[h, keep:], tw[h, keep:]):
            assert bool((t == 7).all())
    assert bool((kept[hkv * keep:] == -5).all())


# sequences that lose rows, that keep them all, empty ones, ones that keep none but fixed rows; with and without one whose rows
# take a cluster of thread blocks, or several chunks of each
RAGGED = {
    "short": ([100, 0, 7, 5000, 333, 64, 1] + [211] * 20, [50, 9, 7, 700, 8, 100, 7] + [30 + s for s in range(20)]),
    "one in a cluster": ([300, 8193, 20, 0, 1000], [100, 3000, 20, 5, 7]),
    "one of several chunks": ([300, 140001, 20, 9000], [299, 30000, 7, 8999]),
}


@pytest.mark.parametrize("name", RAGGED)
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("kind", ["ties", "odd"])
@pytest.mark.parametrize("sinks,recent", [(2, 5), (0, 0)])
def test_ragged_sequences(name, own, kind, sinks, recent):
    """In one view or a view each at row offsets, with and without weights that move; other rows stay as they were."""
    k_len, keep = RAGGED[name]
    g, hkv, S = gen(241 + sorted(RAGGED).index(name)), 3, len(k_len)
    n = [min(a, b) for a, b in zip(k_len, keep)]
    # (a view each: [row][head][D + 8]; one view: [head][row][D])
    at, row0 = ([s % 3 for s in range(S)], [s % 4 for s in range(S)]) if own else ([sum(n[:s]) + s for s in range(S)], [sum(k_len[:s]) for s in range(S)])
    if own:
        ks, vs = ([normal(g, K + 5, hkv, D + 8).transpose(0, 1) for K in k_len] for _ in range(2))
        ws = [kinds(g, kind, hkv, K + 5) for K in k_len]
        tk, tv = ([torch.full((hkv, m + 4, D), 7.0, dtype=torch.bfloat16, device=DEV) for m in n] for _ in range(2))
        tw = [torch.full((hkv, m + 4), 7.0, device=DEV) for m in n]
        views = [fq.fq_kv_view(a.data_ptr(), b.data_ptr(), K + 5, hkv * (D + 8), D + 8) for a, b, K in zip(ks, vs, k_len)]
        to = [fq.fq_kv_view(a.data_ptr(), b.data_ptr(), m + 4, D, (m + 4) * D) for a, b, m in zip(tk, tv, n)]
        w, to_w = [weights(x) for x in ws], [weights(x) for x in tw]
    else:
        R, N = sum(k_len), sum(n) + S
        ks, vs, ws = [normal(g, hkv, R, D)] * S, [normal(g, hkv, R, D)] * S, [kinds(g, kind, hkv, R)] * S
        tk, tv = ([torch.full((hkv, N, D), 7.0, dtype=torch.bfloat16, device=DEV)] * S for _ in range(2))
        tw = [torch.full((hkv, N), 7.0, device=DEV)] * S
        views = fq.fq_kv_view(ks[0].data_ptr(), vs[0].data_ptr(), R, D, R * D)
        to = fq.fq_kv_view(tk[0].data_ptr(), tv[0].data_ptr(), N, D, N * D)
        w, to_w = weights(ws[0]), weights(tw[0])
    for moved in (None, to_w):
        kept = torch.full((hkv * sum(n) + 2,), -5, dtype=torch.int32, device=DEV)
        fq.fq_kv_evict(views, w, row0, k_len, keep, sinks, recent, hkv, to, moved, at, kept.data_ptr(), stream())
        used = [torch.zeros(t.shape[:2], dtype=torch.bool, device=DEV) for t in (tk if own else tk[:1])]
        for s in range(S):
            rows, put = slice(row0[s], row0[s] + k_len[s]), slice(at[s], at[s] + n[s])
            used[s if own else 0][:, put] = True
            for h in range(hkv):
                a, b, x = ks[s][h, rows, :D], vs[s][h, rows, :D], ws[s][h, rows]
                want = chosen(x, n[s], sinks, recent)
                first = hkv * sum(n[:s]) + h * n[s]
                assert bool((kept[first:first + n[s]] == want).all()), (s, h)
                assert bool((tk[s][h, put] == a[want]).all()) and bool((tv[s][h, put] == b[want]).all())
                if moved is not None:
                    assert bool((bits(tw[s][h, put]) == bits(x[want])).all())
        assert bool((kept[hkv * sum(n):] == -5).all())
        for i, u in enumerate(used):
            assert bool((tk[i][~u] == 7).all()) and bool((tv[i][~u] == 7).all())
            assert bool((tw[i][~u] == 7).all()) if moved is not None else bool((tw[i] == 7).all())
