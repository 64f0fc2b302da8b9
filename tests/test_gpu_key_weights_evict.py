"""The attention weights that keys receive, and caches made shorter by them, on the GPU against plain 64-bit forms, at the
sizes, masks, layouts and ties where they can go wrong."""
import math

import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, NAN, SCALE, junk, log_sum, run_window, stream, visible
from tests.prompt_ops_util import gen, normal

pytestmark = pytest.mark.gpu

HEADS = [(4, 4), (4, 2), (8, 2), (8, 1)]
# single tokens, up to two and more blocks of 128 packed rows, whole prompts (cut into several units), ragged and empty
# ones, more queries than keys
LENGTHS = [([1], [1]), ([1], [5000]), ([1, 0, 2, 1], [300, 77, 129, 4096]), ([31, 64, 33], [31, 640, 333]), ([127, 128, 129], [127, 128, 129]),
           ([300], [40]), ([9, 4, 3], [2, 0, 3]), ([500], [3000]), ([2100], [2100])]
MASKS = [(0, 0), (1, 0), (16, 4), (129, 300), (700, 17)]


def view(k):
    return fq.fq_kv_view(k.data_ptr(), k.data_ptr(), k.shape[1], D, k.shape[1] * D)


def weights(w):
    return fq.fq_key_weights(w.data_ptr(), w.shape[1])


def log_sums(q, k_of, q_len, k_len, hq, hkv, window, sinks, scale=SCALE):
    out, r = [], 0
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        seen = visible(L, K, window, sinks)
        out.append(torch.stack([log_sum(q[r:r + L, h], k_of(s, h // (hq // hkv)), seen, scale)[0] for h in range(hq)], dim=1)
                   if L else torch.zeros(0, hq, dtype=torch.float64, device=DEV))
        r += L
    return torch.cat(out).float()


def gathered(q, lse, k, seen, scale):
    """One sequence and kv head: what its keys receive from q [L, G, D], in 64 bits, and the bound of the error.

    A weight 2^x, x = c q.k - log2(e) lse: the dot product carries at most 128 2^-24 sum_d |q_d k_d| scale, c and the
    product with it three roundings of the score, lse's product two of lse, the subtraction one of both; exp2 2^-21.  The
    weights of a tile are added up in 8 sums of 16 and these in 3 steps; tiles by compensated addition, whose error is 2 steps; 16
    partial sums of thread blocks and what the key had at most, a step each."""
    out, bound = (torch.zeros(k.shape[0], dtype=torch.float64, device=DEV) for _ in range(2))
    k = torch.where(seen.any(dim=0)[:, None], k.double(), 0.0)
    for g in range(q.shape[1]):
        x = q[:, g].double()
        s, e = x @ k.T * scale, lse[:, g, None].double()
        p = torch.where(seen, torch.exp(torch.where(seen, s - e, 0.0)), 0.0)
        dx = x.abs() @ k.abs().T * abs(scale) * 128 + 4 * s.abs() + torch.where(torch.isinf(e), 0.0, 3 * e.abs())
        out += p.sum(dim=0)
        bound += (p * (dx * 2.0 ** -24 + 2.0 ** -21)).sum(dim=0)
    return out, bound + out * (16 + 3 + 2 + 17) * 2.0 ** -24


def run(q, lse, views, q_len, k_len, hq, hkv, window, sinks, before, after, scale=SCALE, **kw):
    ws = junk(fq.fq_attn_key_weights_workspace(q_len, k_len, hq, hkv, window, sinks))
    fq.fq_attn_key_weights(q.data_ptr(), lse.data_ptr(), views, q_len, k_len, hq, hkv, window, sinks, scale, before, after,
                           ws.data_ptr(), ws.numel() * 4, stream(), **kw)
    fq.fq_attn_check(stream())


def assert_weights(got, was, ref, bound, what=""):
    tol = bound + 2.0 ** -23 * (ref + was.double().abs()) + 1e-37
    err = (got.double() - (ref + was.double())).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst {float((err / tol).max()):.3g} of it, " \
        f"first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("q_len,k_len", LENGTHS)
@pytest.mark.parametrize("window,sinks", MASKS)
def test_key_weights(hq, hkv, q_len, k_len, window, sinks):
    g = gen(hash((hq, tuple(q_len), tuple(k_len), window)) % 2 ** 31)
    q, rows = normal(g, sum(q_len), hq, D), sum(k_len)
    k = torch.full((hkv, rows + 130, D), NAN, dtype=torch.bfloat16, device=DEV)
    k[:, :rows] = normal(g, hkv, rows, D)
    first = [sum(k_len[:s]) for s in range(len(k_len))]
    k_of = lambda s, h: k[h, first[s]:first[s] + k_len[s]]  # noqa: E731
    lse = log_sums(q, k_of, q_len, k_len, hq, hkv, window, sinks)
    was = torch.rand(hkv, rows + 130, generator=g, device=DEV)
    got = torch.full((hkv, rows + 133), 5.0, device=DEV)
    run(q, lse, view(k), q_len, k_len, hq, hkv, window, sinks, weights(was), weights(got))
    zeros = torch.full((hkv, rows + 130), 5.0, device=DEV)
    run(q, lse, view(k), q_len, k_len, hq, hkv, window, sinks, None, weights(zeros))
    r = 0
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        seen = visible(L, K, window, sinks)
        at = slice(first[s], first[s] + K)
        for h in range(hkv):
            G = hq // hkv
            ref, bound = gathered(q[r:r + L, h * G:(h + 1) * G], lse[r:r + L, h * G:(h + 1) * G], k_of(s, h), seen, SCALE)
            assert_weights(got[h, at], was[h, at], ref, bound, f"sequence {s} head {h}")
            assert_weights(zeros[h, at], torch.zeros_like(was[h, at]), ref, bound, f"sequence {s} head {h} from zeros")
        r += L
    assert bool((got[:, rows:] == 5).all())
    run(q, lse, view(k), q_len, k_len, hq, hkv, window, sinks, weights(was), weights(was))   # in place, the same bits
    assert bool((was[:, :rows] == got[:, :rows]).all())


@pytest.mark.parametrize("hq,hkv,q_len,k_len", [(520, 520, [200, 1], [300, 700]), (1, 1, [9000, 3], [700, 90000]),
                                                (8, 1, [12] * 40, [30 * i for i in range(40)])])
def test_key_weights_many_and_few_heads(hq, hkv, q_len, k_len):
    """More kv heads than thread blocks; one, whose work all of them share out."""
    g = gen(33)
    q, rows = normal(g, sum(q_len), hq, D), sum(k_len)
    k = normal(g, hkv, rows, D)
    first = [sum(k_len[:s]) for s in range(len(k_len))]
    k_of = lambda s, h: k[h, first[s]:first[s] + k_len[s]]  # noqa: E731
    lse = log_sums(q, k_of, q_len, k_len, hq, hkv, 0, 0)
    w, again = torch.empty(hkv, rows, device=DEV), torch.empty(hkv, rows, device=DEV)
    run(q, lse, view(k), q_len, k_len, hq, hkv, 0, 0, None, weights(w))
    run(q, lse, view(k), q_len, k_len, hq, hkv, 0, 0, None, weights(again))
    assert bool((w == again).all())
    r, G = 0, hq // hkv
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        seen = visible(L, K, 0, 0)
        at = slice(first[s], first[s] + K)
        for h in range(0, hkv, max(1, hkv // 40)):
            ref, bound = gathered(q[r:r + L, h * G:(h + 1) * G], lse[r:r + L, h * G:(h + 1) * G], k_of(s, h), seen, SCALE)
            # (the sums of up to 152 parts of a line, a step each)
            assert_weights(w[h, at], torch.zeros_like(w[h, at]), ref, bound + ref * 152 * 2.0 ** -24, f"sequence {s} head {h}")
        r += L


def test_key_weights_of_one_row_sum_to_one():
    """Over its keys, a row's weights with the log-sum that fq_attn_window gave."""
    g, hq, hkv, q_len, k_len = gen(5), 8, 2, [1, 200], [3000, 1500]
    q, rows = normal(g, sum(q_len), hq, D), sum(k_len)
    k, v = normal(g, hkv, rows, D), normal(g, hkv, rows, D)
    for window, sinks in ((0, 0), (100, 4)):
        _, lse = run_window(q, fq.fq_kv_view(k.data_ptr(), v.data_ptr(), rows, D, rows * D), q_len, k_len, hq, hkv, window, sinks)
        w = torch.empty(hkv, rows, device=DEV)
        run(q, lse, view(k), q_len, k_len, hq, hkv, window, sinks, None, weights(w))
        r = 0
        for L, K in zip(q_len, k_len):
            total = w[:, r:r + K].double().sum(dim=1)
            # (a weight is off by the scores' and log-sums' errors, some 1e-5 at these sizes)
            assert float((total / (L * hq / hkv) - 1).abs().max()) < 2e-5
            r += K


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_key_weights_scales(scale):
    g, hq, hkv, L, K = gen(7), 4, 2, 200, 333
    q, k = normal(g, L, hq, D), normal(g, hkv, K, D)
    lse = log_sums(q, lambda s, h: k[h], [L], [K], hq, hkv, 90, 3, scale)
    w = torch.empty(hkv, K, device=DEV)
    run(q, lse, view(k), [L], [K], hq, hkv, 90, 3, None, weights(w), scale=scale)
    for h in range(hkv):
        ref, bound = gathered(q[:, 2 * h:2 * h + 2], lse[:, 2 * h:2 * h + 2], k[h], visible(L, K, 90, 3), scale)
        assert_weights(w[h], torch.zeros_like(w[h]), ref, bound)


def test_key_weights_views_rows_strides_and_many_sequences():
    """64 sequences with a view and weights of their own, row offsets, a row stride of q; other weights stay."""
    g, hq, hkv = gen(9), 8, 2
    q_len, k_len = [1, 0, 3, 70] * 16, [900, 5, 40, 300] * 15 + [2000, 0, 1, 800]
    row0 = [s % 5 for s in range(64)]
    T = sum(q_len)
    q = normal(g, T, hq * D + 8)
    heads = q[:, :hq * D].reshape(T, hq, D)
    ks = [normal(g, hkv, K + 7, D) for K in k_len]
    k_of = lambda s, h: ks[s][h, row0[s]:row0[s] + k_len[s]]  # noqa: E731
    lse = log_sums(heads, k_of, q_len, k_len, hq, hkv, 0, 0)
    was = [torch.rand(hkv, K + 7, generator=g, device=DEV) for K in k_len]
    got = [w.clone() for w in was]
    run(q, lse, [view(k) for k in ks], q_len, k_len, hq, hkv, 0, 0, [weights(w) for w in was], [weights(w) for w in got],
        kv_row0=row0, q_stride=hq * D + 8)
    r = 0
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        for h in range(hkv):
            ref, bound = gathered(heads[r:r + L, 4 * h:4 * h + 4], lse[r:r + L, 4 * h:4 * h + 4], k_of(s, h), visible(L, K, 0, 0), SCALE)
            at = slice(row0[s], row0[s] + K)
            assert_weights(got[s][h, at], was[s][h, at], ref, bound, f"sequence {s}")
            rest = [i for i in range(K + 7) if not row0[s] <= i < row0[s] + K]
            assert bool((got[s][h, rest] == was[s][h, rest]).all())
        r += L


@pytest.mark.parametrize("bad", [NAN, math.inf])
@pytest.mark.parametrize("L,K,window", [(200, 200, 50), (3, 300, 20), (300, 900, 100)])
def test_key_weights_rows_that_do_not_see_a_key(bad, L, K, window):
    """Query rows, keys and log-sums that are not finite reach only the keys whose sums they belong to; so do those of the
    sequence behind."""
    g, hq, hkv = gen(13), 4, 2
    q, k = normal(g, 2 * L, hq, D), normal(g, hkv, 2 * K, D)
    k_of = lambda s, h: k[h, s * K:(s + 1) * K]  # noqa: E731
    lse = log_sums(q, k_of, [L, L], [K, K], hq, hkv, window, 2)
    ref = [[gathered(q[s * L:(s + 1) * L, 2 * h:2 * h + 2], lse[s * L:(s + 1) * L, 2 * h:2 * h + 2], k_of(s, h), visible(L, K, window, 2), SCALE)
            for h in range(hkv)] for s in range(2)]
    row = L // 2
    q[row, 0, 7] = bad          # head 0 of kv head 0
    lse[L + row, 3] = NAN       # head 1 of kv head 1, second sequence
    k[1, 5, 9] = bad
    w = torch.empty(hkv, 2 * K, device=DEV)
    run(q, lse, view(k), [L, L], [K, K], hq, hkv, window, 2, None, weights(w))
    sees = visible(L, K, window, 2)[row]
    for s in range(2):
        for h in range(hkv):
            touched = torch.zeros(K, dtype=torch.bool, device=DEV)
            if (s, h) in ((0, 0), (1, 1)):
                touched |= sees
            if (s, h) == (0, 1):
                touched[5] = True
            part = w[h, s * K:(s + 1) * K]
            r, b = ref[s][h]
            assert_weights(part[~touched], torch.zeros_like(part[~touched]), r[~touched], b[~touched], f"{s} {h}")


@pytest.mark.parametrize("L,K", [(1, 300), (20, 500), (700, 900), (4000, 4000)])
@pytest.mark.parametrize("low", [-math.inf, -1e6])
def test_weights_beyond_f32_are_infinite(L, K, low):
    """A log-sum far below its row's scores: the formula is infinite in f32 for every key that the row sees, and stays so
    whatever is added behind it; the other head's keys have what they had."""
    g, hq, hkv = gen(17), 4, 2
    q, k = normal(g, L, hq, D), normal(g, hkv, K, D)
    lse = log_sums(q, lambda s, h: k[h], [L], [K], hq, hkv, 0, 0)
    row = L // 3
    lse[row, 1] = low
    w = torch.empty(hkv, K, device=DEV)
    run(q, lse, view(k), [L], [K], hq, hkv, 0, 0, None, weights(w))
    seen = visible(L, K, 0, 0)
    assert bool((w[0, seen[row]] == math.inf).all())
    ref, bound = gathered(q[:, :2], lse[:, :2], k[0], seen, SCALE)
    rest = ~seen[row]
    assert_weights(w[0, rest], torch.zeros_like(w[0, rest]), ref[rest], bound[rest])
    ref, bound = gathered(q[:, 2:], lse[:, 2:], k[1], seen, SCALE)
    assert_weights(w[1], torch.zeros_like(w[1]), ref, bound)


def plain_evict(w, n, sinks, recent):
    """The rows of one head that stay, by sorting."""
    K = w.shape[0]
    if n == K:
        return torch.arange(K, device=w.device)
    x = w.clone()
    x[torch.isnan(x)] = math.inf
    nan, x = torch.isnan(w).tolist(), x.tolist()
    # NaN first, then by weight, then by row
    ranked = sorted(range(sinks, K - recent), key=lambda j: (not nan[j], -x[j], j))[:n - sinks - recent]
    return torch.tensor(sorted(ranked + list(range(sinks)) + list(range(K - recent, K))), device=w.device, dtype=torch.long)


def kinds(g, kind, hkv, K):
    w = torch.rand(hkv, K, generator=g, device=DEV)
    if kind == "ties":
        return (w * 4).floor()
    if kind == "same":
        return torch.full_like(w, 0.5)
    if kind == "odd":      # infinities, NaN, zeros of both signs, negative and tiny numbers
        w = torch.where(w < 0.1, -0.0, torch.where(w < 0.2, 0.0, (w - 0.6) * 1e-39 if K % 2 else w - 0.6))
        w[:, ::7] = math.inf
        w[:, 3::11] = -math.inf
        w[:, 5::97] = NAN
        return w
    return w ** 8


@pytest.mark.parametrize("kind", ["wide", "ties", "same", "odd"])
@pytest.mark.parametrize("K,keep,sinks,recent", [(1, 1, 0, 0), (2, 1, 0, 0), (2, 1, 1, 0), (5, 0, 0, 0), (300, 300, 4, 4), (300, 400, 500, 4),
                                                 (300, 299, 4, 32), (513, 100, 0, 100), (513, 100, 100, 0), (4096, 1000, 4, 32),
                                                 (4097, 4000, 4, 32), (9001, 17, 0, 1), (40000, 12345, 100, 300)])
def test_evict(kind, K, keep, sinks, recent):
    g, hkv = gen(hash((kind, K, keep)) % 2 ** 31), 2
    k, v = normal(g, hkv, K, D), normal(g, hkv, K, D)
    w = kinds(g, kind, hkv, K)
    n = min(K, keep)
    tk, tv = (torch.full((hkv, n + 3, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tw = torch.full((hkv, n + 3), 7.0, device=DEV)
    kept = torch.full((hkv * n + 4,), -5, dtype=torch.int32, device=DEV)
    fq.fq_kv_evict(fq.fq_kv_view(k.data_ptr(), v.data_ptr(), K, D, K * D), weights(w), None, [K], [keep], sinks, recent, hkv,
                   fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), n + 3, D, (n + 3) * D), weights(tw), None, kept.data_ptr(), stream())
    for h in range(hkv):
        want = plain_evict(w[h], n, sinks, recent)
        assert kept[h * n:(h + 1) * n].tolist() == want.tolist()
        assert bool((tk[h, :n] == k[h, want]).all()) and bool((tv[h, :n] == v[h, want]).all())
        assert bool((tw[h, :n].view(torch.int32) == w[h, want].view(torch.int32)).all())
        for t in (tk[h, n:], tv[h, n:], tw[h, n:]):
            assert bool((t == 7).all())
    assert bool((kept[hkv * n:] == -5).all())


@pytest.mark.parametrize("own", [False, True])
def test_evict_many_sequences(own):
    """Ragged sequences, empty ones among them, in one view or a view each, at row offsets, with and without weights."""
    g, hkv, sinks, recent = gen(17), 3, 2, 5
    k_len = [100, 0, 7, 5000, 333, 64, 1] + [211] * 57
    keep = [50, 9, 7, 700, 7, 100, 0] + [30 + s for s in range(57)]
    sinks, recent = 0, 0
    n = [min(a, b) for a, b in zip(k_len, keep)]
    S = len(k_len)
    kept = torch.full((hkv * sum(n),), -5, dtype=torch.int32, device=DEV)
    if own:
        row0, at = [s % 4 for s in range(S)], [s % 3 for s in range(S)]
        ks, vs = ([normal(g, K + 5, hkv, D + 8) for K in k_len] for _ in range(2))     # [row][head][D + 8]
        ws = [kinds(g, "ties", hkv, K + 5) for K in k_len]
        tk, tv = ([torch.zeros(hkv, m + 4, D, dtype=torch.bfloat16, device=DEV) for m in n] for _ in range(2))
        fq.fq_kv_evict([fq.fq_kv_view(a.data_ptr(), b.data_ptr(), K + 5, hkv * (D + 8), D + 8) for a, b, K in zip(ks, vs, k_len)],
                       [weights(w) for w in ws], row0, k_len, keep, sinks, recent, hkv,
                       [fq.fq_kv_view(a.data_ptr(), b.data_ptr(), m + 4, D, (m + 4) * D) for a, b, m in zip(tk, tv, n)], None, at,
                       kept.data_ptr(), stream())
        src = lambda s, h: (ks[s][row0[s]:, h, :D], vs[s][row0[s]:, h, :D], ws[s][h, row0[s]:row0[s] + k_len[s]])  # noqa: E731
        dst = lambda s, h: (tk[s][h, at[s]:at[s] + n[s]], tv[s][h, at[s]:at[s] + n[s]])  # noqa: E731
    else:
        R, N = sum(k_len), sum(n)
        k, v, w = normal(g, hkv, R, D), normal(g, hkv, R, D), kinds(g, "wide", hkv, R)
        tk, tv = (torch.zeros(hkv, N, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        fq.fq_kv_evict(fq.fq_kv_view(k.data_ptr(), v.data_ptr(), R, D, R * D), weights(w), None, k_len, keep, sinks, recent, hkv,
                       fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), N, D, N * D), None, None, kept.data_ptr(), stream())
        src = lambda s, h: tuple(t[h, sum(k_len[:s]):sum(k_len[:s + 1])] for t in (k, v, w))  # noqa: E731
        dst = lambda s, h: tuple(t[h, sum(n[:s]):sum(n[:s + 1])] for t in (tk, tv))  # noqa: E731
    for s in range(S):
        for h in range(hkv):
            a, b, x = src(s, h)
            want = plain_evict(x, n[s], sinks, recent)
            first = hkv * sum(n[:s]) + h * n[s]
            assert kept[first:first + n[s]].tolist() == want.tolist(), s
            c, d = dst(s, h)
            assert bool((c == a[want]).all()) and bool((d == b[want]).all())


def test_captured_and_replayed():
    """The weights and the eviction in one graph, replayed with other queries."""
    g, hq, hkv, L, K, keep = gen(19), 8, 2, 300, 2000, 500
    q, k, v = normal(g, L, hq, D), normal(g, hkv, K, D), normal(g, hkv, K, D)
    lse = torch.empty(L, hq, device=DEV)
    w = torch.empty(hkv, K, device=DEV)
    tk, tv = (torch.empty(hkv, keep, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kept = torch.empty(hkv * keep, dtype=torch.int32, device=DEV)
    ws = junk(fq.fq_attn_key_weights_workspace([L], [K], hq, hkv, 0, 0))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        s = torch.cuda.current_stream(DEV).cuda_stream
        fq.fq_attn_key_weights(q.data_ptr(), lse.data_ptr(), view(k), [L], [K], hq, hkv, 0, 0, SCALE, None, weights(w), ws.data_ptr(),
                               ws.numel() * 4, s)
        fq.fq_kv_evict(fq.fq_kv_view(k.data_ptr(), v.data_ptr(), K, D, K * D), weights(w), None, [K], [keep], 4, 32, hkv,
                       fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), keep, D, keep * D), None, None, kept.data_ptr(), s)
    for _ in range(2):
        q.copy_(normal(g, L, hq, D))
        lse.copy_(log_sums(q, lambda s, h: k[h], [L], [K], hq, hkv, 0, 0))
        graph.replay()
        torch.cuda.synchronize()
        fq.fq_attn_check(stream())
        for h in range(hkv):
            ref, bound = gathered(q[:, 4 * h:4 * h + 4], lse[:, 4 * h:4 * h + 4], k[h], visible(L, K, 0, 0), SCALE)
            assert_weights(w[h], torch.zeros_like(w[h]), ref, bound)
            assert kept[h * keep:(h + 1) * keep].tolist() == plain_evict(w[h], keep, 4, 32).tolist()


def test_a_shortened_cache_in_use():
    """A prompt with its log-sums, the weights of its last rows, the cache made shorter, and tokens that attend to what
    stayed: against attention over the rows that stayed, head by head."""
    g, hq, hkv, P, keep, sinks, recent = gen(23), 8, 2, 700, 200, 4, 32
    q, k, v = normal(g, P, hq, D), normal(g, hkv, P, D), normal(g, hkv, P, D)
    whole = fq.fq_kv_view(k.data_ptr(), v.data_ptr(), P, D, P * D)
    _, lse = run_window(q, whole, [P], [P], hq, hkv, 0, 0)
    w = torch.empty(hkv, P, device=DEV)
    last = 64
    run(q[P - last:], lse[P - last:], view(k), [last], [P], hq, hkv, 0, 0, None, weights(w))
    cap = keep + 50
    tk, tv = (torch.full((hkv, cap, D), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tw = torch.zeros(hkv, cap, device=DEV)
    kept = torch.empty(hkv * keep, dtype=torch.int32, device=DEV)
    short = fq.fq_kv_view(tk.data_ptr(), tv.data_ptr(), cap, D, cap * D)
    fq.fq_kv_evict(whole, weights(w), None, [P], [keep], sinks, recent, hkv, short, weights(tw), None, kept.data_ptr(), stream())
    for i in range(3):
        at = keep + i
        tk[:, at], tv[:, at] = normal(g, hkv, D), normal(g, hkv, D)
        x = normal(g, 1, hq, D)
        out, e = run_window(x, short, [1], [at + 1], hq, hkv, 0, 0, out_dtype="f32")
        was = tw.clone()
        run(x, e, fq.fq_kv_view(tk.data_ptr(), 0, cap, D, cap * D), [1], [at + 1], hq, hkv, 0, 0, weights(was), weights(tw))
        for h in range(hkv):
            rows = kept[h * keep:(h + 1) * keep].long()
            assert rows.tolist() == plain_evict(w[h], keep, sinks, recent).tolist()
            kk, vv = torch.cat((k[h, rows], tk[h, keep:at + 1])).double(), torch.cat((v[h, rows], tv[h, keep:at + 1])).double()
            p = torch.softmax(x[0, 4 * h:4 * h + 4].double() @ kk.T * SCALE, dim=1)
            # (weights are rounded to bf16 for the product with V: 2^-8 of them at most)
            assert bool(((out[0, 4 * h:4 * h + 4].double() - p @ vv).abs() <= 1.1 * 2.0 ** -8 * (p @ vv.abs())).all())
            assert float((tw[h, :at + 1].double() - was[h, :at + 1].double() - p.sum(dim=0)).abs().max()) < 1e-4
