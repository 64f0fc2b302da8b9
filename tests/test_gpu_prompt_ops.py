"""The prompt and shared-prompt attention operators on the GPU against plain 64-bit forms, at
the sizes, masks, layouts and streams where they can go wrong."""
import math

import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.prompt_ops_util import BF16_HALF_STEP, D, DEV, assert_within, attend, causal, gen, normal

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(D)
NAN = float("nan")


def stream():
    return torch.cuda.current_stream(DEV).cuda_stream


def workspace(n, fill=NAN):
    """A workspace whose contents are junk."""
    return torch.full((max(1, -(-n // 4)),), fill, dtype=torch.float32, device=DEV)


def layer(g, rows, hkv, layout="cache", pad=0, fill=NAN):
    """K or V storage of `rows` rows plus `pad` rows of `fill`, as [hkv, rows + pad, D] (cache layer) or
    [rows + pad, hkv, D] (packed), and its (row, head) strides."""
    if layout == "cache":
        t = torch.full((hkv, rows + pad, D), fill, dtype=torch.bfloat16, device=DEV)
        t[:, :rows] = normal(g, hkv, rows, D)
        return t, t, D, (rows + pad) * D
    t = torch.full((rows + pad, hkv, D + 16), fill, dtype=torch.bfloat16, device=DEV)
    t[:rows, :, :D] = normal(g, rows, hkv, D)
    return t, t.transpose(0, 1)[:, :, :D], hkv * (D + 16), D + 16


def view_of(k, v, rows, rs, hs):
    return fq.fq_kv_view(k.data_ptr(), v.data_ptr(), rows, rs, hs)


def run_prompt(q, views, q_len, k_len, hq, hkv, kv_row0=None, out=None, out_dtype="bf16", q_stride=0, out_stride=0,
               scale=SCALE):
    ws = workspace(fq.fq_attn_prompt_workspace(q_len, k_len, hq, hkv))
    if out is None:
        out = torch.full((sum(q_len), hq, D), NAN, device=DEV, dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    fq.fq_attn_prompt(q.data_ptr(), views, q_len, k_len, hq, hkv, scale, out.data_ptr(), ws.data_ptr(), ws.numel() * 4,
                      stream(), kv_row0=kv_row0, q_stride=q_stride, out_stride=out_stride, out_dtype=out_dtype)
    fq.fq_attn_check(stream())
    return out


def reference_prompt(q, kv, q_len, k_len, hq, hkv, scale=SCALE):
    """kv(s, h) -> (k, v) [k_len, D] of sequence s and kv head h."""
    out, bound, r = [], [], 0
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        o, b = torch.zeros(L, hq, D, dtype=torch.float64, device=DEV), torch.zeros(L, hq, D, dtype=torch.float64, device=DEV)
        for h in range(hq):
            k, v = kv(s, h // (hq // hkv))
            o[:, h], b[:, h] = attend(q[r:r + L, h], k, v, causal(L, K), scale)
        out.append(o)
        bound.append(b)
        r += L
    return torch.cat(out), torch.cat(bound)


HEADS = [(4, 4), (4, 2), (8, 2), (8, 1)]
# (query lengths, key lengths): whole prompts of one token, around the tile sizes, ragged and
# empty ones; chunks behind cached rows; more queries than keys (rows that see nothing); few
# rows over many keys; no keys at all
LENGTHS = [([1], [1]), ([2], [2]), ([31, 1, 33], [31, 1, 33]), ([127, 128, 129], [127, 128, 129]),
           ([255, 0, 257, 5], [255, 0, 257, 5]), ([640], [640]), ([1000, 3], [1000, 3]), ([17, 40], [217, 1000]),
           ([1, 1, 2, 1], [1, 300, 129, 4096]), ([300], [40]), ([9, 4, 3], [2, 0, 3]), ([130], [3000]),
           ([64], [20000]), ([1], [30000])]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("q_len,k_len", LENGTHS)
@pytest.mark.parametrize("layout,out_dtype", [("cache", "bf16"), ("packed", "f32")])
def test_prompt(hq, hkv, q_len, k_len, layout, out_dtype):
    g = gen(hash((hq, hkv, tuple(q_len))) % 2 ** 31)
    q = normal(g, sum(q_len), hq, D)
    rows = sum(k_len)
    ks, k, rs, hs = layer(g, rows, hkv, layout, pad=200)
    vs, v, _, _ = layer(g, rows, hkv, layout, pad=200)
    got = run_prompt(q, view_of(ks, vs, rows + 200, rs, hs), q_len, k_len, hq, hkv, out_dtype=out_dtype)
    k0 = [sum(k_len[:s]) for s in range(len(k_len))]
    ref, bound = reference_prompt(q, lambda s, h: (k[h, k0[s]:k0[s] + k_len[s]], v[h, k0[s]:k0[s] + k_len[s]]), q_len, k_len, hq, hkv)
    assert_within(got, ref, bound, out_dtype == "bf16", f"{hq}/{hkv} {q_len} {k_len}")


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("own_views", [False, True])
def test_prompt_few_rows_beside_long_ones(hq, hkv, own_views):
    """Sequences of a few rows next to one that is split along its keys: short ones take part in its
    kernel (and are split too), long ones run beside it; one view for all, or a view each."""
    g = gen(91 + hq + own_views)
    q_len, k_len = [60, 1, 2, 0, 1, 1], [4000, 1000, 700, 5, 3000, 0]
    q = normal(g, sum(q_len), hq, D)
    if own_views:
        stores = [(layer(g, max(K, 1), hkv, pad=150), layer(g, max(K, 1), hkv, pad=150)) for K in k_len]
        views = [view_of(k[0], v[0], max(K, 1) + 150, k[2], k[3]) for (k, v), K in zip(stores, k_len)]
        kv = lambda s, h: tuple(t[1][h, :k_len[s]] for t in stores[s])  # noqa: E731
    else:
        k, v = layer(g, sum(k_len), hkv, pad=150), layer(g, sum(k_len), hkv, pad=150)
        views = view_of(k[0], v[0], sum(k_len) + 150, k[2], k[3])
        kv = lambda s, h: tuple(t[1][h, sum(k_len[:s]):sum(k_len[:s + 1])] for t in (k, v))  # noqa: E731
    ref, bound = reference_prompt(q, kv, q_len, k_len, hq, hkv)
    for out_dtype in ("bf16", "f32"):
        got = run_prompt(q, views, q_len, k_len, hq, hkv, out_dtype=out_dtype)
        assert_within(got, ref, bound, out_dtype == "bf16", f"{hq}/{hkv} {out_dtype}")


def test_prompt_views_rows_and_strides():
    """A view per sequence (one of them used twice, at overlapping rows), row offsets, row strides of q and
    out; what lies between the rows of out and behind them stays."""
    g, hq, hkv = gen(5), 8, 2
    q_len, k_len, row0 = [40, 200, 1, 77], [140, 200, 500, 77], [3, 0, 9, 100]
    caps = [150, 200, 520, 200]
    stores = [(layer(g, c, hkv), layer(g, c, hkv)) for c in caps[:3]]
    stores.append(stores[1])   # the second sequence's cache again
    views = [view_of(k[0], v[0], c, k[2], k[3]) for (k, v), c in zip(stores, caps)]
    T = sum(q_len)
    q = normal(g, T, hq * D + 8)
    out = torch.full((T + 3, hq * D + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    run_prompt(q, views, q_len, k_len, hq, hkv, kv_row0=[3, 0, 9, 100], out=out, q_stride=hq * D + 8, out_stride=hq * D + 24)
    kv = lambda s, h: tuple(t[1][h, row0[s]:row0[s] + k_len[s]] for t in stores[s])  # noqa: E731
    ref, bound = reference_prompt(q[:, :hq * D].reshape(T, hq, D), kv, q_len, k_len, hq, hkv)
    assert_within(out[:T, :hq * D].reshape(T, hq, D), ref, bound, True)
    assert bool((out[T:] == 7).all()) and bool((out[:, hq * D:] == 7).all())


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("where", ["k", "v", "kv"])
@pytest.mark.parametrize("hq,hkv,at,L,K", [(4, 4, 100, 300, 300), (4, 2, 128, 300, 300), (8, 1, 299, 300, 300),
                                           (4, 2, 0, 300, 300), (8, 2, 250, 20, 260), (8, 2, 255, 3, 256)])
def test_prompt_future_values_do_not_leak(bad, where, hq, hkv, at, L, K):
    """A key that a row does not see has no influence on it, whatever it holds.  Rows that see it
    give what the definition gives: checked where that is finite or NaN throughout."""
    g = gen(11)
    q = normal(g, L, hq, D)
    k, v = normal(g, hkv, K, D), normal(g, hkv, K, D)
    if "k" in where:
        k[:, at, 5:9] = bad
    if "v" in where:
        v[:, at, 60:70] = bad
    got = run_prompt(q, view_of(k, v, K, D, K * D), [L], [K], hq, hkv)
    kc, vc = k.clone(), v.clone()
    kc[:, at], vc[:, at] = 0, 0
    ref, bound = reference_prompt(q, lambda s, h: (kc[h], vc[h]), [L], [K], hq, hkv)
    blind = max(0, at - (K - L))   # rows before the key
    assert_within(got[:blind], ref[:blind], bound[:blind], True, "rows before the key")
    if math.isnan(bad):
        if "k" in where:
            assert bool(got[blind:].isnan().all())
        else:
            assert bool(got[blind:, :, 60:70].isnan().all())
            assert not bool(got[blind:, :, :60].isnan().any()) and not bool(got[blind:, :, 70:].isnan().any())
    elif where == "v" and math.isinf(bad):   # a positive weight times an infinity
        assert bool((got[blind:, :, 60:70] == bad).all())


def test_prompt_scores_of_minus_infinity_and_large_ones():
    """Keys whose scores are -inf weigh nothing; a row with nothing else is 0 / 0 as the definition
    says.  Scores of +-1e4 select single keys without overflow; a row's scores may all be equal."""
    g, hq, hkv, L = gen(13), 4, 2, 200
    q = normal(g, L, hq, D).abs() + 0.5
    k, v = normal(g, hkv, L, D), normal(g, hkv, L, D)
    k[:, 0:50] = -math.inf
    got = run_prompt(q, view_of(k, v, L, D, L * D), [L], [L], hq, hkv)
    assert bool(got[:50].isnan().all())
    kc = k[:, 50:]
    ref, bound = reference_prompt(q[50:], lambda s, h: (kc[h], v[h, 50:]), [L - 50], [L - 50], hq, hkv)
    assert_within(got[50:], ref, bound, True, "rows with finite scores")
    q = normal(g, L, hq, D) * 30
    k = normal(g, hkv, L, D) * 30
    got = run_prompt(q, view_of(k, v, L, D, L * D), [L], [L], hq, hkv)
    ref, bound = reference_prompt(q, lambda s, h: (k[h], v[h]), [L], [L], hq, hkv)
    assert_within(got, ref, bound, True, "large scores")
    k[:] = 0
    got = run_prompt(q, view_of(k, v, L, D, L * D), [L], [L], hq, hkv)
    ref, bound = reference_prompt(q, lambda s, h: (k[h], v[h]), [L], [L], hq, hkv)
    assert_within(got, ref, bound, True, "equal scores")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_prompt_scale(scale):
    g, hq, hkv, L = gen(17), 4, 2, 150
    q, k, v = normal(g, L, hq, D), normal(g, hkv, L, D), normal(g, hkv, L, D)
    got = run_prompt(q, view_of(k, v, L, D, L * D), [L], [L], hq, hkv, scale=scale)
    ref, bound = reference_prompt(q, lambda s, h: (k[h], v[h]), [L], [L], hq, hkv, scale)
    assert_within(got, ref, bound, True)


def test_prompt_growing_scores():
    """Scores that keep growing along the keys: the running maximum moves at every tile."""
    g, hq, hkv, L = gen(19), 4, 2, 1500
    q, v = normal(g, L, hq, D), normal(g, hkv, L, D)
    q[:, :, 0] = 8.0
    k = normal(g, hkv, L, D) * 0.1
    k[:, :, 0] = torch.linspace(-40, 40, L, device=DEV)
    got = run_prompt(q, view_of(k, v, L, D, L * D), [L], [L], hq, hkv)
    ref, bound = reference_prompt(q, lambda s, h: (k[h], v[h]), [L], [L], hq, hkv)
    assert_within(got, ref, bound, True)


def test_prompt_many_calls_in_a_row():
    """Calls queued behind one another: the same bits every time and no wait that gave up.  Lengths whose
    last units have an empty second tile, single tokens, one-tile units and splits among them."""
    g, hq, hkv = gen(29), 32, 8
    q_len = [1, 37, 129, 255, 64, 640, 771, 901, 65, 1187]
    rows, T = sum(q_len), sum(q_len)
    k, v = normal(g, hkv, rows, D), normal(g, hkv, rows, D)
    qs = [normal(g, T, hq, D) for _ in range(2)]
    ws = workspace(fq.fq_attn_prompt_workspace(q_len, q_len, hq, hkv))
    outs = [torch.empty_like(qs[0]) for _ in range(4)]
    for i in range(400):
        fq.fq_attn_prompt(qs[i & 1].data_ptr(), view_of(k, v, rows, D, rows * D), q_len, q_len, hq, hkv, SCALE,
                          outs[i & 1 if i < 2 else 2 + (i & 1)].data_ptr(), ws.data_ptr(), ws.numel() * 4, stream())
    fq.fq_attn_check(stream())
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    k0 = [sum(q_len[:s]) for s in range(len(q_len))]
    ref, bound = reference_prompt(qs[1], lambda s, h: (k[h, k0[s]:k0[s] + q_len[s]], v[h, k0[s]:k0[s] + q_len[s]]), q_len, q_len, hq, hkv)
    assert_within(outs[3], ref, bound, True)


def test_prompt_long_cache_offsets():
    """Rows and heads whose element offsets pass 2^32."""
    g, hq, hkv = gen(23), 4, 2
    rows, used = (1 << 31) // D + 4096, 1300   # one head alone has more than 2^31 elements, two pass 2^32
    k = torch.empty(hkv, rows, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    r0 = rows - used
    k[:, r0:], v[:, r0:] = normal(g, hkv, used, D), normal(g, hkv, used, D)
    for q_len in ([used], [3]):
        q = normal(g, q_len[0], hq, D)
        got = run_prompt(q, view_of(k, v, rows, D, rows * D), q_len, [used], hq, hkv, kv_row0=[r0])
        ref, bound = reference_prompt(q, lambda s, h: (k[h, r0:], v[h, r0:]), q_len, [used], hq, hkv)
        assert_within(got, ref, bound, True)


def run_shared(q, prefix, prefix_len, tails, tail_len, hq, hkv, out=None, out_dtype="bf16", scale=SCALE, **kw):
    ws = workspace(fq.fq_attn_shared_workspace(prefix_len, tail_len, hq, hkv))
    if out is None:
        out = torch.full((len(tail_len), hq, D), NAN, device=DEV, dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    fq.fq_attn_shared(q.data_ptr(), prefix, prefix_len, tails, tail_len, hq, hkv, scale, out.data_ptr(), ws.data_ptr(),
                      ws.numel() * 4, stream(), out_dtype=out_dtype, **kw)
    fq.fq_attn_check(stream())
    return out


def reference_shared(q, pk, pv, tk, tv, tail_len, hq, hkv, scale=SCALE):
    """pk, pv [hkv, P, D]; tk[s], tv[s] [hkv, >= tail_len[s], D]"""
    out = torch.zeros(len(tail_len), hq, D, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(out)
    for s, t in enumerate(tail_len):
        for h in range(hkv):
            k, v = torch.cat((pk[h], tk[s][h, :t])), torch.cat((pv[h], tv[s][h, :t]))
            hs = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            seen = torch.ones(hq // hkv, k.shape[0], dtype=torch.bool, device=DEV)
            out[s, hs], bound[s, hs] = attend(q[s, hs], k, v, seen, scale)
    return out, bound


# (prefix, tails): one sequence and many, no prefix, no tails, neither, odd lengths, long ones
SHARED = [(1, [0]), (0, [1]), (0, [0, 3]), (128, [0, 0, 0]), (129, [1, 0, 17]), (500, [1, 3, 9, 17]),
          (1000, [5] * 16), (4097, [300, 1, 0, 128, 129]), (777, list(range(64))), (20000, [7, 2000]),
          (3, [4000, 0, 1]), (9000, [0] * 33), (256, [64] * 64)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("P,tail_len", SHARED)
@pytest.mark.parametrize("layout,out_dtype", [("cache", "bf16"), ("packed", "f32")])
def test_shared(hq, hkv, P, tail_len, layout, out_dtype):
    g = gen(P + len(tail_len))
    n = len(tail_len)
    q = normal(g, n, hq, D)
    pks, pk, prs, phs = layer(g, P, hkv, layout, pad=100)
    pvs, pv, _, _ = layer(g, P, hkv, layout, pad=100)
    tk = [layer(g, t, hkv, layout, pad=1 + s % 3) for s, t in enumerate(tail_len)]
    tv = [layer(g, t, hkv, layout, pad=1 + s % 3) for s, t in enumerate(tail_len)]
    tails = [view_of(a[0], b[0], t + 1 + s % 3, a[2], a[3]) for s, (a, b, t) in enumerate(zip(tk, tv, tail_len))]
    got = run_shared(q, view_of(pks, pvs, P + 100, prs, phs), P, tails, tail_len, hq, hkv, out_dtype=out_dtype)
    ref, bound = reference_shared(q, pk[:, :P], pv[:, :P], [a[1] for a in tk], [b[1] for b in tv], tail_len, hq, hkv)
    assert_within(got, ref, bound, out_dtype == "bf16", f"{hq}/{hkv} {P} {tail_len}")


def test_shared_tail_used_twice_strides_and_absent_parts():
    g, hq, hkv, n = gen(31), 8, 2, 5
    tail_len = [40, 7, 0, 40, 130]
    P = 700
    pk, pv = normal(g, hkv, P, D), normal(g, hkv, P, D)
    tk = [normal(g, hkv, 140, D) for _ in range(n)]
    tv = [normal(g, hkv, 140, D) for _ in range(n)]
    tk[3], tv[3] = tk[0], tv[0]   # two sequences over one tail
    tails = [view_of(a, b, 140, D, 140 * D) for a, b in zip(tk, tv)]
    q = normal(g, n, hq * D + 40)
    out = torch.full((n + 2, hq * D + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    q0 = q[:, :hq * D].reshape(n, hq, D)
    run_shared(q, view_of(pk, pv, P, D, P * D), P, tails, tail_len, hq, hkv, out=out, q_stride=hq * D + 40, out_stride=hq * D + 8)
    ref, bound = reference_shared(q0, pk, pv, tk, tv, tail_len, hq, hkv)
    assert_within(out[:n, :hq * D].reshape(n, hq, D), ref, bound, True)
    assert bool((out[n:] == 7).all()) and bool((out[:, hq * D:] == 7).all())
    q0 = q0.contiguous()
    got = run_shared(q0, None, 0, tails, tail_len, hq, hkv)   # no prefix
    ref, bound = reference_shared(q0, pk[:, :0], pv[:, :0], tk, tv, tail_len, hq, hkv)
    assert_within(got, ref, bound, True)
    got = run_shared(q0, view_of(pk, pv, P, D, P * D), P, None, [0] * n, hq, hkv)   # no tails
    ref, bound = reference_shared(q0, pk, pv, tk, tv, [0] * n, hq, hkv)
    assert_within(got, ref, bound, True)
    assert bool((run_shared(q0, None, 0, None, [0] * n, hq, hkv) == 0).all())   # no keys


@pytest.mark.parametrize("bad", [NAN, math.inf])
def test_shared_rows_behind_the_ends_do_not_leak(bad):
    g, hq, hkv, P = gen(37), 8, 2, 333
    tail_len = [1, 15, 16, 17, 33, 0]
    pk, pv = normal(g, hkv, 400, D), normal(g, hkv, 400, D)
    pk[:, P:], pv[:, P:] = bad, bad
    tk, tv = normal(g, 6, hkv, 40, D), normal(g, 6, hkv, 40, D)
    for s, t in enumerate(tail_len):
        tk[s, :, t:], tv[s, :, t:] = bad, bad
    q = normal(g, 6, hq, D)
    tails = [view_of(tk[s], tv[s], 40, D, 40 * D) for s in range(6)]
    got = run_shared(q, view_of(pk, pv, 400, D, 400 * D), P, tails, tail_len, hq, hkv)
    ref, bound = reference_shared(q, pk[:, :P], pv[:, :P], tk, tv, tail_len, hq, hkv)
    assert_within(got, ref, bound, True)
    tv[1, :, 3, 7] = bad   # a value that sequence 1 sees: its own column only
    got2 = run_shared(q, view_of(pk, pv, 400, D, 400 * D), P, tails, tail_len, hq, hkv)
    hit = torch.zeros(6, hq, D, dtype=torch.bool, device=DEV)
    hit[1, :, 7] = True
    assert torch.equal(got2[~hit], got[~hit])
    assert bool((got2[hit].isnan() if math.isnan(bad) else got2[hit] == bad).all())


def rows_case(g, lens, hq, hkv):
    T = sum(lens)
    return normal(g, T, (hq + 2 * hkv) * D, dtype=torch.float32) * 3, 1 + 0.1 * normal(g, D, dtype=torch.float32), \
        1 + 0.1 * normal(g, D, dtype=torch.float32)


def rope_table(n, theta=1e6):
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * theta ** (-torch.arange(0, D, 2, dtype=torch.float64, device=DEV) / D)
    return torch.stack((a.cos(), a.sin()), dim=-1).float().contiguous()


def reference_rows(qkv, qn, kn, eps, rope, pos, hq, hkv):
    """q, k, v in 64 bits and the bound before rounding to bf16: the 128-term sum of squares and the
    roundings of the norm (128 + 8 halves of 2^-23, one half of the sum's error reaches the root) and the
    rotation's two products and sum, relative to |a c| + |b s|."""
    x = qkv.double().reshape(-1, hq + 2 * hkv, D)
    y = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps)
    y[:, :hq] *= qn.double()
    y[:, hq:hq + hkv] *= kn.double()
    c, s = rope[pos].double()[:, None, :, 0], rope[pos].double()[:, None, :, 1]
    a, b = y[..., :64], y[..., 64:]
    z = torch.cat((a * c - b * s, a * s + b * c), dim=-1)
    bound = torch.cat(((a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()), dim=-1) * (128 + 16) * 2.0 ** -24
    return (z[:, :hq], bound[:, :hq]), (z[:, hq:hq + hkv], bound[:, hq:hq + hkv]), x[:, hq + hkv:]


@pytest.mark.parametrize("hq,hkv", HEADS + [(16, 8), (3, 3)])
@pytest.mark.parametrize("lens,pos0", [([1], [0]), ([1], [39999]), ([5, 0, 2], [7, 3, 30000]), ([1] * 64, list(range(64))),
                                       ([200, 33], [0, 1000])])
def test_rows(hq, hkv, lens, pos0):
    g = gen(41)
    qkv, qn, kn = rows_case(g, lens, hq, hkv)
    rope = rope_table(40000)
    T, cap = sum(lens), sum(lens) + 20
    k, v = (torch.full((hkv, cap, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    row0 = [3 + sum(lens[:i]) for i in range(len(lens))]
    q = torch.full((T + 1, hq * D + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    fq.fq_qk_norm_rope(qkv.data_ptr(), lens, pos0, view_of(k, v, cap, D, cap * D), row0, hq, hkv, qn.data_ptr(), kn.data_ptr(),
                       1e-6, rope.data_ptr(), 40000, q.data_ptr(), stream(), q_stride=hq * D + 8)
    torch.cuda.synchronize()
    pos = torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(pos0, lens)])
    (rq, bq), (rk, bk), rv = reference_rows(qkv, qn, kn, 1e-6, rope, pos, hq, hkv)
    assert_within(q[:T, :hq * D].reshape(T, hq, D), rq, bq, True, "q")
    assert_within(k[:, 3:3 + T].transpose(0, 1), rk, bk, True, "k")
    assert torch.equal(v[:, 3:3 + T].transpose(0, 1), rv.float().to(torch.bfloat16))
    assert bool((q[T:] == 7).all()) and bool((q[:, hq * D:] == 7).all())
    for t in (k, v):
        assert bool((t[:, :3] == 7).all()) and bool((t[:, 3 + T:] == 7).all())


def test_rows_views_per_sequence_and_packed_layout():
    g, hq, hkv, lens, pos0 = gen(43), 8, 2, [3, 1, 10], [100, 5, 0]
    qkv, qn, kn = rows_case(g, lens, hq, hkv)
    wide = torch.full((sum(lens), (hq + 2 * hkv) * D + 12), NAN, device=DEV)
    wide[:, :(hq + 2 * hkv) * D] = qkv
    rope = rope_table(200)
    ks = [torch.full((20, hkv, D + 8), 7.0, dtype=torch.bfloat16, device=DEV) for _ in lens]
    vs = [torch.full((20, hkv, D + 8), 7.0, dtype=torch.bfloat16, device=DEV) for _ in lens]
    views = [view_of(k, v, 20, hkv * (D + 8), D + 8) for k, v in zip(ks, vs)]
    q = torch.empty(sum(lens), hq, D, dtype=torch.bfloat16, device=DEV)
    fq.fq_qk_norm_rope(wide.data_ptr(), lens, pos0, views, [10, 0, 5], hq, hkv, qn.data_ptr(), kn.data_ptr(), 1e-6,
                       rope.data_ptr(), 200, q.data_ptr(), stream(), qkv_stride=wide.shape[1])
    torch.cuda.synchronize()
    pos = torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(pos0, lens)])
    (rq, bq), (rk, bk), rv = reference_rows(qkv, qn, kn, 1e-6, rope, pos, hq, hkv)
    assert_within(q, rq, bq, True, "q")
    r = 0
    for s, (n, r0) in enumerate(zip(lens, [10, 0, 5])):
        assert_within(ks[s][r0:r0 + n, :, :D], rk[r:r + n], bk[r:r + n], True, "k")
        assert torch.equal(vs[s][r0:r0 + n, :, :D], rv[r:r + n].float().to(torch.bfloat16))
        for t in (ks[s], vs[s]):
            assert bool((t[:r0] == 7).all()) and bool((t[r0 + n:] == 7).all()) and bool((t[:, :, D:] == 7).all())
        r += n


def test_rows_zero_and_nan_rows():
    """A head of zeros stays zero with eps > 0; NaN and infinite rows stay in their head."""
    g, hq, hkv = gen(47), 4, 2
    qkv, qn, kn = rows_case(g, [4], hq, hkv)
    qkv = qkv.reshape(4, hq + 2 * hkv, D)
    qkv[0, 1], qkv[1, 2, 3], qkv[2, hq + hkv, 9] = 0, NAN, math.inf
    rope = rope_table(4)
    k, v = (torch.empty(hkv, 4, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.empty(4, hq, D, dtype=torch.bfloat16, device=DEV)
    fq.fq_qk_norm_rope(qkv.data_ptr(), [4], [0], view_of(k, v, 4, D, 4 * D), [0], hq, hkv, qn.data_ptr(), kn.data_ptr(), 1e-6,
                       rope.data_ptr(), 4, q.data_ptr(), stream())
    torch.cuda.synchronize()
    assert bool((q[0, 1] == 0).all()) and bool(q[1, 2].isnan().all()) and float(v[0, 2, 9]) == math.inf
    assert int(q.isnan().any(dim=2).sum()) == 1 and not bool(k.isnan().any()) and not bool(v.isnan().any())


# ---------------------------------------------------------------- used together, streams and graphs

class Together:
    """Rows -> prompt attention of two prompts, then rows -> shared attention of five answers to the
    first prompt, all on caller-held buffers."""

    def __init__(self, seed, hq=8, hkv=2, lens=(300, 45), n=5):
        g = gen(seed)
        self.hq, self.hkv, self.lens, self.n = hq, hkv, list(lens), n
        self.T = sum(lens)
        self.qkv, self.qn, self.kn = rows_case(g, self.lens, hq, hkv)
        self.qkv1, _, _ = rows_case(g, [n], hq, hkv)
        self.rope = rope_table(1024)
        self.k, self.v = (torch.full((hkv, self.T, D), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.tk, self.tv = (torch.full((n, hkv, 4, D), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.q = torch.empty(self.T, hq, D, dtype=torch.bfloat16, device=DEV)
        self.q1 = torch.empty(n, hq, D, dtype=torch.bfloat16, device=DEV)
        self.out, self.out1 = torch.empty_like(self.q), torch.empty_like(self.q1)
        self.view = view_of(self.k, self.v, self.T, D, self.T * D)
        self.tails = fq.kv_view_array([view_of(self.tk[i], self.tv[i], 4, D, 4 * D) for i in range(n)])
        self.ws = workspace(max(fq.fq_attn_prompt_workspace(self.lens, self.lens, hq, hkv),
                                fq.fq_attn_shared_workspace(lens[0], [1] * n, hq, hkv)))

    def launch(self):
        hq, hkv, st = self.hq, self.hkv, stream()
        norm = (self.qn.data_ptr(), self.kn.data_ptr(), 1e-6, self.rope.data_ptr(), 1024)
        fq.fq_qk_norm_rope(self.qkv.data_ptr(), self.lens, [0, 0], self.view, [0, self.lens[0]], hq, hkv, *norm, self.q.data_ptr(), st)
        fq.fq_attn_prompt(self.q.data_ptr(), self.view, self.lens, self.lens, hq, hkv, SCALE, self.out.data_ptr(),
                          self.ws.data_ptr(), self.ws.numel() * 4, st)
        fq.fq_qk_norm_rope(self.qkv1.data_ptr(), [1] * self.n, [self.lens[0]] * self.n, self.tails, [0] * self.n, hq, hkv, *norm,
                           self.q1.data_ptr(), st)
        fq.fq_attn_shared(self.q1.data_ptr(), self.view, self.lens[0], self.tails, [1] * self.n, hq, hkv, SCALE,
                          self.out1.data_ptr(), self.ws.data_ptr(), self.ws.numel() * 4, st)

    def check(self):
        torch.cuda.synchronize()
        hq, hkv = self.hq, self.hkv
        pos = torch.cat([torch.arange(n, device=DEV) for n in self.lens])
        (rq, bq), (rk, bk), rv = reference_rows(self.qkv, self.qn, self.kn, 1e-6, self.rope, pos, hq, hkv)
        assert_within(self.q, rq, bq, True, "q")
        assert_within(self.k.transpose(0, 1), rk, bk, True, "k")
        k0 = [0, self.lens[0]]
        kv = lambda s, h: (self.k[h, k0[s]:k0[s] + self.lens[s]], self.v[h, k0[s]:k0[s] + self.lens[s]])  # noqa: E731
        ref, bound = reference_prompt(self.q, kv, self.lens, self.lens, hq, hkv)
        assert_within(self.out, ref, bound, True, "prompt")
        pos = torch.full((self.n,), self.lens[0], device=DEV)
        (rq, bq), (rk, bk), rv = reference_rows(self.qkv1, self.qn, self.kn, 1e-6, self.rope, pos, hq, hkv)
        assert_within(self.q1, rq, bq, True, "q of the answers")
        assert_within(self.tk[:, :, 0], rk, bk, True, "k of the answers")
        P = self.lens[0]
        ref, bound = reference_shared(self.q1, self.k[:, :P], self.v[:, :P], self.tk, self.tv, [1] * self.n, hq, hkv)
        assert_within(self.out1, ref, bound, True, "answers")
        return self.out.clone(), self.out1.clone()


def test_together():
    c = Together(1)
    c.launch()
    a = c.check()
    c.out.fill_(NAN)
    c.launch()   # again on the same buffers: the same bits
    b = c.check()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_together_captured_and_replayed():
    """Two captured runs with workspaces of their own, replayed on two streams at once."""
    cs = [Together(2), Together(3, hq=4, hkv=4, lens=(150, 260), n=3)]
    for c in cs:
        c.launch()
    torch.cuda.synchronize()
    graphs = []
    for c in cs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.launch()
        graphs.append(gr)
    g = gen(9)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for c in cs:   # new inputs in the same buffers
            c.qkv.copy_(normal(g, *c.qkv.shape, dtype=torch.float32))
            c.qkv1.copy_(normal(g, *c.qkv1.shape, dtype=torch.float32))
            c.out.fill_(NAN)
            c.out1.fill_(NAN)
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        for c in cs:
            c.check()


def test_together_on_other_streams():
    cs = [Together(4 + i) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, st in zip(cs, streams):
            with torch.cuda.stream(st):
                c.launch()
    for c in cs:
        c.check()


def test_calls_from_two_threads():
    import threading
    cs = [Together(8), Together(9, hq=8, hkv=1)]
    torch.cuda.synchronize()
    errors = []

    def work(c):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    c.launch()
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(c,)) for c in cs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
    for c in cs:
        c.check()
