"""Attention with windows and sinks over views and over pages, and the append into pages, on the GPU against plain 64-bit
forms, at the sizes, masks, layouts and streams where they can go wrong."""
import math

import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import (D, DEV, NAN, SCALE, Pool, assert_lse, junk, reference, run_paged, run_window, stream,
                                  visible)
from tests.prompt_ops_util import assert_within, attend, gen, normal

pytestmark = pytest.mark.gpu

HEADS = [(4, 4), (4, 2), (8, 2), (8, 1)]
# whole prompts around the tile sizes, ragged and empty ones, chunks behind cached rows, more queries than keys, few rows
# over many keys, rows beside tiles
LENGTHS = [([1], [1]), ([31, 1, 33], [31, 1, 33]), ([127, 128, 129], [127, 128, 129]), ([255, 0, 257, 5], [255, 0, 257, 5]),
           ([1000, 3], [1000, 3]), ([17, 40], [217, 1000]), ([1, 1, 2, 1], [1, 300, 129, 4096]), ([300], [40]),
           ([9, 4, 3], [2, 0, 3]), ([64], [20000]), ([1, 150], [3000, 1500])]
MASKS = [(0, 0), (1, 0), (1, 1), (16, 4), (100, 0), (128, 128), (129, 300), (700, 17), (100000, 5)]


def cache(g, rows, hkv, pad=200, fill=NAN):
    """K or V of a cache layer: `rows` rows, then rows of junk."""
    t = torch.full((hkv, rows + pad, D), fill, dtype=torch.bfloat16, device=DEV)
    t[:, :rows] = normal(g, hkv, rows, D)
    return t


def view(k, v):
    rows = k.shape[1]
    return fq.fq_kv_view(k.data_ptr(), v.data_ptr(), rows, D, rows * D)


def packed(k, v, k_len):
    """The rows of sequences that follow one another in a view."""
    first = [sum(k_len[:s]) for s in range(len(k_len))]
    return lambda s, h: (k[h, first[s]:first[s] + k_len[s]], v[h, first[s]:first[s] + k_len[s]])


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("q_len,k_len", LENGTHS)
@pytest.mark.parametrize("window,sinks", MASKS)
def test_window(hq, hkv, q_len, k_len, window, sinks):
    g = gen(hash((hq, hkv, tuple(q_len), window, sinks)) % 2 ** 31)
    q = normal(g, sum(q_len), hq, D)
    k, v = cache(g, sum(k_len), hkv), cache(g, sum(k_len), hkv)
    ref, bound, lse, lse_bound = reference(q, packed(k, v, k_len), q_len, k_len, hq, hkv, window, sinks)
    f32 = (window + sinks + hq) % 2 == 1
    got, e = run_window(q, view(k, v), q_len, k_len, hq, hkv, window, sinks, out_dtype="f32" if f32 else "bf16")
    assert_within(got, ref, bound, not f32, f"{hq}/{hkv} {q_len} {k_len} {window} {sinks}")
    assert_lse(e, lse, lse_bound)


@pytest.mark.parametrize("hq,hkv,q_len,k_len", [(520, 520, [1, 3, 40], [300, 500, 200]), (2, 1, [1] * 64, [64 * i for i in range(64)]),
                                                (1, 1, [1, 1, 8], [70000, 1, 129])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
def test_many_and_few_heads(hq, hkv, q_len, k_len, window, sinks):
    """More kv heads than thread blocks run at once; one, whose keys all of them share out."""
    g = gen(31)
    q = normal(g, sum(q_len), hq, D)
    k, v = cache(g, sum(k_len), hkv), cache(g, sum(k_len), hkv)
    ref, bound, lse, lse_bound = reference(q, packed(k, v, k_len), q_len, k_len, hq, hkv, window, sinks)
    got, e = run_window(q, view(k, v), q_len, k_len, hq, hkv, window, sinks)
    assert_within(got, ref, bound, True, f"{hq}/{hkv} {window} {sinks}")
    assert_lse(e, lse, lse_bound)
    again, _ = run_window(q, view(k, v), q_len, k_len, hq, hkv, window, sinks)
    assert bool((got == again).all())


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("q_len,k_len", LENGTHS)
@pytest.mark.parametrize("page,layout", [(16, "head"), (32, "row"), (64, "head"), (128, "row"), (256, "head")])
def test_paged(hq, hkv, q_len, k_len, page, layout):
    window, sinks = MASKS[(sum(k_len) + page // 16 + hq) % len(MASKS)]
    g = gen(hash((hq, hkv, tuple(q_len), page)) % 2 ** 31)
    q = normal(g, sum(q_len), hq, D)
    pool = Pool(g, k_len, hkv, page, layout)
    for w, s in {(0, 0), (window, sinks)}:
        ref, bound, lse, lse_bound = reference(q, pool.rows, q_len, k_len, hq, hkv, w, s)
        got, e = run_paged(q, pool, q_len, k_len, hq, hkv, w, s)
        assert_within(got, ref, bound, True, f"{hq}/{hkv} {q_len} {k_len} page {page} {w} {s}")
        assert_lse(e, lse, lse_bound)


def test_without_a_window_is_prompt_attention():
    """window 0, and one that reaches every key: the same numbers as fq_attn_prompt, bit for bit.  But for the single token
    over 3000 keys (row 700), whose keys the two calls cut at other places: the weights of a cut are rounded to 8 bits
    against its own largest score, so both are within the bound of their roundings and need not be equal."""
    g, hq, hkv, q_len, k_len = gen(3), 8, 2, [700, 1, 40, 9], [700, 3000, 1040, 9]
    q = normal(g, sum(q_len), hq, D)
    k, v = cache(g, sum(k_len), hkv), cache(g, sum(k_len), hkv)
    ws = junk(fq.fq_attn_prompt_workspace(q_len, k_len, hq, hkv))
    want = torch.empty(sum(q_len), hq, D, dtype=torch.bfloat16, device=DEV)
    fq.fq_attn_prompt(q.data_ptr(), view(k, v), q_len, k_len, hq, hkv, SCALE, want.data_ptr(), ws.data_ptr(), ws.numel() * 4, stream())
    for window, sinks in ((0, 0), (0, 7), (5000, 0), (2 ** 32 - 1, 2 ** 32 - 1)):
        got, _ = run_window(q, view(k, v), q_len, k_len, hq, hkv, window, sinks, lse=False)
        same = [r for r in range(sum(q_len)) if r != 700]
        assert bool((got[same] == want[same]).all()), (window, sinks)
        ref, bound, _, _ = reference(q, packed(k, v, k_len), q_len, k_len, hq, hkv, 0, 0)
        assert_within(got, ref, bound, True, f"window {window} {sinks}")


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 3.0])
def test_scales(paged, scale):
    g, hq, hkv, q_len, k_len = gen(17), 4, 2, [200, 1], [333, 900]
    q = normal(g, sum(q_len), hq, D)
    if paged:
        pool = Pool(g, k_len, hkv, 32)
        ref, bound, lse, lb = reference(q, pool.rows, q_len, k_len, hq, hkv, 90, 3, scale)
        got, e = run_paged(q, pool, q_len, k_len, hq, hkv, 90, 3, scale=scale, out_dtype="f32")
    else:
        k, v = cache(g, sum(k_len), hkv), cache(g, sum(k_len), hkv)
        ref, bound, lse, lb = reference(q, packed(k, v, k_len), q_len, k_len, hq, hkv, 90, 3, scale)
        got, e = run_window(q, view(k, v), q_len, k_len, hq, hkv, 90, 3, scale=scale, out_dtype="f32")
    assert_within(got, ref, bound, False)
    assert_lse(e, lse, lb)


def test_window_views_rows_and_strides():
    """A view per sequence, row offsets, row strides of q and out; what lies between and behind out's rows stays."""
    g, hq, hkv = gen(5), 8, 2
    q_len, k_len, row0, caps = [40, 200, 1, 77], [140, 200, 500, 77], [3, 0, 9, 100], [150, 200, 520, 200]
    stores = [(cache(g, c, hkv, 0), cache(g, c, hkv, 0)) for c in caps]
    T = sum(q_len)
    q = normal(g, T, hq * D + 8)
    out = torch.full((T + 3, hq * D + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = junk(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, 60, 2))
    fq.fq_attn_window(q.data_ptr(), [view(*s) for s in stores], q_len, k_len, hq, hkv, 60, 2, SCALE, out.data_ptr(), ws.data_ptr(),
                      ws.numel() * 4, stream(), kv_row0=row0, q_stride=hq * D + 8, out_stride=hq * D + 24)
    fq.fq_attn_check(stream())
    kv = lambda s, h: tuple(t[h, row0[s]:row0[s] + k_len[s]] for t in stores[s])  # noqa: E731
    ref, bound, _, _ = reference(q[:, :hq * D].reshape(T, hq, D), kv, q_len, k_len, hq, hkv, 60, 2)
    assert_within(out[:T, :hq * D].reshape(T, hq, D), ref, bound, True)
    assert bool((out[T:] == 7).all()) and bool((out[:, hq * D:] == 7).all())


@pytest.mark.parametrize("hq,hkv", HEADS)
def test_window_many_views(hq, hkv):
    """64 sequences with a view each, long ones among them, so that units are split and rows run beside them."""
    g = gen(41)
    q_len = [1, 0, 3, 40] * 16
    k_len = [900, 5, 40, 300] * 15 + [5000, 0, 9000, 8000]
    stores = [(cache(g, max(K, 1), hkv, 0), cache(g, max(K, 1), hkv, 0)) for K in k_len]
    q = normal(g, sum(q_len), hq, D)
    kv = lambda s, h: tuple(t[h, :k_len[s]] for t in stores[s])  # noqa: E731
    for window, sinks in ((0, 0), (333, 20)):
        got, e = run_window(q, [view(*s) for s in stores], q_len, k_len, hq, hkv, window, sinks)
        ref, bound, lse, lb = reference(q, kv, q_len, k_len, hq, hkv, window, sinks)
        assert_within(got, ref, bound, True)
        assert_lse(e, lse, lb)


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("hq,hkv,at,L,K,window,sinks", [
    (4, 4, [100], 300, 300, 50, 0), (4, 2, [128, 130], 300, 300, 128, 4), (8, 1, [299, 2], 300, 300, 40, 8),
    (4, 2, [0, 3, 4], 300, 300, 64, 4), (8, 2, [250, 100], 20, 260, 33, 3), (8, 2, [255, 0], 1, 256, 16, 1),
    (4, 4, [90, 200], 2, 300, 100, 91), (8, 8, [5], 3, 2000, 1500, 0), (4, 2, [700, 701, 1100], 700, 1500, 300, 20)])
def test_values_that_a_row_does_not_see_do_not_leak(bad, where, paged, hq, hkv, at, L, K, window, sinks):
    """A key outside a row's window has no influence on it, whatever it holds, on either side of the window and between
    the sinks and the window.  Rows that see one give what the definition gives: checked where that is finite or NaN
    throughout."""
    g = gen(11)
    q = normal(g, L, hq, D)
    if paged:
        pool = Pool(g, [K], hkv, 32)
        k, v = (torch.stack([pool.rows(0, h)[i] for h in range(hkv)]) for i in range(2))
    else:
        k, v = (t[:, :K].contiguous() for t in (cache(g, K, hkv, 0), cache(g, K, hkv, 0)))
    t = k if where == "k" else v
    for i, key in enumerate(at):
        t[i % hkv, key, 5:9] = bad
    if paged:
        pool.put(pool.k, 0, 0, k)
        pool.put(pool.v, 0, 0, v)
        got, _ = run_paged(q, pool, [L], [K], hq, hkv, window, sinks, out_dtype="f32")
    else:
        got, _ = run_window(q, view(k, v), [L], [K], hq, hkv, window, sinks, out_dtype="f32")
    seen = visible(L, K, window, sinks)
    for h in range(hq):
        kh = h // (hq // hkv)
        touched = torch.zeros(L, dtype=torch.bool, device=DEV)
        for i, key in enumerate(at):
            if i % hkv == kh:
                touched |= seen[:, key]
        clean_k = torch.where(torch.isfinite(k[kh].float()) & (k[kh].float().abs() < 1e30), k[kh], 0)
        clean_v = torch.where(torch.isfinite(v[kh].float()) & (v[kh].float().abs() < 1e30), v[kh], 0)
        ref, bound = attend(q[:, h], clean_k, clean_v, seen, SCALE)
        assert_within(got[~touched, h], ref[~touched], bound[~touched], False, f"head {h}: rows that do not see it")
        if where == "v" and bool(touched.any()):
            other = [d for d in range(D) if not 5 <= d < 9]
            assert_within(got[touched][:, h][:, other], ref[touched][:, other], bound[touched][:, other], False, "other dims")
            hit = got[touched][:, h, 5:9]
            if math.isnan(bad):
                assert bool(torch.isnan(hit).all())
            elif math.isinf(bad):
                assert bool((hit == bad).all())


@pytest.mark.parametrize("page", [16, 64, 256])
def test_paged_shared_pages_and_junk_entries(page):
    """Sequences that begin with the same pages; entries that no row looks into name no page, and no error is recorded
    for them: beyond the end, and between the sinks and the window."""
    g, hq, hkv = gen(23), 8, 2
    q_len, k_len, window, sinks = [1, 70, 2, 300], [900, 1100, 3000, 1200], 200, 5
    pool = Pool(g, k_len, hkv, page)
    same = 512 // page
    pool.table[1, :same] = pool.table[0, :same]
    pool.table[3, :same] = pool.table[0, :same]
    q = normal(g, sum(q_len), hq, D)
    for w, s in ((0, 0), (window, sinks)):
        ref, bound, lse, lb = reference(q, pool.rows, q_len, k_len, hq, hkv, w, s)
        if w:   # pages that the window has left behind are given away
            for i, (L, K) in enumerate(zip(q_len, k_len)):
                first = max(0, K - L + 1 - w)
                for p in range(-(-s // page), first // page):
                    pool.table[i, p] = -1 if i % 2 else pool.n_pages
        got, e = run_paged(q, pool, q_len, k_len, hq, hkv, w, s)
        assert_within(got, ref, bound, True)
        assert_lse(e, lse, lb)


@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1, -2 ** 31, "n"])
@pytest.mark.parametrize("q_len,k_len", [([1], [300]), ([200], [300])])
def test_paged_entries_without_a_page_are_recorded(entry, q_len, k_len):
    """The call reads nothing for them and fq_attn_check tells; the next call is as ever."""
    g, hq, hkv = gen(29), 4, 2
    pool = Pool(g, k_len, hkv, 32)
    q = normal(g, sum(q_len), hq, D)
    good = pool.table[0, 3].clone()
    pool.table[0, 3] = pool.n_pages if entry == "n" else entry
    run_paged(q, pool, q_len, k_len, hq, hkv, 0, 0, check=False)
    with pytest.raises(fq.FqError) as e:
        fq.fq_attn_check(stream())
    assert e.value.status == fq.INVALID_ARGUMENT and "page" in str(e.value)
    fq.fq_attn_check(stream())
    pool.table[0, 3] = good
    got, _ = run_paged(q, pool, q_len, k_len, hq, hkv, 0, 0)
    ref, bound, _, _ = reference(q, pool.rows, q_len, k_len, hq, hkv, 0, 0)
    assert_within(got, ref, bound, True)


def rope_table(rows):
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * 1e6 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    return torch.stack((a.cos(), a.sin()), dim=-1).float().contiguous()


def normed(x, gain, cs, eps=1e-6):
    """In 64 bits, and the bound of the f32 computation before rounding to bf16: the sum of 128 squares and its root (70
    roundings at half weight), the gain, the rotation of two values."""
    x = x.double()
    y = x / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + eps) * gain.double()
    a, b = y[..., :64], y[..., 64:]
    c, s = cs[..., 0].double()[:, None], cs[..., 1].double()[:, None]
    out = torch.cat((a * c - b * s, a * s + b * c), dim=-1)
    size = torch.cat((a.abs() * c.abs() + b.abs() * s.abs(), a.abs() * s.abs() + b.abs() * c.abs()), dim=-1)
    return out, size * 80 * 2.0 ** -24


@pytest.mark.parametrize("hq,hkv", HEADS + [(24, 3)])
@pytest.mark.parametrize("lens,row0,page", [([1], [0], 16), ([1, 1, 1], [5, 16, 47], 16), ([33, 0, 5], [15, 3, 64], 32),
                                            ([300, 17], [0, 129], 128), ([257], [250], 256)])
def test_append(hq, hkv, lens, row0, page):
    """q, and the rows of K and V in their pages; every other row of the pool stays as it was."""
    g = gen(hash((hq, tuple(lens), page)) % 2 ** 31)
    pool = Pool(g, [r + n for r, n in zip(row0, lens)], hkv, page, "row" if page == 32 else "head", fill=3.0)
    before = [t.clone() for t in pool.store]
    T, pos0 = sum(lens), [7 * i + 3 for i in range(len(lens))]
    rope = rope_table(max(p + n for p, n in zip(pos0, lens)) + 1)
    qkv = torch.randn(T, (hq + 2 * hkv) * D + 4, generator=g, device=DEV)
    qn, kn = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    qo = torch.full((T, hq * D + 8), 9.0, dtype=torch.bfloat16, device=DEV)
    fq.fq_qk_norm_rope_paged(qkv.data_ptr(), lens, pos0, pool.pages(), pool.table.data_ptr(), pool.stride, row0, hq, hkv,
                             qn.data_ptr(), kn.data_ptr(), 1e-6, rope.data_ptr(), rope.shape[0], qo.data_ptr(), stream(),
                             qkv_stride=(hq + 2 * hkv) * D + 4, q_stride=hq * D + 8)
    fq.fq_attn_check(stream())
    x = qkv[:, :(hq + 2 * hkv) * D].reshape(T, hq + 2 * hkv, D)
    at = torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(pos0, lens)])
    q, qb = normed(x[:, :hq], qn, rope[at])
    k, kb = normed(x[:, hq:hq + hkv], kn, rope[at])
    v = x[:, hq + hkv:].to(torch.bfloat16)
    assert_within(qo[:, :hq * D].reshape(T, hq, D), q, qb, True)
    assert bool((qo[:, hq * D:] == 9).all())
    r = 0
    for s, n in enumerate(lens):
        for h in range(hkv):
            gk, gv = pool.rows(s, h, n, row0[s])
            assert_within(gk, k[r:r + n, h], kb[r:r + n, h], True)
            assert bool((gv == v[r:r + n, h]).all())
        r += n
    after = [t.clone() for t in pool.store]
    for t, b in zip(after, before):   # put the rows back: nothing else has changed
        now = t.as_strided(pool.k.shape, pool.k.stride())
        old = b.as_strided(pool.k.shape, pool.k.stride())
        for s, n in enumerate(lens):
            page_, row_ = pool.where(s, row0[s], n)
            now[page_, :, row_] = old[page_, :, row_]
        assert bool((t == b).all())


def test_append_entries_without_a_page():
    """Rows whose entry names no page are not written; q and the other rows are."""
    g, hq, hkv, page = gen(31), 4, 2, 16
    pool = Pool(g, [40], hkv, page, fill=3.0)
    before = [t.clone() for t in pool.store]
    pool.table[0, 1] = pool.n_pages
    rope = rope_table(40)
    qkv = torch.randn(40, (hq + 2 * hkv) * D, generator=g, device=DEV)
    one = torch.ones(D, device=DEV)
    qo = torch.full((40, hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    fq.fq_qk_norm_rope_paged(qkv.data_ptr(), [40], [0], pool.pages(), pool.table.data_ptr(), pool.stride, [0], hq, hkv, one.data_ptr(),
                             one.data_ptr(), 1e-6, rope.data_ptr(), 40, qo.data_ptr(), stream())
    with pytest.raises(fq.FqError) as e:
        fq.fq_attn_check(stream())
    assert e.value.status == fq.INVALID_ARGUMENT
    q, qb = normed(qkv.reshape(40, -1, D)[:, :hq], one, rope)
    assert_within(qo, q, qb, True)
    v = qkv.reshape(40, -1, D)[:, hq + hkv:].to(torch.bfloat16)
    ids = pool.table[0].tolist()
    for i in (0, 2):
        n = min(page, 40 - i * page)
        assert bool((pool.v[ids[i], :, :n].transpose(0, 1) == v[i * page:i * page + n]).all())
        pool.v[ids[i], :, :n] = before[1][ids[i], :, :n]
    assert bool((pool.v == before[1]).all())


@pytest.mark.parametrize("paged", [False, True])
def test_captured_and_replayed(paged):
    """A captured call: new values (and another page table of the same lengths) at a replay, a workspace of its own."""
    g, hq, hkv, q_len, k_len, window, sinks = gen(37), 8, 2, [150, 1, 4], [1150, 3000, 700], 500, 4
    q = normal(g, sum(q_len), hq, D)
    pool = Pool(g, k_len, hkv, 64) if paged else None
    k, v = cache(g, sum(k_len), hkv), cache(g, sum(k_len), hkv)
    ws = junk(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, window, sinks))
    out = torch.empty(sum(q_len), hq, D, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream(DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        s = torch.cuda.current_stream(DEV).cuda_stream
        if paged:
            fq.fq_attn_paged(q.data_ptr(), pool.pages(), pool.table.data_ptr(), pool.stride, q_len, k_len, hq, hkv, window, sinks,
                             SCALE, out.data_ptr(), ws.data_ptr(), ws.numel() * 4, s)
        else:
            fq.fq_attn_window(q.data_ptr(), view(k, v), q_len, k_len, hq, hkv, window, sinks, SCALE, out.data_ptr(), ws.data_ptr(),
                              ws.numel() * 4, s)
    for turn in range(2):
        q.copy_(normal(g, sum(q_len), hq, D))
        if paged:
            pool.table[0, :18] = pool.table[0, :18].flip(0) if turn else pool.table[0, :18]
        else:
            k[:, :sum(k_len)] = normal(g, hkv, sum(k_len), D)
        out.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        fq.fq_attn_check(stream())
        ref, bound, _, _ = reference(q, pool.rows if paged else packed(k, v, k_len), q_len, k_len, hq, hkv, window, sinks)
        assert_within(out, ref, bound, True)


def test_prompt_and_tokens_through_pages():
    """As a program uses them: a prompt's rows into pages and its attention, then tokens one after the other, against
    the same through fq_qk_norm_rope and fq_attn_window on a cache."""
    g, hq, hkv, page, window, sinks, n_prompt, n_tok = gen(43), 8, 2, 16, 64, 4, 150, 40
    total = n_prompt + n_tok
    pool = Pool(g, [total], hkv, page, fill=0.0)
    k, v = (torch.zeros(hkv, total, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for t in pool.store:
        t.zero_()
    rope = rope_table(total)
    qn, kn = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    at = 0
    for n in [n_prompt] + [1] * n_tok:
        qkv = torch.randn(n, (hq + 2 * hkv) * D, generator=g, device=DEV)
        qs = [torch.empty(n, hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        fq.fq_qk_norm_rope_paged(qkv.data_ptr(), [n], [at], pool.pages(), pool.table.data_ptr(), pool.stride, [at], hq, hkv,
                                 qn.data_ptr(), kn.data_ptr(), 1e-6, rope.data_ptr(), total, qs[0].data_ptr(), stream())
        fq.fq_qk_norm_rope(qkv.data_ptr(), [n], [at], view(k, v), [at], hq, hkv, qn.data_ptr(), kn.data_ptr(), 1e-6,
                           rope.data_ptr(), total, qs[1].data_ptr(), stream())
        at += n
        a, _ = run_paged(qs[0], pool, [n], [at], hq, hkv, window, sinks)
        b, _ = run_window(qs[1], view(k, v), [n], [at], hq, hkv, window, sinks)
        assert bool((qs[0] == qs[1]).all()) and bool((a == b).all()), at
    for h in range(hkv):
        pk, pv = pool.rows(0, h)
        assert bool((pk == k[h]).all()) and bool((pv == v[h]).all())


@pytest.mark.parametrize("q_len", [[1], [3, 1], [300], [300, 1, 40]])
def test_no_keys_at_all(q_len):
    """Rows of sequences without keys: zeros and -infinity, through views and through a pool that has no pages."""
    g, hq, hkv = gen(53), 8, 2
    k_len = [0] * len(q_len)
    q = normal(g, sum(q_len), hq, D)
    k = cache(g, 1, hkv)
    out, lse = run_window(q, view(k, k), q_len, k_len, hq, hkv, 5, 2)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    ws = junk(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, 0, 0))
    out.fill_(NAN)
    fq.fq_attn_paged(q.data_ptr(), fq.fq_kv_pages(0, 0, 0, 16, 0, 0, 0), 0, 0, q_len, k_len, hq, hkv, 0, 0, SCALE, out.data_ptr(),
                     ws.data_ptr(), ws.numel() * 4, stream())
    fq.fq_attn_check(stream())
    assert bool((out == 0).all())
