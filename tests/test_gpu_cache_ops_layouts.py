"""Caches in the layouts that programs have (K and V in one storage, heads of a row side by side), sequences that share rows or lie in
another order than the call's, outputs with strides of their own, evictions within one storage: on the GPU against plain 64-bit forms."""
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, NAN, SCALE, assert_lse, junk, reference, stream, visible
from tests.prompt_ops_util import assert_within, gen, normal
from tests.test_gpu_evict_more import bits, chosen
from tests.test_gpu_key_weights_evict import assert_weights, gathered, kinds, weights

pytestmark = pytest.mark.gpu

ROWS = 3000


def storage(g, order, hkv):
    """One array with K and V in the given order of its dims: the view, K and V as [head][row][D]."""
    size = {"kv": 2, "row": ROWS, "head": hkv}
    dims = order.split()
    store = normal(g, *[size[d] for d in dims], D)
    stride = dict(zip(dims, store.stride()))
    kv = [store.as_strided((hkv, ROWS, D), (stride["head"], stride["row"], 1), i * stride["kv"]) for i in range(2)]
    return store, fq.fq_kv_view(store.data_ptr(), store.data_ptr() + 2 * stride["kv"], ROWS, stride["row"], stride["head"]), kv


ORDERS = ["kv head row", "kv row head", "row kv head", "row head kv", "head kv row", "head row kv"]
# rows of the sequences: apart and in another order than the call's; shared ones (attention alone)
CALLS = {"apart": ([1, 150, 0, 3, 70], [2000, 300, 5, 90, 70], [1000, 0, 500, 400, 700]),
         "shared": ([1, 1, 2, 200, 40], [1500, 700, 1500, 900, 40], [0, 0, 0, 100, 60])}


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 5)])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_attention_and_weights(order, name, window, sinks, out_dtype):
    q_len, k_len, row0 = CALLS[name]
    g, hq, hkv = gen(601), 8, 2
    store, view, (k, v) = storage(g, order, hkv)
    T, f32 = sum(q_len), out_dtype == "f32"
    q = normal(g, T, hq, D)
    width = hq * D + (4 if f32 else 8)   # (rows of f32 outputs on 16 bytes, not on 32)
    out = torch.full((T, width), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    lse = torch.full((T, hq), NAN, device=DEV)
    ws = junk(max(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, window, sinks), fq.fq_attn_key_weights_workspace(q_len, k_len, hq, hkv, window, sinks)))
    fq.fq_attn_window(q.data_ptr(), view, q_len, k_len, hq, hkv, window, sinks, SCALE, out.data_ptr(), ws.data_ptr(), ws.numel() * 4, stream(),
                      kv_row0=row0, out_stride=width, out_dtype=out_dtype, lse_ptr=lse.data_ptr())
    fq.fq_attn_check(stream())
    rows = lambda t, s, h: t[h, row0[s]:row0[s] + k_len[s]]  # noqa: E731
    ref, bound, e, eb = reference(q, lambda s, h: (rows(k, s, h), rows(v, s, h)), q_len, k_len, hq, hkv, window, sinks)
    assert_within(out[:, :hq * D].reshape(T, hq, D), ref, bound, not f32)
    assert bool((out[:, hq * D:] == 7).all())
    assert_lse(lse, e, eb)
    if name == "shared":
        return
    # in place; rows of no sequence, and of sequences without query rows, keep what they had
    was = torch.rand(hkv, ROWS + 11, generator=g, device=DEV)
    w = was.clone()
    fq.fq_attn_key_weights(q.data_ptr(), lse.data_ptr(), view, q_len, k_len, hq, hkv, window, sinks, SCALE, weights(w), weights(w), ws.data_ptr(),
                           ws.numel() * 4, stream(), kv_row0=row0)
    fq.fq_attn_check(stream())
    rest, r, G = torch.ones(ROWS + 11, dtype=torch.bool, device=DEV), 0, hq // hkv
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        at = slice(row0[s], row0[s] + K)
        rest[at] = L == 0
        for h in range(hkv):
            x, b = gathered(q[r:r + L, h * G:(h + 1) * G], lse[r:r + L, h * G:(h + 1) * G], rows(k, s, h), visible(L, K, window, sinks), SCALE)
            assert_weights(w[h, at], was[h, at], x, b, f"sequence {s} head {h}")
        r += L
    assert bool((w[:, rest] == was[:, rest]).all())


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("kind", ["wide", "ties"])
def test_evict_within_one_storage(order, kind):
    """Sequences move to rows of the same view that none is read from, their weights to floats of the same array."""
    g, hkv, sinks, recent = gen(611), 3, 3, 20
    store, view, (k, v) = storage(g, order, hkv)
    k_len, keep, row0, at = [700, 5, 300], [200, 9, 100], [1500, 0, 900], [10, 300, 1300]
    n = [min(a, b) for a, b in zip(k_len, keep)]
    w = kinds(g, kind, hkv, ROWS)
    before, wb = store.clone(), w.clone()
    bk, bv = (before.as_strided(t.shape, t.stride(), t.storage_offset()) for t in (k, v))
    kept = torch.full((hkv * sum(n),), -5, dtype=torch.int32, device=DEV)
    fq.fq_kv_evict(view, weights(w), row0, k_len, keep, sinks, recent, hkv, view, weights(w), at, kept.data_ptr(), stream())
    torch.cuda.synchronize()
    for s in range(3):
        src, dst = slice(row0[s], row0[s] + k_len[s]), slice(at[s], at[s] + n[s])
        for h in range(hkv):
            want = chosen(wb[h, src], n[s], sinks, recent)
            first = hkv * sum(n[:s]) + h * n[s]
            assert bool((kept[first:first + n[s]] == want).all())
            assert bool((k[h, dst] == bk[h, src][want]).all()) and bool((v[h, dst] == bv[h, src][want]).all())
            assert bool((bits(w[h, dst]) == bits(wb[h, src][want])).all())
        for t, b in ((k, bk), (v, bv)):   # put the rows back: nothing else has changed
            t[:, dst] = b[:, dst]
        w[:, dst] = wb[:, dst]
    assert bool((store == before).all()) and bool((w == wb).all())
