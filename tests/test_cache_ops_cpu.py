"""Refusals of the operators on windows, pages and caches made shorter: every check runs on the host before anything is
launched, so none of these needs a GPU.  Addresses are made up."""
import math

import pytest

from quantized_decoder_decode_gb300 import build as fqbuild
from quantized_decoder_decode_gb300 import fq
from tests.test_prompt_ops_cpu import HEADS, IO, VIEWS, P, refused, view

FAR = 1 << 40   # an address far from P


@pytest.fixture(scope="module", autouse=True)
def lib():
    fqbuild.build()
    return fq.lib()


def pool(k=P, v=P, n_pages=8, page_rows=16, page_stride=2 * 16 * 128, row_stride=128, head_stride=16 * 128):
    return fq.fq_kv_pages(k, v, n_pages, page_rows, page_stride, row_stride, head_stride)


def window(q=P, views=None, q_len=(4,), k_len=(4,), hq=4, hkv=2, window=3, sinks=1, scale=0.1, out=P, ws=P, ws_bytes=1 << 30, **kw):
    fq.fq_attn_window(q, view() if views is None else views, q_len, k_len, hq, hkv, window, sinks, scale, out, ws, ws_bytes, 0, **kw)


def paged(q=P, pages=None, table=P, stride=4, q_len=(4,), k_len=(4,), hq=4, hkv=2, window=0, sinks=0, scale=0.1, out=P, ws=P,
          ws_bytes=1 << 30, **kw):
    fq.fq_attn_paged(q, pool() if pages is None else pages, table, stride, q_len, k_len, hq, hkv, window, sinks, scale, out, ws, ws_bytes, 0,
                     **kw)


def append(qkv=P, lens=(4, 3), pos0=(0, 9), pages=None, table=P, stride=4, kv_row0=(0, 4), hq=4, hkv=2, qn=P, kn=P, eps=1e-6,
           rope=P, rope_rows=64, q=P, **kw):
    fq.fq_qk_norm_rope_paged(qkv, lens, pos0, pool() if pages is None else pages, table, stride, kv_row0, hq, hkv, qn, kn, eps, rope,
                             rope_rows, q, 0, **kw)


def weights(q=P, lse=P, views=None, q_len=(4,), k_len=(4,), hq=4, hkv=2, window=0, sinks=0, scale=0.1, before=None, after=None, ws=P,
            ws_bytes=1 << 30, **kw):
    fq.fq_attn_key_weights(q, lse, view() if views is None else views, q_len, k_len, hq, hkv, window, sinks, scale, before,
                           fq.fq_key_weights(P, 64) if after is None else after, ws, ws_bytes, 0, **kw)


def evict(views=None, w=None, row0=None, k_len=(40,), keep=(20,), sinks=2, recent=3, hkv=2, to=None, to_w=None, to_row0=None, kept=P):
    fq.fq_kv_evict(view() if views is None else views, fq.fq_key_weights(P, 64) if w is None else w, row0, k_len, keep, sinks, recent,
                   hkv, view(k=FAR, v=FAR + (1 << 30)) if to is None else to, to_w, to_row0, kept, 0)


@pytest.mark.parametrize("kw,status", HEADS + IO + [(dict(lse_ptr=P + 2), fq.INVALID_ARGUMENT)])
def test_window_and_paged_refusals(kw, status):
    refused(window, status, **kw)
    refused(paged, status, **kw)


@pytest.mark.parametrize("kw,status", VIEWS)
def test_window_view_refusals(kw, status):
    refused(window, status, views=view(**kw))
    refused(window, status, views=[view(), view(**kw)], q_len=(4, 4), k_len=(4, 4))


PAGES = [(dict(k=0), fq.INVALID_ARGUMENT), (dict(v=0), fq.INVALID_ARGUMENT), (dict(k=P + 8), fq.INVALID_ARGUMENT),
         (dict(v=P + 2), fq.INVALID_ARGUMENT), (dict(n_pages=0), fq.KV_CACHE_OVERFLOW), (dict(n_pages=1 << 31), fq.INVALID_ARGUMENT),
         (dict(page_rows=0), fq.INVALID_ARGUMENT), (dict(page_rows=8), fq.INVALID_ARGUMENT), (dict(page_rows=24), fq.INVALID_ARGUMENT),
         (dict(page_rows=512), fq.INVALID_ARGUMENT), (dict(row_stride=132), fq.INVALID_ARGUMENT),
         (dict(row_stride=0), fq.INVALID_ARGUMENT), (dict(head_stride=64), fq.INVALID_ARGUMENT),
         (dict(page_stride=1 << 40), fq.INVALID_ARGUMENT), (dict(page_stride=4), fq.INVALID_ARGUMENT),
         (dict(n_pages=1 << 30, page_stride=1 << 30), fq.INVALID_ARGUMENT)]


@pytest.mark.parametrize("kw,status", PAGES)
def test_pool_refusals(kw, status):
    refused(paged, status, pages=pool(**kw))
    refused(append, status, pages=pool(**kw))


def test_table_refusals():
    for call in (paged, append):
        refused(call, fq.INVALID_ARGUMENT, table=0)
        refused(call, fq.INVALID_ARGUMENT, table=P + 2)
        refused(call, fq.INVALID_ARGUMENT, stride=1 << 37)
        refused(call, fq.KV_CACHE_OVERFLOW, stride=0)
    refused(paged, fq.KV_CACHE_OVERFLOW, stride=4, k_len=(65,))        # 5 pages of 16
    refused(paged, fq.INVALID_ARGUMENT, k_len=((1 << 30) + 1,), stride=1 << 30)
    refused(append, fq.KV_CACHE_OVERFLOW, kv_row0=(0, 62))
    refused(append, fq.KV_CACHE_OVERFLOW, kv_row0=(0, 2 ** 32 - 1))    # no 32-bit wrap
    refused(append, fq.INVALID_ARGUMENT, kv_row0=(0, 2 ** 32 - 1), stride=1 << 32)


def test_pool_of_one_page_and_one_head():
    """Strides that are not looked at may hold anything: the call gets past them to the next refusal."""
    refused(paged, fq.INVALID_ARGUMENT, pages=pool(n_pages=1, page_stride=3), scale=math.nan)
    refused(paged, fq.INVALID_ARGUMENT, pages=pool(head_stride=3), hq=2, hkv=1, scale=math.nan)
    with pytest.raises(fq.FqError) as e:
        paged(pages=pool(n_pages=1, page_stride=3), scale=math.nan)
    assert "scale" in str(e.value)


def test_counts_and_lengths():
    for call in (window, paged, weights):
        refused(call, fq.INVALID_SEQUENCE_LENGTH, q_len=(), k_len=())
        refused(call, fq.INVALID_ARGUMENT, q_len=(1,) * 65, k_len=(1,) * 65)
        refused(call, fq.INVALID_ARGUMENT, q_len=(1 << 30, 1 << 30), k_len=(4, 4))
        with pytest.raises(ValueError):
            call(q_len=(1,), k_len=(1, 2))
        for bad in (-1, 1 << 32):
            with pytest.raises(ValueError):
                call(window=bad)
            with pytest.raises(ValueError):
                call(sinks=bad)
            with pytest.raises(ValueError):
                call(k_len=(bad,))
    refused(window, fq.KV_CACHE_OVERFLOW, q_len=(1, 1), k_len=(60, 5))
    refused(window, fq.INVALID_ARGUMENT, views=[view()] * 2, q_len=(1,) * 3, k_len=(1,) * 3)


def test_workspaces():
    assert fq.fq_attn_window_workspace((64,), (1 << 16,), 4, 2, 0, 0) > 0
    assert fq.fq_attn_window_workspace((64,), (1 << 16,), 4, 2, 100, 4) == 0       # (few keys are looked at)
    assert fq.fq_attn_key_weights_workspace((4096,), (4096,), 32, 8, 0, 0) > 0
    assert fq.fq_attn_key_weights_workspace((1,), (1 << 16,), 32, 8, 0, 0) == 0
    big = dict(q_len=(64,), k_len=(1 << 16,), hq=4, hkv=2)
    need = fq.fq_attn_window_workspace((64,), (1 << 16,), 4, 2, 0, 0)
    refused(paged, fq.INVALID_ARGUMENT, stride=1 << 12, ws_bytes=need - 1, **big)
    refused(paged, fq.INVALID_ARGUMENT, stride=1 << 12, ws=P + 16, **big)
    refused(window, fq.INVALID_ARGUMENT, views=view(rows=1 << 16), window=0, ws=0, **big)
    with pytest.raises(fq.FqError) as e:   # more work than a call is cut into
        fq.fq_attn_key_weights_workspace((1 << 30,), (1 << 30,), 8, 1, 0, 0)
    assert e.value.status == fq.INVALID_ARGUMENT
    with pytest.raises(fq.FqError) as e:   # (of many sequences: before they are listed)
        fq.fq_attn_key_weights_workspace((1000,) * 64, (1 << 30,) * 64, 8, 1, 0, 0)
    assert e.value.status == fq.INVALID_ARGUMENT
    long = dict(q_len=(4096,), k_len=(4096,), hq=32, hkv=8, views=view(rows=4096))
    refused(weights, fq.INVALID_ARGUMENT, after=fq.fq_key_weights(P, 4096), ws_bytes=64, **long)
    for call in (fq.fq_attn_window_workspace, fq.fq_attn_key_weights_workspace):
        for args, status in ((((), (), 4, 2, 0, 0), fq.INVALID_SEQUENCE_LENGTH), (((1,), (1,), 6, 2, 0, 0), fq.UNSUPPORTED),
                             (((1,) * 65, (1,) * 65, 4, 2, 0, 0), fq.INVALID_ARGUMENT)):
            with pytest.raises(fq.FqError) as e:
                call(*args)
            assert e.value.status == status


@pytest.mark.parametrize("kw,status", [(dict(eps=-1.0), fq.INVALID_ARGUMENT), (dict(eps=math.nan), fq.INVALID_ARGUMENT),
                                       (dict(qkv=0), fq.INVALID_ARGUMENT), (dict(q=0), fq.INVALID_ARGUMENT),
                                       (dict(rope=P + 4), fq.INVALID_ARGUMENT), (dict(qn=0), fq.INVALID_ARGUMENT),
                                       (dict(rope_rows=11), fq.INVALID_SEQUENCE_LENGTH), (dict(qkv_stride=512), fq.INVALID_ARGUMENT),
                                       (dict(q_stride=516), fq.INVALID_ARGUMENT), (dict(hq=6), fq.UNSUPPORTED)])
def test_append_refusals(kw, status):
    refused(append, status, **kw)


@pytest.mark.parametrize("kw,status", HEADS + [(dict(q=0), fq.INVALID_ARGUMENT), (dict(q=P + 8), fq.INVALID_ARGUMENT),
                                               (dict(lse=0), fq.INVALID_ARGUMENT), (dict(lse=P + 2), fq.INVALID_ARGUMENT),
                                               (dict(q_stride=516), fq.INVALID_ARGUMENT), (dict(scale=math.inf), fq.INVALID_ARGUMENT)])
def test_key_weights_refusals(kw, status):
    refused(weights, status, **kw)


def test_key_weights_buffers():
    w = fq.fq_key_weights
    refused(weights, fq.INVALID_ARGUMENT, after=w(0, 64))
    refused(weights, fq.INVALID_ARGUMENT, after=w(P + 2, 64))
    refused(weights, fq.INVALID_ARGUMENT, after=w(P, 3))                     # shorter than the rows used
    refused(weights, fq.INVALID_ARGUMENT, after=w(P, 8), kv_row0=(5,))
    refused(weights, fq.INVALID_ARGUMENT, before=w(0, 64))
    refused(weights, fq.INVALID_ARGUMENT, before=w(P, 3))
    refused(weights, fq.INVALID_ARGUMENT, views=view(k=0))
    two = dict(q_len=(1, 1), k_len=(40, 40))
    refused(weights, fq.INVALID_ARGUMENT, kv_row0=(0, 20), **two)            # rows of one view twice
    refused(weights, fq.INVALID_ARGUMENT, views=[view(), view(k=FAR)], after=[w(P, 64), w(P + 39 * 4, 64)], **two)
    refused(weights, fq.INVALID_ARGUMENT, views=[view(), view(k=FAR)], after=[w(P, 64), w(P + 64 * 4 + 156, 64)], **two)   # head 1 and head 0
    refused(weights, fq.INVALID_ARGUMENT, views=[view(), view(k=FAR)], after=[w(P, 64), w(P + 50 * 4, 72)], **two)   # other strides
    with pytest.raises(ValueError):
        weights(after=[w(P, 64)] * 2)
    with pytest.raises(ValueError):
        weights(views=[view(), view()], after=w(P, 64), **two)


EVICT = [(dict(hkv=0), fq.INVALID_ARGUMENT), (dict(hkv=1025), fq.INVALID_ARGUMENT), (dict(k_len=(), keep=()), fq.INVALID_SEQUENCE_LENGTH),
         (dict(k_len=(1,) * 65, keep=(1,) * 65), fq.INVALID_ARGUMENT), (dict(k_len=(65,)), fq.KV_CACHE_OVERFLOW),
         (dict(row0=(30,)), fq.KV_CACHE_OVERFLOW), (dict(to_row0=(50,)), fq.KV_CACHE_OVERFLOW), (dict(keep=(4,)), fq.INVALID_ARGUMENT),
         (dict(sinks=2 ** 32 - 1, recent=2 ** 32 - 1), fq.INVALID_ARGUMENT), (dict(kept=0), fq.INVALID_ARGUMENT),
         (dict(kept=P + 1), fq.INVALID_ARGUMENT), (dict(w=fq.fq_key_weights(0, 64)), fq.INVALID_ARGUMENT),
         (dict(w=fq.fq_key_weights(P, 39)), fq.INVALID_ARGUMENT), (dict(to_w=fq.fq_key_weights(P, 19)), fq.INVALID_ARGUMENT),
         (dict(to_w=fq.fq_key_weights(P + 2, 64)), fq.INVALID_ARGUMENT)]


@pytest.mark.parametrize("kw,status", EVICT)
def test_evict_refusals(kw, status):
    refused(evict, status, **kw)


@pytest.mark.parametrize("kw,status", [c for c in VIEWS if "rows" not in c[0]])
def test_evict_view_refusals(kw, status):
    refused(evict, status, views=view(**kw))
    refused(evict, status, to=view(**kw))


def test_evict_rows_that_would_race():
    w = fq.fq_key_weights
    refused(evict, fq.INVALID_ARGUMENT, to=view())                                            # in place
    refused(evict, fq.INVALID_ARGUMENT, to=view(k=P + 39 * 256, v=FAR))                       # K over the last row that is read
    refused(evict, fq.INVALID_ARGUMENT, to=view(k=FAR, v=FAR))                                # K and V to the same rows
    two = dict(k_len=(20, 20), keep=(10, 10))
    refused(evict, fq.INVALID_ARGUMENT, to_row0=(0, 9), **two)
    refused(evict, fq.INVALID_ARGUMENT, to=[view(k=FAR, v=FAR + (1 << 30))] * 2, **two)
    refused(evict, fq.INVALID_ARGUMENT, to_w=w(FAR, 64), to_row0=(0, 5), **two)
    refused(evict, fq.INVALID_ARGUMENT, to=[view(k=FAR, v=FAR + (1 << 30)), view(k=FAR + (1 << 31), v=FAR + (1 << 32))],
            to_w=[w(FAR, 64), w(FAR + 36, 64)], **two)
    far = dict(to=view(k=FAR, v=FAR + (1 << 30)))
    refused(evict, fq.INVALID_ARGUMENT, to_w=w(P, 64), **far)                                  # weights in place
    refused(evict, fq.INVALID_ARGUMENT, to_w=w(P + 39 * 4, 64), **far)
    refused(evict, fq.INVALID_ARGUMENT, to_w=w(P, 64), to_row0=(30,), **far)
    with pytest.raises(ValueError):
        evict(k_len=(1, 2), keep=(1,))
    for bad in (-1, 1 << 32):
        for name in ("sinks", "recent"):
            with pytest.raises(ValueError):
                evict(**{name: bad})


def test_nothing_to_do():
    """No rows at all: nothing is launched and no buffer is asked for."""
    fq.fq_attn_window(0, view(), (0, 0), (4, 0), 4, 2, 1, 1, 0.1, 0)
    fq.fq_attn_paged(0, pool(), P, 1, (0,), (4,), 4, 2, 0, 0, 0.1, 0)
    fq.fq_attn_paged(0, pool(k=0, v=0, n_pages=0), 0, 0, (0,), (0,), 4, 2, 0, 0, 0.1, 0)
    fq.fq_qk_norm_rope_paged(0, (0,), (0,), pool(), 0, 0, (0,), 4, 2, 0, 0, 1e-6, 0, 0, 0)
    fq.fq_kv_evict(view(), fq.fq_key_weights(P, 64), None, (5, 0), (0, 7), 0, 0, 2, view(), None, None, 0)
