"""Refusals of the prompt and shared-prompt attention operators: every check runs on the host
before anything is launched, so none of these needs a GPU.  Addresses are made up."""
import math

import pytest

from quantized_decoder_decode_gb300 import build as fqbuild
from quantized_decoder_decode_gb300 import fq

P = 0x10000   # a 16-byte aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def lib():
    fqbuild.build()
    return fq.lib()


def view(k=P, v=P, rows=64, row_stride=128, head_stride=64 * 128):
    return fq.fq_kv_view(k, v, rows, row_stride, head_stride)


def prompt(q=P, views=None, q_len=(4,), k_len=(4,), hq=4, hkv=2, scale=0.1, out=P, ws=P, ws_bytes=1 << 30, **kw):
    fq.fq_attn_prompt(q, view() if views is None else views, q_len, k_len, hq, hkv, scale, out, ws, ws_bytes, 0, **kw)


def shared(q=P, prefix=None, prefix_len=5, tails=None, tail_len=(3, 2), hq=4, hkv=2, scale=0.1, out=P, ws=P,
           ws_bytes=1 << 30, **kw):
    fq.fq_attn_shared(q, view() if prefix is None else prefix, prefix_len, [view(), view()] if tails is None else tails,
                      tail_len, hq, hkv, scale, out, ws, ws_bytes, 0, **kw)


def rows(qkv=P, lens=(4, 3), pos0=(0, 9), views=None, kv_row0=(0, 4), hq=4, hkv=2, qn=P, kn=P, eps=1e-6, rope=P,
         rope_rows=64, q=P, **kw):
    fq.fq_qk_norm_rope(qkv, lens, pos0, view() if views is None else views, kv_row0, hq, hkv, qn, kn, eps, rope,
                       rope_rows, q, 0, **kw)


def refused(call, status, **kw):
    with pytest.raises(fq.FqError) as e:
        call(**kw)
    assert e.value.status == status, kw


HEADS = [(dict(hq=0), fq.INVALID_ARGUMENT), (dict(hkv=0), fq.INVALID_ARGUMENT), (dict(hq=5), fq.INVALID_ARGUMENT),
         (dict(hq=6, hkv=2), fq.UNSUPPORTED), (dict(hq=16, hkv=1), fq.UNSUPPORTED),
         (dict(hq=2048, hkv=2048), fq.INVALID_ARGUMENT)]
VIEWS = [(dict(k=0), fq.INVALID_ARGUMENT), (dict(v=0), fq.INVALID_ARGUMENT), (dict(k=P + 8), fq.INVALID_ARGUMENT),
         (dict(v=P + 2), fq.INVALID_ARGUMENT), (dict(rows=2), fq.KV_CACHE_OVERFLOW),
         (dict(row_stride=132), fq.INVALID_ARGUMENT), (dict(row_stride=120), fq.INVALID_ARGUMENT),
         (dict(head_stride=100), fq.INVALID_ARGUMENT), (dict(head_stride=64), fq.INVALID_ARGUMENT),
         (dict(row_stride=1 << 40), fq.INVALID_ARGUMENT)]
IO = [(dict(q=0), fq.INVALID_ARGUMENT), (dict(out=0), fq.INVALID_ARGUMENT), (dict(q=P + 8), fq.INVALID_ARGUMENT),
      (dict(out=P + 4), fq.INVALID_ARGUMENT), (dict(q_stride=256), fq.INVALID_ARGUMENT),
      (dict(q_stride=516), fq.INVALID_ARGUMENT), (dict(out_stride=514), fq.INVALID_ARGUMENT),
      (dict(out_stride=128), fq.INVALID_ARGUMENT), (dict(out_dtype="q8_0"), fq.UNSUPPORTED),
      (dict(scale=math.nan), fq.INVALID_ARGUMENT), (dict(scale=math.inf), fq.INVALID_ARGUMENT)]


@pytest.mark.parametrize("kw,status", HEADS + IO)
def test_prompt_refusals(kw, status):
    refused(prompt, status, **kw)


@pytest.mark.parametrize("kw,status", VIEWS)
def test_prompt_view_refusals(kw, status):
    refused(prompt, status, views=view(**kw))
    refused(prompt, status, views=[view(), view(**kw)], q_len=(4, 4), k_len=(4, 4))


def test_prompt_counts():
    refused(prompt, fq.INVALID_SEQUENCE_LENGTH, q_len=(), k_len=())
    refused(prompt, fq.INVALID_ARGUMENT, q_len=(1,) * 65, k_len=(1,) * 65)
    refused(prompt, fq.INVALID_ARGUMENT, views=[view()] * 2, q_len=(1,) * 3, k_len=(1,) * 3)
    refused(prompt, fq.KV_CACHE_OVERFLOW, q_len=(1, 1), k_len=(60, 5))              # 60 + 5 rows of 64
    refused(prompt, fq.KV_CACHE_OVERFLOW, q_len=(1,), k_len=(60,), kv_row0=(5,))
    refused(prompt, fq.INVALID_ARGUMENT, q_len=(1 << 30, 1 << 30), k_len=(4, 4))
    refused(prompt, fq.INVALID_ARGUMENT, views=view(rows=1 << 31), q_len=(1,), k_len=(1 << 31,))
    refused(prompt, fq.KV_CACHE_OVERFLOW, q_len=(1,), k_len=(2,), kv_row0=(2 ** 32 - 1,))   # no 32-bit wrap
    with pytest.raises(ValueError):
        prompt(q_len=(1, 2), k_len=(1,))
    prompt(q=0, out=0, q_len=(0, 0), k_len=(3, 0))   # no query rows: nothing to do


def test_workspace_is_checked():
    q_len, k_len = (64,), (1 << 16,)   # few rows over many keys: the keys are split
    v = view(rows=1 << 16, head_stride=(1 << 16) * 128)
    need = fq.fq_attn_prompt_workspace(q_len, k_len, 4, 2)
    if need:
        refused(prompt, fq.INVALID_ARGUMENT, views=v, q_len=q_len, k_len=k_len, ws_bytes=need - 1)
        refused(prompt, fq.INVALID_ARGUMENT, views=v, q_len=q_len, k_len=k_len, ws=0)
        refused(prompt, fq.INVALID_ARGUMENT, views=v, q_len=q_len, k_len=k_len, ws=P + 8)
    need = fq.fq_attn_shared_workspace(1 << 16, (3, 2), 4, 2)
    if need:
        refused(shared, fq.INVALID_ARGUMENT, prefix=v, prefix_len=1 << 16, ws_bytes=need - 1)
    for call in (lambda: fq.fq_attn_prompt_workspace((), (), 4, 2), lambda: fq.fq_attn_shared_workspace(4, (), 4, 2)):
        refused(call, fq.INVALID_SEQUENCE_LENGTH)
    refused(lambda: fq.fq_attn_prompt_workspace((1,), (1,), 6, 2), fq.UNSUPPORTED)
    refused(lambda: fq.fq_attn_shared_workspace(4, (1,), 5, 2), fq.INVALID_ARGUMENT)


@pytest.mark.parametrize("kw,status", HEADS + IO)
def test_shared_refusals(kw, status):
    refused(shared, status, **kw)


@pytest.mark.parametrize("kw,status", VIEWS)
def test_shared_view_refusals(kw, status):
    refused(shared, status, prefix=view(**kw))
    refused(shared, status, tails=[view(), view(**kw)], tail_len=(3, 3))


def test_shared_counts():
    refused(shared, fq.INVALID_SEQUENCE_LENGTH, tails=[], tail_len=())
    refused(shared, fq.INVALID_ARGUMENT, tails=[view()] * 65, tail_len=(1,) * 65)
    refused(lambda: fq.fq_attn_shared(P, None, 3, [view()], (1,), 4, 2, 0.1, P, P, 1 << 30), fq.INVALID_ARGUMENT)
    refused(lambda: fq.fq_attn_shared(P, view(), 3, None, (1,), 4, 2, 0.1, P, P, 1 << 30), fq.INVALID_ARGUMENT)
    refused(shared, fq.KV_CACHE_OVERFLOW, prefix_len=65)
    with pytest.raises(ValueError):
        shared(tails=[view()], tail_len=(1, 2))


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(qkv=0), fq.INVALID_ARGUMENT), (dict(qkv=P + 4), fq.INVALID_ARGUMENT), (dict(q=0), fq.INVALID_ARGUMENT),
    (dict(q=P + 2), fq.INVALID_ARGUMENT), (dict(qn=0), fq.INVALID_ARGUMENT), (dict(kn=P + 4), fq.INVALID_ARGUMENT),
    (dict(rope=0), fq.INVALID_ARGUMENT), (dict(eps=-1.0), fq.INVALID_ARGUMENT), (dict(eps=math.nan), fq.INVALID_ARGUMENT),
    (dict(qkv_stride=1022), fq.INVALID_ARGUMENT), (dict(qkv_stride=512), fq.INVALID_ARGUMENT),
    (dict(q_stride=500), fq.INVALID_ARGUMENT), (dict(rope_rows=11), fq.INVALID_SEQUENCE_LENGTH),
    (dict(pos0=(0, 2 ** 32 - 2)), fq.INVALID_SEQUENCE_LENGTH), (dict(kv_row0=(0, 62)), fq.KV_CACHE_OVERFLOW),
    (dict(kv_row0=(0, 3)), fq.INVALID_ARGUMENT),                      # rows 3 .. of both sequences
    (dict(lens=(), pos0=(), kv_row0=()), fq.INVALID_SEQUENCE_LENGTH)])
def test_rows_refusals(kw, status):
    refused(rows, status, **kw)


@pytest.mark.parametrize("kw,status", VIEWS)
def test_rows_view_refusals(kw, status):
    refused(rows, status, views=view(**kw))
    refused(rows, status, views=[view(), view(**kw)], kv_row0=(0, 0))


def test_rows_counts():
    refused(rows, fq.INVALID_ARGUMENT, views=[view()] * 3)
    refused(rows, fq.INVALID_ARGUMENT, lens=(1,) * 65, pos0=(0,) * 65, kv_row0=(0,) * 65)
    # the same cache given twice under two views
    refused(rows, fq.INVALID_ARGUMENT, views=[view(), view()], kv_row0=(0, 1))
    rows(qkv=0, q=0, qn=0, kn=0, rope=0, lens=(0, 0), kv_row0=(0, 0))   # no rows: nothing to do


def test_layer_view_refusals():
    refused(lambda: fq.fq_kv_layer_view(None, 0), fq.INVALID_ARGUMENT)


def test_rows_beyond_a_device():
    n = 1 << 23   # x 512 heads
    refused(rows, fq.INVALID_ARGUMENT, hq=256, hkv=128, lens=(n,), pos0=(0,), kv_row0=(0,),
            views=view(rows=n, head_stride=n * 128), rope_rows=n)


def test_steps_of_operators_refusals():
    """What is refused before the model is looked at (the rest needs caches, hence a GPU)."""
    refused(lambda: fq.fq_forward_step_packed(0, [P], [1], [1]), fq.INVALID_ARGUMENT)
    refused(lambda: fq.fq_forward_step_packed(0, [P, P], [1, 2], [2]), fq.INVALID_ARGUMENT)
    refused(lambda: fq.fq_forward_step_packed(0, [P], [1, 2], [1]), fq.INVALID_ARGUMENT)
    refused(lambda: fq.fq_decode_step_shared(0, 0, [P], [1]), fq.INVALID_ARGUMENT)
    refused(lambda: fq.fq_decode_step_shared(0, 0, [P], [1, 2]), fq.INVALID_ARGUMENT)
