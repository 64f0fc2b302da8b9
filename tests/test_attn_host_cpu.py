"""Host side of the prompt and shared-prompt attention operators, without a GPU: what is refused before
anything is launched.  Addresses are made up."""
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


def refused(call, status, **kw):
    with pytest.raises(fq.FqError) as e:
        call(**kw)
    assert e.value.status == status, kw


def wait_timeout(q=P, v=None, q_len=4, k_len=4, hq=4, hkv=2, out=P, starve=1, cycles=0):
    fq.fq_debug_attn_wait_timeout(q, view() if v is None else v, q_len, k_len, hq, hkv, out, starve, cycles, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), fq.INVALID_ARGUMENT), (dict(q=P + 8), fq.INVALID_ARGUMENT), (dict(out=0), fq.INVALID_ARGUMENT),
    (dict(k_len=65), fq.KV_CACHE_OVERFLOW), (dict(q_len=0), fq.INVALID_SEQUENCE_LENGTH), (dict(hq=5), fq.INVALID_ARGUMENT),
    (dict(hq=6), fq.UNSUPPORTED), (dict(starve=3), fq.INVALID_ARGUMENT), (dict(cycles=(1 << 29) + 1), fq.INVALID_ARGUMENT),
    (dict(v=view(k=P + 2)), fq.INVALID_ARGUMENT)])
def test_wait_timeout_hook_refusals(kw, status):
    refused(wait_timeout, status, **kw)


@pytest.mark.parametrize("bad", [2 ** 32 + 4, -1, -2 ** 32 + 4, 4.5, 4.0, "4", None])
def test_lengths_do_not_wrap_around(bad):
    """What 32 bits do not hold is refused: a ctypes array would take 2^32 + 4 for 4."""
    v = view()
    for call in (lambda: fq.u32_array([4, bad]),
                 lambda: fq.fq_attn_prompt(P, v, [bad], [4], 4, 2, 0.1, P),
                 lambda: fq.fq_attn_prompt(P, v, [4], [bad], 4, 2, 0.1, P),
                 lambda: fq.fq_attn_prompt(P, v, [4], [4], 4, 2, 0.1, P, kv_row0=[bad]),
                 lambda: fq.fq_attn_prompt_workspace([4], [bad], 4, 2),
                 lambda: fq.fq_attn_shared(P, v, 4, [v], [bad], 4, 2, 0.1, P),
                 lambda: fq.fq_attn_shared_workspace(4, [bad], 4, 2),
                 lambda: fq.fq_qk_norm_rope(P, [bad], [0], v, [0], 4, 2, P, P, 1e-6, P, 64, P),
                 lambda: fq.fq_qk_norm_rope(P, [4], [bad], v, [0], 4, 2, P, P, 1e-6, P, 64, P),
                 lambda: fq.fq_qk_norm_rope(P, [4], [0], v, [bad], 4, 2, P, P, 1e-6, P, 64, P)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fq.fq_attn_shared(P, v, bad, [v], [4], 4, 2, 0.1, P),
                 lambda: fq.fq_attn_shared_workspace(bad, [4], 4, 2),
                 lambda: fq.fq_qk_norm_rope(P, [4], [0], v, [0], 4, 2, P, P, 1e-6, P, bad, P)):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_lengths_as_they_come():
    import numpy as np
    for values in ([], [0], [1, 2 ** 32 - 1], (3, 4), np.array([5, 6]), np.array([7], dtype=np.uint32)):
        a = fq.u32_array(values)
        assert list(a) == [int(v) for v in values] and fq.u32_array(a) is a
