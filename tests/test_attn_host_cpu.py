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
