"""Host side of the prompt and shared-prompt attention operators, without a GPU: what is refused before
anything is launched, and (with launches that are only written down) what is not.  Addresses are made up."""
import random

import pytest

from quantized_decoder_decode_gb300 import fq
from tests import attn_host_util

P = 0x10000   # a 16-byte aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def host(tmp_path_factory):
    return attn_host_util.build(tmp_path_factory.mktemp("attn_host"))


@pytest.fixture
def launches(host):
    with attn_host_util.recorded(host) as f:
        yield f


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


# ---- rows that one fq_qk_norm_rope call would write twice

B = 1 << 30   # bytes between made-up buffers


def elements(views, kv_row0, lens, hkv):
    """Every eighth element that the call writes, K and V of every sequence, as a list of addresses / 2."""
    out = []
    for s, n in enumerate(lens):
        v = views[s] if isinstance(views, list) else views
        for base in (v.k, v.v):
            out += [base // 2 + (kv_row0[s] + r) * v.row_stride + h * v.head_stride + d
                    for r in range(n) for h in range(hkv) for d in range(0, 128, 8)]
    return out


def written_twice(views, kv_row0, lens, hkv):
    e = elements(views, kv_row0, lens, hkv)
    return len(set(e)) < len(e)


def is_refused(launches, views, kv_row0, lens, hkv):
    try:
        fq.fq_qk_norm_rope(P, lens, [0] * len(lens), views, kv_row0, 2 * hkv, hkv, P, P, 1e-6, P, 1 << 20, P)
    except fq.FqError as e:
        assert e.status == fq.INVALID_ARGUMENT and ("same rows" in str(e) or "overlap" in str(e)), e
        assert launches() == []
        return True
    assert launches() == [[3, sum(lens)]]
    return False


def cache(k, cap=64):
    """A cache layer, [kv head][row][128], V at some distance from K."""
    return fq.fq_kv_view(k, k + B, cap, 128, cap * 128)


A = cache(P)
SHIFTED = fq.fq_kv_view(P + 16 * 256, P + B + 16 * 256, 48, 128, 64 * 128)   # rows 16 .. of the same layer
BETWEEN = fq.fq_kv_view(P + 256, P + 2 * B, 9, 256, 64 * 128)                # every second row of the layer's K, from 1
SIDE = fq.fq_kv_view(P, P + 2 * 256, 64, 4 * 128, 128)                       # K | V of two heads side by side in a row


@pytest.mark.parametrize("views,row0,lens,hkv,bad", [
    (A, [0, 4], [4, 4], 2, False), (A, [4, 0], [4, 5], 2, True), (A, [0, 0, 9], [0, 4, 1], 2, False),
    ([A, SHIFTED], [0, 0], [16, 4], 2, False), ([A, SHIFTED], [0, 0], [17, 4], 2, True),
    ([A, SHIFTED], [20, 3], [2, 1], 2, False), ([A, SHIFTED], [20, 5], [2, 1], 2, True),
    (SIDE, [0, 7], [7, 3], 2, False), ([SIDE, SIDE], [0, 7], [7, 3], 2, False), (SIDE, [0], [5], 3, True),
    (fq.fq_kv_view(P, P, 64, 128, 64 * 128), [0], [1], 2, True),         # K and V in one place
    (fq.fq_kv_view(P, P + B, 64, 128, 128), [0], [2], 2, True),          # head 1 of row 0 is row 1 of head 0
    (fq.fq_kv_view(P, P + B, 64, 128, 128), [0], [1], 2, False),
    (fq.fq_kv_view(P, P + B, 64, 256, 136), [0], [1], 2, False), (fq.fq_kv_view(P, P + B, 64, 256, 136), [0], [2], 2, True),
    ([A, cache(P + B)], [0, 0], [4, 4], 2, True),                        # V of one, K of the other
    ([A, cache(P + 2 * B)], [0, 0], [4, 4], 2, False),
    ([A, BETWEEN], [0, 0], [1, 4], 2, False), ([A, BETWEEN], [2, 0], [1, 4], 2, False), ([A, BETWEEN], [3, 0], [1, 4], 2, True)])
def test_rows_written_twice_are_refused(launches, views, row0, lens, hkv, bad):
    assert written_twice(views, row0, lens, hkv) == bad
    assert is_refused(launches, views, row0, lens, hkv) == bad


def test_rows_written_twice_in_random_layouts(launches):
    rng, seen = random.Random(5), [0, 0]
    for _ in range(4000):
        hkv, n = rng.choice((1, 2, 3, 4)), rng.randint(1, 4)
        rs, hs = rng.choice(((128, 12 * 128), (hkv * 128, 128), (2 * hkv * 128, 128), (136, 2000), (hkv * 136, 136), (256, 136)))

        def make():
            k = P + 16 * rng.choice((0, 1, 16, 32, 33, 16 * hkv, 16 * 12, rng.randint(0, 900), rng.randint(0, 9000)))
            wider = 8 if n < 3 and rng.random() < .3 else 0
            return fq.fq_kv_view(k, k + rng.choice((0, B, B, B, 256 * hkv)), 12, rs + wider, hs)
        views = make() if rng.random() < .4 else [make() for _ in range(n)]
        lens, row0 = [rng.choice((0, 1, 2, 5)) for _ in range(n)], [rng.randint(0, 7) for _ in range(n)]
        if sum(lens):
            bad = written_twice(views, row0, lens, hkv)
            seen[bad] += 1
            assert is_refused(launches, views, row0, lens, hkv) == bad, (views, row0, lens, hkv)
    assert min(seen) > 600, seen


def test_long_interleaved_rows_of_other_strides_are_refused_at_once(launches):
    """Two views of other strides whose rows lie between each other: found apart row by row where that is quick,
    refused where it is not."""
    for hkv, n, bad in ((2, 500, False), (64, 100000, True)):
        a = fq.fq_kv_view(P, P + B * 4096, n, 512, 512 * n)
        b = fq.fq_kv_view(P + 512, P + 2 * B * 4096, n, 1024, 512 * n)
        assert is_refused(launches, [a, b], [0, 0], [n // 4, n // 4], hkv) == bad


def test_rows_beyond_any_memory(launches):
    v = fq.fq_kv_view(P, P + B, 1 << 30, 1 << 36, 128)
    refused(lambda: fq.fq_qk_norm_rope(P, [1], [0], v, [1 << 20], 4, 2, P, P, 1e-6, P, 64, P), fq.INVALID_ARGUMENT)
    refused(lambda: fq.fq_attn_prompt(P, v, [1], [1], 4, 2, .1, P, P, 1 << 30, kv_row0=[1 << 20]), fq.INVALID_ARGUMENT)
    assert launches() == []


@pytest.mark.parametrize("head_stride", [0, 3, 1 << 37, 2 ** 64 - 1])
def test_one_kv_head_has_no_head_stride(launches, head_stride):
    v, w = fq.fq_kv_view(P, P + B, 64, 128, head_stride), fq.fq_kv_view(P + 2 * B, P + 3 * B, 64, 128, 128)
    fq.fq_qk_norm_rope(P, [3, 2], [0, 0], [v, w], [0, 0], 4, 1, P, P, 1e-6, P, 64, P)
    fq.fq_attn_prompt(P, [v, w], [3, 2], [3, 2], 4, 1, .1, P, P, 1 << 30)
    fq.fq_attn_shared(P, v, 5, [w], [3], 4, 1, .1, P, P, 1 << 30)
    assert len(launches()) >= 3
    refused(lambda: fq.fq_attn_prompt(P, v, [3], [3], 4, 2, .1, P, P, 1 << 30), fq.INVALID_ARGUMENT)
