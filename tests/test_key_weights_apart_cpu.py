"""What a call of fq_attn_key_weights reads and writes of gathered weights, without a GPU (launches are only written down):
weights that one sequence or head adds to while another writes them are refused, and no others."""
import itertools
import random

import pytest

from quantized_decoder_decode_gb300 import fq
from tests.test_cache_plan_cpu import BIG, host, recorded, view  # noqa: F401

P = 0x10000
HQ, HKV = 8, 4


def call(k_len, before, after, row0=None, hkv=HKV):
    n = len(k_len)
    views = view(1000, hkv) if len(after) == 1 else [view(1000, hkv, P + (s << 42)) for s in range(n)]
    fq.fq_attn_key_weights(P, P, views, [1] * n, k_len, 2 * hkv, hkv, 0, 0, 0.1, before, after, P, 1 << 30, kv_row0=row0)


def refused(host, *a, **kw):  # noqa: F811
    with recorded(host) as launches:
        try:
            call(*a, **kw)
        except fq.FqError as e:
            assert e.status == fq.INVALID_ARGUMENT and "weights" in str(e) and not launches(), str(e)
            return True
        assert launches()
    return False


def w(floats, stride):
    return fq.fq_key_weights(BIG + 4 * floats, stride)


def test_before_and_after_the_same(host):  # noqa: F811
    assert not refused(host, [300], [w(0, 400)], [w(0, 400)])
    assert not refused(host, [100, 0, 50], [w(0, 400)], [w(0, 400)])
    assert not refused(host, [100, 50], [w(0, 100), w(1000, 70)], [w(0, 100), w(1000, 70)])
    assert not refused(host, [100, 50], None, [w(0, 100), w(1000, 70)])


def test_before_and_after_apart(host):  # noqa: F811
    assert not refused(host, [300], [w(10000, 300)], [w(0, 400)])
    assert not refused(host, [300], [w(400, 800)], [w(0, 800)])                 # [head][before, after][rows]
    assert not refused(host, [100, 50], [w(0, 400)], [w(200, 400)])             # behind one another in a head
    assert not refused(host, [100, 100], [w(0, 400)], [w(100, 400)], row0=[0, 200])
    assert not refused(host, [100, 50], [w(0, 100), w(1000, 70)], [w(0, 100), w(2000, 70)])   # one of them in place
    assert not refused(host, [10, 10], [w(0, 100), w(1000, 70)], [w(20, 130), w(2000, 70)])   # strides of their own, heads in between


@pytest.mark.parametrize("k_len,before,after,row0", [
    ([300], [w(1, 400)], [w(0, 400)], None),                       # a row further
    ([300], [w(400, 400)], [w(0, 400)], None),                     # a head further
    ([300], [w(299, 800)], [w(0, 800)], None),
    ([300], [w(0, 401)], [w(0, 400)], None),                       # another stride
    ([100, 100], [w(0, 400)], [w(100, 400)], None),                # one sequence writes what the other reads
    ([100, 100], [w(0, 400)], [w(199, 400)], [0, 200]),
    ([100, 50], [w(1000, 70), w(0, 100)], [w(0, 100), w(1000, 70)], None),
    ([100, 50], [w(0, 100), w(5000, 70)], [w(0, 100), w(5049, 70)], None)])
def test_before_and_after_that_meet(host, k_len, before, after, row0):  # noqa: F811
    assert refused(host, k_len, before, after, row0)


def test_one_head(host):  # noqa: F811
    """Strides are not looked at."""
    assert not refused(host, [300], [w(0, 7)], [w(0, 9)], hkv=1)
    assert not refused(host, [300], [w(300, 1)], [w(0, 1)], hkv=1)
    assert refused(host, [300], [w(299, 1)], [w(0, 1)], hkv=1)


@pytest.mark.parametrize("seed", range(4))
def test_random_calls_against_the_list_of_weights(host, seed):  # noqa: F811
    rng = random.Random(seed)
    seen = {False: 0, True: 0}
    for _ in range(300):
        n, hkv = rng.randint(1, 3), rng.randint(1, 4)
        k_len = [rng.randint(0, 12) for _ in range(n)]
        strides = [rng.randint(max(k_len + [1]), 40) for _ in range(2)]
        at = [[rng.randint(0, 150) for _ in range(n)] for _ in range(2)]
        stride = [[rng.choice(strides) for _ in range(n)] for _ in range(2)]
        if rng.random() < .5:   # in place, but for one perhaps
            at[0], stride[0] = list(at[1]), list(stride[1])
            if rng.random() < .5:
                at[0][rng.randrange(n)] += rng.randint(-3, 3) + 500 * rng.randint(0, 1)
                at[0] = [max(0, x) for x in at[0]]
        floats = [[[{at[i][s] + h * stride[i][s] + r for r in range(k_len[s])} for h in range(hkv)] for s in range(n)] for i in range(2)]
        same = [at[0][s] == at[1][s] and (hkv == 1 or stride[0][s] == stride[1][s]) for s in range(n)]
        pairs = [(x, y) for x in itertools.product(range(n), range(hkv)) for y in itertools.product(range(n), range(hkv))]
        want = any(floats[1][s][h] & floats[1][t][g] and (s, h) != (t, g) or
                   floats[0][s][h] & floats[1][t][g] and not ((s, h) == (t, g) and same[s]) for (s, h), (t, g) in pairs)
        before, after = ([w(at[i][s], stride[i][s]) for s in range(n)] for i in range(2))
        if sum(k_len):
            assert refused(host, k_len, before, after, hkv=hkv) == want, (k_len, hkv, at, stride)
            seen[want] += 1
    assert min(seen.values()) > 30, seen
