"""A pool that rows are appended to: pages, rows and heads that share elements are refused, and no others, without a GPU
(launches are only written down)."""
import itertools
import random

import pytest

from quantized_decoder_decode_gb300 import fq
from tests.test_cache_plan_cpu import host, recorded  # noqa: F401

P, D = 0x10000, 128


def append(pages, hkv, n=3):
    fq.fq_qk_norm_rope_paged(P, (n,), (0,), pages, P, 4, (5,), 2 * hkv, hkv, P, P, 1e-6, P, 64, P, 0)


def refused(host, pages, hkv):  # noqa: F811
    with recorded(host) as launches:
        try:
            append(pages, hkv)
        except fq.FqError as e:
            assert e.status == fq.INVALID_ARGUMENT and not launches(), str(e)
            return True
        assert [v[0] for v in launches()] == [3]
    return False


def meet(k, v, n_pages, rows, strides, hkv):
    """Do two rows of the pool share elements?  By the list of all of them."""
    ps, rs, hs = strides
    at = sorted(base // 2 + p * ps + r * rs + h * hs
                for base in (k, v) for p in range(n_pages) for r in range(rows) for h in range(hkv))
    return any(b - a < D for a, b in zip(at, at[1:]))


FAR = 1 << 40
N, R, H = 6, 16, 4     # pages, rows, heads
LAYOUTS = {            # k -> v in elements, page, row and head stride
    "page head row": (FAR, H * R * D, D, R * D),
    "page row head": (FAR, H * R * D, H * D, D),
    "head page row": (FAR, R * D, D, N * R * D),
    "row head page": (FAR, D, N * H * D, N * D),
    "with gaps": (FAR, H * (R * (D + 8) + 24), D + 8, R * (D + 8) + 16),
    "page kv head row": (H * R * D, 2 * H * R * D, D, R * D),
    "page row kv head": (H * D, 2 * R * H * D, 2 * H * D, D),
    "page row head kv": (D, 2 * R * H * D, 2 * H * D, 2 * D),
    "kv page row head": (N * R * H * D, R * H * D, H * D, D),
    "page layer kv head row": (H * R * D, 10 * H * R * D, D, R * D),
    "v a few pages and a row of heads behind k": (3 * 4 * R * H * D + H * D, 4 * R * H * D, 2 * H * D, D),
    "k behind v": (-H * D, 2 * R * H * D, 2 * H * D, D),
}


@pytest.mark.parametrize("name", LAYOUTS)
def test_layouts_that_programs_have(host, name):  # noqa: F811
    c, ps, rs, hs = LAYOUTS[name]
    k = P + (1 << 30)
    pages = fq.fq_kv_pages(k, k + 2 * c, N, R, ps, rs, hs)
    assert not meet(k, k + 2 * c, N, R, (ps, rs, hs), H)
    assert not refused(host, pages, H)


@pytest.mark.parametrize("c,ps,rs,hs", [
    (0, H * R * D, D, R * D),                 # K and V are the same rows
    (FAR, D, D, R * D),                       # pages a row apart
    (FAR, H * R * D - 8, D, R * D),           # .. whose last row ends in the next
    (FAR, H * R * D, D, D),                   # rows and heads of one stride
    (FAR, H * R * D, R * D, R * D),
    (FAR, H * R * D, D, (R - 1) * D),         # a head's last row is the next one's first
    (FAR, H * R * D, H * D - 8, D),
    (H * R * D, H * R * D, D, R * D),         # K's next page is V's page
    (D, H * R * D, H * D, D),                 # V a head behind K
    (H * R * D - 8, 2 * H * R * D, D, R * D),
    (-64, H * R * D, D, R * D),
    (5 * H * R * D, H * R * D, D, R * D)])    # K's last page is V's first
def test_rows_that_share_elements(host, c, ps, rs, hs):  # noqa: F811
    k = P + (1 << 30)
    assert meet(k, k + 2 * c, N, R, (ps, rs, hs), H)
    assert refused(host, fq.fq_kv_pages(k, k + 2 * c, N, R, ps, rs, hs), H)


def test_strides_that_are_not_looked_at(host):  # noqa: F811
    """Of one page, of one head: whatever they are."""
    assert not refused(host, fq.fq_kv_pages(P, FAR, 1, R, 8, D, R * D), H)
    assert not refused(host, fq.fq_kv_pages(P, FAR, N, R, R * D, D, 8), 1)
    assert refused(host, fq.fq_kv_pages(P, P, 1, R, 8, D, R * D), H)


def test_large_pools(host):  # noqa: F811
    for n_pages, rows, hkv in itertools.product((1 << 20, 1 << 28), (16, 256), (1, 8, 512)):
        ps = rows * hkv * D
        if n_pages * ps > 1 << 46:
            continue
        k = P + (1 << 50)
        assert not refused(host, fq.fq_kv_pages(k, k + 2 * n_pages * ps, n_pages, rows, ps, D, rows * D), hkv)
        assert not refused(host, fq.fq_kv_pages(k, k - 2 * n_pages * ps, n_pages, rows, ps, hkv * D, D), hkv)
        assert not refused(host, fq.fq_kv_pages(k, k + 2 * ps, n_pages, rows, 2 * ps, D, rows * D), hkv)
        assert refused(host, fq.fq_kv_pages(k, k + 2 * n_pages * ps - 16, n_pages, rows, ps, D, rows * D), hkv)
        if n_pages > 1 << 20:
            continue
        # pages innermost; and V among K's rows, which no nest of strides shows
        ps = (n_pages + 1) * D
        assert not refused(host, fq.fq_kv_pages(k, k + 2 * rows * ps, n_pages, rows, D, ps, D), 1)
        assert not refused(host, fq.fq_kv_pages(k, k + 2 * (2 * ps + n_pages * D), n_pages, rows, D, 4 * ps, D), 1)
        assert refused(host, fq.fq_kv_pages(k, k + 2 * (4 * ps + n_pages * D - 8), n_pages, rows, D, 4 * ps, D), 1)


@pytest.mark.parametrize("seed", range(4))
def test_random_pools_against_the_list_of_rows(host, seed):  # noqa: F811
    """Nests of the dimensions in any order, some strides and offsets a little off."""
    rng = random.Random(seed)
    seen = {False: 0, True: 0}
    for _ in range(400):
        hkv, n_pages = rng.randint(1, 4), rng.randint(1, 5)
        dims, stride, at = {"page": n_pages, "row": R, "head": hkv, "kv": 2}, {}, D
        for d in rng.sample(sorted(dims), 4):
            stride[d] = max(D, at + rng.choice((0, 0, 0, 8, 40, -8, D, rng.randint(-8, 8) * D)))
            at = stride[d] * dims[d]
        if rng.random() < .3:
            stride["kv"] = rng.choice((1, -1)) * rng.randint(0, 3 * at // 8) * 8
        k = P + (1 << 30)
        v = k + 2 * stride["kv"]
        strides = tuple(stride[d] for d in ("page", "row", "head"))
        want = meet(k, v, n_pages, R, strides, hkv)
        assert refused(host, fq.fq_kv_pages(k, v, n_pages, R, *strides), hkv) == want, (dims, stride)
        seen[want] += 1
    assert min(seen.values()) > 40, seen
