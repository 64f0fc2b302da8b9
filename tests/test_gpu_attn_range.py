"""Values and scores at the ends of the number range in the prompt and shared-prompt attention operators:
outputs are finite and right wherever the definition's are."""
import math

import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.prompt_ops_util import D, DEV, assert_within, gen, normal
from tests.test_gpu_prompt_ops import reference_prompt, reference_shared, run_prompt, run_shared, view_of

pytestmark = pytest.mark.gpu

# whole prompts (pairs of tiles, single ones), keys that are split, few rows over keys in one chunk and in
# several, short sequences beside long ones
LENGTHS = [([300], [300]), ([30, 700], [30, 700]), ([40], [9000]), ([1], [20]), ([2, 1], [5000, 700]), ([200, 1], [200, 900])]


@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (8, 1)])
@pytest.mark.parametrize("q_len,k_len", LENGTHS)
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_large_values(hq, hkv, q_len, k_len, out_dtype):
    """Values of up to 2^126 and more: their sums over the keys pass the f32 range, their means do not.  The scores are
    such that the reference maximum stays behind the maximum too."""
    g, rows = gen(61), sum(k_len)
    q, k = normal(g, sum(q_len), hq, D) * 2, normal(g, hkv, rows, D)
    v = (normal(g, hkv, rows, D, dtype=torch.float32).clamp(-4, 4).abs() * 2.0 ** 125).to(torch.bfloat16)
    got = run_prompt(q, view_of(k, v, rows, D, rows * D), q_len, k_len, hq, hkv, out_dtype=out_dtype)
    k0 = [sum(k_len[:s]) for s in range(len(k_len))]
    kv = lambda s, h: (k[h, k0[s]:k0[s] + k_len[s]], v[h, k0[s]:k0[s] + k_len[s]])  # noqa: E731
    ref, bound = reference_prompt(q, kv, q_len, k_len, hq, hkv)
    assert bool(got.isfinite().all())
    assert_within(got, ref, bound, out_dtype == "bf16")


@pytest.mark.parametrize("P,tail_len", [(700, [3, 0, 150]), (3000, [40] * 20), (0, [1, 600])])
def test_large_values_behind_a_shared_prefix(P, tail_len):
    g, hq, hkv, n = gen(62), 8, 2, len(tail_len)
    cap = max(tail_len) + 1
    big = lambda *s: (normal(g, *s, dtype=torch.float32).clamp(-4, 4).abs() * 2.0 ** 125).to(torch.bfloat16)  # noqa: E731
    q, pk, tk = normal(g, n, hq, D) * 2, normal(g, hkv, P, D), normal(g, n, hkv, cap, D)
    pv, tv = big(hkv, P, D), big(n, hkv, cap, D)
    tails = [view_of(tk[i], tv[i], cap, D, cap * D) for i in range(n)]
    got = run_shared(q, view_of(pk, pv, P, D, P * D) if P else None, P, tails, tail_len, hq, hkv)
    ref, bound = reference_shared(q, pk, pv, tk, tv, tail_len, hq, hkv)
    assert bool(got.isfinite().all())
    assert_within(got, ref, bound, True)


@pytest.mark.parametrize("L,K", [(300, 300), (3, 500), (1, 1)])
def test_the_largest_value_everywhere(L, K):
    """Equal scores and one value: the output is that value."""
    hq, hkv, top = 4, 2, 2.0 ** 127
    q, k = torch.zeros(L, hq, D, dtype=torch.bfloat16, device=DEV), torch.ones(hkv, K, D, dtype=torch.bfloat16, device=DEV)
    v = torch.full_like(k, top)
    got = run_prompt(q, view_of(k, v, K, D, K * D), [L], [K], hq, hkv)
    assert bool((got.float() == top).all())


@pytest.mark.parametrize("scale", [0.0, 1e-39, -1e-39, 2e-38])
@pytest.mark.parametrize("L,K", [(300, 300), (3, 500), (30, 9000)])
def test_tiny_scales_of_large_scores(scale, L, K):
    """Scores of up to 1e38 with scales from 0 to the smallest normal numbers: every scale counts as it is."""
    g, hq, hkv = gen(63), 4, 2
    q = (normal(g, L, hq, D, dtype=torch.float32).clamp(-3, 3) * 1.5e18).to(torch.bfloat16)
    k = (normal(g, hkv, K, D, dtype=torch.float32).clamp(-3, 3) * 1.5e18).to(torch.bfloat16)
    v = normal(g, hkv, K, D)
    got = run_prompt(q, view_of(k, v, K, D, K * D), [L], [K], hq, hkv, scale=scale)
    ref, bound = reference_prompt(q, lambda s, h: (k[h], v[h]), [L], [K], hq, hkv, scale)
    assert_within(got, ref, bound, True)


@pytest.mark.parametrize("bad", [3e38, -3e38])
@pytest.mark.parametrize("hq,hkv,at,L,K", [(4, 4, 100, 300, 300), (8, 1, 299, 300, 300), (4, 2, 0, 300, 300), (8, 2, 250, 20, 260),
                                           (8, 2, 255, 3, 256), (8, 2, 5000, 20, 9000), (8, 2, 100, 1, 3000)])
def test_one_large_value_among_ordinary_ones(bad, hq, hkv, at, L, K):
    """A finite value near the largest at one key: rows that see the key give what the definition gives, the others
    what they give without it."""
    g = gen(64)
    q, k, v = normal(g, L, hq, D), normal(g, hkv, K, D), normal(g, hkv, K, D)
    v[:, at, 60:70] = bad
    got = run_prompt(q, view_of(k, v, K, D, K * D), [L], [K], hq, hkv)
    ref, bound = reference_prompt(q, lambda s, h: (k[h], v[h]), [L], [K], hq, hkv)
    assert_within(got, ref, bound, True)
