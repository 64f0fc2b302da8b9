"""Calls whose work lists are long (the kernels' larger arguments, lists of several launches that use one workspace in turn, sums that
a later launch adds to) on the GPU against plain 64-bit forms."""
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_lists_util import ATTENTION, KEY_WEIGHTS, MANY_ROWS
from tests.cache_ops_util import D, DEV, NAN, SCALE, Pool, assert_lse, reference, run_paged, run_window, visible
from tests.prompt_ops_util import assert_within, gen, normal
from tests.test_gpu_key_weights_evict import assert_weights, gathered, log_sums, run, view, weights

pytestmark = pytest.mark.gpu

# Beyond what gathered() bounds: the sums of up to 152 thread blocks' parts of a key, of each of two launches, a step each.
PARTS = 2 * 152 * 2.0 ** -24


@pytest.mark.parametrize("name", KEY_WEIGHTS)
def test_key_weights(name):
    q_len, k_len, hq, hkv, window, sinks, own, _ = KEY_WEIGHTS[name]
    g, S, G = gen(101 + sorted(KEY_WEIGHTS).index(name)), len(k_len), hq // hkv
    q = normal(g, sum(q_len), hq, D)
    ks = [normal(g, hkv, K, D) for K in k_len] if own else normal(g, hkv, sum(k_len), D).split(k_len, dim=1)
    lse = log_sums(q, lambda s, h: ks[s][h], q_len, k_len, hq, hkv, window, sinks)
    was = [torch.rand(hkv, K, generator=g, device=DEV) for K in k_len]
    if own:
        views = [view(k) for k in ks]
        got = [torch.full_like(w, NAN) for w in was]
        before, after = [weights(w) for w in was], [weights(w) for w in got]
    else:
        store = torch.cat(list(ks), dim=1).contiguous()
        views, all_was, all_got = view(store), torch.cat(was, dim=1).contiguous(), torch.full((hkv, sum(k_len)), NAN, device=DEV)
        got = all_got.split(k_len, dim=1)
        before, after = weights(all_was), weights(all_got)
    run(q, lse, views, q_len, k_len, hq, hkv, window, sinks, before, after)
    r = 0
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        seen = visible(L, K, window, sinks)
        for h in range(hkv):
            ref, bound = gathered(q[r:r + L, h * G:(h + 1) * G], lse[r:r + L, h * G:(h + 1) * G], ks[s][h], seen, SCALE)
            assert_weights(got[s][h], was[s][h], ref, bound + ref * PARTS, f"sequence {s} head {h}")
        r += L
    run(q, lse, views, q_len, k_len, hq, hkv, window, sinks, before, before)   # in place, the same bits
    now = was if own else all_was.split(k_len, dim=1)
    for s in range(S):
        assert bool((now[s] == got[s]).all())


def test_key_weights_of_many_rows():
    """Every row sees the sinks: more blocks of query rows than an entry has, so that a second launch adds to what the first one
    left; from zeros, on top of what was there, and in place."""
    c, g = MANY_ROWS, gen(131)
    L, hq, window, sinks = c["L"], c["hq"], c["window"], c["sinks"]
    q, k = normal(g, L, hq, D), normal(g, 1, L, D)
    lse = torch.empty(L, hq, device=DEV)
    ref, bound = (torch.zeros(L, dtype=torch.float64, device=DEV) for _ in range(2))
    for t in range(0, L, 2000):   # rows t .. and the keys that they see
        rows = torch.arange(t, min(L, t + 2000), device=DEV)
        keys = torch.cat((torch.arange(min(sinks, max(0, t - window)), device=DEV), torch.arange(max(0, t - window), int(rows[-1]) + 1, device=DEV)))
        seen = (keys[None] <= rows[:, None]) & ((keys[None] > rows[:, None] - window) | (keys[None] < sinks))
        for h in range(hq):
            s = torch.where(seen, q[rows, h].double() @ k[0, keys].double().T * SCALE, -torch.inf)
            lse[rows, h] = torch.logsumexp(s, dim=1).float()
        r, b = gathered(q[rows], lse[rows], k[0, keys], seen, SCALE)
        ref.index_add_(0, keys, r)
        bound.index_add_(0, keys, b)
    bound += ref * PARTS
    was = torch.rand(1, L, generator=g, device=DEV) * 100
    got, zeros = (torch.full((1, L), NAN, device=DEV) for _ in range(2))
    call = lambda before, after: run(q, lse, view(k), [L], [L], hq, 1, window, sinks, before, after)  # noqa: E731
    call(weights(was), weights(got))
    call(None, weights(zeros))
    assert_weights(got[0], was[0], ref, bound)
    assert_weights(zeros[0], torch.zeros_like(zeros[0]), ref, bound)
    call(weights(was), weights(was))
    assert bool((was == got).all())


@pytest.mark.parametrize("name", ATTENTION)
def test_attention(name):
    q_len, k_len, hq, hkv, window, sinks, kind, _ = ATTENTION[name]
    g = gen(151 + sorted(ATTENTION).index(name))
    q = normal(g, sum(q_len), hq, D)
    if kind == "pages":
        pool = Pool(g, k_len, hkv, 32)
        kv = pool.rows
        got, e = run_paged(q, pool, q_len, k_len, hq, hkv, window, sinks)
    else:
        ks, vs = ([normal(g, hkv, K, D) for K in k_len] for _ in range(2))
        kv = lambda s, h: (ks[s][h], vs[s][h])  # noqa: E731
        if kind == "views":
            views = [fq.fq_kv_view(a.data_ptr(), b.data_ptr(), K, D, K * D) for a, b, K in zip(ks, vs, k_len)]
        else:
            k, v, rows = torch.cat(ks, dim=1).contiguous(), torch.cat(vs, dim=1).contiguous(), sum(k_len)
            views = fq.fq_kv_view(k.data_ptr(), v.data_ptr(), rows, D, rows * D)
        got, e = run_window(q, views, q_len, k_len, hq, hkv, window, sinks)
    ref, bound, lse, lse_bound = reference(q, kv, q_len, k_len, hq, hkv, window, sinks)
    assert_within(got, ref, bound, True, name)
    assert_lse(e, lse, lse_bound, name)
