"""Values that are not finite, seen by some rows and not by others, through every way that outputs of windows and pages take: bf16
and f32, whole units, units whose keys are split, few rows.  And what the roundings leave of all others."""
import math

import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.cache_ops_util import D, DEV, SCALE, Pool, run_paged, run_window, visible
from tests.prompt_ops_util import assert_within, attend, gen, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("hq,hkv,at,L,K,window,sinks", [
    (4, 4, [100], 300, 300, 50, 0), (4, 2, [128, 130], 300, 300, 128, 4), (4, 2, [0, 3, 4], 300, 300, 64, 4),
    (8, 2, [250, 100], 20, 260, 33, 3), (8, 2, [255, 0], 1, 256, 16, 1), (4, 4, [90, 200], 2, 300, 100, 91),
    (4, 2, [700, 701, 1100], 700, 1500, 300, 20), (4, 2, [3, 2970, 8100, 11990], 64, 12000, 9000, 20), (2, 1, [100, 39000, 59999], 2, 60000, 21000, 200)])
def test_rows_get_the_values_that_they_see(out_dtype, paged, hq, hkv, at, L, K, window, sinks):
    """+inf, -inf and NaN in different dims of keys here and there: a row that sees one has it in its output, both infinities
    give NaN, other rows and dims are within the bound of the roundings."""
    g, G, bf16 = gen(311), hq // hkv, out_dtype == "bf16"
    q, k, v = normal(g, L, hq, D), normal(g, hkv, K, D), normal(g, hkv, K, D)
    clean = v.clone()
    odd = {5: math.inf, 6: -math.inf, 127: math.nan, 64: math.inf}   # dim: value
    for i, key in enumerate(at):
        for d, x in odd.items():
            v[i % hkv, key, d] = -x if d == 64 and i // hkv % 2 else x   # (dim 64: infinities of both signs)
            clean[i % hkv, key, d] = 0
    if paged:
        pool = Pool(g, [K], hkv, 32)
        pool.put(pool.k, 0, 0, k)
        pool.put(pool.v, 0, 0, v)
        got, _ = run_paged(q, pool, [L], [K], hq, hkv, window, sinks, out_dtype=out_dtype)
    else:
        got, _ = run_window(q, fq.fq_kv_view(k.data_ptr(), v.data_ptr(), K, D, K * D), [L], [K], hq, hkv, window, sinks, out_dtype=out_dtype)
    seen = visible(L, K, window, sinks)
    for h in range(hq):
        kh = h // G
        ref, bound = attend(q[:, h], k[kh], clean[kh], seen, SCALE)
        want = torch.zeros(L, D, device=DEV)
        for i, key in enumerate(at):
            if i % hkv == kh:
                for d in odd:
                    want[:, d] += torch.where(seen[:, key], v[kh, key, d].float(), 0.0)
        plain = want == 0
        assert_within(got[:, h][plain], ref[plain], bound[plain], bf16, f"head {h}")
        x, y = got[:, h][~plain].float(), want[~plain]
        assert bool((torch.isnan(x) == torch.isnan(y)).all()) and bool((x[~torch.isnan(y)] == y[~torch.isnan(y)]).all()), f"head {h}"


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len,k_len,hq,hkv,window,sinks", [
    ([17], [1017], 16, 8, 256, 4), ([1] * 16, [512 + 479 * i for i in range(16)], 32, 8, 2048, 4), ([1] * 7 + [333], [2048, 17, 901, 1500, 333, 4096, 129, 1333], 16, 8, 0, 0),
    ([1500], [1500], 8, 8, 700, 4)])
def test_roundings(out_dtype, q_len, k_len, hq, hkv, window, sinks):
    """Root mean square of the error, relative to that of the outputs.  A rounding to bf16 is off by at most 2^-8 of the value, evenly, so
    by 2^-8 / sqrt(3) of it in the mean.  With independent values of V of one variance the weights' roundings leave as much in
    sum_j p_j e_j v_j as one rounding of it, and the output's own comes on top: sqrt(2) of it together.  And a call
    gives the same bits every time."""
    g = gen(331)
    q, rows = normal(g, sum(q_len), hq, D), sum(k_len)
    k, v = normal(g, hkv, rows, D), normal(g, hkv, rows, D)
    view = fq.fq_kv_view(k.data_ptr(), v.data_ptr(), rows, D, rows * D)
    got, lse = run_window(q, view, q_len, k_len, hq, hkv, window, sinks, out_dtype=out_dtype)
    err = size = 0.0
    r = c = 0
    for L, K in zip(q_len, k_len):
        for h in range(hq):
            kv = h // (hq // hkv)
            ref, _ = attend(q[r:r + L, h], k[kv, c:c + K], v[kv, c:c + K], visible(L, K, window, sinks), SCALE)
            err += float((got[r:r + L, h].double() - ref).square().sum())
            size += float(ref.square().sum())
        r, c = r + L, c + K
    assert math.sqrt(err / size) < 2.0 ** -8 / math.sqrt(3) * (math.sqrt(2) if out_dtype == "bf16" else 1)
    for _ in range(4):
        again, e = run_window(q, view, q_len, k_len, hq, hkv, window, sinks, out_dtype=out_dtype)
        assert bool((again == got).all()) and bool((e == lse).all())
