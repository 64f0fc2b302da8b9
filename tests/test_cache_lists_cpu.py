"""The launches that calls with long work lists make, without a GPU (launches are only written down); the lists themselves are
followed pair by pair."""
import pytest

from quantized_decoder_decode_gb300 import fq
from tests.cache_lists_util import ATTENTION, KEY_WEIGHTS, MANY_ROWS
from tests.test_cache_plan_cpu import BIG, P, check_weights, check_window, host, recorded, view  # noqa: F401


@pytest.mark.parametrize("name", KEY_WEIGHTS)
def test_key_weights(host, name):  # noqa: F811
    q_len, k_len, hq, hkv, window, sinks, own, want = KEY_WEIGHTS[name]
    with recorded(host) as launches:
        rows = sum(k_len)
        views = [view(rows, hkv, P + (s << 42)) for s in range(len(k_len))] if own else view(rows, hkv)
        after = [fq.fq_key_weights(BIG + (s << 32), rows) for s in range(len(k_len))] if own else fq.fq_key_weights(BIG, rows)
        fq.fq_attn_key_weights(P, P, views, q_len, k_len, hq, hkv, window, sinks, 0.1, None, after, P, 1 << 40)
        assert [(v[1], v[2]) for v in launches() if v[0] == 4] == want
    check_weights(host, q_len, k_len, hq, hkv, window, sinks, own)


def test_key_weights_of_many_rows(host):  # noqa: F811
    c = MANY_ROWS
    with recorded(host) as launches:
        fq.fq_attn_key_weights(P, P, view(c["L"], c["hkv"]), [c["L"]], [c["L"]], c["hq"], c["hkv"], c["window"], c["sinks"], 0.1, None,
                               fq.fq_key_weights(BIG, c["L"]), P, 1 << 40)
        more = [v[10 + 9 * u + 3] for v in launches() if v[0] == 4 for u in range(v[9])]
    assert 0 in more and 1 in more
    check_weights(host, [c["L"]], [c["L"]], c["hq"], c["hkv"], c["window"], c["sinks"], False)


@pytest.mark.parametrize("name", ATTENTION)
def test_attention(host, name):  # noqa: F811
    q_len, k_len, hq, hkv, window, sinks, kind, want = ATTENTION[name]
    with recorded(host) as launches:
        if kind == "pages":
            pages = fq.fq_kv_pages(P, P, 1 << 20, 16, 16 * 128 * hkv, 128, 16 * 128)
            fq.fq_attn_paged(P, pages, P, 1 << 27, q_len, k_len, hq, hkv, window, sinks, 0.1, BIG, P, 1 << 40)
        else:
            rows = sum(k_len)
            views = [view(rows, hkv, P + (s << 42)) for s in range(len(k_len))] if kind == "views" else view(rows, hkv)
            fq.fq_attn_window(P, views, q_len, k_len, hq, hkv, window, sinks, 0.1, BIG, P, 1 << 40)
        raw = launches()
    assert [(v[1], v[2]) for v in raw if v[0] == 0] == want
    assert any(v[0] == 2 for v in raw) == ("cut" in name)
    check_window(host, q_len, k_len, hq, hkv, window, sinks, kind == "pages", kind == "views")
