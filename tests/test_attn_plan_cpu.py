"""The work lists of the attention operators, without a GPU: every (query row, key) pair once, every partial
result joined once, inside the workspace and the bounds of a launch."""
import random

import pytest

from quantized_decoder_decode_gb300 import fq
from tests import attn_host_util
from tests.attn_plan_util import MANY, prompt, shared

HEADS = [(4, 4), (4, 2), (8, 2), (8, 1), (16, 8), (32, 8), (32, 4), (3, 3), (64, 64)]


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return attn_host_util.build(tmp_path_factory.mktemp("attn_plan"))


@pytest.fixture
def launches(host):
    with attn_host_util.recorded(host) as f:
        yield f


def length(rng):
    return rng.choice((0, 1, 2, 3, rng.randint(0, 40), rng.randint(0, 300), rng.randint(0, 3000)))


@pytest.mark.parametrize("seed", range(6))
def test_every_pair_once_in_random_prompts(launches, seed):
    rng = random.Random(seed)
    for _ in range(120):
        n = rng.choice((1, 1, 2, 3, 5, 17, 18, 30, 64))
        q = [length(rng) for _ in range(n)]
        k = [rng.choice((m, m, m + length(rng), length(rng), m + rng.randint(0, 30000))) for m in q]
        prompt(launches, q, k, *rng.choice(HEADS), rng.random() < .5)


@pytest.mark.parametrize("seed", range(4))
def test_every_pair_once_behind_random_prefixes(launches, seed):
    rng = random.Random(100 + seed)
    for _ in range(150):
        n = rng.choice((1, 2, 3, 5, 17, 33, 64))
        shared(launches, rng.choice((0, 1, length(rng), rng.randint(0, 30000))),
               [rng.choice((0, length(rng))) for _ in range(n)], *rng.choice(HEADS))


@pytest.mark.parametrize("name", MANY)
def test_calls_of_many_entries(launches, name):
    q_len, k_len, hq, hkv, own_views, want = MANY[name]
    reached = [r[:2] if r[0] != "rows" else r[:1] for r in prompt(launches, q_len, k_len, hq, hkv, own_views)]
    assert reached == want


def test_largest_lengths(launches):
    """The most rows of a call, in one sequence and in 64."""
    for q, k in (([1], [1 << 30]), ([64], [1 << 30]), ([1] * 64, [1 << 30] * 64)):
        prompt(launches, q, k, 8, 1, True)
    shared(launches, 1 << 29, [1 << 29] * 64, 8, 1)


def test_split_calls_need_a_workspace():
    """The lengths at which the refusal of a small workspace is tested do need one."""
    assert fq.fq_attn_prompt_workspace((64,), (1 << 16,), 4, 2) > 0
    assert fq.fq_attn_shared_workspace(1 << 16, (3, 2), 4, 2) > 0
