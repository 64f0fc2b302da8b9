"""Calls of the prompt attention whose lists need the larger parameter blocks or more than one launch (a CPU test says
which), and the packed step that makes such calls."""
import math

import numpy as np
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.attn_plan_util import MANY
from tests.gpu_util import assert_logits_close
from tests.prompt_ops_util import D, DEV, assert_within, attend, causal, gen, normal
from tests.test_gpu_packed_steps import assert_rows, packed, tokens_of
from tests.test_gpu_parity import SMALL, SMALL_G4, pair_factory, workload  # noqa: F401
from tests.test_gpu_prompt_ops import run_prompt, stream, view_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", MANY)
def test_calls_of_many_entries(name, out_dtype):
    q_len, k_len, hq, hkv, own_views, _ = MANY[name]
    g, n, scale = gen(len(name)), len(q_len), 1 / math.sqrt(D)
    q = normal(g, sum(q_len), hq, D)
    k0 = [sum(k_len[:s]) for s in range(n)]
    if own_views:   # with rows behind the keys that hold NaN
        ks, vs = ([torch.full((hkv, K + 130, D), math.nan, dtype=torch.bfloat16, device=DEV) for K in k_len] for _ in range(2))
        for s, K in enumerate(k_len):
            ks[s][:, :K], vs[s][:, :K] = normal(g, hkv, K, D), normal(g, hkv, K, D)
        views = [view_of(a, b, K + 130, D, (K + 130) * D) for a, b, K in zip(ks, vs, k_len)]
        kv = lambda s, h: (ks[s][h, :k_len[s]], vs[s][h, :k_len[s]])  # noqa: E731
    else:
        k, v = normal(g, hkv, sum(k_len), D), normal(g, hkv, sum(k_len), D)
        views = view_of(k, v, sum(k_len), D, sum(k_len) * D)
        kv = lambda s, h: (k[h, k0[s]:k0[s] + k_len[s]], v[h, k0[s]:k0[s] + k_len[s]])  # noqa: E731
    got = run_prompt(q, views, q_len, k_len, hq, hkv, out_dtype=out_dtype)
    again = run_prompt(q, views, q_len, k_len, hq, hkv, out_dtype=out_dtype)
    assert torch.equal(got, again) and bool(got.isfinite().all())
    r = 0
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        some = torch.arange(0, L, 1 if L * K < 1 << 21 else 13, device=DEV)   # rows looked at: every tile of tokens
        some = torch.unique(torch.cat((some, torch.tensor([L - 1], device=DEV))))
        for h in range(hq):
            ref, bound = attend(q[r + some, h], *kv(s, h // (hq // hkv)), causal(L, K)[some], scale)
            assert_within(got[r + some, h], ref, bound, out_dtype == "bf16", f"{name}: sequence {s} head {h}")
        r += L


@pytest.mark.parametrize("dims,n", [(SMALL, 40), (SMALL_G4, 64)])
def test_packed_step_of_many_prompts(pair_factory, dims, n):  # noqa: F811
    """40 and 64 prompts of different lengths in one step: what a forwardStep per sequence gives."""
    p = pair_factory(workload(dims, "q8_0", "bf16", seed=91), max_positions=256, with_oracle=False)
    lens, ctx = [20 + (7 * i * i) % 41 for i in range(n)], [(11 * i) % 70 for i in range(n)]
    seqs = [tokens_of(dims, 91, i, L) for i, L in enumerate(lens)]
    a, b = [[p.new_seq(capacity=c + L, ctx=c, seq=i, oracle_cache=False)[0] for i, (L, c) in enumerate(zip(lens, ctx))] for _ in range(2)]
    got = packed(p, a, seqs)
    ref = torch.empty(dims.vocab_size, device=DEV)
    for i in range(n):
        fq.fq_forward_step(p.model, b[i], seqs[i], ctx[i], ref.data_ptr(), stream())
        torch.cuda.synchronize()
        assert_logits_close(got[i], ref.cpu().numpy(), f"sequence {i}")
        for L in range(dims.num_layers):
            for x, y in zip(p.read_kv(a[i], L, ctx[i], lens[i]), p.read_kv(b[i], L, ctx[i], lens[i])):
                assert_rows(np.asarray(x), np.asarray(y), L, f"sequence {i} layer {L}")
