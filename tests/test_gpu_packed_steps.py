"""The packed forwardStep and the shared-prefix decode step: the steps that are made of the prompt
and shared-prompt attention operators, against the oracle and against the steps that they are
equal to up to rounding.

Tolerances.  Besides the f32 arithmetic of the other steps these round q (half a bf16 step, 2^-8)
and the softmax weights (2^-8 each).  In a 64-bit form of the models below, roundings of a whole
2^-8 with random signs everywhere move the logits by up to 0.012 (200 tokens) and the K and V rows
of the second layer by up to 7.5 times the absolute part of the row tolerance, on top of one bf16
step of the row: the logits keep their 2e-2, rows above the first layer get 16 times the absolute
part."""
import numpy as np
import pytest
import torch

import synth
import synth.workloads as wl
from quantized_decoder_decode_gb300 import fq
from tests.gpu_util import DEV, assert_logits_close, stream
from tests.test_gpu_parity import SMALL, SMALL_G4, SMALL_MOE, pair_factory, workload  # noqa: F401

pytestmark = pytest.mark.gpu


def tokens_of(dims, seed, i, n):
    return [int(t) for t in synth.uniform_i32(seed, 100 + i, n, 0, dims.vocab_size)]


def assert_rows(got, ref, layer, what):
    tol = 2.0 ** -7 * np.abs(ref) + (1 if layer == 0 else 16) * (1e-3 * float(np.abs(ref).max()) + 1e-4)
    assert np.all(np.abs(got - ref) <= tol), what


def check_rows(p, kv, oc, gpu_row0, oracle_row0, n, what):
    for L in range(p.dims.num_layers):
        for got, ref, name in zip(p.read_kv(kv, L, gpu_row0, n), oc.read(L, oracle_row0, n), "kv"):
            assert_rows(got, ref, L, f"{what} layer {L} {name}")


def read_rows(p, kv, row0, n):
    """The rows of every layer, as bits."""
    return [x.view(np.uint32) for L in range(p.dims.num_layers if n else 0) for x in p.read_kv(kv, L, row0, n)]


def same(a, b):
    return len(a) == len(b) and all(np.array_equal(x, y) for x, y in zip(a, b))


def packed(p, kvs, seqs, logits=True, s=None):
    out = torch.full((len(kvs), p.dims.vocab_size), float("nan"), device=DEV) if logits else None
    fq.fq_forward_step_packed(p.model, kvs, [t for q in seqs for t in q], [len(q) for q in seqs],
                              out.data_ptr() if logits else 0, stream() if s is None else s)
    torch.cuda.synchronize()
    fq.fq_check_device(p.model, stream())
    return out.cpu().numpy() if logits else None


@pytest.mark.parametrize("dims,wtype,seed,lens,ctx", [
    (SMALL, "q8_0", 37, (77, 1, 40), (0, 0, 0)),          # whole prompts
    (SMALL, "q8_0", 37, (5, 129, 33), (130, 9, 0)),       # chunks behind cached rows
    (SMALL_G4, "q4_k", 37, (40, 1, 2), (0, 63, 127)),
    (SMALL, "q4_k", 37, (1,), (0,)),                      # one token of one sequence
    (SMALL_MOE, "q8_0", 40, (5, 1, 3), (0, 0, 0)),        # router gaps of 0.04, moved by up to 0.007
])
def test_packed_step_matches_oracle(pair_factory, dims, wtype, seed, lens, ctx):
    p = pair_factory(workload(dims, wtype, "bf16", seed=seed), max_positions=512)
    kvs, ocs = zip(*[p.new_seq(capacity=c + n + 3, ctx=c, seq=i) for i, (n, c) in enumerate(zip(lens, ctx))])
    seqs = [tokens_of(dims, seed, i, n) for i, n in enumerate(lens)]
    prior = [read_rows(p, kv, 0, c) for kv, c in zip(kvs, ctx)]
    behind = [read_rows(p, kv, c + n, 3) for kv, n, c in zip(kvs, lens, ctx)]
    got = packed(p, kvs, seqs)
    for i, (kv, oc, n, c) in enumerate(zip(kvs, ocs, lens, ctx)):
        assert fq.fq_kv_len(kv) == c + n
        for j, t in enumerate(seqs[i]):
            z = p.om.decode_step(oc, t, c + j, logits=j == n - 1)
        assert_logits_close(got[i], z, f"sequence {i}")
        check_rows(p, kv, oc, c, c, n, f"sequence {i}")
        # other rows stay as they were
        assert same(prior[i], read_rows(p, kv, 0, c)) and same(behind[i], read_rows(p, kv, c + n, 3))


def test_packed_step_in_passes(pair_factory):
    """2310 rows run in two passes, the second sequence split between them; equal to a forwardStep
    per sequence, and the same bits in a second run and without logits."""
    p = pair_factory(workload(SMALL, "q8_0", "bf16", seed=41), max_positions=2048, with_oracle=False)
    lens = (1500, 800, 10)
    seqs = [tokens_of(SMALL, 41, i, n) for i, n in enumerate(lens)]
    new = lambda: [p.new_seq(capacity=n, ctx=0, seq=i, oracle_cache=False)[0] for i, n in enumerate(lens)]  # noqa: E731
    a, b, c = new(), new(), new()
    got = packed(p, a, seqs)
    again = packed(p, b, seqs)
    packed(p, c, seqs, logits=False)
    assert np.array_equal(got, again)
    ref = torch.empty(SMALL.vocab_size, device=DEV)
    for i, n in enumerate(lens):
        for other in (b, c):
            assert same(read_rows(p, a[i], 0, n), read_rows(p, other[i], 0, n))
        kv, _ = p.new_seq(capacity=n, ctx=0, seq=i, oracle_cache=False)
        fq.fq_forward_step(p.model, kv, seqs[i], 0, ref.data_ptr(), stream())
        torch.cuda.synchronize()
        assert_logits_close(got[i], ref.cpu().numpy(), f"sequence {i}")
        for L in range(SMALL.num_layers):
            for x, y in zip(p.read_kv(a[i], L, 0, n), p.read_kv(kv, L, 0, n)):
                assert_rows(x, y, L, f"sequence {i} layer {L}")


def shared_seqs(p, n, P, own, capacity=8):
    """The prefix cache of P prior rows and n caches with `own` prior rows behind it; the oracle's
    caches hold both, one after the other."""
    prefix, _ = p.new_seq(capacity=max(P, 1), ctx=P, seq=0, oracle_cache=False)
    kvs, ocs = [], []
    for i in range(n):
        kv, _ = p.new_seq(capacity=own + capacity, ctx=own, seq=1 + i, oracle_cache=False)
        oc = p.om.new_cache(P + own + capacity) if p.om else None
        for L in range(p.dims.num_layers if oc else 0):
            for seq, row0, rows in ((0, 0, P), (1 + i, P, own)):
                if rows:
                    oc.write(L, row0, *wl.make_kv_prior(p.w, seq, L, rows))
        if oc:
            oc.set_len(P + own)
        kvs.append(kv)
        ocs.append(oc)
    return prefix, kvs, ocs


def shared_step(p, prefix, kvs, toks, logits=True, s=None):
    out = torch.full((len(kvs), p.dims.vocab_size), float("nan"), device=DEV) if logits else None
    fq.fq_decode_step_shared(p.model, prefix, kvs, toks, out.data_ptr() if logits else 0, stream() if s is None else s)
    torch.cuda.synchronize()
    fq.fq_check_device(p.model, stream())
    return out.cpu().numpy() if logits else None


@pytest.mark.parametrize("dims,wtype,seed,n,P,own", [
    (SMALL, "q8_0", 37, 1, 130, 0), (SMALL, "q8_0", 37, 5, 300, 3), (SMALL_G4, "q4_k", 37, 9, 128, 0),
    (SMALL, "q8_0", 37, 33, 40, 1), (SMALL, "q8_0", 37, 3, 0, 2), (SMALL, "q4_k", 37, 64, 129, 0),
    (SMALL_MOE, "q8_0", 55, 2, 50, 0),                    # router gaps of 0.16
])
def test_shared_step_matches_oracle(pair_factory, dims, wtype, seed, n, P, own):
    p = pair_factory(workload(dims, wtype, "bf16", seed=seed), max_positions=512)
    prefix, kvs, ocs = shared_seqs(p, n, P, own)
    before = read_rows(p, prefix, 0, P)
    checked = range(n) if n < 10 else (0, 1, 31, n - 1)   # of the oracle; their rows and logits
    for step in range(2):
        toks = tokens_of(dims, seed + step, 1, n)
        got = shared_step(p, prefix, kvs, toks)
        assert np.isfinite(got).all()
        for i in checked:
            z = p.om.decode_step(ocs[i], toks[i], P + own + step)
            assert_logits_close(got[i], z, f"step {step} sequence {i}")
            check_rows(p, kvs[i], ocs[i], own + step, P + own + step, 1, f"step {step} sequence {i}")
        assert all(fq.fq_kv_len(kv) == own + step + 1 for kv in kvs)
    assert fq.fq_kv_len(prefix) == P and same(before, read_rows(p, prefix, 0, P))


def test_prompt_then_answers(pair_factory):
    """As they are used together, on a stream of its own: one prompt, then several answers behind it."""
    p = pair_factory(workload(SMALL, "q8_0", "bf16", seed=43), max_positions=512)
    P, n = 150, 3
    prompt = tokens_of(SMALL, 43, 0, P)
    prefix, _ = p.new_seq(capacity=P, ctx=0, seq=0, oracle_cache=False)
    kvs = [p.new_seq(capacity=4, ctx=0, seq=0, oracle_cache=False)[0] for _ in range(n)]
    s = torch.cuda.Stream(DEV)
    first = packed(p, [prefix], [prompt], s=s.cuda_stream)
    answers = [tokens_of(SMALL, 43, 1 + i, 3) for i in range(n)]
    got = [shared_step(p, prefix, kvs, [a[j] for a in answers], s=s.cuda_stream) for j in range(3)]
    for i in range(n):
        oc = p.om.new_cache(P + 4)
        for j, t in enumerate(prompt):
            z = p.om.decode_step(oc, t, j, logits=j == P - 1)
        assert_logits_close(first[0], z, "prompt")
        for j, t in enumerate(answers[i]):
            assert_logits_close(got[j][i], p.om.decode_step(oc, t, P + j), f"answer {i} token {j}")
        check_rows(p, kvs[i], oc, 0, P, 3, f"answer {i}")


def test_steps_without_logits(pair_factory):
    """Logits may be left out: the same rows are appended."""
    p = pair_factory(workload(SMALL, "q8_0", "bf16", seed=44), max_positions=512, with_oracle=False)
    rows = []
    for logits in (True, False):
        prefix, kvs, _ = shared_seqs(p, 4, 60, 0)
        shared_step(p, prefix, kvs, [1, 2, 3, 4], logits)
        rows.append([x for kv in kvs for x in read_rows(p, kv, 0, 1)])
    assert same(*rows)


def refused(call, status):
    with pytest.raises(fq.FqError) as e:
        call()
    assert e.value.status == status


def test_packed_step_contract(pair_factory):
    p = pair_factory(workload(SMALL, "q8_0", "bf16", seed=38), max_positions=512, with_oracle=False)
    other = pair_factory(workload(SMALL, "q8_0", "bf16", seed=39), max_positions=512, with_oracle=False)
    q8 = pair_factory(workload(SMALL, "q8_0", "q8_0", seed=38), max_positions=512, with_oracle=False)
    a, b = [p.new_seq(capacity=40, ctx=10, seq=i, oracle_cache=False)[0] for i in range(2)]
    foreign = other.new_seq(capacity=40, ctx=0, seq=0, oracle_cache=False)[0]
    c8 = q8.new_seq(capacity=40, ctx=0, seq=0, oracle_cache=False)[0]
    call = lambda kvs, toks, lens, m=p.model: fq.fq_forward_step_packed(m, kvs, toks, lens, 0, stream())  # noqa: E731
    for kvs, toks, lens, status in [
            ([], [], [], fq.INVALID_SEQUENCE_LENGTH), ([a, b], [1], [1, 0], fq.INVALID_SEQUENCE_LENGTH),
            ([a, b], [1] * 32, [1, 31], fq.KV_CACHE_OVERFLOW), ([a, a], [1, 2], [1, 1], fq.MISMATCHED_KV_CACHES),
            ([a, foreign], [1, 2], [1, 1], fq.MISMATCHED_KV_CACHES), ([a, b], [1, -1], [1, 1], fq.INVALID_ARGUMENT),
            ([a, b], [1, SMALL.vocab_size], [1, 1], fq.INVALID_ARGUMENT), ([a, b], [1, 2], [2], fq.INVALID_ARGUMENT),
            ([a, b], [1, 2, 3], [1, 1], fq.INVALID_ARGUMENT), ([a] * 65, [1] * 65, [1] * 65, fq.INVALID_ARGUMENT)]:
        refused(lambda: call(kvs, toks, lens), status)
        assert fq.fq_kv_len(a) == fq.fq_kv_len(b) == 10
    refused(lambda: call([c8], [1], [1], q8.model), fq.UNSUPPORTED)
    call([a, b], [1] * 31, [30, 1])   # up to the capacity
    torch.cuda.synchronize()
    assert fq.fq_kv_len(a) == 40 and fq.fq_kv_len(b) == 11
    refused(lambda: call([b, a], [1, 1], [1, 1]), fq.KV_CACHE_OVERFLOW)


def test_shared_step_contract(pair_factory):
    p = pair_factory(workload(SMALL, "q8_0", "bf16", seed=38), max_positions=64, with_oracle=False)
    other = pair_factory(workload(SMALL, "q8_0", "bf16", seed=39), max_positions=64, with_oracle=False)
    q8 = pair_factory(workload(SMALL, "q8_0", "q8_0", seed=38), max_positions=64, with_oracle=False)
    prefix = p.new_seq(capacity=60, ctx=60, seq=9, oracle_cache=False)[0]
    a, b = [p.new_seq(capacity=10, ctx=i, seq=i, oracle_cache=False)[0] for i in range(2)]
    full = p.new_seq(capacity=2, ctx=2, seq=3, oracle_cache=False)[0]
    late = p.new_seq(capacity=10, ctx=4, seq=4, oracle_cache=False)[0]   # its next position is max_positions
    foreign = other.new_seq(capacity=40, ctx=0, seq=0, oracle_cache=False)[0]
    c8, d8 = [q8.new_seq(capacity=40, ctx=0, seq=0, oracle_cache=False)[0] for _ in range(2)]
    call = lambda pre, kvs, toks, m=p.model: fq.fq_decode_step_shared(m, pre, kvs, toks, 0, stream())  # noqa: E731
    for pre, kvs, toks, status in [
            (prefix, [], [], fq.INVALID_SEQUENCE_LENGTH), (0, [a], [1], fq.INVALID_ARGUMENT),
            (prefix, [a, a], [1, 2], fq.MISMATCHED_KV_CACHES), (prefix, [a, prefix], [1, 2], fq.KV_CACHE_OVERFLOW),
            (b, [a, b], [1, 2], fq.MISMATCHED_KV_CACHES), (foreign, [a], [1], fq.MISMATCHED_KV_CACHES),
            (prefix, [a, foreign], [1, 2], fq.MISMATCHED_KV_CACHES), (prefix, [a, full], [1, 2], fq.KV_CACHE_OVERFLOW),
            (prefix, [a, late], [1, 2], fq.INVALID_SEQUENCE_LENGTH), (prefix, [a, b], [1, -1], fq.INVALID_ARGUMENT),
            (prefix, [a, b], [1, SMALL.vocab_size], fq.INVALID_ARGUMENT), (prefix, [a, b], [1], fq.INVALID_ARGUMENT)]:
        refused(lambda: call(pre, kvs, toks), status)
        assert fq.fq_kv_len(a) == 0 and fq.fq_kv_len(b) == 1 and fq.fq_kv_len(prefix) == 60
    refused(lambda: call(c8, [d8], [1], q8.model), fq.UNSUPPORTED)
    call(prefix, [a, b], [1, 2])
    torch.cuda.synchronize()
    assert fq.fq_kv_len(a) == 1 and fq.fq_kv_len(b) == 2


def test_one_token_each_equals_the_batch_step(pair_factory):
    """64 sequences with one token each: what fq_decode_step_batch computes, up to rounding."""
    p = pair_factory(workload(SMALL_G4, "q8_0", "bf16", seed=45), max_positions=512, with_oracle=False)
    ctx = [(7 * i * i) % 200 for i in range(64)]
    a, b = [[p.new_seq(capacity=c + 1, ctx=c, seq=i, oracle_cache=False)[0] for i, c in enumerate(ctx)] for _ in range(2)]
    toks = tokens_of(SMALL_G4, 45, 0, 64)
    got = packed(p, a, [[t] for t in toks])
    ref = torch.empty(64, SMALL_G4.vocab_size, device=DEV)
    fq.fq_decode_step_batch(p.model, b, toks, ref.data_ptr(), stream())
    torch.cuda.synchronize()
    assert_logits_close(got, ref.cpu().numpy(), "logits")
    for i, (x, y, c) in enumerate(zip(a, b, ctx)):
        for L in range(SMALL_G4.num_layers):
            for u, v in zip(p.read_kv(x, L, c, 1), p.read_kv(y, L, c, 1)):
                assert_rows(u, v, L, f"sequence {i} layer {L}")


def test_steps_at_once_on_two_streams(pair_factory):
    """A workspace belongs to a stream: two threads with a stream each, the prefix shared, get what
    one after the other gets."""
    import threading
    p = pair_factory(workload(SMALL, "q8_0", "bf16", seed=46), max_positions=512, with_oracle=False)
    prompts = [tokens_of(SMALL, 46, i, 90 + 31 * i) for i in range(2)]
    prefix, alone, _ = shared_seqs(p, 6, 100, 0)
    kvs = [shared_seqs(p, 6, 100, 0)[1] for _ in range(2)]
    ref_p = []
    for q in prompts:
        kv, _ = p.new_seq(capacity=200, ctx=0, seq=0, oracle_cache=False)
        ref_p.append(packed(p, [kv], [q]))
    toks = tokens_of(SMALL, 46, 9, 6)
    ref_s = shared_step(p, prefix, alone, toks)
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    outs = [[] for _ in range(2)]
    caches = [[p.new_seq(capacity=200, ctx=0, seq=0, oracle_cache=False)[0] for _ in range(3)] for _ in range(2)]
    torch.cuda.synchronize()

    def work(i):
        s = streams[i].cuda_stream
        with torch.cuda.stream(streams[i]):
            for kv in caches[i]:
                o = torch.empty(1, SMALL.vocab_size, device=DEV)
                fq.fq_forward_step_packed(p.model, [kv], prompts[i], [len(prompts[i])], o.data_ptr(), s)
                outs[i].append(o)
            o = torch.empty(6, SMALL.vocab_size, device=DEV)
            fq.fq_decode_step_shared(p.model, prefix, kvs[i], toks, o.data_ptr(), s)
            outs[i].append(o)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    fq.fq_check_device(p.model, stream())
    for i in range(2):
        for o in outs[i][:3]:
            assert np.array_equal(o.cpu().numpy(), ref_p[i])
        assert np.array_equal(outs[i][3].cpu().numpy(), ref_s)
