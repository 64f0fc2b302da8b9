"""The failure path of the attention operators' bounded waits, made to run out on purpose without any
fault: a tile kernel whose loader leaves out one tile of K or V and whose waits may take half a
millisecond.  Every role has to give up and leave, the failure is reported once, and the calls behind it
are right."""
import math
import threading

import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.gpu_util import assert_logits_close
from tests.test_gpu_parity import SMALL, pair_factory, workload  # noqa: F401
from tests.prompt_ops_util import D, DEV, assert_within, attend, causal, gen, normal

pytestmark = pytest.mark.gpu

HALF_MS = 1 << 20   # cycles


def stream():
    return torch.cuda.current_stream(DEV).cuda_stream


class Case:
    """Prompt attention of one sequence, its reference, and the call with and without a tile left out."""

    def __init__(self, hq, hkv, L, K, seed=3):
        g = gen(seed)
        self.hq, self.hkv, self.L, self.K = hq, hkv, L, K
        self.q, self.k, self.v = normal(g, L, hq, D), normal(g, hkv, K, D), normal(g, hkv, K, D)
        self.view = fq.fq_kv_view(self.k.data_ptr(), self.v.data_ptr(), K, D, K * D)
        self.out = torch.empty_like(self.q)

    def starved(self, starve, cycles=HALF_MS, model=0):
        fq.fq_debug_attn_wait_timeout(self.q.data_ptr(), self.view, self.L, self.K, self.hq, self.hkv, self.out.data_ptr(),
                                      starve, cycles, stream(), model)

    def run(self):
        need = fq.fq_attn_prompt_workspace([self.L], [self.K], self.hq, self.hkv)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
        self.out.fill_(float("nan"))
        fq.fq_attn_prompt(self.q.data_ptr(), self.view, [self.L], [self.K], self.hq, self.hkv, 1 / math.sqrt(D),
                          self.out.data_ptr(), ws.data_ptr(), ws.numel(), stream())

    def check(self):
        for h in range(self.hq):
            k, v = self.k[h // (self.hq // self.hkv)], self.v[h // (self.hq // self.hkv)]
            ref, bound = attend(self.q[:, h], k, v, causal(self.L, self.K), 1 / math.sqrt(D))
            assert_within(self.out[:, h], ref, bound, True, f"head {h}")


def reported(call):
    with pytest.raises(fq.FqError) as e:
        call()
    assert e.value.status == fq.DEVICE_TIMEOUT


# pairs of query tiles, single tiles; tiles that every row sees and tiles that some rows see in part; one
# unit per CTA and several
@pytest.mark.parametrize("starve", [1, 2])
@pytest.mark.parametrize("hq,hkv,L,K", [(4, 2, 100, 600), (4, 4, 50, 300), (8, 1, 16, 1500), (4, 2, 700, 700), (32, 8, 1500, 2000)])
def test_left_out_tile_is_reported_and_later_calls_are_right(starve, hq, hkv, L, K):
    c = Case(hq, hkv, L, K)
    c.starved(0)
    fq.fq_attn_check(stream())
    c.check()
    c.starved(starve)
    reported(lambda: fq.fq_attn_check(stream()))
    fq.fq_attn_check(stream())   # once
    c.run()
    fq.fq_attn_check(stream())
    c.check()
    c.starved(starve)            # the call right behind it on the stream is right too
    c.run()
    reported(lambda: fq.fq_attn_check(stream()))
    c.check()


def test_a_model_answers_for_its_own_waits(pair_factory):  # noqa: F811
    """fq_check_device of one model and fq_attn_check take no failure away from another model or from calls
    outside the steps, and report none of theirs."""
    a, b = (pair_factory(workload(SMALL, "q8_0", "bf16", seed=s), max_positions=256) for s in (71, 72))
    c = Case(4, 2, 100, 600)
    c.starved(1)
    fq.fq_check_device(a.model, stream())
    reported(lambda: fq.fq_attn_check(stream()))
    c.starved(1, model=a.model)
    fq.fq_attn_check(stream())
    fq.fq_check_device(b.model, stream())
    reported(lambda: fq.fq_check_device(a.model, stream()))
    fq.fq_check_device(a.model, stream())
    kv, oc = a.new_seq(capacity=64, ctx=10, seq=0)   # the model's steps run as before
    out = torch.empty(1, SMALL.vocab_size, device=DEV)
    fq.fq_forward_step_packed(a.model, [kv], [3, 5], [2], out.data_ptr(), stream())
    fq.fq_check_device(a.model, stream())
    a.om.decode_step(oc, 3, 10, logits=False)
    assert_logits_close(out.cpu().numpy()[0], a.om.decode_step(oc, 5, 11), "step after the failure")


def test_every_thread_is_told_of_a_failure():
    """A check on one thread hides nothing from another that has launched or checked before."""
    c = Case(4, 2, 100, 600)
    torch.cuda.synchronize()
    fq.fq_attn_check(stream())
    ready, failed, told = threading.Event(), threading.Event(), []

    def other():
        torch.cuda.set_device(DEV)
        fq.fq_attn_check(stream())
        ready.set()
        assert failed.wait(60)
        for _ in range(2):
            try:
                fq.fq_attn_check(stream())
                told.append(fq.OK)
            except fq.FqError as e:
                told.append(e.status)

    t = threading.Thread(target=other)
    t.start()
    assert ready.wait(60)
    c.starved(2)
    reported(lambda: fq.fq_attn_check(stream()))
    failed.set()
    t.join()
    assert told == [fq.DEVICE_TIMEOUT, fq.OK]
    fq.fq_attn_check(stream())
    late = []   # a thread that comes later is not told again
    t = threading.Thread(target=lambda: (torch.cuda.set_device(DEV), fq.fq_attn_check(stream()), late.append(fq.OK)))
    t.start()
    t.join()
    assert late == [fq.OK]


@pytest.mark.parametrize("hq,hkv,L,K", [(4, 2, 60, 1 << 16), (4, 4, 200, 50000)])
def test_units_longer_than_the_limit_of_a_wait(hq, hkv, L, K):
    """What a wait's limit bounds is the time without progress, not the length of a unit: units of 300 us and
    more whose outputs wait for their end under a limit of 65 us."""
    c = Case(hq, hkv, L, K)
    c.starved(0, 1 << 17)
    fq.fq_attn_check(stream())
    c.check()
