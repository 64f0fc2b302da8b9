"""The packed and the shared-prefix step on a stream that is being captured: refused, with the caches and the
capture as they were."""
import pytest
import torch

from quantized_decoder_decode_gb300 import fq
from tests.gpu_util import DEV, stream
from tests.test_gpu_packed_steps import packed, read_rows, same, shared_seqs, shared_step
from tests.test_gpu_parity import SMALL, pair_factory, workload  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("warm", [False, True])
def test_captured_steps_are_refused(pair_factory, warm):  # noqa: F811
    p = pair_factory(workload(SMALL, "q8_0", "bf16", seed=81 + warm), max_positions=256, with_oracle=False)
    prefix, kvs, _ = shared_seqs(p, 3, 40, 2)
    side = torch.cuda.Stream(DEV)
    if warm:   # the stream's buffers are there already
        shared_step(p, prefix, kvs, [1, 2, 3], s=side.cuda_stream)
        packed(p, kvs, [[4], [5, 6], [7]], s=side.cuda_stream)
    lens = [fq.fq_kv_len(kv) for kv in kvs]
    before = [read_rows(p, kv, 0, n) for kv, n in zip(kvs, lens)]
    x = torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        x += 1
        for call in (lambda: fq.fq_decode_step_shared(p.model, prefix, kvs, [1, 2, 3], 0, stream()),
                     lambda: fq.fq_forward_step_packed(p.model, kvs, [1, 2, 3], [1, 1, 1], 0, stream())):
            with pytest.raises(fq.FqError) as e:
                call()
            assert e.value.status == fq.UNSUPPORTED
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert bool((x == 2).all())
    assert [fq.fq_kv_len(kv) for kv in kvs] == lens
    assert all(same(b, read_rows(p, kv, 0, n)) for b, kv, n in zip(before, kvs, lens))
    shared_step(p, prefix, kvs, [1, 2, 3], s=side.cuda_stream)   # and uncaptured it runs
    assert [fq.fq_kv_len(kv) for kv in kvs] == [n + 1 for n in lens]
