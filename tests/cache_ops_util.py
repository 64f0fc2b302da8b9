"""Plain 64-bit forms of the operators on windows, pages and caches made shorter, and the bounds that their outputs may
be off by."""
import math

import torch

from quantized_decoder_decode_gb300 import fq
from tests.prompt_ops_util import BF16_HALF_STEP, D, DEV, attend, normal

NAN = float("nan")
SCALE = 1.0 / math.sqrt(D)


def stream():
    return torch.cuda.current_stream(DEV).cuda_stream


def visible(L, K, window, sinks, dev=DEV):
    """[L, K]: which keys a query row sees."""
    own = torch.arange(L, device=dev)[:, None] + (K - L)
    key = torch.arange(K, device=dev)[None, :]
    return (key <= own) & ((key > own - window) | (key < sinks) if window else torch.ones_like(key, dtype=torch.bool))


def log_sum(q, k, seen, scale):
    """One head in 64 bits: log sum exp of the seen scores, and the bound of its error.

    The score of the largest weight carries at most 128 2^-24 sum_d |q_d k_d| scale of the f32 dot product and three
    roundings (as in attend); a weight exp2's error of 2^-21 and the sum of K of them K 2^-24; the logarithm, the
    reference maximum (in base 2) and the offset that the weights are held at are added and multiplied in f32: four
    roundings of at most 1.5 |s| + 60; and the result's own."""
    s = torch.where(seen, q.double() @ torch.where(seen.any(dim=0)[:, None], k.double(), 0.0).T * scale, -math.inf)
    out = torch.logsumexp(s, dim=1) if s.shape[1] else torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    kk = torch.where(seen.any(dim=0)[:, None], k.double(), 0.0).abs()
    ds = torch.where(seen, q.double().abs() @ kk.T * abs(scale), 0.0)
    ds = (ds.amax(dim=1) if s.shape[1] else torch.zeros_like(out)) * (128 + 3) * 2.0 ** -24
    top = torch.where(seen, s.abs(), 0.0).amax(dim=1) if s.shape[1] else torch.zeros_like(out)
    bound = ds + 2.0 ** -21 + (2 * s.shape[1] + 16) * 2.0 ** -24 + 5 * 2.0 ** -24 * (1.5 * top + 60)
    return out, bound


def reference(q, kv, q_len, k_len, hq, hkv, window, sinks, scale=SCALE):
    """kv(s, h) -> (k, v) [k_len, D].  Outputs, their bound, log-sums, their bound."""
    outs, r = [], 0
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        o, b = (torch.zeros(L, hq, D, dtype=torch.float64, device=DEV) for _ in range(2))
        e, eb = (torch.zeros(L, hq, dtype=torch.float64, device=DEV) for _ in range(2))
        seen = visible(L, K, window, sinks)
        for h in range(hq):
            k, v = kv(s, h // (hq // hkv))
            o[:, h], b[:, h] = attend(q[r:r + L, h], k, v, seen, scale)
            e[:, h], eb[:, h] = log_sum(q[r:r + L, h], k, seen, scale)
        outs.append((o, b, e, eb))
        r += L
    return tuple(torch.cat(x) for x in zip(*outs))


def assert_lse(got, ref, bound, what=""):
    none = torch.isinf(ref)
    assert bool((got[none] == -math.inf).all()), f"{what}: a row without keys has a log-sum"
    err = (got.double() - ref).abs()[~none]
    bad = ~(err <= bound[~none])
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} log-sums beyond the bound, worst {float((err / bound[~none]).max()):.3g} of it"


def junk(n):
    """A workspace whose contents are junk."""
    return torch.full((max(1, -(-n // 4)),), NAN, dtype=torch.float32, device=DEV)


class Pool:
    """A pool of pages with rows of given sequences at scattered pages; every row that is nobody's holds `fill`."""

    def __init__(self, g, lengths, hkv, page, layout="head", fill=NAN, extra=3, room=0):
        need = [-(-(n + room) // page) for n in lengths]
        self.page, self.hkv, self.lengths = page, hkv, list(lengths)
        self.n_pages = sum(need) + extra
        ids = torch.randperm(self.n_pages, generator=g, device=DEV)
        self.stride = max(need + [1]) + 2
        self.table = torch.full((len(lengths), self.stride), -7, dtype=torch.int32, device=DEV)   # (nobody's entries name no page)
        for s, n in enumerate(need):
            self.table[s, :n] = ids[sum(need[:s]):sum(need[:s]) + n].int()
        if layout == "head":     # [page][head][row][D]
            self.store = [torch.full((self.n_pages, hkv, page, D), fill, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            self.k, self.v = self.store
            self.strides = (hkv * page * D, D, page * D)
        else:                    # [page][row][head][D + 8], a gap behind every page
            self.store = [torch.full((self.n_pages, page * hkv * (D + 8) + 16), fill, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            self.k, self.v = (t.as_strided((self.n_pages, hkv, page, D), (page * hkv * (D + 8) + 16, D + 8, hkv * (D + 8), 1))
                              for t in self.store)
            self.strides = (page * hkv * (D + 8) + 16, hkv * (D + 8), D + 8)
        for s, n in enumerate(lengths):
            for t in (self.k, self.v):
                self.put(t, s, 0, normal(g, hkv, n, D))

    def where(self, s, first, n):
        at = torch.arange(first, first + n, device=DEV)
        return self.table[s, at // self.page].long(), at % self.page

    def put(self, t, s, first, rows):
        page, row = self.where(s, first, rows.shape[1])
        t[page, :, row] = rows.transpose(0, 1)

    def rows(self, s, h, n=None, first=0):
        page, row = self.where(s, first, self.lengths[s] if n is None else n)
        return self.k[page, h, row], self.v[page, h, row]

    def pages(self):
        return fq.fq_kv_pages(self.store[0].data_ptr(), self.store[1].data_ptr(), self.n_pages, self.page, *self.strides)


def run_window(q, views, q_len, k_len, hq, hkv, window, sinks, out_dtype="bf16", scale=SCALE, lse=True, **kw):
    ws = junk(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, window, sinks))
    out = torch.full((sum(q_len), hq, D), NAN, device=DEV, dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    e = torch.full((sum(q_len), hq), NAN, device=DEV) if lse else None
    fq.fq_attn_window(q.data_ptr(), views, q_len, k_len, hq, hkv, window, sinks, scale, out.data_ptr(), ws.data_ptr(),
                      ws.numel() * 4, stream(), out_dtype=out_dtype, lse_ptr=e.data_ptr() if lse else 0, **kw)
    fq.fq_attn_check(stream())
    return out, e


def run_paged(q, pool, q_len, k_len, hq, hkv, window, sinks, out_dtype="bf16", scale=SCALE, lse=True, check=True, **kw):
    ws = junk(fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, window, sinks))
    out = torch.full((sum(q_len), hq, D), NAN, device=DEV, dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    e = torch.full((sum(q_len), hq), NAN, device=DEV) if lse else None
    fq.fq_attn_paged(q.data_ptr(), pool.pages(), pool.table.data_ptr(), pool.stride, q_len, k_len, hq, hkv, window, sinks, scale,
                     out.data_ptr(), ws.data_ptr(), ws.numel() * 4, stream(), out_dtype=out_dtype,
                     lse_ptr=e.data_ptr() if lse else 0, **kw)
    if check:
        fq.fq_attn_check(stream())
    return out, e


__all__ = ["BF16_HALF_STEP", "D", "DEV", "NAN", "SCALE", "Pool", "assert_lse", "junk", "log_sum", "normal", "reference",
           "run_paged", "run_window", "stream", "visible"]
