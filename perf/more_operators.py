"""The bounded-cache and paged-cache operators as measurable cases.

Five operators that keep the cache of a long sequence small or in pages, over bf16 K/V rows of
head_dim 128:

  window   ``fq_attn_window``: grouped-query attention of packed sequences in which a row sees the
           last ``window`` keys up to its own and the first ``sinks`` keys of its sequence;
  paged    ``fq_attn_paged``: the same over K/V rows that lie in pages, found through a page table;
  append   ``fq_qk_norm_rope_paged``: raw q | k | v projections -> RMSNorm and rotary embedding per
           head, q rounded to bf16, k and v rounded into the rows' pages;
  weights  ``fq_attn_key_weights``: the attention weight that each key receives, summed over query
           rows and the heads of its group, added to what the key has gathered before;
  evict    ``fq_kv_evict``: per kv head the keys with the largest gathered weight stay, with the
           first and the most recent ones, and move to a smaller cache in their order.

``run`` computes them in their plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where ``own`` is true, through the framework's entry points.
"""
import math

import torch

own = False

D = 128
EPS = 1e-6
THETA = 1e6
SCALE = 1.0 / math.sqrt(D)


def _ints(text):
    return [int(t) for t in text.split(",")]


def _text(values):
    return ",".join(str(int(v)) for v in values)


def listed():
    return [
        # a chat turn behind a short conversation: latency of one small call
        {"name": "window-turn", "op": "window", "hq": 16, "hkv": 8, "q": "17", "k": "1017", "window": 256, "sinks": 4},
        # one prompt of the 8B workload's context, a window of half of it
        {"name": "window-8192", "op": "window", "hq": 32, "hkv": 8, "q": "8192", "k": "8192", "window": 4096, "sinks": 4},
        # one token per sequence, long caches of which only the window and the sinks are read
        {"name": "window-tokens", "op": "window", "hq": 32, "hkv": 8, "q": _text([1] * 16),
         "k": _text([512 + 479 * i for i in range(16)]), "window": 2048, "sinks": 4},
        # one token per sequence against ragged caches in small pages
        {"name": "paged-tokens", "op": "paged", "hq": 32, "hkv": 8, "q": _text([1] * 32),
         "k": _text([301 + 119 * i for i in range(32)]), "page": 16, "window": 0, "sinks": 0},
        # decode tokens of seven sequences in one pass with a part of an eighth's prompt
        {"name": "paged-mixed", "op": "paged", "hq": 16, "hkv": 8, "q": "1,1,1,1,1,1,1,333",
         "k": "2048,17,901,1500,333,4096,129,1333", "page": 32, "window": 0, "sinks": 0},
        # the next chunk of a long prompt behind its cached beginning
        {"name": "paged-chunk", "op": "paged", "hq": 32, "hkv": 8, "q": "2048", "k": "8192", "page": 64, "window": 0, "sinks": 0},
        # the rows of one decode step of 16 sequences
        {"name": "append-16", "op": "append", "hq": 32, "hkv": 4, "n": _text([1] * 16),
         "at": _text([4090 + i for i in range(16)]), "page": 16},
        # the rows of three prompts' parts at the 8B shape
        {"name": "append-4097", "op": "append", "hq": 32, "hkv": 8, "n": "2001,1023,1073", "at": "0,517,3001", "page": 64},
        # one token per sequence: a decode step's weights
        {"name": "weights-tokens", "op": "weights", "hq": 32, "hkv": 8, "q": _text([1] * 16),
         "k": _text([512 + 239 * i for i in range(16)]), "window": 0, "sinks": 0},
        # all rows of a prompt of the 8B workload's context
        {"name": "weights-8192", "op": "weights", "hq": 32, "hkv": 8, "q": "8192", "k": "8192", "window": 0, "sinks": 0},
        # one prompt of the 8B workload's context down to a quarter
        {"name": "evict-8192", "op": "evict", "hkv": 8, "k": "8192", "keep": "2048", "sinks": 4, "recent": 32},
        # sixteen ragged caches down to 1024 rows each; some are shorter and stay whole
        {"name": "evict-16", "op": "evict", "hkv": 8, "k": _text([701 + 359 * i for i in range(16)]),
         "keep": _text([1024] * 16), "sinks": 4, "recent": 128},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def _split(rng, total, n):
    """total as n ragged positive parts."""
    cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _draw_lengths(rng, most):
    """Query and key lengths: whole prompts, chunks behind cached rows, single tokens."""
    kind = rng.choice(("whole", "chunk", "tokens"))
    if kind == "whole":
        total = _log_int(rng, 2, most)
        q = _split(rng, total, min(total, _log_int(rng, 1, 24)))
        return q, q
    if kind == "chunk":
        total = _log_int(rng, 2, 1500)
        q = _split(rng, total, min(total, rng.randint(1, 3)))
        return q, [n + rng.randint(0, 6000) for n in q]
    q = [rng.choice((1, 1, 1, 2, 4)) for _ in range(_log_int(rng, 1, 48))]
    return q, [m + _log_int(rng, 1, 6000) for m in q]


def draw(rng):
    op = rng.choice(("window", "window", "paged", "paged", "append", "weights", "weights", "evict"))
    hq, hkv = rng.choice(((16, 8), (32, 8), (32, 4), (8, 8)))
    page = rng.choice((16, 32, 64, 128, 256))
    if op in ("window", "paged", "weights"):
        q, k = _draw_lengths(rng, 8000)
        case = {"op": op, "hq": hq, "hkv": hkv, "q": _text(q), "k": _text(k), "window": 0, "sinks": 0}
        if op == "window" or rng.random() < 0.3:
            case["window"], case["sinks"] = _log_int(rng, 1, 4096), rng.choice((0, 1, 4, rng.randint(1, 300)))
        if op == "paged":
            case["page"] = page
        return case
    if op == "append":
        total = _log_int(rng, 2, 8000)
        n = _split(rng, total, min(total, _log_int(rng, 1, 32)))
        return {"op": op, "hq": hq, "hkv": hkv, "n": _text(n), "at": _text([rng.choice((0, rng.randint(0, 6000))) for _ in n]),
                "page": page}
    k = [_log_int(rng, 1, 16384) for _ in range(rng.randint(1, 16))]
    sinks, recent = rng.choice((0, 4, rng.randint(0, 100))), rng.choice((0, 32, rng.randint(0, 300)))
    return {"op": op, "hkv": hkv, "k": _text(k), "sinks": sinks, "recent": recent,
            "keep": _text([sinks + recent + _log_int(rng, 1, n) for n in k])}


def _rope_table(rows, dev):
    """cos and sin of position * theta^(-2 i / 128), made in 64 bits."""
    angle = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * \
        THETA ** (-torch.arange(0, D, 2, device=dev, dtype=torch.float64) / D)[None, :]
    return torch.stack((angle.cos(), angle.sin()), dim=-1).float().contiguous()


def _visible(first, last, K, window, sinks, past, dev):
    """Which of the first K keys the query rows first .. last - 1 see; row i has the position i + past."""
    at = torch.arange(first, last, device=dev)[:, None] + past
    key = torch.arange(K, device=dev)[None, :]
    seen = key <= at
    if window:
        seen &= (key > at - window) | (key < sinks)
    return seen


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    def pages_for(lengths):
        """A pool with a few pages more than the sequences need, and a table of scattered pages."""
        need = [-(-n // case["page"]) for n in lengths]
        n_pages = sum(need) + 5
        ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32, device=dev)   # (entries that nothing reads)
        for s, n in enumerate(need):
            table[s, :n] = ids[sum(need[:s]):sum(need[:s]) + n]
        return n_pages, table

    hkv = case["hkv"]
    s = {"op": case["op"], "hkv": hkv}
    if case["op"] == "evict":
        s["k_len"], s["keep"] = _ints(case["k"]), _ints(case["keep"])
        s["sinks"], s["recent"] = case["sinks"], case["recent"]
        s["n"] = [min(a, b) for a, b in zip(s["k_len"], s["keep"])]
        rows, kept = sum(s["k_len"]), sum(s["n"])
        # one layer of a cache, [kv head][row][128], and the gathered weights of its keys: a few large
        # ones, many small ones, some that no query has looked at
        s["k"], s["v"] = normal(hkv, rows, D), normal(hkv, rows, D)
        w = torch.rand(hkv, rows, generator=g, device=dev)
        s["w"] = torch.where(w < 0.1, 0.0, w ** 8 * 20)
        s["dk"], s["dv"] = torch.empty_like(s["k"][:, :kept]).contiguous(), torch.empty_like(s["v"][:, :kept]).contiguous()
        s["dw"] = torch.empty(hkv, kept, device=dev)
        s["kept"] = torch.empty(hkv * kept, dtype=torch.int32, device=dev)
        return s
    hq = s["hq"] = case["hq"]
    if case["op"] == "append":
        s["n"], s["pos"], s["page"] = _ints(case["n"]), _ints(case["at"]), case["page"]
        rows = sum(s["n"])
        s["qkv"] = normal(rows, (hq + 2 * hkv) * D, dtype=torch.float32)
        s["q_norm"] = 1.0 + 0.1 * normal(D, dtype=torch.float32)
        s["k_norm"] = 1.0 + 0.1 * normal(D, dtype=torch.float32)
        ends = [p + n for p, n in zip(s["pos"], s["n"])]
        s["rope"] = _rope_table(max(ends), dev)
        s["at"] = torch.cat([torch.arange(p, e, device=dev) for p, e in zip(s["pos"], ends)])
        s["seq"] = torch.cat([torch.full((n,), i, device=dev) for i, n in enumerate(s["n"])])
        # one layer of a pool of pages, [page][kv head][row][128]
        s["n_pages"], s["table"] = pages_for(ends)
        s["k"], s["v"] = (torch.zeros(s["n_pages"], hkv, s["page"], D, device=dev, dtype=torch.bfloat16) for _ in range(2))
        return s
    s["q_len"], s["k_len"] = _ints(case["q"]), _ints(case["k"])
    s["window"], s["sinks"] = case["window"], case["sinks"]
    s["q"] = normal(sum(s["q_len"]), hq, D)
    if case["op"] == "paged":
        s["page"] = case["page"]
        s["n_pages"], s["table"] = pages_for(s["k_len"])
        s["k"], s["v"] = normal(s["n_pages"], hkv, s["page"], D), normal(s["n_pages"], hkv, s["page"], D)
        return s
    rows = sum(s["k_len"])
    # one layer of a cache, [kv head][row][128]; the sequences' rows follow one another
    s["k"] = normal(hkv, rows, D)
    if case["op"] == "window":
        s["v"] = normal(hkv, rows, D)
        return s
    # the logarithm of every row's sum of exponentials, as the attention of the same rows leaves it,
    # and what the keys have gathered so far
    s["lse"] = torch.empty(s["q"].shape[:2], device=dev)
    q0 = k0 = 0
    for L, K in zip(s["q_len"], s["k_len"]):
        seen = _visible(0, L, K, s["window"], s["sinks"], K - L, dev)
        for h in range(hq):
            scores = s["q"][q0:q0 + L, h].float() @ s["k"][h * hkv // hq, k0:k0 + K].float().T * SCALE
            s["lse"][q0:q0 + L, h] = torch.logsumexp(scores.masked_fill_(~seen, float("-inf")), dim=1)
        q0, k0 = q0 + L, k0 + K
    s["w"] = torch.rand(hkv, rows, generator=g, device=dev) * 0.01
    return s


# ---------------------------------------------------------------- plain forms

def _plain_sequence(q, k, v, window, sinks):
    """q [L, hkv, G, D], k and v [hkv, K, D], all f32; the last query row sees the last key."""
    L, K = q.shape[0], k.shape[1]
    scores = torch.einsum("lhgd,hkd->hglk", q, k) * SCALE
    seen = _visible(0, L, K, window, sinks, K - L, q.device)
    scores = scores.masked_fill(~seen, float("-inf"))
    e = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    e = e.masked_fill(~seen, 0.0)
    return torch.einsum("hglk,hkd->lhgd", e / e.sum(dim=-1, keepdim=True), v)


def _plain_window(s):
    hq, hkv = s["hq"], s["hkv"]
    q = s["q"].float().reshape(-1, hkv, hq // hkv, D).split(s["q_len"])
    k, v = s["k"].float().split(s["k_len"], dim=1), s["v"].float().split(s["k_len"], dim=1)
    out = torch.cat([_plain_sequence(a, b, c, s["window"], s["sinks"]) for a, b, c in zip(q, k, v)])
    return out.reshape(-1, hq, D).to(torch.bfloat16)


def _plain_paged(s):
    hq, hkv = s["hq"], s["hkv"]
    q = s["q"].float().reshape(-1, hkv, hq // hkv, D).split(s["q_len"])
    out = []
    for i, (a, n) in enumerate(zip(q, s["k_len"])):
        ids = s["table"][i, :-(-n // s["page"])].long()
        k, v = (t[ids].transpose(0, 1).reshape(hkv, -1, D)[:, :n].float() for t in (s["k"], s["v"]))
        out.append(_plain_sequence(a, k, v, s["window"], s["sinks"]))
    return torch.cat(out).reshape(-1, hq, D).to(torch.bfloat16)


def _plain_append(s):
    hq, hkv = s["hq"], s["hkv"]
    q, k, v = s["qkv"].reshape(-1, hq + 2 * hkv, D).split((hq, hkv, hkv), dim=1)
    cos, sin = s["rope"][s["at"]][:, None, :, 0], s["rope"][s["at"]][:, None, :, 1]

    def turned(x, gain):
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * gain
        a, b = x[..., : D // 2], x[..., D // 2:]
        return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1).to(torch.bfloat16)

    page, row = s["table"][s["seq"], s["at"] // s["page"]].long(), s["at"] % s["page"]
    s["k"][page, :, row] = turned(k, s["k_norm"])
    s["v"][page, :, row] = v.to(torch.bfloat16)
    return {"q": turned(q, s["q_norm"]), "k": s["k"], "v": s["v"]}


def _plain_weights(s):
    hq, hkv = s["hq"], s["hkv"]
    q = s["q"].float().reshape(-1, hkv, hq // hkv, D).split(s["q_len"])
    lse = s["lse"].reshape(-1, hkv, hq // hkv).split(s["q_len"])
    out = []
    for a, b, k in zip(q, lse, s["k"].float().split(s["k_len"], dim=1)):
        L, K = a.shape[0], k.shape[1]
        scores = torch.einsum("lhgd,hkd->hglk", a, k) * SCALE
        seen = _visible(0, L, K, s["window"], s["sinks"], K - L, a.device)
        p = torch.exp(scores - b.permute(1, 2, 0)[..., None]).masked_fill(~seen, 0.0)
        out.append(p.sum(dim=(1, 2)))
    return s["w"] + torch.cat(out, dim=1)


def _plain_evict(s):
    hkv, dev = s["hkv"], s["k"].device
    kept = []
    k0 = d0 = 0
    for K, n in zip(s["k_len"], s["n"]):
        w = s["w"][:, k0:k0 + K].clone()
        at = torch.arange(K, device=dev)
        w[:, (at < s["sinks"]) | (at >= K - s["recent"])] = float("inf")
        best = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :n]   # equal ones: the lower index first
        idx = torch.sort(best, dim=1).values
        take = (idx + k0)[..., None].expand(hkv, n, D)
        s["dk"][:, d0:d0 + n] = s["k"].gather(1, take)
        s["dv"][:, d0:d0 + n] = s["v"].gather(1, take)
        s["dw"][:, d0:d0 + n] = s["w"].gather(1, idx + k0)
        kept.append(idx.to(torch.int32).reshape(-1))
        k0, d0 = k0 + K, d0 + n
    return {"kept": torch.cat(kept), "k": s["dk"], "v": s["dv"], "w": s["dw"]}


# ---------------------------------------------------------------- the framework's calls

def _stream():
    return torch.cuda.current_stream().cuda_stream


def _own_window(s):
    from quantized_decoder_decode_gb300 import fq
    hq, hkv, q = s["hq"], s["hkv"], s["q"]
    if "view" not in s:   # what a program keeps with its cache: the view of the layer, the lengths, a workspace
        rows = s["k"].shape[1]
        s["view"] = fq.fq_kv_view(s["k"].data_ptr(), s["v"].data_ptr(), rows, D, rows * D)
        s["lens"] = fq.u32_array(s["q_len"]), fq.u32_array(s["k_len"])
        need = fq.fq_attn_window_workspace(*s["lens"], hq, hkv, s["window"], s["sinks"])
        s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q)
    fq.fq_attn_window(q.data_ptr(), s["view"], *s["lens"], hq, hkv, s["window"], s["sinks"], SCALE, out.data_ptr(),
                      s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return out


def _pages(fq, s):
    p, hkv = s["page"], s["hkv"]
    return fq.fq_kv_pages(s["k"].data_ptr(), s["v"].data_ptr(), s["n_pages"], p, hkv * p * D, D, p * D)


def _own_paged(s):
    from quantized_decoder_decode_gb300 import fq
    hq, hkv, q = s["hq"], s["hkv"], s["q"]
    if "pages" not in s:
        s["pages"] = _pages(fq, s)
        s["lens"] = fq.u32_array(s["q_len"]), fq.u32_array(s["k_len"])
        need = fq.fq_attn_window_workspace(*s["lens"], hq, hkv, s["window"], s["sinks"])
        s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q)
    fq.fq_attn_paged(q.data_ptr(), s["pages"], s["table"].data_ptr(), s["table"].shape[1], *s["lens"], hq, hkv, s["window"],
                     s["sinks"], SCALE, out.data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return out


def _own_append(s):
    from quantized_decoder_decode_gb300 import fq
    hq, hkv, qkv = s["hq"], s["hkv"], s["qkv"]
    if "pages" not in s:
        s["pages"] = _pages(fq, s)
        s["lens"] = fq.u32_array(s["n"]), fq.u32_array(s["pos"])
    q = torch.empty(qkv.shape[0], hq, D, dtype=torch.bfloat16, device=qkv.device)
    fq.fq_qk_norm_rope_paged(qkv.data_ptr(), *s["lens"], s["pages"], s["table"].data_ptr(), s["table"].shape[1], s["lens"][1],
                             hq, hkv, s["q_norm"].data_ptr(), s["k_norm"].data_ptr(), EPS, s["rope"].data_ptr(),
                             s["rope"].shape[0], q.data_ptr(), _stream())
    return {"q": q, "k": s["k"], "v": s["v"]}


def _own_weights(s):
    from quantized_decoder_decode_gb300 import fq
    hq, hkv, q = s["hq"], s["hkv"], s["q"]
    rows = s["k"].shape[1]
    if "view" not in s:
        s["view"] = fq.fq_kv_view(s["k"].data_ptr(), s["k"].data_ptr(), rows, D, rows * D)   # (V is not looked at)
        s["lens"] = fq.u32_array(s["q_len"]), fq.u32_array(s["k_len"])
        need = fq.fq_attn_key_weights_workspace(*s["lens"], hq, hkv, s["window"], s["sinks"])
        s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        s["before"] = fq.fq_key_weights(s["w"].data_ptr(), rows)
    w = torch.empty_like(s["w"])
    fq.fq_attn_key_weights(q.data_ptr(), s["lse"].data_ptr(), s["view"], *s["lens"], hq, hkv, s["window"], s["sinks"], SCALE,
                           s["before"], fq.fq_key_weights(w.data_ptr(), rows), s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return w


def _own_evict(s):
    from quantized_decoder_decode_gb300 import fq
    hkv = s["hkv"]
    if "view" not in s:
        rows, kept = s["k"].shape[1], s["dk"].shape[1]
        s["view"] = fq.fq_kv_view(s["k"].data_ptr(), s["v"].data_ptr(), rows, D, rows * D)
        s["to"] = fq.fq_kv_view(s["dk"].data_ptr(), s["dv"].data_ptr(), kept, D, kept * D)
        s["of"], s["ow"] = fq.fq_key_weights(s["w"].data_ptr(), rows), fq.fq_key_weights(s["dw"].data_ptr(), kept)
        s["lens"] = fq.u32_array(s["k_len"]), fq.u32_array(s["keep"])
        s["at"] = fq.u32_array([sum(s["k_len"][:i]) for i in range(len(s["k_len"]))])
        s["to_at"] = fq.u32_array([sum(s["n"][:i]) for i in range(len(s["n"]))])
    fq.fq_kv_evict(s["view"], s["of"], s["at"], *s["lens"], s["sinks"], s["recent"], hkv, s["to"], s["ow"], s["to_at"],
                   s["kept"].data_ptr(), _stream())
    return {"kept": s["kept"], "k": s["dk"], "v": s["dv"], "w": s["dw"]}


def run(state):
    if own:
        return {"window": _own_window, "paged": _own_paged, "append": _own_append, "weights": _own_weights,
                "evict": _own_evict}[state["op"]](state)
    return {"window": _plain_window, "paged": _plain_paged, "append": _plain_append, "weights": _plain_weights,
            "evict": _plain_evict}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _seen_counts(L, K, window, sinks):
    """(query, key) pairs that the mask keeps, and keys that any row sees."""
    W = window or K + 1
    pairs, past = 0, K - L
    # rows whose whole past is in the window, and the others (the window and the sinks before it)
    whole = max(0, min(L, W - past))
    pairs += whole * past + whole * (whole + 1) // 2
    for i in range(whole, L):
        pairs += W + min(sinks, i + past + 1 - W)
    first = max(0, past + 1 - W)   # the first row's window begins here
    return pairs, K - first + min(sinks, first)


def work(case):
    hkv = case["hkv"]
    if case["op"] == "evict":
        k, n = _ints(case["k"]), [min(a, b) for a, b in zip(_ints(case["k"]), _ints(case["keep"]))]
        # the weights; per kept row its number, its weight, and K and V read and written
        return {"bytes": hkv * (4 * sum(k) + sum(n) * (4 + 4 + 2 * 2 * 2 * D)), "flops": 0}
    hq = case["hq"]
    if case["op"] == "append":
        n, at = _ints(case["n"]), _ints(case["at"])
        last = len(set().union(*(range(p, p + m) for p, m in zip(at, n))))   # rows of the rotary table that are read
        pages = sum((p + m - 1) // case["page"] - p // case["page"] + 1 for p, m in zip(at, n))
        return {"bytes": sum(n) * (hq + 2 * hkv) * D * (4 + 2) + last * D * 4 + 2 * D * 4 + 4 * pages,
                "flops": sum(n) * (hq + hkv) * D * 8}
    counts = [_seen_counts(L, K, case["window"], case["sinks"]) for L, K in zip(_ints(case["q"]), _ints(case["k"]))]
    pairs, keys, rows = sum(c[0] for c in counts), sum(c[1] for c in counts), sum(_ints(case["q"]))
    if case["op"] == "weights":
        return {"bytes": rows * hq * (2 * D + 4) + keys * hkv * (2 * D + 8), "flops": 2 * D * hq * pairs}
    table = 4 * sum(-(-n // case["page"]) for n in _ints(case["k"])) if case["op"] == "paged" and not case["window"] else 0
    return {"bytes": 2 * D * (2 * rows * hq + 2 * keys * hkv) + table, "flops": 4 * D * hq * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits

BLOCK = 1024   # query rows at a time


def _key_range(i, n, K, L, window, sinks):
    """The keys that query rows i .. i + n - 1 may see, as indexes, and the rows' own mask over them."""
    own_key = [j + K - L for j in range(i, i + n)]
    first = max(0, own_key[0] - window + 1) if window else 0
    keys = torch.cat((torch.arange(min(sinks, first)), torch.arange(first, own_key[-1] + 1))) if window else \
        torch.arange(own_key[-1] + 1)
    at = torch.tensor(own_key)[:, None]
    hidden = keys[None, :] > at
    if window:
        hidden = hidden | ((at - keys[None, :] >= window) & (keys[None, :] >= sinks))
    return keys.cuda(), hidden.cuda()


def _exact_sequence(q, k, v, window, sinks):
    """q [L, hq, D], k and v [hkv, K, D] -> [L, hq, D] in f64."""
    L, hq, _ = q.shape
    hkv, K, _ = k.shape
    out = torch.empty(L, hq, D, dtype=torch.float64, device=q.device)
    for i in range(0, L, BLOCK):
        n = min(BLOCK, L - i)
        keys, hidden = _key_range(i, n, K, L, window, sinks)
        for h in range(hq):
            kk, vv = k[h // (hq // hkv), keys].double(), v[h // (hq // hkv), keys].double()
            w = torch.where(hidden, -math.inf, q[i:i + n, h].double() @ kk.T / math.sqrt(D))
            out[i:i + n, h] = torch.exp(w - torch.logsumexp(w, dim=1, keepdim=True)) @ vv
    return out


def _exact_weights(q, lse, k, window, sinks):
    """The weights that the K keys receive, [hkv, K] in f64."""
    L, hq, _ = q.shape
    hkv, K, _ = k.shape
    out = torch.zeros(hkv, K, dtype=torch.float64, device=q.device)
    for i in range(0, L, BLOCK):
        n = min(BLOCK, L - i)
        keys, hidden = _key_range(i, n, K, L, window, sinks)
        for h in range(hq):
            w = q[i:i + n, h].double() @ k[h // (hq // hkv), keys].double().T / math.sqrt(D)
            p = torch.where(hidden, 0.0, torch.exp(w - lse[i:i + n, h, None].double()))
            out[h // (hq // hkv), keys] += p.sum(dim=0)
    return out


def _exact_evict(s):
    kept, k, v, w = [], [], [], []
    k0 = 0
    for K, n in zip(s["k_len"], s["n"]):
        for h in range(s["hkv"]):
            weight = s["w"][h, k0:k0 + K].tolist()
            free = range(s["sinks"], max(s["sinks"], K - s["recent"]))
            if n == K:
                rows = list(range(K))
            else:
                best = sorted(free, key=lambda j: (-weight[j], j))[:n - s["sinks"] - s["recent"]]
                rows = sorted(set(best) | set(range(s["sinks"])) | set(range(K - s["recent"], K)))
            kept.append(torch.tensor(rows, dtype=torch.int32, device="cuda"))
        idx = torch.stack(kept[-s["hkv"]:]).long() + k0
        heads = torch.arange(s["hkv"], device="cuda")[:, None]
        k.append(s["k"][heads, idx])
        v.append(s["v"][heads, idx])
        w.append(s["w"][heads, idx])
        k0 += K
    return {"kept": torch.cat(kept), "k": torch.cat(k, dim=1).double(), "v": torch.cat(v, dim=1).double(),
            "w": torch.cat(w, dim=1).double()}


def exact(case, seed):
    s = prepare(case, seed)
    hkv = s["hkv"]
    if case["op"] == "evict":
        return _exact_evict(s)
    hq = s["hq"]
    if case["op"] == "append":
        x = s["qkv"].double().view(-1, hq + 2 * hkv, D)
        angle = torch.view_as_complex(s["rope"].double())[s["at"]].unsqueeze(1)
        x[:, :hq + hkv] /= torch.sqrt(x[:, :hq + hkv].pow(2).sum(dim=-1, keepdim=True) / D + EPS)
        x[:, :hq] *= s["q_norm"].double()
        x[:, hq:hq + hkv] *= s["k_norm"].double()
        z = torch.complex(x[..., : D // 2], x[..., D // 2:])[:, :hq + hkv] * angle
        y = torch.cat((z.real, z.imag), dim=-1)
        k, v = s["k"].double(), s["v"].double()
        row = 0
        for i, (n, p) in enumerate(zip(s["n"], s["pos"])):
            ids = s["table"][i].tolist()
            j = 0
            while j < n:   # to the end of a page
                r, m = (p + j) % s["page"], min(n - j, s["page"] - (p + j) % s["page"])
                page = ids[(p + j) // s["page"]]
                k[page, :, r:r + m] = y[row + j:row + j + m, hq:].transpose(0, 1)
                v[page, :, r:r + m] = x[row + j:row + j + m, hq + hkv:].transpose(0, 1)
                j += m
            row += n
        return {"q": y[:, :hq], "k": k, "v": v}
    out = []
    q0 = k0 = 0
    for i, (L, K) in enumerate(zip(s["q_len"], s["k_len"])):
        q = s["q"][q0:q0 + L]
        if case["op"] == "paged":
            ids = s["table"][i, :-(-K // s["page"])].tolist()
            k, v = (torch.cat([t[p] for p in ids], dim=1)[:, :K] for t in (s["k"], s["v"]))
            out.append(_exact_sequence(q, k, v, s["window"], s["sinks"]))
        elif case["op"] == "window":
            out.append(_exact_sequence(q, s["k"][:, k0:k0 + K], s["v"][:, k0:k0 + K], s["window"], s["sinks"]))
        else:
            w = _exact_weights(q, s["lse"][q0:q0 + L], s["k"][:, k0:k0 + K], s["window"], s["sinks"])
            out.append(s["w"][:, k0:k0 + K].double() + w)
        q0, k0 = q0 + L, k0 + K
    return torch.cat(out, dim=1 if case["op"] == "weights" else 0)
