"""The prompt and shared-prompt attention operators as measurable cases.

Three operators that serve a prompt and the answers to it, over bf16 K/V rows of head_dim 128:

  rows     ``fq_qk_norm_rope``: raw q | k | v projections -> RMSNorm and rotary embedding per
           head, q rounded to bf16, k and v rounded into the rows of a cache layer;
  prompt   ``fq_attn_prompt``: causal grouped-query attention of packed sequences of different
           lengths, each over its own rows of a cache (the last query row sees every key);
  shared   ``fq_attn_shared``: one query token per sequence over a prefix that all sequences
           share and over each sequence's own tail.

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
        # a short chat turn: latency of one small call
        {"name": "prompt-short", "op": "prompt", "hq": 16, "hkv": 8, "q": "17", "k": "17"},
        # one prompt of the 0.6B workload's context
        {"name": "prompt-2048", "op": "prompt", "hq": 16, "hkv": 8, "q": "2048", "k": "2048"},
        # requests of different lengths packed into one pass, odd lengths and one single token
        {"name": "prompt-packed", "op": "prompt", "hq": 32, "hkv": 8,
         "q": "1,37,129,255,511,640,771,901,1023,1187", "k": "1,37,129,255,511,640,771,901,1023,1187"},
        # one prompt of the 8B workload's context
        {"name": "prompt-8192", "op": "prompt", "hq": 32, "hkv": 8, "q": "8192", "k": "8192"},
        # the next chunk of a long prompt behind its cached beginning
        {"name": "prompt-chunk", "op": "prompt", "hq": 32, "hkv": 4, "q": "333", "k": "7333"},
        # one token per sequence against ragged caches
        {"name": "prompt-tokens", "op": "prompt", "hq": 32, "hkv": 8, "q": _text([1] * 16),
         "k": _text([512 + 239 * i for i in range(16)])},
        # four answers to one medium prompt, just begun
        {"name": "shared-small", "op": "shared", "hq": 16, "hkv": 8, "prefix": 500, "tails": "1,3,9,17"},
        # a batch of 32 behind one system prompt, answers of up to 512 tokens
        {"name": "shared-32", "op": "shared", "hq": 32, "hkv": 8, "prefix": 4096,
         "tails": _text([(37 * i * i + 11 * i) % 513 for i in range(32)])},
        # the largest batch behind one long document, groups of 8 query heads
        {"name": "shared-64", "op": "shared", "hq": 32, "hkv": 4, "prefix": 16384,
         "tails": _text([(61 * i * i + 5 * i) % 1025 for i in range(64)])},
        # the rows of one decode step of 16 sequences
        {"name": "rows-16", "op": "rows", "hq": 32, "hkv": 4, "n": _text([1] * 16), "pos": _text([4096 + i for i in range(16)])},
        # one prompt's rows at the 0.6B shape
        {"name": "rows-2048", "op": "rows", "hq": 16, "hkv": 8, "n": "2048", "pos": "0"},
        # three prompts' rows at the 8B shape, one behind a cached beginning
        {"name": "rows-8191", "op": "rows", "hq": 32, "hkv": 8, "n": "4001,1023,3167", "pos": "0,517,0"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def _split(rng, total, n):
    """total as n ragged positive parts."""
    cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(("prompt", "prompt", "shared", "rows"))
    hq, hkv = rng.choice(((16, 8), (32, 8), (32, 4), (8, 8)))
    if op == "prompt":
        kind = rng.choice(("whole", "chunk", "tokens"))
        if kind == "whole":
            total = _log_int(rng, 2, 8000)
            q = _split(rng, total, min(total, _log_int(rng, 1, 24)))
            k = q
        elif kind == "chunk":
            total = _log_int(rng, 2, 2000)
            q = _split(rng, total, min(total, rng.randint(1, 3)))
            k = [n + rng.randint(0, 6000) for n in q]
        else:
            n = _log_int(rng, 1, 48)
            q = [rng.choice((1, 1, 1, 2, 4)) for _ in range(n)]
            k = [m + _log_int(rng, 1, 6000) for m in q]
        return {"op": op, "hq": hq, "hkv": hkv, "q": _text(q), "k": _text(k)}
    if op == "shared":
        n, most = _log_int(rng, 1, 64), _log_int(rng, 1, 1024)
        return {"op": op, "hq": hq, "hkv": hkv, "prefix": _log_int(rng, 1, 16384),
                "tails": _text([rng.randint(0, most) for _ in range(n)])}
    total = _log_int(rng, 2, 8000)
    n = _split(rng, total, min(total, _log_int(rng, 1, 32)))
    return {"op": op, "hq": hq, "hkv": hkv, "n": _text(n), "pos": _text([rng.choice((0, rng.randint(0, 8000))) for _ in n])}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    hq, hkv = case["hq"], case["hkv"]
    s = {"op": case["op"], "hq": hq, "hkv": hkv}
    if case["op"] == "prompt":
        s["q_len"], s["k_len"] = _ints(case["q"]), _ints(case["k"])
        rows = sum(s["k_len"])
        s["q"] = normal(sum(s["q_len"]), hq, D)
        # one layer of a cache, [kv head][row][128]; the sequences' rows follow one another
        s["k"], s["v"] = normal(hkv, rows, D), normal(hkv, rows, D)
    elif case["op"] == "shared":
        s["prefix"], s["tail_len"] = case["prefix"], _ints(case["tails"])
        n, cap = len(s["tail_len"]), max(1, max(s["tail_len"])) + 16
        s["q"] = normal(n, hq, D)
        s["k"], s["v"] = normal(hkv, case["prefix"], D), normal(hkv, case["prefix"], D)
        # every sequence's own cache layer, [kv head][capacity][128], filled up to its length
        s["tk"], s["tv"] = normal(n, hkv, cap, D), normal(n, hkv, cap, D)
    else:
        s["n"], s["pos"] = _ints(case["n"]), _ints(case["pos"])
        rows = sum(s["n"])
        s["qkv"] = normal(rows, (hq + 2 * hkv) * D, dtype=torch.float32)
        s["q_norm"] = 1.0 + 0.1 * normal(D, dtype=torch.float32)
        s["k_norm"] = 1.0 + 0.1 * normal(D, dtype=torch.float32)
        last = max(p + n for p, n in zip(s["pos"], s["n"]))
        # cos and sin of position * theta^(-2 i / 128), made in 64 bits
        angle = torch.arange(last, device=dev, dtype=torch.float64)[:, None] * \
            THETA ** (-torch.arange(0, D, 2, device=dev, dtype=torch.float64) / D)[None, :]
        s["rope"] = torch.stack((angle.cos(), angle.sin()), dim=-1).float().contiguous()
        # the rows' positions, and a cache layer [kv head][row][128] that takes them one after the other
        s["at"] = torch.cat([torch.arange(p, p + n, device=dev) for p, n in zip(s["pos"], s["n"])])
        s["k"], s["v"] = torch.zeros(hkv, rows, D, device=dev, dtype=torch.bfloat16), \
            torch.zeros(hkv, rows, D, device=dev, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_sequence(q, k, v):
    """q [L, hkv, G, D], k and v [hkv, K, D], all f32: causal, the last query row sees every key."""
    L, K = q.shape[0], k.shape[1]
    scores = torch.einsum("lhgd,hkd->hglk", q, k) * SCALE
    seen = torch.arange(K, device=q.device)[None, :] <= torch.arange(L, device=q.device)[:, None] + (K - L)
    scores = scores.masked_fill(~seen, float("-inf"))
    e = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    e = e.masked_fill(~seen, 0.0)
    return torch.einsum("hglk,hkd->lhgd", e / e.sum(dim=-1, keepdim=True), v)


def _plain_prompt(s):
    hq, hkv = s["hq"], s["hkv"]
    q = s["q"].float().reshape(-1, hkv, hq // hkv, D).split(s["q_len"])
    k, v = s["k"].float().split(s["k_len"], dim=1), s["v"].float().split(s["k_len"], dim=1)
    out = torch.cat([_plain_sequence(a, b, c) for a, b, c in zip(q, k, v)])
    return out.reshape(-1, hq, D).to(torch.bfloat16)


def _plain_shared(s):
    hq, hkv = s["hq"], s["hkv"]
    q = s["q"].float().reshape(-1, hkv, hq // hkv, D)
    cap = s["tk"].shape[2]
    lens = torch.tensor(s["tail_len"], device=q.device)
    seen = torch.arange(cap, device=q.device)[None, :] < lens[:, None]
    first = torch.einsum("nhgd,hkd->nhgk", q, s["k"].float()) * SCALE
    then = torch.einsum("nhgd,nhkd->nhgk", q, s["tk"].float()) * SCALE
    then = then.masked_fill(~seen[:, None, None, :], float("-inf"))
    top = torch.maximum(first.amax(dim=-1, keepdim=True), then.amax(dim=-1, keepdim=True))
    first, then = torch.exp(first - top), torch.exp(then - top)
    total = first.sum(dim=-1, keepdim=True) + then.sum(dim=-1, keepdim=True)
    out = torch.einsum("nhgk,hkd->nhgd", first / total, s["v"].float()) + \
        torch.einsum("nhgk,nhkd->nhgd", then / total, s["tv"].float())
    return out.reshape(-1, hq, D).to(torch.bfloat16)


def _plain_rows(s):
    hq, hkv = s["hq"], s["hkv"]
    q, k, v = s["qkv"].reshape(-1, hq + 2 * hkv, D).split((hq, hkv, hkv), dim=1)
    cos, sin = s["rope"][s["at"]][:, None, :, 0], s["rope"][s["at"]][:, None, :, 1]

    def turned(x, gain):
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * gain
        a, b = x[..., : D // 2], x[..., D // 2:]
        return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1).to(torch.bfloat16)

    s["k"].copy_(turned(k, s["k_norm"]).transpose(0, 1))
    s["v"].copy_(v.to(torch.bfloat16).transpose(0, 1))
    return {"q": turned(q, s["q_norm"]), "k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------- the framework's calls

def _own_prompt(s):
    from quantized_decoder_decode_gb300 import fq
    hq, hkv, q = s["hq"], s["hkv"], s["q"]
    if "view" not in s:   # what a program keeps with its cache: the view of the layer, the lengths, a workspace
        rows = s["k"].shape[1]
        s["view"] = fq.fq_kv_view(s["k"].data_ptr(), s["v"].data_ptr(), rows, D, rows * D)
        s["lens"] = fq.u32_array(s["q_len"]), fq.u32_array(s["k_len"])
        need = fq.fq_attn_prompt_workspace(*s["lens"], hq, hkv)
        s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q)
    fq.fq_attn_prompt(q.data_ptr(), s["view"], *s["lens"], hq, hkv, SCALE, out.data_ptr(), s["ws"].data_ptr(),
                      s["ws"].numel(), torch.cuda.current_stream().cuda_stream)
    return out


def _own_shared(s):
    from quantized_decoder_decode_gb300 import fq
    hq, hkv, q = s["hq"], s["hkv"], s["q"]
    if "view" not in s:
        rows, (n, _, cap, _) = s["prefix"], s["tk"].shape
        s["view"] = fq.fq_kv_view(s["k"].data_ptr(), s["v"].data_ptr(), rows, D, rows * D)
        s["tails"] = fq.kv_view_array([fq.fq_kv_view(s["tk"][i].data_ptr(), s["tv"][i].data_ptr(), cap, D, cap * D)
                                       for i in range(n)])
        s["lens"] = fq.u32_array(s["tail_len"])
        need = fq.fq_attn_shared_workspace(rows, s["lens"], hq, hkv)
        s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q)
    fq.fq_attn_shared(q.data_ptr(), s["view"], s["prefix"], s["tails"], s["lens"], hq, hkv, SCALE, out.data_ptr(),
                      s["ws"].data_ptr(), s["ws"].numel(), torch.cuda.current_stream().cuda_stream)
    return out


def _own_rows(s):
    from quantized_decoder_decode_gb300 import fq
    hq, hkv, qkv = s["hq"], s["hkv"], s["qkv"]
    if "view" not in s:
        rows = s["k"].shape[1]
        s["view"] = fq.fq_kv_view(s["k"].data_ptr(), s["v"].data_ptr(), rows, D, rows * D)
        s["lens"] = fq.u32_array(s["n"]), fq.u32_array(s["pos"])
        s["row0"] = fq.u32_array([sum(s["n"][:i]) for i in range(len(s["n"]))])
    q = torch.empty(qkv.shape[0], hq, D, dtype=torch.bfloat16, device=qkv.device)
    fq.fq_qk_norm_rope(qkv.data_ptr(), *s["lens"], s["view"], s["row0"], hq, hkv, s["q_norm"].data_ptr(),
                       s["k_norm"].data_ptr(), EPS, s["rope"].data_ptr(), s["rope"].shape[0], q.data_ptr(),
                       torch.cuda.current_stream().cuda_stream)
    return {"q": q, "k": s["k"], "v": s["v"]}


def run(state):
    if own:
        return {"prompt": _own_prompt, "shared": _own_shared, "rows": _own_rows}[state["op"]](state)
    return {"prompt": _plain_prompt, "shared": _plain_shared, "rows": _plain_rows}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "prompt":
        q, k = _ints(case["q"]), _ints(case["k"])
        pairs = sum(L * (K - L) + L * (L + 1) // 2 for L, K in zip(q, k))   # (query, key) pairs that the mask keeps
        return {"bytes": 2 * D * (2 * sum(q) * hq + 2 * sum(k) * hkv), "flops": 4 * D * hq * pairs}
    if case["op"] == "shared":
        tails = _ints(case["tails"])
        keys = case["prefix"] + sum(tails)
        return {"bytes": 2 * D * (2 * len(tails) * hq + 2 * keys * hkv),
                "flops": 4 * D * hq * (len(tails) * case["prefix"] + sum(tails))}
    n, pos = _ints(case["n"]), _ints(case["pos"])
    last = len(set().union(*(range(p, p + m) for p, m in zip(pos, n))))   # rows of the rotary table that are read
    return {"bytes": sum(n) * (hq + 2 * hkv) * D * (4 + 2) + last * D * 4 + 2 * D * 4, "flops": sum(n) * (hq + hkv) * D * 8}


# ---------------------------------------------------------------- the definitions in 64 bits

def _softmax_values(scores, v):
    """scores [rows, keys] and v [keys, D] in f64 -> sum_j softmax(scores)_j v_j."""
    return torch.exp(scores - torch.logsumexp(scores, dim=1, keepdim=True)) @ v


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv = case["hq"], case["hkv"]
    group = hq // hkv
    if case["op"] == "prompt":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        q0 = k0 = 0
        for L, K in zip(s["q_len"], s["k_len"]):
            above = torch.ones(L, K, dtype=torch.bool, device=out.device).triu(K - L + 1)
            for h in range(hq):
                q, k = s["q"][q0:q0 + L, h].double(), s["k"][h // group, k0:k0 + K].double()
                w = torch.where(above, -math.inf, (q @ k.T) / math.sqrt(D))
                out[q0:q0 + L, h] = _softmax_values(w, s["v"][h // group, k0:k0 + K].double())
            q0, k0 = q0 + L, k0 + K
        return out
    if case["op"] == "shared":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        for h in range(hkv):
            pk, pv = s["k"][h].double(), s["v"][h].double()
            for i, t in enumerate(s["tail_len"]):
                q = s["q"][i, h * group:(h + 1) * group].double()
                w = torch.cat((q @ pk.T, q @ s["tk"][i, h, :t].double().T), dim=1) / math.sqrt(D)
                out[i, h * group:(h + 1) * group] = _softmax_values(w, torch.cat((pv, s["tv"][i, h, :t].double())))
        return out
    x = s["qkv"].double().view(-1, hq + 2 * hkv, D)
    angle = torch.view_as_complex(s["rope"].double())[s["at"]].unsqueeze(1)
    x[:, :hq + hkv] /= torch.sqrt(x[:, :hq + hkv].pow(2).sum(dim=-1, keepdim=True) / D + EPS)
    x[:, :hq] *= s["q_norm"].double()
    x[:, hq:hq + hkv] *= s["k_norm"].double()
    z = torch.complex(x[..., : D // 2], x[..., D // 2:])[:, :hq + hkv] * angle
    y = torch.cat((z.real, z.imag), dim=-1)
    return {"q": y[:, :hq], "k": y[:, hq:].transpose(0, 1).contiguous(), "v": x[:, hq + hkv:].transpose(0, 1).contiguous()}
