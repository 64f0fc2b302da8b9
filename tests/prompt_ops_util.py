"""Plain 64-bit forms of the prompt and shared-prompt attention operators, and the bound that
an output may be off by."""
import math

import torch

DEV = torch.device("cuda:0")
D = 128
BF16_HALF_STEP = 2.0 ** -8   # rounding to bf16, relative to the value


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def attend(q, k, v, seen, scale):
    """One head in 64 bits.  q [L, D], k and v [K, D], seen [L, K] bool.  Returns the outputs and
    the bound of |error| before the output's own rounding.

    Bound, to first order: a weight p_j = exp(s_j) / sum carries
      * its rounding to bf16 for the product with V: 2^-8;
      * twice the error of its score (numerator and denominator): the f32 dot product of 128
        exact bf16 products, at most 128 2^-24 sum_d |q_d k_d| scale, the product with
        log2(e) scale and the subtraction of the maximum (3 roundings of |s|);
      * exp2's error, 2^-21, and the sums over up to K keys, K 2^-24 each of numerator and
        denominator, and a few roundings of rescaling and joining (16 of them)."""
    L, K = q.shape[0], k.shape[0]
    out = torch.zeros(L, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    rows = seen.any(dim=1)
    if K == 0 or not bool(rows.any()):
        return out, bound
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T) * scale
    s = torch.where(seen, s, -math.inf)
    top = torch.where(rows, s.amax(dim=1), 0.0)
    p = torch.where(seen, torch.exp(s - top[:, None]), 0.0)
    p = p / p.sum(dim=1, keepdim=True)
    kk, vv = torch.where(seen.any(dim=0)[:, None], k, 0.0), torch.where(seen.any(dim=0)[:, None], v, 0.0)
    out[rows] = (p @ vv)[rows]
    ds = torch.where(seen, (q.abs() @ kk.abs().T) * abs(scale), 0.0).amax(dim=1) * (128 + 3) * 2.0 ** -24
    rel = BF16_HALF_STEP + 2 * ds + 2.0 ** -21 + (2 * K + 16) * 2.0 ** -24
    bound[rows] = ((p @ vv.abs()) * rel[:, None])[rows]
    return out, bound


def causal(L, K, dev=DEV):
    return torch.arange(K, device=dev)[None, :] <= torch.arange(L, device=dev)[:, None] + (K - L)


def assert_within(got, ref, bound, bf16_out, what=""):
    """|got - ref| <= bound (+ half a bf16 step of the value where the output is bf16)."""
    ref, bound = ref.to(got.device), bound.to(got.device)
    tol = bound + (BF16_HALF_STEP * (ref.abs() + bound) if bf16_out else 2.0 ** -24 * ref.abs()) + 1e-37
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; worst " \
        f"{float(torch.nan_to_num(err / tol, nan=math.inf).max()):.3g} of it, first at {bad.nonzero()[0].tolist()}"
