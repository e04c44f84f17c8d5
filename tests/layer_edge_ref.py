"""64-bit forms of lora whose first product is exact, so that the second is held to a
bound of its own (torch on the CPU; nothing of the library)."""
from __future__ import annotations

import torch

from step_ref import BF16, F16, F32, draw


def pick_case(rng, M, N, rank, K, n, t, dense):
    """(A, B, scale, ids, base, picked): every row of every A holds a single 1, at column
    picked[adapter][row], so that t is an activation times scale, rounded to fp32 twice and
    nowhere else.  B: one value to an output (dense: all), with all the bits of its type."""
    picked = torch.from_numpy(rng.integers(0, K, (n, rank)))
    A = torch.zeros(n, rank, K).scatter_(2, picked[..., None], 1.0).to(t)
    B = draw(rng, (n, N, rank)).to(t)
    if not dense:
        one = torch.from_numpy(rng.permutation(N) % rank)
        B = B * (torch.arange(rank)[None, None] == one[None, :, None]).to(t)
    scale = torch.from_numpy(rng.uniform(0.5, 2, n).astype("float32"))
    ids = torch.from_numpy(rng.integers(-1, n, M).astype("int32"))
    base = 2.0 ** -30 * draw(rng, (M, N))   # (its addition leaves the bits of the products)
    return A, B, scale, ids, base, picked


def picked_t(qs, d, bs, scale, ids, picked):
    """t [M][rank] as fp32 has it: (qs * d) rounded, times scale rounded."""
    rows = torch.arange(qs.shape[0])[:, None]
    at = picked[ids.clamp(min=0).long()]                        # [M][rank]
    return (qs[rows, at].to(F32) * d[rows, at // bs]) * scale[ids.clamp(min=0).long()][:, None]


def second(t, B, ids, base, dense):
    """(out, bound) of base + B t.  Every product of a part of t and a part of B is exact in
    fp32, and products below 2^-24 of the whole may be left out.  What is left are the additions,
    each off by at most 2^-23 of the sum of magnitudes (2^-23: a matrix core need not round to
    nearest inside): a value of t and one of B have 3 products of parts, 5 where B's is
    float16 (two parts), and base is one more."""
    has = (ids >= 0)[:, None]
    b = B[ids.clamp(min=0).long()].double()                     # [M][N][rank]
    td = t.double()[:, None]
    out = base.double() + torch.where(has, (b * td).sum(-1), 0.0)
    size = torch.where(has, (b * td).abs().sum(-1), 0.0) + base.double().abs()
    additions = (t.shape[1] if dense else 1) * (5 if B.dtype == F16 else 3) + 1.5   # (and the products left out)
    return out, torch.where(has, additions * 2.0 ** -23 * size, 0.0)


def parts(t, n):
    """t as the sum of its first n parts of 8 bits."""
    out, left = torch.zeros_like(t), t.clone()
    for _ in range(n):
        p = left.to(BF16).to(F32)
        out, left = out + p, left - p
    return out
