"""Plain 64-bit forms of the operators around the products of a layer
(norm_quantize, attn_chunk, lora), with bounds worked out from the roundings of
each step (torch on the CPU; nothing of the library)."""
from __future__ import annotations

import math

import torch

from step_ref import ROUND, TINY

EPS32 = 2.0 ** -24


def norm(x, r, w, eps):
    """(s, y) in float64 and a bound on what fp32 may change of y: s and the two products
    round once each, the sum of K squares is off by at most the depth of its tree
    (64 in a lane, 6 steps in a wave, 16 waves), halved by the root, and mean, eps, root
    and inverse round once each: under 100 roundings."""
    s = x.double() if r is None else x.double() + r.double()
    mean = s.pow(2).mean(-1, keepdim=True) + eps
    y = s / mean.clamp(min=1e-300).sqrt()
    if w is not None:
        y = y * w.double()
    return s, y, 100 * EPS32 * y.abs()


def check_quantized(y, bound, qs, d, bs):
    """qs [M][K] int8 and d [M][K / bs] as the quantization of y within bound: the scale is
    amax / 127, and every value is within half a step of y."""
    M, K = y.shape
    yb, bb = y.view(M, K // bs, bs), bound.view(M, K // bs, bs)
    q, d = qs.double().view(M, K // bs, bs), d.double()
    step = yb.abs().amax(-1) / 127
    near = bb.amax(-1) / 127 + 4 * EPS32 * step
    assert ((d - step).abs() <= near).all(), ("d", ((d - step).abs() / near.clamp(min=1e-300)).max())
    # d itself is off by near, 127 times at most; x * (127 / amax) rounds twice in fp32
    off = (q * d[..., None] - yb).abs()
    most = 0.5 * step[..., None] + bb + (127 + 0.5) * near[..., None] + 4 * EPS32 * yb.abs()
    assert (off <= most).all(), ("values", (off / most.clamp(min=1e-300)).max())
    assert (qs.abs() <= 127).all()
    return (off / most.clamp(min=1e-300)).max().item()


def seen(old, T, window, sinks):
    """[T][old + T]: which slots each new row sees."""
    pos = old + torch.arange(T)[:, None]
    slot = torch.arange(old + T)[None, :]
    on = slot <= pos
    if window:
        on &= (slot > pos - window) | (slot < sinks)
    return on


def chunk(step, k, v, q, window, sinks, scale, k_scale=1.0, v_scale=1.0):
    """(out, bound on what rounding p to q's type and fp32 sums may change)."""
    M, hq, dim = q.shape
    G = hq // k.shape[1]
    out = torch.zeros((M, hq, dim), dtype=torch.float64)
    bound = torch.zeros((M, hq, dim), dtype=torch.float64)
    u = ROUND[q.dtype]
    for b in range(len(step.lens)):
        T, L = int(step.new[b]), int(step.lens[b])
        if not T:
            continue
        p, at = step.where(b, torch.arange(L + T).numpy())
        on = seen(L, T, window, sinks)
        r = step.rows(b)
        for h in range(hq):
            kk, vv = k[p, h // G, at].double() * k_scale, v[p, h // G, :, at].double() * v_scale
            # (what no row sees may be anything; what only some see is 0 times p here)
            vis = on.any(0)
            kk, vv = torch.where(vis[:, None], kk, 0.0), torch.where(vis[:, None], vv, 0.0)
            qq = q[r, h].double()
            w = (qq @ kk.t() * scale).masked_fill(~on, -math.inf).softmax(-1)
            # a score is a sum of dim products in fp32 (each step off by 2^-24 of the sum of
            # magnitudes), so p is off by that times p; rounding p adds u p.  The weights are divided
            # by the sum of the rounded ones: with w_i (1 + e_i), |e_i| <= u, the result is off by
            # sum w_i e_i (v_i - out) to first order, at most u (sum w_i |v_i| + |out|)
            most = (qq.abs() @ kk.abs().t() * abs(scale)).masked_fill(~on, 0.0).amax(-1, keepdim=True)
            rel = u + EPS32 * (dim + 16) * (1.0 + most) + 2.0 ** -18
            out[r, h] = w @ vv
            bound[r, h] = rel * (w @ vv.abs()) + u * out[r, h].abs() + TINY[q.dtype] * (L + T) * vv.abs().amax()
    return out, bound


def lora(qs, d, bs, A, B, scale, ids, base):
    """(out, bound): every product of int8 and 16-bit values is exact in fp32; a sum of n terms
    in fp32, in any order, is off by at most n 2^-23 of the sum of magnitudes (2^-23: a
    matrix core need not round to nearest inside)."""
    M, K = qs.shape
    x = qs.double() * d.double().repeat_interleave(bs, 1)
    n, r, _ = A.shape
    N = B.shape[1]
    out = torch.zeros((M, N), dtype=torch.float64) if base is None else base.double().clone()
    bound = out.abs() * 2 * EPS32
    for i in range(n):
        rows = (ids == i).nonzero()[:, 0]
        if len(rows):
            a, b, s = A[i].double(), B[i].double(), 1.0 if scale is None else float(scale[i])
            out[rows] += s * (x[rows] @ a.t()) @ b.t()
            bound[rows] += abs(s) * (x[rows].abs() @ a.abs().t()) @ b.abs().t() * 2.0 ** -23 * (K + r + 8)
    return out, bound
