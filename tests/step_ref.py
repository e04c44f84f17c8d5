"""Plain 64-bit forms of the operators between two products of a layer, and
seeded inputs for them (numpy and torch on the CPU; nothing of the library)."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16, F16, F8, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32
# half the distance of two neighbours, relative to the value
ROUND = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F8: 2.0 ** -4, F32: 2.0 ** -24}
# half the smallest distance of two values (reached among the smallest)
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F8: 2.0 ** -10, F32: 2.0 ** -150}
F8_MAX = 448.0


class Step:
    """Sequences with `lens` cached and `new` new tokens over a shuffled page
    table whose unused places point anywhere in the cache."""

    def __init__(self, seed, lens, new, page, spare=2, n_pages=None):
        rng = np.random.default_rng(seed)
        self.rng, self.page = rng, page
        self.lens, self.new = np.asarray(lens), np.asarray(new)
        need = -(-(self.lens + self.new) // page)
        used = int(need.sum())
        self.n_pages = n_pages or used + spare
        order = rng.permutation(self.n_pages)
        self.pages = rng.integers(0, self.n_pages, (len(lens), max(1, int(need.max()) + 1))).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.pages[b, :n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.M = int(self.offsets[-1])
        self.max_len = int((self.lens + self.new).max())
        self.max_new = int(self.new.max())

    def batch(self, kq, dev="cuda:0"):
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731
        return kq.Batch(up(self.offsets), up(self.lens), up(self.pages))

    def where(self, b, slots):
        slots = np.asarray(slots)
        return torch.from_numpy(self.pages[b, slots // self.page].astype(np.int64)), torch.from_numpy(slots % self.page)

    def rows(self, b):
        return slice(int(self.offsets[b]), int(self.offsets[b + 1]))


def draw(rng, shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32))


def cast(x, dtype):
    return x.clamp(-F8_MAX, F8_MAX).to(dtype) if dtype == F8 else x.to(dtype)


def empty_cache(n_pages, heads, page, dim, dtype, fill=math.nan):
    """A cache that holds `fill` everywhere."""
    k = torch.full((n_pages, heads, page, dim), fill, dtype=F32).to(dtype)
    v = torch.full((n_pages, heads, dim, page), fill, dtype=F32).to(dtype)
    return k, v


def fill_cache(step, heads, dim, dtype, scale=1.0):
    """Keys and values of every slot in use; all the rest is NaN."""
    k, v = empty_cache(step.n_pages, heads, step.page, dim, dtype)
    kb, vb = k.float(), v.float()
    for b in range(len(step.lens)):
        n = int(step.lens[b] + step.new[b])
        if n:
            p, at = step.where(b, np.arange(n))
            kb[p, :, at] = draw(step.rng, (n, heads, dim), scale)
            vb[p, :, :, at] = draw(step.rng, (n, heads, dim), scale)
    return kb.to(dtype), vb.to(dtype)


def tree_mask(rng, n):
    """Ancestor bits (each its own included) of a random tree of n nodes."""
    m = np.zeros(n, np.uint64)
    for j in range(n):
        p = int(rng.integers(-1, j)) if j else -1
        m[j] = (m[p] if p >= 0 else np.uint64(0)) | np.uint64(1 << j)
    return m


def chain_mask(n):
    return np.array([(2 << j) - 1 for j in range(n)], np.uint64)


def attn(step, k, v, q, mask, scale, k_scale=1.0, v_scale=1.0, heads=None):
    """(out, bound on what rounding p to q's type and fp32 sums may change), in
    float64.  mask: uint64 [M].  heads: only these query heads."""
    M, hq, dim = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    out = torch.zeros((M, hq, dim), dtype=torch.float64)
    bound = torch.zeros((M, hq, dim), dtype=torch.float64)
    u = ROUND[q.dtype]
    for b in range(len(step.lens)):
        T, L = int(step.new[b]), int(step.lens[b])
        if T == 0:
            continue
        p, at = step.where(b, np.arange(L + T))
        bits = mask[step.rows(b)]
        seen = np.ones((T, L + T), bool)
        for j in range(T):
            seen[:, L + j] = (bits >> np.uint64(j)) & np.uint64(1)
        for h in range(hkv):
            kk, vv = k[p, h, at].double() * k_scale, v[p, h, :, at].double() * v_scale
            for i in range(T):
                s = torch.from_numpy(seen[i])
                if not s.any():
                    continue
                qi = q[int(step.offsets[b]) + i, h * G:(h + 1) * G].double()
                ks, vs = kk[s], vv[s]
                w = (qi @ ks.t() * scale).softmax(-1)
                # a score is a sum of dim products in fp32 (each step off by 2^-24 of the sum of
                # magnitudes), so p is off by that times p; rounding p adds u p
                most = (qi.abs() @ ks.abs().t() * abs(scale)).amax()
                rel = u + 2.0 ** -24 * (dim + 16) * (1.0 + float(most)) + 2.0 ** -18
                row = int(step.offsets[b]) + i
                out[row, h * G:(h + 1) * G] = w @ vs
                bound[row, h * G:(h + 1) * G] = rel * (w @ vs.abs()) + TINY[q.dtype] * len(vs) * vs.abs().amax()
    return out, bound


def rope_append(step, x, hq, hkv, dim, rope, rot, pairs, positions, q_norm, k_norm, eps):
    """(q, k, v) [M][heads][dim] in float64, each with a bound on fp32's part."""
    x = x.double().view(-1, hq + 2 * hkv, dim)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    def normed(y, w):
        return y if w is None else y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()

    def turned(y):
        if not rot:
            return y, y.abs()
        c = rope[positions, :rot // 2].double()[:, None]
        s = rope[positions, rot // 2:].double()[:, None]
        out, mag = y.clone(), y.abs()
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if pairs else (j, j + rot // 2)
            out[..., a] = y[..., a] * c[..., j] - y[..., b] * s[..., j]
            out[..., b] = y[..., b] * c[..., j] + y[..., a] * s[..., j]
            both = y[..., a].abs() + y[..., b].abs()
            mag[..., a] = mag[..., b] = both
        return out, mag

    q, qm = turned(normed(q, q_norm))
    k, km = turned(normed(k, k_norm))
    f32 = 2.0 ** -20   # a dozen fp32 roundings, and the sum of dim squares
    return (q, qm * f32), (k, km * f32), (v, v.abs() * f32)


def rounded_bound(y, bound, dtype):
    """How far a value of `dtype` may be from y if its unrounded one is within bound."""
    return bound + ROUND[dtype] * (y.abs() + bound) + TINY[dtype]


def keep(step, k, v, path, counts):
    k, v = k.clone(), v.clone()
    kb = k.view(torch.uint8 if k.element_size() == 1 else torch.int16)
    vb = v.view(torch.uint8 if v.element_size() == 1 else torch.int16)
    for b in range(len(step.lens)):
        n, L = int(counts[b]), int(step.lens[b])
        if not n:
            continue
        src, sat = step.where(b, L + path[step.rows(b)][:n])
        dst, dat = step.where(b, L + np.arange(n))
        kk, vv = kb[src, :, sat].clone(), vb[src, :, :, sat].clone()
        kb[dst, :, dat] = kk
        vb[dst, :, :, dat] = vv
    return k, v


def logprobs(x, tokens, n_top):
    """float64 (logprob, entropy, ids, top logprobs) and a bound for each float."""
    y = x.double()
    V = y.shape[1]
    lse = torch.logsumexp(y, -1, keepdim=True)
    p = (y - lse).exp()
    z = (y - y.amax(-1, keepdim=True)).clamp(min=-1e4)
    entropy = -(torch.where(p > 0, p * (y - lse), 0.0)).sum(-1)
    # a lane adds V / 256 terms one after another in fp32, each off by its exponential
    rel = 2.0 ** -24 * (V / 256 + 64) + 2.0 ** -22
    mean_z = (p * z.abs()).sum(-1)
    entropy_bound = rel * 4 * (1 + mean_z)
    lp, lp_bound = None, None
    if tokens is not None:
        t = tokens.long()
        inside = (t >= 0) & (t < V)
        xt = y.gather(1, t.clamp(0, V - 1))
        lp = torch.where(inside, xt - lse, -math.inf)
        lp_bound = rel * 2 * (1 + mean_z[:, None]) + 2.0 ** -22 * (xt.abs().nan_to_num(posinf=0.0) + lse.abs())
    ids = tops = tb = None
    if n_top:
        f = x.float().numpy()
        order = np.lexsort((np.broadcast_to(np.arange(V), f.shape), -f), -1)[:, :n_top]
        ids = torch.from_numpy(order.astype(np.int32))
        xt = y.gather(1, ids.long())
        tops = xt - lse
        tb = rel * 2 * (1 + mean_z[:, None]) + 2.0 ** -22 * (xt.abs().nan_to_num(posinf=0.0) + lse.abs())
    return (lp, entropy, ids, tops), (lp_bound, entropy_bound, tb)
