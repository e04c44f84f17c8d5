"""Measured cases of the operators between two products of a decoder layer:
rope_append, attn_tree, cache_keep and logprobs.

A case names an operator and its sizes.  prepare() makes the inputs, run() is
one pass through the operator (plain torch operations in fp32, or the library's
kernels where `own` is true), work() the bytes and operations a pass cannot do
without, exact() the result in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "f8": 1}
F8_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one user's next token: one row of a product, 32 query and 8 key heads, norms on both
        dict(name="append one token", op="append", kv="bf16", q="bf16", seqs=1, tokens=1, length=777, q_heads=32,
             kv_heads=8, dim=128, page=64, rot=128, pairs=False, norm=True),
        # a batch of drafted trees going into an 8-bit cache, interleaved rotation over half of each head
        dict(name="append trees f8", op="append", kv="f8", q="bf16", seqs=48, tokens=32, length=1500, q_heads=40,
             kv_heads=8, dim=128, page=32, rot=64, pairs=True, norm=False),
        # prompts: four ragged ones whose caches already hold a prefix, so slots start off any alignment
        dict(name="append prompts", op="append", kv="f16", q="f16", seqs=4, tokens=4096, length=999, q_heads=32,
             kv_heads=8, dim=128, page=16, rot=128, pairs=False, norm=True),
        # one user's next token over a short cache: latency alone
        dict(name="attn one token", op="attn", kv="bf16", q="bf16", seqs=1, tokens=1, length=1000, q_heads=32,
             kv_heads=8, dim=128, page=64),
        # a serving batch, one token each, caches of very different lengths
        dict(name="attn batch", op="attn", kv="bf16", q="bf16", seqs=64, tokens=1, length=8191, q_heads=32,
             kv_heads=8, dim=128, page=16),
        # two users with long documents in an 8-bit cache
        dict(name="attn long f8", op="attn", kv="f8", q="bf16", seqs=2, tokens=1, length=131075, q_heads=64,
             kv_heads=8, dim=128, page=128),
        # a batch of ragged drafted trees, small heads
        dict(name="attn trees f16", op="attn", kv="f16", q="f16", seqs=24, tokens=24, length=4100, q_heads=16,
             kv_heads=4, dim=64, page=32),
        # wide trees over shared heads: 512 query rows to each key head
        dict(name="attn wide trees", op="attn", kv="bf16", q="bf16", seqs=8, tokens=64, length=16384, q_heads=64,
             kv_heads=8, dim=128, page=64),
        # one user's answer token with its alternatives
        dict(name="logprobs one row", op="logprobs", type="f32", rows=1, vocab=128256, given=1, top=20),
        # every row of a verified draft against all its children; rows of an odd length
        dict(name="logprobs drafts", op="logprobs", type="f32", rows=1537, vocab=100277, given=4, top=8),
        # what was accepted of a batch of trees, over the layers of a model
        dict(name="keep layers", op="keep", kv="bf16", seqs=32, tokens=32, length=300, layers=16, kv_heads=8, dim=128,
             page=32),
        # one user's accepted branch, in one layer's cache
        dict(name="keep one layer", op="keep", kv="f8", seqs=1, tokens=15, length=500, layers=1, kv_heads=4, dim=256,
             page=64),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], evenly over its logarithm, so odd ones too."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "logprobs", "keep"])
    if op == "logprobs":
        kind = rng.choice(["f32", "f32", "bf16", "f16"])
        vocab = _spread(rng, 4000, 160000)
        rows = _spread(rng, 1, max(1, min(4096, 150_000_000 // vocab)))
        return dict(op=op, type=kind, rows=rows, vocab=vocab, given=rng.randint(1, 6), top=rng.choice([0, 1, 5, 8, 20, 32]))
    q = rng.choice(["bf16", "f16"])
    kv = rng.choice([q, q, "f8"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    case = dict(op=op, kv=kv, q=q, kv_heads=kv_heads, dim=dim, page=page)
    if op == "append":
        case.update(q_heads=q_heads, seqs=_spread(rng, 1, 64), length=_spread(rng, 1, 4000),
                    rot=rng.choice([dim, dim, dim // 2]), pairs=rng.choice([False, True]), norm=rng.choice([False, True]))
        most = 12_000 * 48 * 128 // ((q_heads + 2 * kv_heads) * dim)
        case["tokens"] = _spread(rng, 1, max(1, min(4096, most // case["seqs"])))
    elif op == "attn":
        case.update(q_heads=q_heads, seqs=_spread(rng, 1, 96))
        case["tokens"] = rng.choice([1, 1, _spread(rng, 2, 64)])
        most = 400_000 * 1024 // (case["seqs"] * kv_heads * dim)
        if case["tokens"] > 1:
            most = min(most, 8 * 16384 * 64 * 64 * 128 // (case["seqs"] * case["tokens"] * q_heads * dim))
        case["length"] = _spread(rng, 1, max(16, min(150_000, most)))
    else:
        del case["q"]
        case.update(seqs=_spread(rng, 1, 32), tokens=_spread(rng, 2, 64), length=_spread(rng, 1, 300),
                    layers=_spread(rng, 1, 16))
        if kv != "f8":
            case["kv"] = q
    return case


# --------------------------------------------------------------------- inputs

def _counts(case):
    """Cached and new tokens of each sequence, the same for every seed: the
    first has the full sizes."""
    n, T, L = case["seqs"], case["tokens"], case["length"]
    rng = np.random.default_rng([n, T, L])
    new = rng.integers(max(1, T // 3), T + 1, n)
    old = rng.integers(L // 4, L + 1, n)
    new[0], old[0] = T, L
    return old.astype(np.int64), new.astype(np.int64)


def _paged(case, seed):
    """Sequences of a step over a paged cache: their lengths, and a page table
    that hands the pages out in no order."""
    rng = np.random.default_rng(seed)
    old, new = _counts(case)
    need = -(-(old + new) // case["page"])
    n_pages = int(need.sum()) + 3
    order = rng.permutation(n_pages)
    pages = np.zeros((case["seqs"], int(need.max())), np.int32)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    offsets = np.concatenate([[0], np.cumsum(new)])
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    return rng, dict(case=case, offsets=up(offsets), lens=up(old), pages=up(pages), n_pages=n_pages,
                     max_tokens=int(new.max()), max_len=int((old + new).max()), M=int(offsets[-1]),
                     old=old, new=new)


def _trees(rng, new):
    """A drafted tree for each sequence: node j hangs off the cache or off an
    earlier node.  (ancestor bits with the node's own, depth), one row each."""
    T = int(new.max())
    bits = np.zeros((len(new), T), np.uint64)
    depth = np.zeros((len(new), T), np.int64)
    rows = np.arange(len(new))
    for j in range(T):
        parent = rng.integers(max(-1, j - 6), j, len(new)) if j else np.full(len(new), -1)
        has = parent >= 0
        p = np.maximum(parent, 0)
        bits[:, j] = np.where(has, bits[rows, p], np.uint64(0)) | np.uint64(1 << j)
        depth[:, j] = np.where(has, depth[rows, p] + 1, 0)
    used = np.arange(T)[None, :] < new[:, None]
    return bits[used], depth[used]


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _cache(gen, case, n_pages, lead=()):
    """Keys [pages][heads][page][dim], values [pages][heads][dim][page]."""
    d, h, p = case["dim"], case["kv_heads"], case["page"]
    dtype = DTYPES[case["kv"]]
    return _normal(gen, (*lead, n_pages, h, p, d), dtype), _normal(gen, (*lead, n_pages, h, d, p), dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) % (1 << 62))
    if case["op"] == "logprobs":
        M, V = case["rows"], case["vocab"]
        # from rows that are nearly sure to rows that are nearly flat
        x = torch.randn((M, V), generator=gen, device=DEV, dtype=torch.float32)
        x *= 0.5 + 3.0 * torch.rand((M, 1), generator=gen, device=DEV)
        # a grammar leaves some rows a part of the vocabulary
        keep = 1 + torch.randint(0, V, (M, 1), generator=gen, device=DEV)
        some = torch.rand((M, 1), generator=gen, device=DEV) < 0.2
        x.masked_fill_((torch.arange(V, device=DEV)[None, :] > keep + 64) & some, float("-inf"))
        tokens = torch.randint(0, V, (M, case["given"]), generator=gen, device=DEV, dtype=torch.int32)
        return dict(case=case, logits=x.to(DTYPES[case["type"]]), tokens=tokens)
    rng, s = _paged(case, seed)
    if case["op"] == "keep":
        s["k"], s["v"] = _cache(gen, case, s["n_pages"], (case["layers"],))
        counts = rng.integers(1, np.maximum(2, s["new"] // 3 + 1))
        path = np.zeros(s["M"], np.int32)
        for b, n in enumerate(counts):
            at = int(s["new"][:b].sum())
            path[at:at + n] = np.sort(rng.permutation(int(s["new"][b]))[:n])
        s["counts"] = torch.from_numpy(counts.astype(np.int32)).to(DEV)
        s["path"] = torch.from_numpy(path).to(DEV)
        return s
    bits, depth = _trees(rng, np.minimum(s["new"], 64))
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "attn":
        s["k"], s["v"] = _cache(gen, case, s["n_pages"])
        s["q"] = (1.5 * _normal(gen, (s["M"], hq, d), torch.float32)).to(DTYPES[case["q"]])
        s["mask"] = torch.from_numpy(bits.view(np.int64)).to(DEV)
        return s
    # append: a prompt is a chain, a draft of up to 64 tokens a tree
    if case["tokens"] > 64:
        depth = np.concatenate([np.arange(n) for n in s["new"]])
    pos = np.repeat(s["old"], s["new"]) + depth
    s["positions"] = torch.from_numpy(pos.astype(np.int32)).to(DEV)
    n_pos = int((s["old"] + s["new"]).max())
    freq = 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64) / (case["rot"] // 2))
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * freq[None, :]
    s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
    s["x"] = 1.3 * _normal(gen, (s["M"], (hq + 2 * hkv) * d), torch.float32)
    s["q_norm"] = 1.0 + 0.1 * _normal(gen, (d,), torch.float32) if case["norm"] else None
    s["k_norm"] = 1.0 + 0.1 * _normal(gen, (d,), torch.float32) if case["norm"] else None
    shape = (s["n_pages"], hkv, case["page"], d)
    s["k"] = torch.zeros(shape, device=DEV, dtype=DTYPES[case["kv"]])
    s["v"] = torch.zeros((s["n_pages"], hkv, d, case["page"]), device=DEV, dtype=DTYPES[case["kv"]])
    s["k_scale"], s["v_scale"] = (0.02, 0.015) if case["kv"] == "f8" else (1.0, 1.0)
    return s


# --------------------------------------------------------------- the plain forms

def _bits(t):
    """The same memory as whole numbers, for indexed stores of any type."""
    return t.view({1: torch.uint8, 2: torch.int16}[t.element_size()])


def _cast(x, dtype):
    if dtype == torch.float8_e4m3fn:
        x = x.clamp(-F8_MAX, F8_MAX)
    return x.to(dtype)


def _slots(s):
    """Page and place in it of every new token."""
    row = torch.arange(s["M"], device=DEV)
    seq = torch.searchsorted(s["offsets"].long(), row, right=True) - 1
    slot = s["lens"].long()[seq] + row - s["offsets"].long()[seq]
    P = s["case"]["page"]
    return s["pages"].long()[seq, slot // P], slot % P


def _rotate(x, s):
    rot = s["case"]["rot"]
    c, n = s["rope"][s["positions"].long()][:, None, :].split(rot // 2, -1)
    r = x[..., :rot]
    if s["case"]["pairs"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _normed(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _append(s):
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["dim"]
    q, k, v = s["x"].view(s["M"], hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    q = _rotate(_normed(q, s["q_norm"]), s).to(DTYPES[c["q"]])
    k = _cast(_rotate(_normed(k, s["k_norm"]), s) / s["k_scale"], s["k"].dtype)
    v = _cast(v / s["v_scale"], s["v"].dtype)
    page, at = _slots(s)
    _bits(s["k"])[page, :, at, :] = _bits(k)
    _bits(s["v"])[page, :, :, at] = _bits(v.contiguous())
    return dict(q=q, k=s["k"], v=s["v"])


def _attn(s):
    c = s["case"]
    hkv, d, P = c["kv_heads"], c["dim"], c["page"]
    G, B, T = c["q_heads"] // hkv, c["seqs"], s["max_tokens"]
    off, lens = s["offsets"].long(), s["lens"].long()
    new = off[1:] - off[:-1]
    L = s["max_len"]
    pages = s["pages"].long()[:, :-(-L // P)]
    k = s["k"][pages].float().permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)[:, :, :L]
    v = s["v"][pages].float().permute(0, 2, 1, 4, 3).reshape(B, hkv, -1, d)[:, :, :L]
    tok = (off[:-1, None] + torch.arange(T, device=DEV)).clamp(max=s["M"] - 1)              # [B][T]
    q = s["q"].float()[tok].view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    score = torch.matmul(q, k.transpose(-1, -2)).view(B, hkv, T, G, L) * (1.0 / math.sqrt(d))
    key = torch.arange(L, device=DEV)
    node = key[None, :] - lens[:, None]                                                      # [B][L]
    bit = (s["mask"][tok][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1                  # [B][T][L]
    seen = (node < 0)[:, None, :] | ((bit != 0) & (node < new[:, None])[:, None, :])
    score = score.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-30)).view(B, hkv, T * G, L)
    o = torch.matmul(p, v).view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, hkv * G, d)
    return o[torch.arange(T, device=DEV)[None, :] < new[:, None]].to(s["q"].dtype)


def _keep(s):
    c, off, P = s["case"], s["offsets"].long(), s["case"]["page"]
    row = torch.arange(s["M"], device=DEV)
    seq = torch.searchsorted(off, row, right=True) - 1
    j = row - off[seq]
    used = j < s["counts"].long()[seq]
    seq, j, src = seq[used], j[used], s["path"].long()[used]
    start, table = s["lens"].long()[seq], s["pages"].long()
    a, b = start + src, start + j
    pa, pb = table[seq, a // P], table[seq, b // P]
    k, v = _bits(s["k"]), _bits(s["v"])
    kept_k, kept_v = k[:, pa, :, a % P, :], v[:, pa, :, :, a % P]
    k[:, pb, :, b % P, :] = kept_k
    v[:, pb, :, :, b % P] = kept_v
    return dict(k=s["k"], v=s["v"])


def _logprobs(s):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    z = x - top
    e = torch.exp(z)
    S = e.sum(-1, keepdim=True)
    lse = top + torch.log(S)
    entropy = (torch.log(S) - torch.where(e > 0, e * z, 0.0).sum(-1, keepdim=True) / S)[:, 0]
    given = x.gather(1, s["tokens"].long()) - lse
    out = dict(logprob=given, entropy=entropy)
    n = s["case"]["top"]
    if n:
        # larger logits first, the lowest index among equal ones
        b = x.view(torch.int32).long()
        key = torch.where(b < 0, -(b & 0x7FFFFFFF), b) * (1 << 32) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=DEV))
        ids = key.topk(n, -1).indices
        out.update(top_ids=ids.int(), top_logprobs=x.gather(1, ids) - lse)
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _append, "attn": _attn, "keep": _keep, "logprobs": _logprobs}[c["op"]](s)
    import block_quantized_matmul_act_amd as kq
    if c["op"] == "logprobs":
        r = kq.logprobs(s["logits"], s["tokens"], n_top=c["top"])
        out = dict(logprob=r.logprob, entropy=r.entropy)
        return dict(out, top_ids=r.top_ids, top_logprobs=r.top_logprobs) if c["top"] else out
    batch = kq.Batch(s["offsets"], s["lens"], s["pages"])
    if c["op"] == "keep":
        kq.cache_keep([kq.PagedCache(k, v) for k, v in zip(s["k"], s["v"])], batch, s["path"], s["counts"])
        return dict(k=s["k"], v=s["v"])
    if c["op"] == "attn":
        return kq.attn_tree(kq.PagedCache(s["k"], s["v"]), batch, s["q"], s["mask"], max_tokens=s["max_tokens"],
                            max_len=s["max_len"])
    cache = kq.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    q = kq.rope_append(cache, batch, s["x"], c["q_heads"], s["rope"], positions=s["positions"], q_norm=s["q_norm"],
                       k_norm=s["k_norm"], eps=EPS, pairs=c["pairs"], q_dtype=DTYPES[c["q"]])
    return dict(q=q, k=s["k"], v=s["v"])


# ------------------------------------------------------------ work and the exact values

def work(case):
    if case["op"] == "logprobs":
        M, V = case["rows"], case["vocab"]
        return dict(bytes=M * V * SIZE[case["type"]] + M * (8 * case["given"] + 4 + 8 * case["top"]), flops=5 * M * V)
    hkv, d, kv = case["kv_heads"], case["dim"], SIZE[case["kv"]]
    old, new = _counts(case)
    if case["op"] == "keep":
        moved = (len(new) + new.sum() / 3) / 2   # each sequence keeps 1 .. a third of its tokens
        return dict(bytes=float(moved * 2 * hkv * d * kv * 2 * case["layers"]), flops=0)
    hq = case["q_heads"]
    if case["op"] == "append":
        heads = hq + 2 * hkv
        n = int(new.sum())
        return dict(bytes=n * d * (4 * heads + 2 * hq + 2 * hkv * kv) + n * 4 * case["rot"], flops=n * d * (hq + hkv) * 8)
    return dict(bytes=float((old + new).sum() * 2 * hkv * d * kv + new.sum() * hq * d * 4),
                flops=float(4 * hq * d * (new * (old + new)).sum()))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    off = [0] + [int(v) for v in np.cumsum(s["new"])]
    table = s["pages"].cpu().numpy()
    P = case["page"]

    def places(b, first, n):
        """(pages, places) of n slots of sequence b from slot `first` on."""
        slot = np.arange(first, first + n)
        return (torch.from_numpy(table[b, slot // P].astype(np.int64)).to(DEV),
                torch.from_numpy((slot % P).astype(np.int64)).to(DEV))

    k, v = s["k"].double(), s["v"].double()
    hkv, d = case["kv_heads"], case["dim"]
    if case["op"] == "keep":
        path, counts = s["path"].cpu().numpy(), s["counts"].cpu().numpy()
        for b in range(case["seqs"]):
            for j in range(int(counts[b])):   # rising sources: no slot is read after it is written
                (pa, a), (pb, t) = (places(b, int(s["old"][b]) + i, 1) for i in (int(path[off[b] + j]), j))
                k[:, pb[0], :, t[0], :] = k[:, pa[0], :, a[0], :]
                v[:, pb[0], :, :, t[0]] = v[:, pa[0], :, :, a[0]]
        return dict(k=k, v=v)
    hq = case["q_heads"]
    G = hq // hkv
    if case["op"] == "attn":
        q, out = s["q"].double(), torch.empty((s["M"], hq, d), dtype=torch.float64, device=DEV)
        bits = s["mask"].cpu().numpy().view(np.uint64)
        for b in range(case["seqs"]):
            T, L0 = int(s["new"][b]), int(s["old"][b])
            pg, at = places(b, 0, L0 + T)
            seen = np.ones((T, L0 + T), bool)
            for j in range(T):
                seen[:, L0 + j] = (bits[off[b]:off[b + 1]] >> np.uint64(j)) & np.uint64(1)
            seen = torch.from_numpy(seen).to(DEV)
            for h in range(hkv):
                rows = q[off[b]:off[b + 1], h * G:(h + 1) * G].reshape(T * G, d)
                w = rows @ k[pg, h, at].t() / math.sqrt(d)
                w = torch.where(seen.repeat_interleave(G, 0), w, -math.inf).softmax(-1)
                out[off[b]:off[b + 1], h * G:(h + 1) * G] = (w @ v[pg, h, :, at]).view(T, G, d)
        return out
    x = s["x"].double().view(s["M"], hq + 2 * hkv, d)
    half = case["rot"] // 2
    pos = s["positions"].long()
    turn = torch.complex(s["rope"][pos, :half].double(), s["rope"][pos, half:].double())[:, None, :]

    def turned(y, w):
        y = y.clone()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
        first = slice(0, 2 * half, 2) if case["pairs"] else slice(0, half)
        second = slice(1, 2 * half, 2) if case["pairs"] else slice(half, 2 * half)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, new_k, new_v = turned(x[:, :hq], s["q_norm"]), turned(x[:, hq:hq + hkv], s["k_norm"]), x[:, hq + hkv:]
    top = F8_MAX if case["kv"] == "f8" else math.inf
    for b in range(case["seqs"]):
        pg, at = places(b, int(s["old"][b]), int(s["new"][b]))
        k[pg, :, at, :] = (new_k[off[b]:off[b + 1]] / s["k_scale"]).clamp(-top, top)
        v[pg, :, :, at] = (new_v[off[b]:off[b + 1]] / s["v_scale"]).clamp(-top, top)
    return dict(q=q, k=k, v=v)


def _exact_logprobs(s):
    c = s["case"]
    given, entropy, tops = [], [], []
    for rows, tokens in zip(s["logits"].split(256), s["tokens"].long().split(256)):
        lp = rows.double().log_softmax(-1)
        given.append(lp.gather(1, tokens))
        entropy.append(-torch.xlogy(lp.exp(), lp.exp()).sum(-1))
        if c["top"]:
            tops.append(lp.topk(c["top"], -1).values)
    out = dict(logprob=torch.cat(given), entropy=torch.cat(entropy))
    return dict(out, top_ids=None, top_logprobs=torch.cat(tops)) if c["top"] else out
