"""Measured cases of three operators of a serving layer: norm_quantize in front
of a product, attn_chunk over the paged cache, lora beside a product.

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
BLOCK = {"q8_k": 256, "q8_128": 128}   # values to a scale of the activation formats
FMT = {"q8_k": 1, "q8_128": 2}
EPS = 1e-6


def listed():
    return [
        # one user's next token: the layer's product, the residual and the input of the next product
        dict(name="norm one row", op="norm", x="f32", r="f32", act="q8_k", rows=1, K=4096, pad=0),
        # a ternary model's drafted trees: a 16-bit residual, rows of a wider product
        dict(name="norm drafts", op="norm", x="f32", r="bf16", act="q8_128", rows=500, K=5120, pad=64),
        # prompts
        dict(name="norm prompts", op="norm", x="f32", r="f32", act="q8_k", rows=4096, K=4096, pad=0),
        # one user's next token far into a text, of which the last 4096 tokens and the first 4 are seen
        dict(name="chunk one token", op="chunk", kv="bf16", q="bf16", seqs=1, tokens=1, mixed=False, length=9000,
             q_heads=32, kv_heads=8, dim=128, page=64, window=4096, sinks=4),
        # a serving batch, one token each, an 8-bit cache under a window
        dict(name="chunk batch f8", op="chunk", kv="f8", q="bf16", seqs=96, tokens=1, mixed=False, length=12000,
             q_heads=64, kv_heads=8, dim=128, page=32, window=2048, sinks=4),
        # a prompt read whole into an empty cache
        dict(name="chunk prompt", op="chunk", kv="bf16", q="bf16", seqs=1, tokens=4096, mixed=False, length=0,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # the next pieces of two long documents
        dict(name="chunk long", op="chunk", kv="f16", q="f16", seqs=2, tokens=512, mixed=False, length=32768,
             q_heads=64, kv_heads=8, dim=128, page=128, window=0, sinks=0),
        # ragged prompts of a model with a window, three query heads to a key head
        dict(name="chunk window", op="chunk", kv="f16", q="f16", seqs=5, tokens=2999, mixed=False, length=700,
             q_heads=24, kv_heads=8, dim=64, page=16, window=1024, sinks=16),
        # one piece of a prompt among users who decode
        dict(name="chunk mixed", op="chunk", kv="bf16", q="bf16", seqs=24, tokens=512, mixed=True, length=6000,
             q_heads=32, kv_heads=8, dim=128, page=32, window=0, sinks=0),
        # one user's next token, one adapter
        dict(name="lora one row", op="lora", type="bf16", act="q8_k", rows=1, requests=1, adapters=8, rank=16, K=4096,
             N=4096),
        # a serving batch in which every user has an adapter of their own, or none
        dict(name="lora batch", op="lora", type="bf16", act="q8_k", rows=64, requests=64, adapters=64, rank=16, K=4096,
             N=14336),
        # ragged prompts of a few adapters
        dict(name="lora prompts", op="lora", type="f16", act="q8_k", rows=2048, requests=7, adapters=6, rank=64, K=4096,
             N=14336),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], evenly over its logarithm, so odd ones too."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "chunk", "chunk", "lora"])
    act = rng.choice(["q8_k", "q8_128"])
    if op == "norm":
        K = BLOCK[act] * _spread(rng, 1, 16384 // BLOCK[act])
        return dict(op=op, x=rng.choice(["f32", "f32", "bf16", "f16"]), r=rng.choice(["f32", "bf16", "f16"]), act=act,
                    rows=_spread(rng, 1, max(1, min(8192, (1 << 24) // K))), K=K, pad=rng.choice([0, 0, 8, 72]))
    if op == "lora":
        K = BLOCK[act] * _spread(rng, 1, 14336 // BLOCK[act])
        N = _spread(rng, 60, 14336)
        rows = _spread(rng, 1, max(1, min(4096, 2048 * 14336 // max(N, K))))
        return dict(op=op, type=rng.choice(["bf16", "f16"]), act=act, rows=rows, requests=_spread(rng, 1, min(rows, 64)),
                    adapters=_spread(rng, 1, 64), rank=rng.choice([8, 16, 32, 64]), K=K, N=N)
    q = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    case = dict(op=op, kv=rng.choice([q, q, "f8"]), q=q, seqs=_spread(rng, 1, 64), tokens=1, mixed=False, length=0,
                q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128, 256]),
                window=rng.choice([0, _spread(rng, 16, 8192)]), sinks=0)
    if case["window"]:
        case["sinks"] = rng.choice([0, 1, 4, _spread(rng, 2, 300)])
    case["mixed"] = rng.choice([False, False, True])
    # scores of at most 4e9 bytes in the plain form, and the work of the largest listed case
    scores = 1_000_000_000 // (case["seqs"] * case["q_heads"])
    scores = min(scores, 2 * 512 * 32768 * 64 * 128 // (case["seqs"] * case["q_heads"] * dim))
    case["tokens"] = rng.choice([1, _spread(rng, 2, max(2, min(4096, int(scores ** 0.5))))])
    cache = 400_000 * 1024 // (case["seqs"] * kv_heads * dim)
    case["length"] = _spread(rng, 1, max(16, min(40_000, scores // case["tokens"] - case["tokens"], cache)))
    return case


# --------------------------------------------------------------------- inputs

def _counts(case):
    """Cached and new tokens of each sequence, the same for every seed: the
    first has the full sizes."""
    n, T, L = case["seqs"], case["tokens"], case["length"]
    rng = np.random.default_rng([n, T, L])
    new = rng.integers(max(1, T // 3), T + 1, n)
    old = rng.integers(L // 4, L + 1, n)
    if case["mixed"]:
        new[:] = 1
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
    return dict(case=case, offsets=up(offsets), lens=up(old), pages=up(pages), n_pages=n_pages,
                max_tokens=int(new.max()), max_len=int((old + new).max()), M=int(offsets[-1]), old=old, new=new)


def _requests(case):
    """Rows of each request of a lora case, the same for every seed."""
    n = case["requests"]
    cuts = np.sort(np.random.default_rng([n, case["rows"]]).permutation(case["rows"] - 1)[:n - 1] + 1)
    return np.diff(np.concatenate([[0], cuts, [case["rows"]]]))


def _ids(case, seed):
    """The adapter of each request: all different while there are enough; one request in 8 has none."""
    rng = np.random.default_rng([case["requests"], case["adapters"], seed])
    ids = np.resize(rng.permutation(case["adapters"]), case["requests"])
    ids[7::8] = -1
    return ids


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _up256(n):
    return (n + 255) // 256 * 256


def _activations(gen, case):
    """Quantized activations as the products take them (one buffer), and the views of its
    values [M][K] and scales [K / block][M].  The sums behind them, which only the products
    read, stay zero."""
    M, K, bs = case["rows"], case["K"], BLOCK[case["act"]]
    x = _normal(gen, (M, K // bs, bs), torch.float32)
    d = x.abs().amax(-1) / 127.0
    at_d = _up256(M * K)
    size = at_d + _up256(4 * M * (K // bs))
    if bs == 256:
        size += _up256(2 * M * (K // 16)) + _up256(32 * M * (K // 256))
    buf = torch.zeros(size, dtype=torch.uint8, device=DEV)
    qs = buf[:M * K].view(torch.int8).view(M, K)
    qs.copy_((x / d[..., None]).round().view(M, K))
    scales = buf[at_d:at_d + 4 * M * (K // bs)].view(torch.float32).view(K // bs, M)
    scales.copy_(d.t())
    return buf, qs, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) % (1 << 62))
    if case["op"] == "norm":
        M, K = case["rows"], case["K"]
        # a few features are far larger than the others, as in real residual streams
        big = 1.0 + 20.0 * (torch.rand(K, generator=gen, device=DEV) < 0.002)
        return dict(case=case, x=(1.3 * _normal(gen, (M, K + case["pad"]), torch.float32)).to(DTYPES[case["x"]])[:, :K],
                    r=(2.0 * big * _normal(gen, (M, K), torch.float32)).to(DTYPES[case["r"]]),
                    sum=torch.empty((M, K), device=DEV, dtype=DTYPES[case["r"]]),
                    w=1.0 + 0.2 * _normal(gen, (K,), torch.float32))
    if case["op"] == "lora":
        t, n, r = DTYPES[case["type"]], case["adapters"], case["rank"]
        buf, qs, d = _activations(gen, case)
        ids = np.repeat(_ids(case, seed), _requests(case)).astype(np.int32)
        return dict(case=case, a_q8=buf, qs=qs, d=d,
                    A=(_normal(gen, (n, r, case["K"]), torch.float32) / math.sqrt(case["K"])).to(t),
                    B=(_normal(gen, (n, case["N"], r), torch.float32) / math.sqrt(r)).to(t),
                    scale=0.5 + torch.rand(n, generator=gen, device=DEV), ids=torch.from_numpy(ids).to(DEV),
                    base=_normal(gen, (case["rows"], case["N"]), torch.float32))
    s = _paged(case, seed)
    hq, hkv, d, p = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    s["k"] = _normal(gen, (s["n_pages"], hkv, p, d), DTYPES[case["kv"]])
    s["v"] = _normal(gen, (s["n_pages"], hkv, d, p), DTYPES[case["kv"]])
    s["q"] = (1.5 * _normal(gen, (s["M"], hq, d), torch.float32)).to(DTYPES[case["q"]])
    return s


# --------------------------------------------------------------- the plain forms

def _norm(s):
    c = s["case"]
    M, K, bs = c["rows"], c["K"], BLOCK[c["act"]]
    x = s["x"].float() + s["r"].float()
    s["sum"].copy_(x)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    y = y.view(M, K // bs, bs)
    top = y.abs().amax(-1, keepdim=True)
    q = (y * (127.0 / top)).round().clamp(-127, 127)
    return dict(sum=s["sum"], values=(q * (top / 127.0)).to(torch.bfloat16).view(M, K))


def _chunk(s):
    c = s["case"]
    hkv, d, P = c["kv_heads"], c["dim"], c["page"]
    G, B, T, L = c["q_heads"] // hkv, c["seqs"], s["max_tokens"], s["max_len"]
    off, lens = s["offsets"].long(), s["lens"].long()
    new = off[1:] - off[:-1]
    pages = s["pages"].long()[:, :-(-L // P)]
    k = s["k"][pages].float().permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)[:, :, :L]
    v = s["v"][pages].float().permute(0, 2, 1, 4, 3).reshape(B, hkv, -1, d)[:, :, :L]
    tok = (off[:-1, None] + torch.arange(T, device=DEV)).clamp(max=s["M"] - 1)              # [B][T]
    q = s["q"].float()[tok].view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    score = torch.matmul(q, k.transpose(-1, -2)).view(B, hkv, T, G, L).mul_(1.0 / math.sqrt(d))
    key, place = torch.arange(L, device=DEV), lens[:, None] + torch.arange(T, device=DEV)    # [B][T]
    seen = key <= place[..., None]
    if c["window"]:
        seen &= (key > place[..., None] - c["window"]) | (key < c["sinks"])
    score.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(B, hkv, T * G, L)
    o = torch.matmul(p, v).view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, hkv * G, d)
    return o[torch.arange(T, device=DEV)[None, :] < new[:, None]].to(s["q"].dtype)


def _lora(s):
    c = s["case"]
    M, K, n, r, bs = c["rows"], c["K"], c["adapters"], c["rank"], BLOCK[c["act"]]
    x = (s["qs"].view(M, K // bs, bs).float() * s["d"].t()[..., None]).view(M, K)
    t = (x @ s["A"].view(n * r, K).float().t()).view(M, n, r) * s["scale"][None, :, None]
    mine = s["ids"][:, None] == torch.arange(n, device=DEV, dtype=torch.int32)              # [M][n]
    t = torch.where(mine[..., None], t, 0.0).view(M, n * r)
    return s["base"] + t @ s["B"].float().permute(0, 2, 1).reshape(n * r, c["N"])


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _norm, "chunk": _chunk, "lora": _lora}[c["op"]](s)
    import block_quantized_matmul_act_amd as kq
    if c["op"] == "norm":
        M, K, bs = c["rows"], c["K"], BLOCK[c["act"]]
        a_q8 = kq.norm_quantize(s["x"], s["r"], s["w"], EPS, FMT[c["act"]], sum_out=s["sum"])
        qs, d, _ = kq.act_views(a_q8, FMT[c["act"]], M, K)
        # the 8-bit values as what they stand for, in a type finer than they are
        values = torch.empty((M, K // bs, bs), dtype=torch.bfloat16, device=DEV)
        torch.mul(qs.view(M, K // bs, bs), d[..., None], out=values)
        return dict(sum=s["sum"], values=values.view(M, K))
    if c["op"] == "lora":
        return kq.lora(s["a_q8"], s["A"], s["B"], s["ids"], s["scale"], base=s["base"], act_fmt=FMT[c["act"]])
    return kq.attn_chunk(kq.PagedCache(s["k"], s["v"]), kq.Batch(s["offsets"], s["lens"], s["pages"]), s["q"],
                         window=c["window"], sinks=c["sinks"], max_tokens=s["max_tokens"], max_len=s["max_len"])


# ------------------------------------------------------------ work and the exact values

def work(case):
    if case["op"] == "norm":
        M, K, bs = case["rows"], case["K"], BLOCK[case["act"]]
        behind = 2 / 16 + 32 / 256 if bs == 256 else 0   # sums that the products read
        each = SIZE[case["x"]] + 2 * SIZE[case["r"]] + 1 + 4 / bs + behind
        return dict(bytes=M * K * each + 4 * K, flops=8 * M * K)
    if case["op"] == "lora":
        M, K, N, r = case["rows"], case["K"], case["N"], case["rank"]
        used = len(set(_ids(case, 0).tolist()) - {-1})   # as many of them for every seed
        return dict(bytes=float(M * K * (1 + 4 / BLOCK[case["act"]]) + used * r * (K + N) * 2 + M * N * 8),
                    flops=float(2 * M * r * (K + N)))
    hq, hkv, d, kv = case["q_heads"], case["kv_heads"], case["dim"], SIZE[case["kv"]]
    W, S = case["window"], case["sinks"]
    slots = pairs = 0
    for old, new in zip(*_counts(case)):
        place = np.arange(old, old + new)
        if W:
            pairs += int((np.minimum(place + 1, W) + np.clip(place + 1 - W, 0, S)).sum())
            first = max(0, int(old) - W + 1)
            slots += int(old + new) - first + min(first, S)
        else:
            pairs += int((place + 1).sum())
            slots += int(old + new)
    M = int(_counts(case)[1].sum())
    return dict(bytes=float(slots * 2 * hkv * d * kv + M * hq * d * 4), flops=float(4 * hq * d * pairs))


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "chunk": _exact_chunk, "lora": _exact_lora}[case["op"]](s)


def _exact_norm(s):
    bs = BLOCK[s["case"]["act"]]
    z = torch.add(s["x"].double(), s["r"].double())
    blocks = (z / (z.pow(2).sum(1, keepdim=True) / z.shape[1] + EPS).sqrt() * s["w"].double()).unflatten(1, (-1, bs))
    step = blocks.abs().max(2, keepdim=True).values / 127.0
    return dict(sum=z, values=(torch.round(blocks / step) * step).flatten(1))


def _exact_chunk(s):
    c = s["case"]
    P, hq, G = c["page"], c["q_heads"], c["q_heads"] // c["kv_heads"]
    W, S = c["window"] or (1 << 40), c["sinks"]
    out = torch.empty((s["M"], hq, c["dim"]), dtype=torch.float64, device=DEV)
    table, at = s["pages"].cpu().numpy(), 0
    for b in range(c["seqs"]):
        L0, T = int(s["old"][b]), int(s["new"][b])
        slot = np.arange(L0 + T)
        pg = torch.from_numpy(table[b, slot // P].astype(np.int64)).to(DEV)
        pl = torch.from_numpy(slot % P).to(DEV)
        slot = torch.from_numpy(slot).to(DEV)
        own_slot = L0 + torch.arange(T, device=DEV)[:, None]
        back = own_slot - slot
        hidden = (back < 0) | ((back >= W) & (slot >= S))
        for h in range(hq):
            kk, vv = s["k"][pg, h // G, pl].double(), s["v"][pg, h // G, :, pl].double()
            w = s["q"][at:at + T, h].double() @ kk.t() / math.sqrt(c["dim"])
            out[at:at + T, h] = w.masked_fill_(hidden, -math.inf).softmax(-1) @ vv
        at += T
    return out


def _exact_lora(s):
    c = s["case"]
    x = s["qs"].double() * s["d"].double().t().repeat_interleave(BLOCK[c["act"]], 1)
    out = s["base"].double()
    for i in range(c["adapters"]):
        rows = (s["ids"] == i).nonzero()[:, 0]
        if len(rows):
            out[rows] += s["scale"][i].double() * ((x[rows] @ s["A"][i].double().t()) @ s["B"][i].double().t())
    return out
