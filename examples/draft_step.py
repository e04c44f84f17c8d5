"""Decoding with drafted tokens: a small random model with Q4_K weights.

A step takes, for each sequence, a tree of token rows: its last token and under
it the branches that a drafter proposes.  One pass of the model over all rows
(kq_quantize_act, kq_gemm, rope_append, attn_tree) gives every row's logits;
logprobs gives every row's best token; the branch that agrees with them is
accepted, cache_keep moves its keys and values together, and the sequence grows
by one token more than was accepted.  The tokens are those of greedy decoding.

    python examples/draft_step.py [--seqs 4] [--prompt 100] [--new 64] [--cache bf16|f16|f8]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

CHUNK = 64  # rows of a sequence in one pass at most


# ------------------------------------------------------------- trees, on the host

def draft(history, depth=4, branches=2):
    """The tree of the next step, as (tokens, parents): the last token of the
    history, and under it what followed this token's latest other occurrences
    there, up to `depth` tokens each.  Branches share what they have in common."""
    tokens, parents = [history[-1]], [-1]
    seen = 0
    for at in range(len(history) - 2, -1, -1):
        if seen == branches:
            break
        if history[at] != history[-1]:
            continue
        node = 0
        for t in history[at + 1:at + 1 + depth]:
            child = [i for i, p in enumerate(parents) if p == node and tokens[i] == t]
            if not child:
                tokens.append(t)
                parents.append(node)
            node = child[0] if child else len(tokens) - 1
        seen += 1
    return tokens, parents


def ancestry(parents):
    """Each row's depth and its bits: itself and the rows above it."""
    depth, bits = [], []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        bits.append((0 if p < 0 else bits[p]) | 1 << i)
    return depth, bits


def accepted(tokens, parents, best):
    """The rows from the root down that the model agrees with, given each row's
    best next token."""
    path = [0]
    while True:
        child = [i for i, p in enumerate(parents) if p == path[-1] and tokens[i] == best[path[-1]]]
        if not child:
            return path
        path.append(child[0])


# ---------------------------------------------------------------------- the model

class Model:
    """A decoder with grouped heads, normed and rotated, and random weights."""

    def __init__(self, layers=2, hidden=512, q_heads=8, heads=2, dim=64, inner=1024, vocab=256, n_pos=4096, seed=1):
        import torch

        import block_quantized_matmul_act_amd as kq
        import datagen

        self.kq, self.torch, self.device = kq, torch, torch.device("cuda:0")
        self.layers, self.hidden, self.vocab = layers, hidden, vocab
        self.q_heads, self.heads, self.dim = q_heads, heads, dim

        def weight(n, k, salt):
            return n, k, torch.from_numpy(datagen.make_weights(kq.KQ_Q4_K, n, k, seed * 1000 + salt)).to(self.device)

        self.qkv = [weight((q_heads + 2 * heads) * dim, hidden, 10 * i) for i in range(layers)]
        self.o = [weight(hidden, q_heads * dim, 10 * i + 1) for i in range(layers)]
        self.up = [weight(2 * inner, hidden, 10 * i + 2) for i in range(layers)]
        self.down = [weight(hidden, inner, 10 * i + 3) for i in range(layers)]
        self.head = weight(vocab, hidden, 999)
        rng = np.random.default_rng(seed)
        # (large against what the layers add: the text then repeats itself, and lookups find something)
        self.embed = torch.from_numpy(8.0 * rng.standard_normal((vocab, hidden), np.float32)).to(self.device)
        angle = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(dim // 2) / (dim // 2))
        table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
        self.rope = torch.from_numpy(table).to(self.device)
        self.ones = torch.ones(dim, device=self.device)

    def norm(self, x):
        return x * self.torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def product(self, x, w):
        n, k, data = w
        kq = self.kq
        return kq.gemm(kq.KQ_Q4_K, data, kq.quantize_act(x.contiguous(), kq.KQ_ACT_Q8_K), x.shape[0], n, k)

    def __call__(self, caches, batch, tokens, positions, mask, max_tokens, max_len):
        """Logits [rows][vocab]; the rows' keys and values are in the caches after it."""
        kq, act = self.kq, self.torch.nn.functional.silu
        x = self.embed[tokens.long()]
        for i in range(self.layers):
            q = kq.rope_append(caches[i], batch, self.product(self.norm(x), self.qkv[i]), self.q_heads, self.rope,
                               positions, self.ones, self.ones)
            a = kq.attn_tree(caches[i], batch, q, mask, max_tokens=max_tokens, max_len=max_len,
                             out_dtype=self.torch.float32)
            x = x + self.norm(self.product(a.flatten(1), self.o[i]))
            gate, up = self.product(self.norm(x), self.up[i]).chunk(2, 1)
            x = x + self.norm(self.product(act(self.norm(gate)) * up, self.down[i]))
        return 3.0 * self.norm(self.product(self.norm(x), self.head))


class Decoder:
    """Sequences and their pages; the lengths are kept on the host, too."""

    def __init__(self, model, prompts, room, page=64, dtype=None):
        torch, kq = model.torch, model.kq
        self.model, self.page = model, page
        self.history = [list(p) for p in prompts]
        self.lens = [0] * len(prompts)
        wide = -(-max(len(p) + room for p in prompts) // page)
        n = wide * len(prompts)
        dtype = dtype or torch.bfloat16
        scale = 0.05 if dtype == torch.float8_e4m3fn else 1.0  # (8 bits: up to 448 times it)

        def cache():
            k = torch.zeros((n, model.heads, page, model.dim), device=model.device).to(dtype)
            return kq.PagedCache(k, k.view(n, model.heads, model.dim, page).clone(), scale, scale)

        self.caches = [cache() for _ in range(model.layers)]
        order = np.random.default_rng(0).permutation(n).astype(np.int32)  # pages lie anywhere
        self.pages = self.up(order.reshape(len(prompts), wide))
        for at in range(0, max(len(p) for p in prompts) - 1, CHUNK):  # all but the last token
            rows = [p[at:min(at + CHUNK, len(p) - 1)] for p in prompts]
            self.forward(rows, [list(range(-1, len(r) - 1)) for r in rows])
            self.lens = [n + len(r) for n, r in zip(self.lens, rows)]

    def up(self, a, dtype=np.int32):
        return self.model.torch.from_numpy(np.ascontiguousarray(a, dtype)).to(self.model.device)

    def forward(self, rows, parents):
        """One pass over each sequence's rows; the logits and the batch."""
        shape = [ancestry(p) for p in parents]
        offsets = np.cumsum([0] + [len(r) for r in rows])
        batch = self.model.kq.Batch(self.up(offsets), self.up(self.lens), self.pages)
        positions = self.up([n + d for n, (depth, _) in zip(self.lens, shape) for d in depth])
        mask = self.up(np.array([b for _, bits in shape for b in bits], np.uint64).view(np.int64), np.int64)
        most = max(map(len, rows))
        logits = self.model(self.caches, batch, self.up(sum(rows, [])), positions, mask, most, max(self.lens) + most)
        return logits, batch

    def step(self, trees):
        """Decode one tree a sequence; the log probabilities of the tokens added."""
        kq = self.model.kq
        logits, batch = self.forward([t for t, _ in trees], [p for _, p in trees])
        found = kq.logprobs(logits, n_top=1, entropy=False)
        best, sure = found.top_ids[:, 0].tolist(), found.top_logprobs[:, 0].tolist()
        path, counts, added, at = [], [], [], 0
        for b, (tokens, parents) in enumerate(trees):
            rows = accepted(tokens, parents, best[at:at + len(tokens)])
            path += rows + [0] * (len(tokens) - len(rows))
            counts.append(len(rows))
            self.history[b] += [best[at + r] for r in rows]
            added.append([sure[at + r] for r in rows])
            at += len(tokens)
        kq.cache_keep(self.caches, batch, self.up(path), self.up(counts))
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        return added


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--seqs", type=int, default=4)
    p.add_argument("--prompt", type=int, default=100)
    p.add_argument("--new", type=int, default=64)
    p.add_argument("--cache", choices=("bf16", "f16", "f8"), default="bf16")
    a = p.parse_args(argv)
    model = Model()
    torch = model.torch
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}[a.cache]
    rng = np.random.default_rng(7)
    # prompts that repeat a phrase, so that there is something to look up
    prompts = [np.resize(rng.integers(0, model.vocab, 12), n).tolist() for n in rng.integers(2, a.prompt + 1, a.seqs)]
    for name, branches in (("one token at a time", 0), ("drafted trees", 2)):
        d = Decoder(model, prompts, a.new + CHUNK, dtype=dtype)
        torch.cuda.synchronize()
        start, steps = time.perf_counter(), 0
        while max(len(h) - len(q) for h, q in zip(d.history, prompts)) < a.new:
            d.step([draft(h, branches=branches) for h in d.history])
            steps += 1
        torch.cuda.synchronize()
        s = time.perf_counter() - start
        made = sum(len(h) - len(q) for h, q in zip(d.history, prompts))
        print(f"{name}: {made} tokens in {steps} steps, {made / steps:.2f} a step, {1e3 * s / steps:.2f} ms a step")


if __name__ == "__main__":
    main()
