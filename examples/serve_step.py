"""Serving requests with adapters of their own: prompts and single tokens in one step.

A step takes a piece of the text of every request: the next part of its prompt while
that lasts, then one token at a time.  Each layer adds its parts to a running sum
and norms and quantizes it in one pass (norm_quantize), multiplies by the shared Q4_K
weights and adds every request's adapter (kq_gemm, lora), stores keys and values
(rope_append) and attends over the cache, however many rows a request brings
(attn_chunk), under a window with a few first tokens if the model has one.

    python examples/serve_step.py [--requests 6] [--prompt 300] [--new 32] [--piece 128] [--window 0] [--sinks 4]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import draft_step  # noqa: E402


class Model(draft_step.Model):
    """The decoder of draft_step.py with an adapter on the first product of each layer, and
    attention under a window (0: none)."""

    def __init__(self, adapters=4, rank=16, window=0, sinks=0, seed=1, **sizes):
        super().__init__(seed=seed, **sizes)
        torch = self.torch
        rng = np.random.default_rng(seed + 17)
        self.window, self.sinks = window, sinks

        def up(*shape):
            scale = 1.0 / np.sqrt(shape[-1])
            return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(self.device).bfloat16()

        self.A = [up(adapters, rank, k) for _, k, _ in self.qkv]
        self.B = [up(adapters, n, rank) for n, _, _ in self.qkv]
        self.scale = torch.from_numpy(rng.uniform(0.5, 1.0, adapters).astype(np.float32)).to(self.device)

    def times(self, a_q8, rows, w):
        n, k, data = w
        return self.kq.gemm(self.kq.KQ_Q4_K, data, a_q8, rows, n, k)

    def __call__(self, caches, batch, tokens, ids, max_tokens, max_len):
        """Logits [rows][vocab]; the rows' keys and values are in the caches after it.
        ids: the adapter of each row (none: below 0)."""
        kq, rows, act = self.kq, tokens.shape[0], self.torch.nn.functional.silu
        total = self.embed[tokens.long()]   # the running sum
        part = self.torch.zeros_like(total)
        for i in range(self.layers):
            a = kq.norm_quantize(part, total)
            qkv = self.times(a, rows, self.qkv[i])
            kq.lora(a, self.A[i], self.B[i], ids, self.scale, base=qkv, out=qkv)
            q = kq.rope_append(caches[i], batch, qkv, self.q_heads, self.rope, None, self.ones, self.ones)
            o = kq.attn_chunk(caches[i], batch, q, self.window, self.sinks, max_tokens=max_tokens, max_len=max_len,
                              out_dtype=self.torch.float32)
            part = self.norm(self.product(o.flatten(1), self.o[i]))
            gate, up = self.times(kq.norm_quantize(part, total), rows, self.up[i]).chunk(2, 1)
            part = self.norm(self.product(act(self.norm(gate)) * up, self.down[i]))
        return 3.0 * self.norm(self.times(kq.norm_quantize(part, total), rows, self.head))


class Server:
    """Requests and their pages; the lengths are kept on the host, too."""

    def __init__(self, model, prompts, adapters, room, page=64, dtype=None):
        torch, kq = model.torch, model.kq
        self.model = model
        self.text = [list(p) for p in prompts]
        self.prompt = [len(p) for p in prompts]
        self.adapters = list(adapters)
        self.lens = [0] * len(prompts)
        wide = -(-max(n + room for n in self.prompt) // page)
        n = wide * len(prompts)
        dtype = dtype or torch.bfloat16
        scale = 0.05 if dtype == torch.float8_e4m3fn else 1.0  # (8 bits: up to 448 times it)

        def cache():
            k = torch.zeros((n, model.heads, page, model.dim), device=model.device).to(dtype)
            return kq.PagedCache(k, k.view(n, model.heads, model.dim, page).clone(), scale, scale)

        self.caches = [cache() for _ in range(model.layers)]
        order = np.random.default_rng(0).permutation(n).astype(np.int32)  # pages lie anywhere
        self.pages = self.up(order.reshape(len(prompts), wide))

    def up(self, a):
        return self.model.torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(self.model.device)

    def forward(self, pieces):
        """One pass over the next `pieces[b]` tokens of each request; the logits."""
        rows = [t[n:n + m] for t, n, m in zip(self.text, self.lens, pieces)]
        batch = self.model.kq.Batch(self.up(np.cumsum([0] + pieces)), self.up(self.lens), self.pages)
        most = max(pieces)
        logits = self.model(self.caches, batch, self.up(sum(rows, [])), self.up(np.repeat(self.adapters, pieces)), most,
                            max(n + m for n, m in zip(self.lens, pieces)))
        self.lens = [n + m for n, m in zip(self.lens, pieces)]
        return logits

    def step(self, piece, new):
        """The next piece of every request that is not done (`new` tokens after its prompt); the
        log probabilities of the tokens added, by request."""
        left = [len(t) - n for t, n in zip(self.text, self.lens)]
        done = [len(t) - p >= new for t, p in zip(self.text, self.prompt)]
        pieces = [0 if d else min(m, piece) for m, d in zip(left, done)]
        logits = self.forward(pieces)
        found = self.model.kq.logprobs(logits, n_top=1, entropy=False)
        best, sure = found.top_ids[:, 0].tolist(), found.top_logprobs[:, 0].tolist()
        added, at = {}, 0
        for b, m in enumerate(pieces):
            at += m
            if m and self.lens[b] == len(self.text[b]):  # its last token so far was read: the next one
                self.text[b].append(best[at - 1])
                added[b] = sure[at - 1]
        return added


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--requests", type=int, default=6)
    p.add_argument("--prompt", type=int, default=300)
    p.add_argument("--new", type=int, default=32)
    p.add_argument("--piece", type=int, default=128)
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=4)
    a = p.parse_args(argv)
    model = Model(window=a.window, sinks=a.sinks)
    rng = np.random.default_rng(7)
    prompts = [rng.integers(0, model.vocab, n).tolist() for n in rng.integers(1, a.prompt + 1, a.requests)]
    server = Server(model, prompts, [i % 5 - 1 for i in range(a.requests)], a.new)
    model.torch.cuda.synchronize()
    start, steps, made = time.perf_counter(), 0, 0
    while any(len(t) - n < a.new for t, n in zip(server.text, server.prompt)):
        made += len(server.step(a.piece, a.new))
        steps += 1
    s = time.perf_counter() - start
    print(f"{sum(server.prompt)} prompt tokens and {made} new ones in {steps} steps, {1e3 * s / steps:.2f} ms a step")


if __name__ == "__main__":
    main()
