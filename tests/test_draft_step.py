"""Decoding with drafted tokens: the trees on the host, and the operators of a
step together on the GPU against the same tokens read one after another."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import draft_step as ds  # noqa: E402


def test_draft_looks_up_and_shares():
    #          0  1  2  3  4  5  6  7
    history = [5, 1, 2, 5, 1, 3, 9, 5]
    assert ds.draft(history, 2, 2) == ([5, 1, 3, 2], [-1, 0, 1, 1])
    assert ds.draft(history, 3, 1) == ([5, 1, 3, 9], [-1, 0, 1, 2])
    assert ds.draft(history, 4, 0) == ([5], [-1])
    assert ds.draft([7], 4, 2) == ([7], [-1])
    assert ds.draft([7, 8], 4, 2) == ([8], [-1])
    assert ds.draft([4, 4], 4, 2) == ([4, 4], [-1, 0])


def test_ancestry_and_acceptance():
    tokens, parents = [5, 1, 3, 2, 6], [-1, 0, 1, 1, 3]
    assert ds.ancestry(parents) == ([0, 1, 2, 2, 3], [1, 3, 7, 11, 27])
    assert ds.accepted(tokens, parents, [1, 2, 0, 6, 8]) == [0, 1, 3, 4]
    assert ds.accepted(tokens, parents, [1, 9, 0, 6, 8]) == [0, 1]
    assert ds.accepted(tokens, parents, [2, 2, 0, 6, 8]) == [0]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float8_e4m3fn"])
def test_drafted_decoding_is_greedy_decoding(kind):
    """What drafted steps produce is read again as prompts, in chunks, into other
    caches: every token is the best one there but for rounding, and its log
    probability the same.

    Logits have mean square 9.  What differs between the two runs is the order of
    fp32 sums, which moves some activations to the next of 255 steps (and in the
    caches to the next value): a step is 1/127 of its block's largest, some 2.5
    deviations for these, so at most 2% of a deviation on an element and, spread
    over a row's elements by independent weights, 2% of a deviation on a logit if
    every element moved, at each of some 8 products one after another: 0.02 * 3 *
    sqrt(8) = 0.17; an 8-bit cache has steps of an eighth, in each of two layers:
    0.53 more.  Foreign or misplaced keys move logits by their own size."""
    torch = pytest.importorskip("torch")
    model = ds.Model()
    rng = np.random.default_rng(3)
    prompts = [np.resize(rng.integers(0, model.vocab, 9), n).tolist() for n in (1, 2, 40, 65, 150)]
    dtype = getattr(torch, kind)
    bound = 0.70 if dtype == torch.float8_e4m3fn else 0.17
    d = ds.Decoder(model, prompts, 400, page=16, dtype=dtype)
    sure = [[] for _ in prompts]
    drafted = 0
    for _ in range(60):
        trees = [ds.draft(h) for h in d.history]
        drafted += sum(len(t) - 1 for t, _ in trees)
        for s, new in zip(sure, d.step(trees)):
            s += new
    made = [len(h) - len(p) for h, p in zip(d.history, prompts)]
    assert made == [len(s) for s in sure] and d.lens == [len(h) - 1 for h in d.history]
    assert drafted > 100 and sum(made) > 60 * len(prompts)  # something was drafted, and some of it accepted

    again = ds.Decoder(model, [[h[0]] for h in d.history], 800, page=32, dtype=dtype)
    at = 0
    while at < max(map(len, d.history)) - 1:
        rows = [h[at:min(at + ds.CHUNK, len(h) - 1)] for h in d.history]
        logits, _ = again.forward(rows, [list(range(-1, len(r) - 1)) for r in rows])
        next_tokens = [t for h, r in zip(d.history, rows) for t in h[at + 1:at + 1 + len(r)]]
        found = model.kq.logprobs(logits, again.up(next_tokens)[:, None], n_top=1)
        row = 0
        for b, r in enumerate(rows):
            for i in range(len(r)):
                k = at + i + 1 - len(prompts[b])  # which of the made tokens
                if k >= 0:
                    lp, top = found.logprob[row + i, 0].item(), found.top_logprobs[row + i, 0].item()
                    assert lp >= top - 2 * bound, (b, k, lp, top)
                    assert abs(lp - sure[b][k]) <= bound, (b, k, lp, sure[b][k])
            row += len(r)
        again.lens = [n + len(r) for n, r in zip(again.lens, rows)]
        at += ds.CHUNK
