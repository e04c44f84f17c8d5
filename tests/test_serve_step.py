"""norm_quantize, lora and attn_chunk together, as a server uses them: prompts in pieces
beside single tokens, against the same texts read whole."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float8_e4m3fn"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_pieces_are_the_whole(kind, window, sinks):
    """What a server made in pieces is read again by another, every text in one piece and with
    other pages: each token is the best one there but for rounding, and its log probability the
    same.

    Logits have mean square 9.  What differs between the two runs is the order of fp32 sums and
    the places where probabilities are rounded, which moves some activations to the next of 255
    steps (and in the caches to the next value): a step is 1/127 of its block's largest, some 2.5
    deviations for these, so at most 2% of a deviation on an element and, spread over a row's
    elements by independent weights, 2% of a deviation on a logit if every element moved, at each of
    some 8 products one after another: 0.02 * 3 * sqrt(8) = 0.17; an 8-bit cache has steps of an
    eighth, in each of two layers: 0.53 more.  Foreign or misplaced keys, another request's
    adapter or another window move logits by their own size."""
    torch = pytest.importorskip("torch")
    import serve_step as ss
    model = ss.Model(window=window, sinks=sinks)
    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, model.vocab, n).tolist() for n in (1, 2, 40, 65, 150, 333)]
    adapters = [0, -1, 3, 1, 0, 2]
    dtype = getattr(torch, kind)
    bound = 0.70 if dtype == torch.float8_e4m3fn else 0.17
    kq = model.kq
    kq.kq_layer_count_reset()
    server = ss.Server(model, prompts, adapters, 40, page=16, dtype=dtype)
    sure = [[] for _ in prompts]
    steps = 0
    while any(len(t) - n < 24 for t, n in zip(server.text, server.prompt)):
        for b, lp in server.step((50, 7, 128)[steps % 3], 24).items():
            sure[b].append(lp)
        steps += 1
    assert [len(t) - n for t, n in zip(server.text, server.prompt)] == [24] * 6 == [len(s) for s in sure]
    counts = kq.layer_counts()
    assert counts["norm_quantize"] and counts["chunk_few"] and counts["chunk_rows"] and counts["lora_few"]

    again = ss.Server(model, [t[:-1] for t in server.text], adapters, 1, page=64, dtype=dtype)
    pieces = [len(t) for t in again.text]
    logits = again.forward(pieces)
    assert logits.shape[0] * 16 > 4096 and kq.layer_counts()["lora_tile"] == model.layers
    nexts = sum((t[1:] for t in server.text), [])
    found = kq.logprobs(logits, again.up(nexts)[:, None], n_top=1)
    at = 0
    for b, m in enumerate(pieces):
        for k, lp_made in enumerate(sure[b]):
            row = at + len(prompts[b]) - 1 + k
            lp, top = found.logprob[row, 0].item(), found.top_logprobs[row, 0].item()
            assert lp >= top - 2 * bound, (b, k, lp, top)
            assert abs(lp - lp_made) <= bound, (b, k, lp, lp_made)
        at += m
    # another adapter gives another text's probabilities
    other = ss.Server(model, [t[:-1] for t in server.text], [a + 1 for a in adapters], 1, page=64, dtype=dtype)
    moved = (other.forward(pieces) - logits).abs().max(-1).values
    assert (moved > 2 * bound).float().mean() > 0.5


@pytest.mark.gpu
def test_example_runs(capsys):
    import serve_step as ss
    ss.main(["--requests", "3", "--prompt", "90", "--new", "3", "--piece", "64", "--window", "30"])
    assert "in " in capsys.readouterr().out
