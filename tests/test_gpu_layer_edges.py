"""GPU tests of the operators around the products of a layer at the edges of their ranges:
scores far from zero, probabilities below the type's smallest, values near the ends of
the range, the bits of lora's second product, workspaces that hold anything."""
from __future__ import annotations

import math

import numpy as np
import pytest

import layer_edge_ref as eref
import layer_ref as lref
import step_ref as ref
from step_ref import BF16, F16, F32, F8, Step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def kq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_act_amd as kq
    kq.lib()
    return kq


def up(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(DEV)


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------- lora

@pytest.mark.parametrize("t", [BF16, F16], ids=str)
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("M,N", [(3, 150), (300, 150), (600, 152)])
@pytest.mark.parametrize("act,K", [(1, 1024), (2, 640)], ids=["q8_k", "q8_128"])
def test_lora_second_product_keeps_24_bits(kq, t, rank, M, N, act, K):
    """The first product exact, the second against the additions alone: by either kernel, with
    rows of N that are 16-byte aligned and not, one value of B to an output and all."""
    bs = 256 if act == 1 else 128
    for dense in (False, True):
        rng = np.random.default_rng(rank + M + dense)
        A, B, scale, ids, base, picked = eref.pick_case(rng, M, N, rank, K, 3, t, dense)
        a = kq.quantize_act(up(ref.draw(rng, (M, K))), act)
        qs, d, _ = kq.act_views(a, act, M, K)
        want, bound = eref.second(eref.picked_t(qs.cpu(), d.cpu(), bs, scale, ids, picked), B, ids, base, dense)
        got = kq.lora(a, up(A), up(B), up(ids), up(scale), base=up(base), act_fmt=act).cpu().double()
        # (the result is rounded once more: 2^-24 of it)
        assert ((got - want).abs() <= bound + 2.0 ** -24 * want.abs()).all(), ((got - want).abs() / (bound + 1e-300)).max()


@pytest.mark.parametrize("M", [7, 300])
@pytest.mark.parametrize("rank", [16, 128])
def test_lora_workspace_may_hold_anything(kq, M, rank):
    """The same bits whatever lies in the workspace, rows without an adapter among them."""
    N, K, n = 100, 512, 3
    rng = np.random.default_rng(M)
    a = kq.quantize_act(up(ref.draw(rng, (M, K))), 1)
    A, B = up(ref.draw(rng, (n, rank, K), 0.05).to(BF16)), up(ref.draw(rng, (n, N, rank), 0.25).to(BF16))
    ids, base = up((np.arange(M) % 5 - 1).astype(np.int32)), up(ref.draw(rng, (M, N)))
    need = kq.kq_lora_workspace(rank, M)
    outs = []
    for fill in (0.0, math.nan, math.inf, -3e38):
        work, out = torch.full((need // 4,), fill, device=DEV), torch.full((M, N), math.nan, device=DEV)
        kq.kq_lora(kq.KQ_T_BF16, rank, A, B, None, n, 1, a, M, N, K, ids, base, N, out, N, work, need)
        outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("t", [BF16, F16], ids=str)
@pytest.mark.parametrize("M,rank", [(3, 16), (600, 8), (300, 64), (70, 128)])
def test_lora_values_between_the_products_at_the_end_of_the_range(kq, t, M, rank):
    """t up to 3.4e38, past the largest bfloat16 but not past fp32, and adapters that bring it back:
    finite, and as near as anywhere."""
    N, K, n = 150, 512, 3
    rng = np.random.default_rng(rank)
    A, B, _, ids, _, picked = eref.pick_case(rng, M, N, rank, K, n, t, dense=False)
    B = (B.float() * 2.0 ** -10).to(t)
    x = torch.from_numpy((3.402e38 * rng.choice([-1.0, 1.0, 0.999, -0.5], (M, K))).astype(np.float32))
    a = kq.quantize_act(up(x), 1)
    qs, d, _ = kq.act_views(a, 1, M, K)
    middle = eref.picked_t(qs.cpu(), d.cpu(), 256, torch.ones(n), ids, picked)
    assert torch.isfinite(middle).all() and (middle.abs() > 3.397e38).any()
    want, bound = eref.second(middle, B, ids, torch.zeros(M, N), dense=False)
    got = kq.lora(a, up(A), up(B), up(ids)).cpu().double()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()


# ----------------------------------------------------------------- attn_chunk

# rows to a key head: the kernels for few, for blocks of 128 and of 256 (heads of 256: 128 too)
ROWS = [(1, 2), (5, 3), (6, 8), (40, 4), (90, 4)]


def far_step(tokens, dim):
    return Step(tokens + dim, [1300, 0, 70, 129], [tokens, tokens, max(1, tokens // 2), tokens], 32)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens,group", ROWS)
@pytest.mark.parametrize("qt,kvt,q0,k0", [(BF16, BF16, 1.0, 2.0 ** 34), (BF16, BF16, 1.0, -2.0 ** 34), (BF16, BF16, 2.0 ** 50, -2.0 ** 56),
                                          (BF16, BF16, 2.0 ** 50, 2.0 ** 56), (F16, F16, 2.0 ** 15, -2.0 ** 14),
                                          (F16, F16, 2.0 ** 15, 2.0 ** 14), (BF16, F8, 2.0 ** 50, 2.0 ** 7),
                                          (BF16, BF16, 1.0, 2.0 ** 22), (F16, F16, 2.0 ** 10, -2.0 ** 13)], ids=str)
@pytest.mark.parametrize("peak", [False, True])
def test_chunk_scores_far_from_zero(kq, dim, tokens, group, qt, kvt, q0, k0, peak):
    """Every other token scores all its keys alike at 2^20 to 2^106 either side of zero (a value
    whose product with the scale is rounded): it gets the mean of the values it sees, or where
    one key scores more that key's value.  The rows between have ordinary scores over the same
    keys.

    Equal scores weigh the same, so the weights are exact and what remains is fp32's sum of
    n <= 1400 values: each is off by half of 2^-23 of the sum of magnitudes at most, and the
    sums of a lane or a product are added in fewer than 128 turns: 2^-17 of it."""
    step = far_step(tokens, dim)
    k, v = (t.float() for t in ref.fill_cache(step, 2, dim, kvt))
    k[..., 0] = k0 * (1 + (2.0 ** -3 if kvt == F8 else 2.0 ** -6))
    at_peak = [1203, None, 5, 128]
    if peak:
        for b, s in enumerate(at_peak):
            if s is not None:
                p, at = step.where(b, [s])
                k[p, :, at, 0] *= 2.0 if k0 > 0 else 0.5
    k, v = k.to(kvt), v.to(kvt)
    q = ref.draw(step.rng, (step.M, 2 * group, dim), 0.3)
    far = np.concatenate([np.arange(n) % 2 == 0 for n in step.new])
    q[far] = 0.0
    q[:, :, 0] = 0.0
    q[far, :, 0] = q0 * (1 + 2.0 ** -7)
    q = q.to(qt)
    scale = 1.0 / 3.0
    k_near = k.clone()
    k_near[..., 0] = 0.0
    want, bound = lref.chunk(step, k_near, v, q, 0, 0, scale)   # (for far rows: the mean over equal scores)
    for b in range(4):
        for i in range(0, int(step.new[b]), 2):
            row = int(step.offsets[b]) + i
            p, at = step.where(b, np.arange(step.lens[b] + i + 1))
            for h in range(2):
                vv = v[p, h, :, at].double()
                if peak and at_peak[b] is not None and at_peak[b] <= step.lens[b] + i:
                    vv = vv[at_peak[b]][None]
                want[row, h * group:(h + 1) * group] = vv.mean(0)
                bound[row, h * group:(h + 1) * group] = 2.0 ** -17 * vv.abs().mean(0)
    for max_len in (step.max_len, 1 << 14):
        got = kq.attn_chunk(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q), scale=scale, max_tokens=tokens,
                            max_len=max_len, out_dtype=F32).cpu().double()
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound).max()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens,group", ROWS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (333, 7)])
def test_chunk_values_near_the_ends_of_the_range(kq, dim, tokens, group, window, sinks):
    """bfloat16 values of 1e38 either sign, whose weighted mean is as far from overflow as
    each of them, and of 1e-30."""
    step = far_step(tokens, dim)
    k, v = ref.fill_cache(step, 2, dim, BF16)
    q = ref.draw(step.rng, (step.M, 2 * group, dim), 1.5).to(BF16)
    for size in (1e38, 1e-30):
        ends = torch.where(v.isnan(), v, torch.where(v > -1.0, size, -size).to(BF16))
        want, bound = lref.chunk(step, k, ends, q, window, sinks, dim ** -0.5)
        for max_len, out in ((step.max_len, F32), (1 << 14, F32), (step.max_len, BF16)):
            got = kq.attn_chunk(kq.PagedCache(up(k), up(ends)), step.batch(kq), up(q), window, sinks, max_tokens=tokens,
                                max_len=max_len, out_dtype=out).cpu().double()
            tol = bound if out == F32 else ref.rounded_bound(want, bound, out)
            assert torch.isfinite(got).all()
            assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


@pytest.mark.parametrize("tokens,group,heads,seqs,dim", [(1, 1, 8, 64, 64), (8, 4, 8, 64, 64), (64, 4, 8, 16, 128), (33, 4, 4, 16, 256)],
                         ids=["one", "rows", "wide", "wide256"])
def test_chunk_f16_small_probabilities_count(kq, tokens, group, heads, seqs, dim):
    """One key 25.05 log2 units above 131071 alike, all values 1: the result is 1, although every
    other probability is below float16's smallest number and together they weigh 0.4%.  (All
    sequences share two pages.)

    The weights are summed as they were rounded, so their roundings leave a mean of ones alone;
    what is left are fp32's sums, off by 2^-23 of the whole for every product that is added (16
    keys at least) and for every pair of weights and every 32 that are added to their sum, over
    n keys.  (Small probabilities that one sum holds and the other does not would show as up
    to 0.4%.)"""
    n, page = 131072, 256
    k = torch.zeros((2, heads, page, dim), dtype=F16)
    k[1, :, 0, 0] = 1.0
    v = torch.ones((2, heads, dim, page), dtype=F16)
    pages = torch.zeros((seqs, n // page), dtype=torch.int32)
    pages[:, 0] = 1
    q = torch.zeros((seqs * tokens, heads * group, dim), dtype=F16)
    q[..., 0] = 1.0
    batch = kq.Batch(i32(np.arange(seqs + 1) * tokens), i32([n - tokens] * seqs), up(pages))
    tol = (n / 16 + n / 32 + 64) * 2.0 ** -23
    assert tol < 0.002   # (half of what the small ones weigh)
    for max_len in (n, 1000):
        got = kq.attn_chunk(kq.PagedCache(up(k), up(v)), batch, up(q), scale=25.05 * math.log(2.0), max_tokens=tokens,
                            max_len=max_len, out_dtype=F32)
        err = (got - 1.0).abs().max().item()
        print(f"{n} keys, {tokens * group} rows: off by {err:.3g} of {tol:.3g}", flush=True)
        assert err <= tol, (err, tol)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("qt,kvt", [(BF16, BF16), (F16, F16), (BF16, F8)], ids=str)
def test_chunk_equals_tree_within_their_roundings(kq, dim, qt, kvt):
    """Up to 64 rows that see all before them: what attn_tree computes, each element within the
    bounds of the two."""
    step = Step(4, [0, 77, 500, 1200], [64, 1, 30, 3], 32)
    k, v = ref.fill_cache(step, 2, dim, kvt)
    q = ref.draw(step.rng, (step.M, 8, dim), 1.5).to(qt)
    bits = np.concatenate([ref.chain_mask(int(n)) for n in step.new])
    _, tree_bound = ref.attn(step, k, v, q, bits, dim ** -0.5)
    _, chunk_bound = lref.chunk(step, k, v, q, 0, 0, dim ** -0.5)
    cache, batch, dq = kq.PagedCache(up(k), up(v)), step.batch(kq), up(q)
    tree = kq.attn_tree(cache, batch, dq, max_tokens=64, max_len=step.max_len, out_dtype=F32).cpu().double()
    for max_len in (step.max_len, 40000):
        got = kq.attn_chunk(cache, batch, dq, max_tokens=64, max_len=max_len, out_dtype=F32).cpu().double()
        assert ((tree - got).abs() <= tree_bound + chunk_bound).all(), ((tree - got).abs() / (tree_bound + chunk_bound)).max()


@pytest.mark.parametrize("tokens,group,dim,kvt", [(1, 4, 128, BF16), (1, 8, 256, BF16), (30, 4, 64, BF16), (40, 4, 128, F8), (90, 4, 128, BF16),
                                                  (90, 4, 256, BF16), (20, 4, 256, F8)])
def test_chunk_workspace_may_hold_anything(kq, tokens, group, dim, kvt):
    """The same bits whatever lies in the workspace, for sequences that are cut, whole and
    empty; rows of no sequence keep what they held."""
    step = Step(13, [5000, 0, 129, 2047, 40], [tokens, tokens, 0, 1, max(1, tokens // 2)], 32)
    k, v = ref.fill_cache(step, 2, dim, kvt)
    cache, batch = kq.PagedCache(up(k), up(v)), step.batch(kq)
    M, hq = step.M + 5, 2 * group
    q = up(ref.draw(step.rng, (M, hq, dim)).to(BF16))
    rows, scale = batch.of(M), dim ** -0.5
    want, bound = lref.chunk(step, k, v, q[:step.M].cpu(), 0, 0, scale)
    need = kq.kq_attn_chunk_workspace(cache.c, rows, hq, 0, 0, tokens, 40000)
    assert need > 0
    outs = []
    for fill in (0, 0xFF, 0x7F):   # (NaN, and 3.4e38 or a count near 2^31)
        work = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        out = torch.full((M, hq, dim), 3.0, device=DEV)
        kq.kq_attn_chunk(cache.c, rows, kq.KQ_T_BF16, q, hq, 0, 0, scale, tokens, 40000, kq.KQ_T_F32, out, work, need)
        torch.cuda.synchronize()
        outs.append(out)
        assert ((out[:step.M].cpu().double() - want).abs() <= bound).all()
        assert (out[step.M:] == 3).all()
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 9, 40, 150])
@pytest.mark.parametrize("qt,kvt", [(BF16, BF16), (F16, F8)], ids=str)
def test_chunk_pages_of_wide_heads(kq, page, tokens, qt, kvt):
    """Heads of 256 over pages of every size, ends of sequences around the ends of pages."""
    step = Step(page, [3, page - 1, page, page + 1, 2 * page + 5, 700], [tokens] * 6, page)
    k, v = ref.fill_cache(step, 2, 256, kvt)
    q = ref.draw(step.rng, (step.M, 6, 256), 1.5).to(qt)
    cache, batch, dq = kq.PagedCache(up(k), up(v)), step.batch(kq), up(q)
    for window, sinks in ((0, 0), (100, 20)):
        want, bound = lref.chunk(step, k, v, q, window, sinks, 1 / 16)
        for max_len in (step.max_len, 5000, 40000):
            got = kq.attn_chunk(cache, batch, dq, window, sinks, max_tokens=tokens, max_len=max_len, out_dtype=F32).cpu().double()
            assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound).max()
