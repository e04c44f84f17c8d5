"""GPU tests of the step operators at the edges of their ranges: scores far
from zero, probabilities below the type's smallest, more rows than the call
allows, arrays that break the contract, many sequences over shared pages."""
from __future__ import annotations

import math

import numpy as np
import pytest

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


# rows to a key head: one wave (whole sequences and parts), 4 waves, 8 waves
ROWS = [(1, 2), (5, 3), (6, 8), (40, 4)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens,group", ROWS)
@pytest.mark.parametrize("qt,q0,k0", [(BF16, 1.0, 2.0 ** 34), (BF16, 1.0, -2.0 ** 34), (BF16, 2.0 ** 50, -2.0 ** 56),
                                      (BF16, 2.0 ** 50, 2.0 ** 56), (F16, 2.0 ** 15, -2.0 ** 14), (F16, 2.0 ** 15, 2.0 ** 14)],
                         ids=str)
@pytest.mark.parametrize("peak", [False, True])
def test_attn_scores_far_from_zero(kq, dim, tokens, group, qt, q0, k0, peak):
    """Every other token scores all its keys alike at 2^30 to 2^106 either side of
    zero (a value whose product with the scale is rounded): it gets the mean of the
    values it sees, or where one key scores more that key's value.  The rows
    between have ordinary scores over the same keys.

    Equal scores weigh the same, so the weights are exact and what remains is
    fp32's sum of n <= 1400 values: each is off by half of 2^-23 of the sum of
    magnitudes at most, and the sums of a lane or a product are added in fewer than
    128 turns: 2^-17 of it."""
    lens, new = [1300, 0, 70, 129], [tokens, tokens, max(1, tokens // 2), tokens]
    step = Step(tokens + dim, lens, new, 32)
    k, v = (t.float() for t in ref.fill_cache(step, 2, dim, qt))
    k[..., 0] = k0 * (1 + 2.0 ** -6)
    at_peak = [1203, None, 5, 128]
    if peak:
        for b, s in enumerate(at_peak):
            if s is not None:
                p, at = step.where(b, [s])
                k[p, :, at, 0] *= 2.0 if k0 > 0 else 0.5
    k, v = k.to(qt), v.to(qt)
    q = ref.draw(step.rng, (step.M, 2 * group, dim), 0.3)
    far = np.concatenate([np.arange(n) % 2 == 0 for n in new])
    q[far] = 0.0
    q[:, :, 0] = 0.0
    q[far, :, 0] = q0 * (1 + 2.0 ** -7)
    q = q.to(qt)
    bits = np.concatenate([ref.chain_mask(n) for n in new])
    scale = 1.0 / 3.0
    k_near = k.clone()
    k_near[..., 0] = 0.0
    want, bound = ref.attn(step, k_near, v, q, bits, scale)   # (for far rows: the mean over equal scores)
    for b in range(4):
        for i in range(new[b]):
            if i % 2 == 0:
                row = int(step.offsets[b]) + i
                p, at = step.where(b, np.arange(lens[b] + i + 1))
                for h in range(2):
                    vv = v[p, h, :, at].double()
                    if peak and at_peak[b] is not None:
                        vv = vv[at_peak[b]][None]
                    want[row, h * group:(h + 1) * group] = vv.mean(0)
                    bound[row, h * group:(h + 1) * group] = 2.0 ** -17 * vv.abs().mean(0)
    for max_len in (step.max_len, 1 << 14):
        got = kq.attn_tree(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q), scale=scale, max_tokens=tokens,
                           max_len=max_len, out_dtype=F32).cpu().double()
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound)[far].max()


@pytest.mark.parametrize("dim", [64, 128])
def test_attn_short_sequence_scores_far_from_zero(kq, dim):
    """The same where a workgroup takes a short sequence whole."""
    step = Step(1, [700], [1], 64)
    k, v = ref.fill_cache(step, 1, dim, BF16)
    k[..., 0] = -2.0 ** 100
    q = torch.zeros((1, 2, dim))
    q[:, :, 0] = 1.25 * 2.0 ** 5
    got = kq.attn_tree(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q.to(BF16)), scale=0.7, max_tokens=1, max_len=701,
                       out_dtype=F32).cpu().double()
    p, at = step.where(0, np.arange(701))
    vv = v[p, 0, :, at].double()
    assert ((got - vv.mean(0)).abs() <= 2.0 ** -17 * vv.abs().mean(0)).all()


@pytest.mark.parametrize("tokens,group,heads,seqs", [(1, 1, 8, 64), (8, 4, 8, 64), (64, 4, 8, 32)], ids=["one", "rows", "wide"])
def test_attn_f16_small_probabilities_count(kq, tokens, group, heads, seqs):
    """One key 25.05 log2 units above 131071 alike, all values 1: the result is 1,
    although every other probability is below float16's smallest number and
    together they weigh 0.4%.  (All sequences share two pages.)

    A wave holds up to N keys: all of them, or where 4 waves take turns a quarter
    with a dominant key for each.  The dominant one has weight 2^7, exactly; of the
    others each is off by 2^-25 (half the spacing of subnormals), so N 2^-32 of the
    dominant; the sums in fp32 are off by 2^-23 of it at most for every product that
    is added (16 keys with waves of 32 rows, 32 with waves of 16) and for every
    tile of 64 keys that is added to the weights' sum."""
    n, dim, page = 131072, 64, 256
    k = torch.zeros((2, heads, page, dim), dtype=F16)
    few = tokens * group <= 16
    k[1, :, [0, 64, 128, 192] if few else [0], 0] = 1.0
    v = torch.ones((2, heads, dim, page), dtype=F16)
    pages = torch.zeros((seqs, n // page), dtype=torch.int32)
    pages[:, 0] = 1
    q = torch.zeros((seqs * tokens, heads * group, dim), dtype=F16)
    q[..., 0] = 1.0
    batch = kq.Batch(i32(np.arange(seqs + 1) * tokens), i32([n - tokens] * seqs), up(pages))
    got = kq.attn_tree(kq.PagedCache(up(k), up(v)), batch, up(q), scale=25.05 * math.log(2.0), max_tokens=tokens,
                       max_len=n, out_dtype=F32)
    N = n // 4 if few else n
    tol = N * 2.0 ** -32 + N / (32 if few else 16) * 2.0 ** -23 + N / 64 * 2.0 ** -23
    err = (got - 1.0).abs().max().item()
    print(f"{n} keys, {tokens * group} rows: off by {err:.3g} of {tol:.3g}", flush=True)
    assert err <= tol, (err, tol)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens,group", ROWS)
def test_attn_values_near_the_ends_of_the_range(kq, dim, tokens, group):
    """bfloat16 values of 1e38 either sign, whose weighted mean is as far from
    overflow as each of them, and of 1e-30."""
    lens, new = [1300, 0, 129, 2], [tokens, tokens, max(1, tokens // 2), tokens]
    step = Step(tokens + dim, lens, new, 32)
    k, v = ref.fill_cache(step, 2, dim, BF16)
    q = ref.draw(step.rng, (step.M, 2 * group, dim), 1.5).to(BF16)
    bits = np.concatenate([ref.chain_mask(n) for n in new])
    for size in (1e38, 1e-30):
        ends = torch.where(v.isnan(), v, torch.where(v > -1.0, size, -size).to(BF16))
        want, bound = ref.attn(step, k, ends, q, bits, dim ** -0.5)
        for out in (F32, BF16):
            got = kq.attn_tree(kq.PagedCache(up(k), up(ends)), step.batch(kq), up(q), max_tokens=tokens, max_len=step.max_len,
                               out_dtype=out).cpu().double()
            tol = bound if out == F32 else ref.rounded_bound(want, bound, out)
            assert torch.isfinite(got).all()
            assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


@pytest.mark.parametrize("dim,group,T", [(64, 2, 4), (128, 6, 6), (256, 4, 9), (128, 8, 20)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_attn_rows_past_the_bound_are_nan(kq, dim, group, T, out):
    """Rows of a sequence past max_tokens come out as NaN, the others as without
    them, in more sequences than a wave has lanes."""
    rng = np.random.default_rng(T)
    new = rng.integers(0, T + 1, 70)
    new[[0, 31, 66]] = T + 3, T + 1, 2 * T
    step = Step(T, rng.integers(0, 200, 70), new, 16)
    k, v = ref.fill_cache(step, 1, dim, BF16)
    q = ref.draw(step.rng, (step.M, group, dim)).to(BF16)
    bits = np.concatenate([ref.chain_mask(min(int(n), 64)) for n in new])
    past = np.concatenate([np.arange(n) >= T for n in new])
    want, bound = ref.attn(step, k, v, q, bits, dim ** -0.5)
    whole = torch.full((step.M + 2, group, dim), 7.0, dtype=out, device=DEV)
    kq.attn_tree(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q), max_tokens=T, max_len=step.max_len, out=whole[1:-1])
    got = whole.cpu().double()
    assert (got[[0, -1]] == 7).all()
    got = got[1:-1]
    assert torch.isnan(got[past]).all()
    tol = bound if out == F32 else ref.rounded_bound(want, bound, out)
    assert ((got - want).abs() <= tol)[~past].all()


@pytest.mark.parametrize("dim,kvt", [(64, F16), (128, F8), (256, BF16)])
@pytest.mark.parametrize("M", [40, 12000])
def test_append_and_keep_stay_inside(kq, dim, kvt, M):
    """Offsets, lengths, pages, positions, paths and counts of nonsense, in a small
    step and in one of whole tiles: what lies before and behind the cache and the
    queries keeps its canaries."""
    heads, q_heads, page, n = 2, 4, 16, 3
    qt = BF16 if kvt == F8 else kvt

    def guarded(shape, dtype):
        pad = 64 * page   # rows of the shape's last dimension's neighbours on each side, a multiple of 16 bytes
        size = math.prod(shape)
        whole = torch.full((size + 2 * pad,), 7.0, dtype=F32, device=DEV).to(dtype)
        return whole, whole[pad:pad + size].view(shape)

    def untouched(whole, inner):
        pad = (whole.numel() - inner.numel()) // 2
        return bool((whole[:pad].float() == 7).all()) and bool((whole[-pad:].float() == 7).all())

    low, high = -2 ** 31, 2 ** 31 - 1
    arrays = [([0, 50, 3], [-9, 1 << 30], [[77, -3]] * 2),
              ([5, -5, 1 << 30], [high, low], [[0, high]] * 2),
              ([0, M // 2, M], [high, high], [[low, high]] * 2),
              ([0, M // 2, M], [(1 << 30) + 1, high - M // 4], [[2, 1]] * 2),
              ([high, low, high], [31, 17], [[high, 1]] * 2),
              ([-3, -2, -1], [0, 31], [[-1, 3]] * 2)]
    x = torch.ones((M, (q_heads + 2 * heads) * dim), device=DEV)
    rope = torch.ones((5, dim), device=DEV)
    for off, lens, pages in arrays:
        print(off, lens, pages, flush=True)
        guards = [guarded((n, heads, page, dim), kvt), guarded((n, heads, dim, page), kvt), guarded((M, q_heads, dim), qt)]
        (_, k), (_, v), (_, q) = guards
        cache, batch = kq.PagedCache(k, v), kq.Batch(i32(off), i32(lens), i32(pages))
        for positions in (None, i32(([high, low, -1, 5] * M)[:M])):
            kq.rope_append(cache, batch, x, q_heads, rope, positions, out=q)
        torch.cuda.synchronize()
        assert all(untouched(*g) for g in guards)
        path = i32(([high, low, -1, 5, M] * M)[:M])
        for counts in ([90, 3], [high, low], [64, 64]):
            kq.cache_keep([cache], batch, path, i32(counts))
        torch.cuda.synchronize()
        assert all(untouched(*g) for g in guards)


@pytest.mark.parametrize("group,dim,qt,kvt", [(6, 128, BF16, BF16), (3, 64, F16, F8), (1, 256, BF16, BF16)])
def test_attn_prompts_as_sequences_over_their_pages(kq, group, dim, qt, kvt):
    """Prompts whose rows are all in the cache attend 64 at a time: sequence i of
    a prompt has its pages, 64 i more cached tokens and the next 64 rows.  85 such
    sequences are more than a wave has lanes, and 64 rows of 6 heads more than a
    workgroup takes at once."""
    lens, new, rows = [37, 0, 300], [4400, 200, 731], 64
    step = Step(group, lens, new, 64)
    k, v = ref.fill_cache(step, 1, dim, kvt)
    q = ref.draw(step.rng, (step.M, group, dim), 1.5).to(qt)
    offsets, cached, pages = [0], [], []
    for b, n in enumerate(new):
        for i in range(0, n, rows):
            cached.append(lens[b] + i)
            pages.append(step.pages[b])
            offsets.append(offsets[-1] + min(rows, n - i))
    assert len(cached) > 64 and offsets[-1] == step.M
    batch = kq.Batch(i32(offsets), i32(cached), up(np.stack(pages)))
    got = kq.attn_tree(kq.PagedCache(up(k), up(v), 0.5, 0.25), batch, up(q), max_len=step.max_len, out_dtype=F32).cpu().double()
    for b, n in enumerate(new):
        L = lens[b] + n
        p, at = step.where(b, np.arange(L))
        kk, vv = 0.5 * k[p, 0, at].double(), 0.25 * v[p, 0, :, at].double()
        unseen = torch.arange(L)[None] > lens[b] + torch.arange(n)[:, None]
        for h in range(group):
            qq = q[step.rows(b), h].double()
            score = qq @ kk.t()
            most = (qq.abs() @ kk.abs().t()).amax() * dim ** -0.5
            w = (score * dim ** -0.5).masked_fill_(unseen, -math.inf).softmax(-1)
            # (the terms of step_ref.attn's bound)
            rel = ref.ROUND[qt] + 2.0 ** -24 * (dim + 16) * (1.0 + float(most)) + 2.0 ** -18
            bound = rel * (w @ vv.abs()) + ref.TINY[qt] * L * vv.abs().amax()
            assert ((got[step.rows(b), h] - w @ vv).abs() <= bound).all(), (b, h)
