"""GPU tests of the operators between two products of a layer (rope_append,
attn_tree, cache_keep, logprobs) against plain 64-bit forms on the CPU.

Tolerances follow from the types (tests/step_ref.py): half a unit in the last
place of the result, what rounding the probabilities to q's type can change,
and fp32 sums.
"""
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


def say(*a):
    print(*a, flush=True)


def up(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(DEV)


def masks(bits):
    return up(bits.view(np.int64))


# ------------------------------------------------------------------ attention

def check_attn(kq, step, hq, hkv, dim, qt, kvt, mask, k=None, v=None, k_scale=1.0, v_scale=1.0, max_len=None, scale=None):
    """One call in q's type and one in float32 against the plain form."""
    if k is None:
        k, v = ref.fill_cache(step, hkv, dim, kvt)
    q = ref.draw(step.rng, (step.M, hq, dim), 1.5).to(qt)
    scale = dim ** -0.5 if scale is None else scale
    bits = ref.chain_mask(64)[np.concatenate([np.arange(n) for n in step.new]).astype(int)] if mask is None else mask
    want, bound = ref.attn(step, k, v, q, bits, scale, k_scale, v_scale)
    cache, batch = kq.PagedCache(up(k), up(v), k_scale, v_scale), step.batch(kq)
    worst = 0.0
    for out_dtype in (qt, F32):
        got = torch.full((step.M, hq, dim), math.nan, dtype=out_dtype, device=DEV)
        kq.attn_tree(cache, batch, up(q), None if mask is None else masks(mask), scale=scale,
                     max_tokens=max(1, step.max_new), max_len=max_len or step.max_len, out=got)
        torch.cuda.synchronize()
        got = got.cpu().double()
        tol = bound if out_dtype == F32 else ref.rounded_bound(want, bound, out_dtype)
        assert torch.isfinite(got).all(), (out_dtype, int((~torch.isfinite(got)).sum()))
        err = ((got - want).abs() / tol.clamp(min=1e-30)).max().item() if got.numel() else 0.0
        assert ((got - want).abs() <= tol).all(), (out_dtype, err)
        worst = max(worst, err)
    return worst


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300]


@pytest.mark.parametrize("qt,kvt", [(BF16, BF16), (F16, F16), (BF16, F8), (F16, F8)], ids=["bf16", "f16", "bf16-f8", "f16-f8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,tokens", [(1, 1), (4, 1), (16, 1), (3, 5), (2, 16), (4, 16), (8, 21), (1, 64)])
def test_attn_lengths_and_rows(kq, qt, kvt, dim, group, tokens):
    """Every length around the tiles' and pages' ends in one ragged batch, with
    each split of the rows over waves and workgroups."""
    rng = np.random.default_rng(dim + group * 7 + tokens)
    new = [tokens] + [int(n) for n in rng.integers(0 if tokens > 1 else 1, tokens + 1, len(LENS) - 1)]
    step = Step(11 + tokens, LENS, new, (16, 32, 64)[dim // 64 % 3])
    mask = np.concatenate([ref.tree_mask(rng, n) for n in new])
    worst = check_attn(kq, step, 2 * group, 2, dim, qt, kvt, mask, k_scale=0.5 if kvt == F8 else 1.0,
                       v_scale=0.25 if kvt == F8 else 1.0)
    say(f"attn {qt} {kvt} dim {dim} group {group} tokens {tokens}: err/tol {worst:.3f}")


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 9])
def test_attn_pages(kq, page, tokens):
    step = Step(page, [3, page - 1, page, page + 1, 2 * page + 5, 700], [tokens] * 6, page)
    check_attn(kq, step, 8, 2, 128, BF16, BF16, None)


@pytest.mark.parametrize("dim,kv", [(64, F8), (64, F16), (128, F8), (128, F16), (256, F16)])
@pytest.mark.parametrize("max_len", [129, 700, 1024, 1025])
def test_attn_short_sequences_whole(kq, dim, kv, max_len):
    """Few rows: sequences up to 1024 slots are not cut; lengths around the
    ends of the waves' turns, masks that see nothing among them."""
    lens = [n for n in (0, 1, 63, 255, 256, 257, 511, 512, 600, 1020) if n + 4 <= max_len]
    step = Step(8, lens, [4] * len(lens), 64)
    check_attn(kq, step, 4, 2, dim, F16, kv, ref.tree_mask(np.random.default_rng(2), 4 * len(lens)) & np.uint64(15), max_len=max_len)


@pytest.mark.parametrize("tokens,group,dim", [(1, 4, 128), (1, 1, 64), (20, 4, 128), (64, 8, 64), (2, 8, 256), (30, 3, 256)])
def test_attn_long_sequences_in_parts(kq, tokens, group, dim):
    """Long and short sequences together: the long ones are cut into parts, the
    short ones reach only the first."""
    lens, new = [5000, 0, 129, 2047], [tokens, tokens, max(1, tokens // 2), tokens]
    step = Step(5, lens, new, 32)
    batch = step.batch(kq)
    c = kq.PagedCache(*(t.to(DEV) for t in ref.empty_cache(2, 1, 32, dim, F16)))
    batch.c.n_tokens = step.M
    assert kq.kq_attn_tree_workspace(c.c, batch.c, group, tokens, step.max_len) > 0
    rng = np.random.default_rng(1)
    mask = np.concatenate([ref.tree_mask(rng, n) for n in new])
    check_attn(kq, step, group, 1, dim, F16, F16, mask)
    check_attn(kq, step, group, 1, dim, F16, F16, None, max_len=step.max_len + 100000)


def test_attn_rows_that_see_nothing_or_only_some(kq):
    """No cached token and an empty mask: 0.  Masks without their own bit, with
    bits past the sequence's rows (which count for nothing)."""
    step = Step(3, [0, 0, 40, 7], [4, 1, 6, 3], 16)
    mask = np.zeros(step.M, np.uint64)
    mask[1] = 1
    mask[2] = 0b1001
    mask[5:11] = np.array([0, 1, 2, 1 << 5, (1 << 64) - 1, (1 << 63) | 4], np.uint64)
    q = ref.draw(step.rng, (step.M, 4, 64)).to(BF16)
    k, v = ref.fill_cache(step, 2, 64, BF16)
    out = kq.attn_tree(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q), masks(mask), max_tokens=6, max_len=64).cpu()
    assert (out[0] == 0).all() and (out[3] == 0).all() and (out[4] == 0).all()
    assert (out[2] != 0).any()
    check_attn(kq, step, 4, 2, 64, BF16, BF16, mask, k, v)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("qt,kvt,dim,group", [(BF16, BF16, 128, 1), (F16, F16, 64, 4), (BF16, F8, 128, 8), (F16, F8, 256, 2)])
def test_attn_what_unseen_slots_hold_does_not_count(kq, bad, qt, kvt, dim, group):
    """A drafted token whose key and value are infinite or NaN reaches the rows
    that see it and no other."""
    step = Step(9, [37, 0, 64], [12, 5, 30], 16)
    k, v = ref.fill_cache(step, 2, dim, kvt)
    kf, vf = k.float(), v.float()
    mask, rotten, clean = [], [], []
    for b, n in enumerate(step.new):
        m = ref.tree_mask(step.rng, int(n))
        for j in (1, int(n) - 2):
            p, at = step.where(b, [int(step.lens[b]) + j])
            vf[p, :, 3:dim:17, at] = bad
            if j == 1:
                kf[p, :, at] = bad
            bit = np.uint64(1 << j)
            m = np.where(np.arange(n) % 3 == 0, m & ~bit, m | bit) if j == 1 else np.where(np.arange(n) % 2 == 0, m & ~bit, m | bit)
        m |= np.uint64(1)
        mask.append(m.astype(np.uint64))
        hit = ((m >> np.uint64(1)) | (m >> np.uint64(int(n) - 2))) & np.uint64(1)
        rotten.append(hit.astype(bool))
    mask, rotten = np.concatenate(mask), np.concatenate(rotten)
    k, v = kf.to(kvt), vf.to(kvt)
    q = ref.draw(step.rng, (step.M, 2 * group, dim)).to(qt)
    want, bound = ref.attn(step, k, v, q, mask, dim ** -0.5)
    got = kq.attn_tree(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q), masks(mask), max_tokens=30, max_len=94).cpu().double()
    clean = ~rotten
    assert clean.sum() > 5 and rotten.sum() > 5
    tol = ref.rounded_bound(want, bound, qt)
    assert torch.isfinite(got[clean]).all()
    assert ((got - want).abs() <= tol)[clean].all()
    assert not torch.isfinite(got[rotten]).all(-1).any()
    # a row that sees only the value of the second one keeps its other features
    second = np.array([not ((m >> np.uint64(1)) & np.uint64(1)) for m in mask]) & rotten
    fine = torch.isfinite(want)
    if second.any() and not math.isnan(bad) and kvt != F8:
        assert (torch.isfinite(got) == fine)[second].all()
        assert ((got - want).abs() <= tol)[torch.from_numpy(second)[:, None, None] & fine].all()


@pytest.mark.parametrize("qt", [BF16, F16])
def test_attn_scores_that_grow_and_dominate(kq, qt):
    """Scores that rise along the keys (the running maximum moves at every tile),
    fall, and one that outweighs all others; large and negative scales."""
    step = Step(2, [900, 900, 900], [1, 3, 2], 64)
    for shape in ("rise", "fall", "spike"):
        k, v = ref.fill_cache(step, 1, 128, qt)
        kf = k.float()
        for b in range(3):
            n = int(step.lens[b] + step.new[b])
            p, at = step.where(b, np.arange(n))
            f = np.linspace(0, 4, n) if shape == "rise" else np.linspace(4, 0, n) if shape == "fall" else np.ones(n)
            if shape == "spike":
                f[n // 2] = 60.0
            kf[p, 0, at] = torch.from_numpy(f.astype(np.float32))[:, None] * (0.2 * ref.draw(step.rng, (n, 128)) + 0.5)
        for scale in (0.5, 0.088, -0.3):
            check_attn(kq, step, 4, 1, 128, qt, qt, None, kf.to(qt), v, scale=scale)


def test_attn_bits_repeat_and_streams_and_graphs(kq):
    step = Step(8, [700, 33, 4000], [5, 1, 8], 32)
    k, v = ref.fill_cache(step, 2, 128, BF16)
    q = up(ref.draw(step.rng, (step.M, 8, 128)).to(BF16))
    cache, batch = kq.PagedCache(up(k), up(v)), step.batch(kq)
    args = dict(max_tokens=8, max_len=step.max_len)
    first = kq.attn_tree(cache, batch, q, **args)
    assert torch.equal(first, kq.attn_tree(cache, batch, q, **args))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = kq.attn_tree(cache, batch, q, stream=side, **args)
    raw = kq.attn_tree(cache, batch, q, stream=side.cuda_stream, **args)
    torch.cuda.synchronize()
    assert torch.equal(first, other) and torch.equal(first, raw)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(first)
    with torch.cuda.graph(graph):
        kq.attn_tree(cache, batch, q, out=out, **args)
    for i in range(4):
        q.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kq.attn_tree(cache, batch, q, **args)), i


def test_attn_past_four_gigabytes(kq):
    """Pages at both ends of a cache of 4.5 GiB for keys and as much for values."""
    heads, dim, page = 8, 128, 64
    n_pages = (9 << 29) // (heads * dim * page * 2)
    step = Step(4, [200, 1000], [1, 7], page, n_pages=64)
    move = np.arange(64)
    move[::2] += n_pages - 64
    k0, v0 = ref.fill_cache(step, heads, dim, BF16)
    k = torch.zeros((n_pages, heads, page, dim), dtype=BF16, device=DEV)
    v = torch.zeros((n_pages, heads, dim, page), dtype=BF16, device=DEV)
    k[up(move)], v[up(move)] = up(k0), up(v0)
    q = ref.draw(step.rng, (step.M, 16, dim)).to(BF16)
    bits = np.concatenate([ref.chain_mask(n) for n in step.new])
    want, bound = ref.attn(step, k0, v0, q, bits, dim ** -0.5)
    step.pages = move[step.pages].astype(np.int32)
    got = kq.attn_tree(kq.PagedCache(k, v), step.batch(kq), up(q), max_tokens=7, max_len=step.max_len).cpu().double()
    assert ((got - want).abs() <= ref.rounded_bound(want, bound, BF16)).all()


def test_attn_arrays_that_break_the_contract_stay_inside(kq):
    """Offsets, lengths and pages of nonsense: the call ends, and memory beside
    the output keeps its canaries."""
    heads, dim, page, M = 2, 64, 16, 12
    k, v = (t.to(DEV) for t in ref.empty_cache(5, heads, page, dim, F16, 0.5))
    q = torch.ones((M, 4, dim), dtype=F16, device=DEV)
    whole = torch.full((M + 16, 4, dim), 7.0, dtype=F16, device=DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    for off, lens, pages in (([0, 9, 3, 12], [-5, 1 << 30, 20], [[99, -4, 7]] * 3),
                             ([-7, 40, 1 << 30, -1], [2 ** 31 - 1, 5, -2 ** 31], [[-1, 2 ** 31 - 1, 0]] * 3)):
        kq.attn_tree(kq.PagedCache(k, v), kq.Batch(i32(off), i32(lens), i32(pages)), q, max_tokens=6, max_len=48,
                     out=whole[8:8 + M])
        torch.cuda.synchronize()
        assert (whole[:8] == 7).all() and (whole[8 + M:] == 7).all()


# ---------------------------------------------------------------- rope_append

def rope_table(n_pos, rot):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def check_append(kq, step, hq, hkv, dim, qt, kvt, rot, pairs, norm, positions=None, k_scale=1.0, v_scale=1.0, pad=0):
    x = ref.draw(step.rng, (step.M, (hq + 2 * hkv) * dim + pad), 2.0)
    slots = np.concatenate([[int(step.lens[b]) + i for i in range(int(step.new[b]))] for b in range(len(step.lens))]).astype(int)
    pos = slots if positions is None else positions
    rope = rope_table(int(pos.max()) + 1 if len(pos) else 1, rot) if rot else None
    wq, wk = (1 + 0.2 * ref.draw(step.rng, (2, dim))) if norm else (None, None)
    part = x[:, :(hq + 2 * hkv) * dim]
    (q, qb), (k, kb), (v, vb) = ref.rope_append(step, part, hq, hkv, dim, rope, rot, pairs, torch.from_numpy(pos), wq, wk, 1e-5)
    k0, v0 = ref.empty_cache(step.n_pages, hkv, step.page, dim, kvt, 0.625)
    cache = kq.PagedCache(up(k0), up(v0), k_scale, v_scale)
    got = kq.rope_append(cache, step.batch(kq), up(x)[:, :(hq + 2 * hkv) * dim], hq, None if rope is None else up(rope),
                         positions=None if positions is None else up(positions.astype(np.int32)),
                         q_norm=None if wq is None else up(wq), k_norm=None if wk is None else up(wk), eps=1e-5,
                         pairs=pairs, q_dtype=qt)
    torch.cuda.synchronize()
    assert ((got.cpu().double() - q).abs() <= ref.rounded_bound(q, qb, qt)).all()
    gk, gv = cache.k.cpu().float(), cache.v.cpu().float()
    k, kb, v, vb = k / k_scale, kb / k_scale, v / v_scale, vb / v_scale
    if kvt == F8:
        k, v = k.clamp(-448, 448), v.clamp(-448, 448)
    for b in range(len(step.lens)):
        if not step.new[b]:
            continue
        p, at = step.where(b, int(step.lens[b]) + np.arange(int(step.new[b])))
        r = step.rows(b)
        assert ((gk[p, :, at].double() - k[r]).abs() <= ref.rounded_bound(k[r], kb[r], kvt)).all(), ("k", b)
        assert ((gv[p, :, :, at].double() - v[r]).abs() <= ref.rounded_bound(v[r], vb[r], kvt)).all(), ("v", b)
        gk[p, :, at] = 0.625
        gv[p, :, :, at] = 0.625
    assert (gk == 0.625).all() and (gv == 0.625).all()   # every other slot as it was


@pytest.mark.parametrize("qt,kvt", [(BF16, BF16), (F16, F16), (BF16, F8), (F16, F8)], ids=["bf16", "f16", "bf16-f8", "f16-f8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rot,pairs,norm", [("all", False, True), ("all", True, False), ("half", False, False),
                                            ("half", True, True), (8, False, True), (0, False, True)])
def test_append(kq, qt, kvt, dim, rot, pairs, norm):
    step = Step(dim, [0, 5, 16, 31, 100], [1, 40, 0, 17, 3], 16)
    rot = dim if rot == "all" else dim // 2 if rot == "half" else rot
    s = (0.02, 0.5) if kvt == F8 else (1.0, 1.0)
    check_append(kq, step, 6, 2, dim, qt, kvt, rot, pairs, norm, k_scale=s[0], v_scale=s[1])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (7, 1), (40, 8), (3, 3)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_heads_pages_strides(kq, hq, hkv, page):
    """Head counts that leave waves partly filled, rows set apart in a wider
    product, positions of a tree (several rows share one)."""
    step = Step(hq + page, [0, 250, 3], [33, 9, 64], page)
    pos = np.concatenate([int(n) + step.rng.integers(0, 5, int(t)) for n, t in zip(step.lens, step.new)])
    check_append(kq, step, hq, hkv, 128, BF16, BF16, 128, False, True, positions=pos, pad=12)


def test_append_many_sequences_and_a_long_prompt(kq):
    rng = np.random.default_rng(0)
    check_append(kq, Step(1, rng.integers(0, 90, 300), rng.integers(0, 3, 300), 16), 4, 2, 64, F16, F16, 64, False, True)
    check_append(kq, Step(2, [13], [700], 128), 4, 2, 128, BF16, BF16, 128, True, True)
    check_append(kq, Step(2, [0, 64], [512, 512], 64), 2, 1, 128, BF16, F8, 64, False, False, k_scale=0.03, v_scale=0.02)


def test_append_clamps(kq):
    """e4m3: values past 448 take 448, not NaN; positions past the table take its
    last row; zero rows scaled by their norm stay zero (eps 0 would divide by 0)."""
    step = Step(6, [2], [4], 16)
    x = torch.full((4, 3 * 64), 1000.0)
    x[1] = -1000.0
    x[2] = 0.0
    k0, v0 = ref.empty_cache(step.n_pages, 1, 16, 64, F8, 0.0)
    cache = kq.PagedCache(up(k0), up(v0))
    rope = rope_table(3, 64)
    kq.rope_append(cache, step.batch(kq), up(x), 1)
    p, at = step.where(0, np.arange(2, 6))
    k, v = cache.k.cpu().float(), cache.v.cpu().float()
    for g in (k[p, 0, at], v[p, 0, :, at]):
        assert (g[0] == 448).all() and (g[1] == -448).all() and (g[2] == 0).all()
    w = up(torch.ones(64))
    q = kq.rope_append(cache, step.batch(kq), up(x), 1, up(rope), positions=up(np.array([1 << 30, -5, 0, 2], np.int32)),
                       q_norm=w).cpu().float()
    assert (q[2] == 0).all()
    c, s = rope[2, :32], rope[2, 32:]
    assert torch.allclose(q[0], torch.cat([c - s, c + s]), atol=2.0 ** -7)
    assert torch.allclose(q[1], torch.full((64,), -1.0), atol=2.0 ** -7)


def test_append_arrays_that_break_the_contract_stay_inside(kq):
    cache = kq.PagedCache(*(t.to(DEV) for t in ref.empty_cache(3, 2, 16, 64, F16, 0.0)))
    x = torch.ones((40, 8 * 64), device=DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    for off, lens, pages in (([0, 50, 3], [-9, 1 << 30], [[77, -3]] * 2), ([5, -5, 1 << 30], [2 ** 31 - 1, -2 ** 31], [[0, 2 ** 31 - 1]] * 2)):
        kq.rope_append(cache, kq.Batch(i32(off), i32(lens), i32(pages)), x, 4)
        kq.cache_keep([cache], kq.Batch(i32(off), i32(lens), i32(pages)), i32([2 ** 31 - 1] * 20 + [-7] * 20), i32([90, 3]))
        torch.cuda.synchronize()


# ------------------------------------------------------------------ cache_keep

@pytest.mark.parametrize("dtype", [BF16, F16, F8])
@pytest.mark.parametrize("dim,page,layers", [(64, 16, 1), (128, 64, 3), (256, 32, 2), (128, 16, 70)])
def test_keep(kq, dtype, dim, page, layers):
    """Bit for bit, sources and destinations overlapping, in any order."""
    step = Step(dim, [0, 7, 16, 130, 63], [64, 9, 0, 30, 1], page)
    counts = np.array([64, 4, 0, 13, 1], np.int32)
    path = np.zeros(step.M, np.int32)
    for b in range(5):
        n, c = int(step.new[b]), int(counts[b])
        path[step.rows(b)][:c] = step.rng.permutation(n)[:c] if b != 3 else np.sort(step.rng.permutation(n)[:c])
    caches, want = [], []
    for i in range(layers):
        k, v = ref.fill_cache(step, 2, dim, dtype)
        want.append(ref.keep(step, k, v, path, counts))
        caches.append(kq.PagedCache(up(k), up(v)))
    kq.cache_keep(caches, step.batch(kq), up(path), up(counts))
    torch.cuda.synchronize()
    bits = torch.uint8 if dtype == F8 else torch.int16
    for c, (k, v) in zip(caches, want):
        assert torch.equal(c.k.cpu().view(bits), k.view(bits)) and torch.equal(c.v.cpu().view(bits), v.view(bits))


# -------------------------------------------------------------------- logprobs

def check_logprobs(kq, x, tokens, n_top, entropy=True, gpu_x=None):
    (lp, ent, ids, tops), (lpb, entb, tb) = ref.logprobs(x, tokens, n_top)
    r = kq.logprobs(up(x) if gpu_x is None else gpu_x, None if tokens is None else up(tokens), n_top=n_top, entropy=entropy)
    torch.cuda.synchronize()

    def near(got, want, bound):
        got = got.cpu().double()
        same = got == want   # infinities
        assert (same | ((got - want).abs() <= bound)).all(), ((got - want).abs() / bound)[~same].max()

    if tokens is not None:
        near(r.logprob, lp, lpb)
    else:
        assert r.logprob is None
    if entropy:
        near(r.entropy, ent, entb)
    else:
        assert r.entropy is None
    if n_top:
        assert torch.equal(r.top_ids.cpu(), ids)
        near(r.top_logprobs, tops, tb)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,V", [(1, 1), (1, 63), (3, 64), (2, 1000), (1, 1024), (5, 1025), (2, 4096), (3, 4097), (1, 50257),
                                 (7, 12289), (700, 333), (1100, 5001), (1, 128256)])
@pytest.mark.parametrize("n_top", [0, 1, 20, 64])
def test_logprobs(kq, dtype, M, V, n_top):
    """Rows whole and in parts, rows of odd lengths (so of any alignment), many
    equal logits (16-bit types), a few rows with part of the vocabulary masked."""
    rng = np.random.default_rng(V + M)
    x = ref.draw(rng, (M, V), 3.0)
    x[:, ::7] = torch.round(x[:, ::7])
    x = x.to(dtype)
    if M > 1 and V > 100:
        x[1, 80:] = -math.inf
    tokens = torch.from_numpy(rng.integers(-1, V + 1, (M, 3)).astype(np.int32))
    check_logprobs(kq, x, tokens, min(n_top, V))


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("order", ["rise", "fall", "equal", "peak", "low"])
def test_logprobs_orders(kq, dtype, order):
    """Logits that rise (each beats all before it), fall, are all equal (the
    lowest indices win), one sure token, values near the type's lowest."""
    V = 40001
    x = torch.linspace(-9, 9, V)[None].repeat(2, 1)
    if order == "fall":
        x = x.flip(1).contiguous()
    elif order == "equal":
        x = torch.full((2, V), -3.25)
    elif order == "peak":
        x = x * 0.01
        x[:, 777] = 90.0
    elif order == "low":
        x[:, 5:] = torch.finfo(dtype).min
    x = x.to(dtype)
    check_logprobs(kq, x, torch.tensor([[0, V - 1, 777], [5, 6, 39999]], dtype=torch.int32), 33)


def test_logprobs_strides_and_parts_of_the_answer(kq):
    rng = np.random.default_rng(4)
    wide = up(ref.draw(rng, (9, 3001), 2.0))
    x = wide[:, 7:2907]
    check_logprobs(kq, x.cpu(), None, 5, gpu_x=x)
    check_logprobs(kq, x.cpu(), torch.zeros((9, 0), dtype=torch.int32), 0, gpu_x=x)
    check_logprobs(kq, x[::2].cpu(), torch.ones((5, 1), dtype=torch.int32), 3, entropy=False, gpu_x=x[::2])


def test_logprobs_rows_without_a_distribution(kq):
    """All -inf, a +inf, a NaN: floats are NaN, ids in range; the row beside is not touched."""
    for V in (100, 9000):
        x = ref.draw(np.random.default_rng(V), (4, V))
        x[0] = -math.inf
        x[1, 50] = math.inf
        x[2, 70] = math.nan
        t = torch.tensor([[3, -1]] * 4, dtype=torch.int32)
        r = kq.logprobs(up(x), up(t), n_top=4)
        torch.cuda.synchronize()
        assert torch.isnan(r.logprob[:3, 0]).all() and torch.isnan(r.entropy[:3]).all()
        assert (r.logprob[:, 1] == -math.inf).all()
        assert torch.isnan(r.top_logprobs[:3]).all()
        assert r.top_ids[0].tolist() == [0, 1, 2, 3] and r.top_ids[1, 0] == 50
        assert ((r.top_ids >= 0) & (r.top_ids < V)).all()
        check_logprobs(kq, x[3:], t[3:], 4)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logprobs_at_the_ends_of_the_range(kq, dtype):
    """Equal logits at the type's lowest and highest value and at a value that
    leaves no bits for the sum's logarithm: log probability -log V and entropy log
    V all the same; and one highest among the lowest is sure."""
    lo, hi = torch.finfo(dtype).min, torch.finfo(dtype).max
    for V in (70, 5000):
        x = torch.tensor([lo, hi, 1e30, -2e38, lo], dtype=dtype)[:, None].repeat(1, V)
        x[4, V // 2] = hi
        t = torch.tensor([[0, V // 2]] * 5, dtype=torch.int32)
        r = kq.logprobs(up(x), up(t), n_top=2)
        torch.cuda.synchronize()
        bound = 2.0 ** -24 * (V / 256 + 64) + 2.0 ** -21 * math.log(V)
        assert ((r.logprob[:4].cpu() + math.log(V)).abs() <= bound).all()
        assert ((r.top_logprobs[:4].cpu() + math.log(V)).abs() <= bound).all()
        assert ((r.entropy[:4].cpu() - math.log(V)).abs() <= bound).all()
        assert r.top_ids[:4].tolist() == [[0, 1]] * 4 and r.top_ids[4].tolist() == [V // 2, 0]
        assert r.logprob[4].tolist() == [-math.inf, 0.0] and r.entropy[4] == 0


def test_logprobs_past_two_gigabytes(kq):
    """Rows at 32-bit-offset ends: 2.2e9 bytes of logits; first and last rows checked."""
    M, V = 5000, 110001
    x = torch.zeros((M, V), device=DEV)
    rng = np.random.default_rng(1)
    some = [0, 1, M // 2, M - 1]
    rows = ref.draw(rng, (4, V), 2.0)
    x[some] = up(rows)
    t = torch.full((M, 1), 11, dtype=torch.int32, device=DEV)
    r = kq.logprobs(x, t, n_top=3)
    (lp, ent, ids, _), (lpb, entb, _) = ref.logprobs(rows, t[some].cpu(), 3)
    assert torch.equal(r.top_ids[some].cpu(), ids)
    assert ((r.logprob[some].cpu() - lp).abs() <= lpb).all() and ((r.entropy[some].cpu() - ent).abs() <= entb).all()
    assert r.top_ids[2].tolist() == [0, 1, 2]


# --------------------------------------------------------------- all of a step

def test_variants_are_counted(kq):
    kq.kq_step_count_reset()
    step = Step(1, [40, 3], [1, 1], 16)
    cache = kq.PagedCache(*(t.to(DEV) for t in ref.empty_cache(step.n_pages, 1, 16, 64, F16, 0.0)))
    q = kq.rope_append(cache, step.batch(kq), torch.ones((2, 10 * 64), device=DEV), 8)
    kq.attn_tree(cache, step.batch(kq), q, max_tokens=1, max_len=41)
    kq.attn_tree(cache, step.batch(kq), q, max_tokens=5, max_len=41)
    kq.cache_keep([cache], step.batch(kq), up(np.zeros(2, np.int32)), up(np.ones(2, np.int32)))
    kq.logprobs(torch.zeros((2, 100), device=DEV))
    kq.logprobs(torch.zeros((2, 10000), device=DEV))
    torch.cuda.synchronize()
    n = kq.step_counts()
    assert [n[v] for v in ("rope_append", "attn_few", "attn_rows", "cache_keep", "logprobs_row", "logprobs_parts")] == [1] * 6
