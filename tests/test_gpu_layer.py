"""GPU tests of the operators around the products of a layer (norm_quantize,
attn_chunk, lora) against plain 64-bit forms on the CPU (tests/layer_ref.py, where
the bounds are worked out)."""
from __future__ import annotations

import math

import numpy as np
import pytest

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


def say(*a):
    print(*a, flush=True)


def up(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(DEV)


def apart(a, pad):
    """The same rows in a wider tensor on the device, foreign values between them."""
    wide = torch.full((a.shape[0], a.shape[1] + pad), 77.0, dtype=a.dtype, device=DEV)
    wide[:, :a.shape[1]] = up(a)
    return wide[:, :a.shape[1]]


# -------------------------------------------------------------- norm_quantize

def check_sums(kq, a_q8, act, M, K):
    """The sums behind the values are those of the values."""
    qs, _, bsums = (None if t is None else t.cpu() for t in kq.act_views(a_q8, act, M, K))
    if act == kq.KQ_ACT_Q8_128:
        return
    assert torch.equal(bsums, qs.view(M, K // 16, 16).sum(-1, dtype=torch.int16))
    part = qs.view(M, K // 256, 8, 32).sum(-1, dtype=torch.int32)                       # [M][K / 256][8]
    alpha = kq.alpha_view(a_q8, M, K).view(torch.bfloat16).cpu().float().to(torch.int32)  # [K / 256][2][M][8]
    low = part.remainder(64)
    assert torch.equal(alpha[:, 0].permute(1, 0, 2), part - low) and torch.equal(alpha[:, 1].permute(1, 0, 2), low)


def check_norm(kq, M, K, xt=F32, rt=F32, act=1, residual=True, weight=True, keep=True, pad=0, eps=1e-6, x=None, r=None,
               in_place=False):
    rng = np.random.default_rng(M * 1000 + K)
    x = (ref.draw(rng, (M, K), 1.5) if x is None else x).to(xt)
    r = (ref.draw(rng, (M, K), 3.0) if r is None else r).to(rt) if residual else None
    w = 1 + 0.3 * ref.draw(rng, (K,)) if weight else None
    s, y, bound = lref.norm(x, r, w, eps)
    dr = None if r is None else apart(r, pad)
    out_t = rt if residual else xt
    total = None if in_place or not keep else torch.full((M, K + pad), 55.0, dtype=out_t, device=DEV)
    a_q8 = kq.norm_quantize(apart(x, pad), dr, None if w is None else up(w), eps, act,
                            sum_out=None if total is None else total[:, :K])
    torch.cuda.synchronize()
    qs, d, _ = kq.act_views(a_q8, act, M, K)
    worst = lref.check_quantized(y, bound, qs.cpu(), d.cpu(), 256 if act == 1 else 128)
    check_sums(kq, a_q8, act, M, K)
    got = dr if total is None else total[:, :K]
    if got is not None and (total is not None or in_place):
        off = (got.cpu().double() - s).abs()
        assert (off <= ref.rounded_bound(s, s.abs() * lref.EPS32, out_t)).all()
    if total is not None and pad:
        assert (total[:, K:] == 55).all()
    if dr is not None and total is not None:
        assert torch.equal(dr.cpu(), r)   # the residual is left alone
    return worst


@pytest.mark.parametrize("act", [1, 2], ids=["q8_k", "q8_128"])
@pytest.mark.parametrize("xt", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("rt", [F32, BF16, F16], ids=str)
def test_norm_types(kq, act, xt, rt):
    say("norm", act, xt, rt, check_norm(kq, 5, 2048, xt, rt, act, pad=8))
    check_norm(kq, 3, 768, xt, rt, act, in_place=True)


@pytest.mark.parametrize("act,K", [(1, 256), (1, 1024), (1, 1280), (1, 4096), (1, 5120), (1, 14336), (1, 16640), (1, 33024),
                                   (1, 65536), (2, 128), (2, 384), (2, 1152), (2, 17408), (2, 40064)])
@pytest.mark.parametrize("M", [1, 2, 7])
def test_norm_sizes(kq, act, K, M):
    """Every number of waves and runs to a row, with rows that end inside them."""
    check_norm(kq, M, K, F32, BF16, act, pad=16)


@pytest.mark.parametrize("residual,weight,keep", [(False, True, False), (False, False, True), (True, False, True), (True, True, True)])
def test_norm_without(kq, residual, weight, keep):
    for act in (1, 2):
        check_norm(kq, 9, 1536, F32, F32, act, residual, weight, keep)
        check_norm(kq, 9, 1536, F16, F32, act, residual, weight, keep)


def test_norm_many_rows(kq):
    check_norm(kq, 1537, 512, F32, F32)
    check_norm(kq, 333, 4096, BF16, BF16)


def test_norm_is_quantize_act_of_the_normed_row(kq):
    """Rows whose mean square is 1 to the last bit need no scaling: the buffer is that of
    quantize_act, bit for bit."""
    x = torch.from_numpy(np.random.default_rng(0).choice([-1.0, 1.0], (6, 4096)).astype(np.float32))
    for act in (1, 2):
        got = kq.norm_quantize(up(x), eps=0.0, act_fmt=act)
        want = kq.quantize_act(up(x), act)
        qs, d, b = kq.act_views(got, act, 6, 4096)
        for g, t in zip((qs, d, b), kq.act_views(want, act, 6, 4096)):
            assert g is None or torch.equal(g, t)
        if act == 1:
            assert torch.equal(kq.alpha_view(got, 6, 4096), kq.alpha_view(want, 6, 4096))


@pytest.mark.parametrize("size,eps", [(1e30, 1e-6), (3e38, 1e-6), (1e-25, 0.0), (1e-38, 0.0), (1e-30, 1e-6), (1e-12, 1e-24)])
@pytest.mark.parametrize("K", [512, 5120])
def test_norm_sizes_of_values(kq, size, eps, K):
    """Sums of squares past both ends of fp32."""
    rng = np.random.default_rng(3)
    x = torch.from_numpy((rng.uniform(-1, 1, (4, K)) * size).astype(np.float32))
    check_norm(kq, 4, K, residual=False, x=x, eps=eps, keep=False)


def test_norm_zeros_and_odd_rows(kq):
    """Rows of zeros are zeros, with an eps of 0 too; a row with an infinity or NaN, in x or in the
    residual, or from their sum, has NaN scales and leaves the rows beside it alone."""
    K = 2560
    for eps in (0.0, 1e-5):
        for act in (1, 2):
            x = ref.draw(np.random.default_rng(1), (8, K))
            r = torch.zeros_like(x)
            x[1] = 0.0
            x[2, 700], x[3, K - 1], r[4, 3] = math.inf, math.nan, -math.inf
            x[5], r[5] = 3e38, 3e38
            x[6, 17], r[6, 17] = math.inf, -math.inf
            s, y, bound = lref.norm(x, r, None, eps)
            a = kq.norm_quantize(up(x), up(r), None, eps, act)
            qs, d, _ = kq.act_views(a, act, 8, K)
            qs, d = qs.cpu(), d.cpu()
            for row in (0, 7):
                lref.check_quantized(y[row:row + 1], bound[row:row + 1], qs[row:row + 1], d[row:row + 1], 256 if act == 1 else 128)
            assert (qs[1] == 0).all() and (d[1] == 0).all()
            for row in (2, 3, 4, 5, 6):
                assert (qs[row] == 0).all() and torch.isnan(d[row]).all(), row
            check_sums(kq, a, act, 8, K)


def test_norm_values_past_fp32(kq):
    """A weight that takes a block past fp32: that block is NaN, the others are not."""
    K = 1024
    x = ref.draw(np.random.default_rng(5), (2, K))
    w = torch.ones(K)
    w[300] = 3e38
    x[:, 300] = 5.0
    qs, d, _ = kq.act_views(kq.norm_quantize(up(x), None, up(w), 1e-6), 1, 2, K)
    assert torch.isnan(d[:, 1]).all() and (qs[:, 256:512] == 0).all()
    assert torch.isfinite(d[:, [0, 2, 3]]).all() and (qs[:, :256] != 0).any()


def test_norm_streams_graphs_and_bits(kq):
    x, r = up(ref.draw(np.random.default_rng(2), (37, 4096))), up(ref.draw(np.random.default_rng(3), (37, 4096)))
    s = torch.empty_like(r)
    # (what lies between the sections of a buffer is not written)
    first = kq.norm_quantize(x, r, sum_out=s, out=torch.zeros(kq.kq_act_bytes(1, 37, 4096), dtype=torch.uint8, device=DEV))
    out = torch.zeros_like(first)
    assert torch.equal(first, kq.norm_quantize(x, r, sum_out=s, out=out))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        other = torch.zeros_like(first)
        torch.cuda.synchronize()
        kq.norm_quantize(x, r, sum_out=s, out=other, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kq.norm_quantize(x, r, sum_out=s, out=out)
    for _ in range(4):
        x.mul_(-0.75)
        graph.replay()
        torch.cuda.synchronize()
        want, total = torch.zeros_like(first), torch.empty_like(s)
        kq.norm_quantize(x, r, sum_out=total, out=want)
        assert torch.equal(out, want) and torch.equal(s, total)


def test_norm_feeds_the_product(kq):
    """norm_quantize and a product against the product of the normed rows, quantized apart."""
    import datagen
    M, N, K = 9, 96, 1024
    x, r = ref.draw(np.random.default_rng(8), (M, K)), ref.draw(np.random.default_rng(9), (M, K))
    for fmt in (kq.KQ_Q4_K, kq.KQ_Q6_K, kq.KQ_TQ, kq.KQ_TQ2):
        W = up(datagen.make_weights(fmt, N, K, 77))
        act = kq.kq_act_fmt_for(fmt)
        a = kq.norm_quantize(up(x), up(r), None, 1e-6, act)
        got = kq.gemm(fmt, W, a, M, N, K).cpu().double()
        _, y, _ = lref.norm(x, r, None, 1e-6)
        want = kq.gemm(fmt, W, kq.quantize_act(up(y.float()), act), M, N, K).cpu().double()
        # a value at the border of two steps may fall to either: a step is at most 1/127 of its
        # block's largest, 4 deviations for these; weights have their own size
        size = want.pow(2).mean().sqrt()
        assert (got - want).abs().max() <= 0.05 * size and (got - want).pow(2).mean().sqrt() <= 0.002 * size


# ----------------------------------------------------------------- attn_chunk

def check_chunk(kq, step, hq, hkv, dim, qt, kvt, window=0, sinks=0, k=None, v=None, k_scale=1.0, v_scale=1.0, scale=None,
                max_tokens=None, max_len=None, types=None, q=None):
    """One call in q's type and one in float32 against the plain form; without a max_len, in q's type
    also as if sequences were longer (larger blocks of rows) and far longer (in runs)."""
    if k is None:
        k, v = ref.fill_cache(step, hkv, dim, kvt)
    q = ref.draw(step.rng, (step.M, hq, dim), 1.5).to(qt) if q is None else q
    scale = dim ** -0.5 if scale is None else scale
    want, bound = lref.chunk(step, k, v, q, window, sinks, scale, k_scale, v_scale)
    cache, batch = kq.PagedCache(up(k), up(v), k_scale, v_scale), step.batch(kq)
    worst = 0.0
    for out_dtype in types or (qt, F32):
        tol = bound if out_dtype == F32 else ref.rounded_bound(want, bound, out_dtype)
        for most in [max_len or step.max_len] + [5000, 40000] * (not max_len and out_dtype == qt):
            got = torch.full((step.M, hq, dim), math.nan, dtype=out_dtype, device=DEV)
            kq.attn_chunk(cache, batch, up(q), window, sinks, scale, max_tokens or max(1, step.max_new), most, out=got)
            torch.cuda.synchronize()
            got = got.cpu().double()
            assert torch.isfinite(got).all(), (out_dtype, most, int((~torch.isfinite(got)).sum()))
            err = ((got - want).abs() / tol.clamp(min=1e-30)).max().item() if got.numel() else 0.0
            assert ((got - want).abs() <= tol).all(), (out_dtype, most, err)
            worst = max(worst, err)
    return worst


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300]
KINDS = [(BF16, BF16), (F16, F16), (BF16, F8), (F16, F8)]


@pytest.mark.parametrize("qt,kvt", KINDS, ids=["bf16", "f16", "bf16-f8", "f16-f8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,tokens", [(1, 1), (4, 1), (16, 1), (3, 5), (2, 40), (4, 32), (5, 90), (8, 130), (1, 300)])
def test_chunk_lengths_and_rows(kq, qt, kvt, dim, group, tokens):
    """Every length around the ends of tiles, units and pages in one ragged batch, with each split
    of the rows over blocks, waves and kernels, under a window and without."""
    rng = np.random.default_rng(dim + group * 7 + tokens)
    new = [tokens] + [int(n) for n in rng.integers(0 if tokens > 1 else 1, min(tokens, 70) + 1, len(LENS) - 1)]
    step = Step(11 + tokens, LENS, new, (16, 32, 64)[dim // 64 % 3])
    s = (0.5, 0.25) if kvt == F8 else (1.0, 1.0)
    for window, sinks in ((0, 0), (70, 5)):
        worst = check_chunk(kq, step, 2 * group, 2, dim, qt, kvt, window, sinks, k_scale=s[0], v_scale=s[1],
                            types=(qt,) if window else None)
        say(f"chunk {qt} {kvt} dim {dim} group {group} tokens {tokens} window {window}: err/tol {worst:.3f}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (63, 64), (64, 1), (65, 200), (128, 63), (200, 4),
                                          (1000, 1000), (1 << 30, 0), (1 << 30, 1 << 30), (7, 1 << 30)])
@pytest.mark.parametrize("dim,group,tokens", [(128, 4, 1), (64, 4, 20), (128, 2, 200), (256, 3, 90), (256, 4, 400)])
def test_chunk_windows(kq, window, sinks, dim, group, tokens):
    """Windows and sinks that meet, overlap, end inside tiles, cover everything and leave one slot."""
    step = Step(window + sinks, [0, 3, 64, 333, 900], [tokens, max(1, tokens // 2), tokens, tokens, 1], 32)
    check_chunk(kq, step, group, 1, dim, BF16, BF16, window, sinks, types=(BF16,))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 9, 150])
@pytest.mark.parametrize("dim", [64, 128])
def test_chunk_pages(kq, page, tokens, dim):
    step = Step(page, [3, page - 1, page, page + 1, 2 * page + 5, 700], [tokens] * 6, page)
    check_chunk(kq, step, 8, 2, dim, BF16, BF16, types=(BF16,))
    check_chunk(kq, step, 8, 2, dim, F16, F8, 100, 20, types=(F16,))


@pytest.mark.parametrize("tokens,group,dim", [(1, 4, 128), (1, 1, 64), (2, 8, 256), (20, 4, 128), (32, 4, 64), (300, 3, 128), (70, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 100)])
def test_chunk_in_parts(kq, tokens, group, dim, window, sinks):
    """Long and short sequences together: the long ones are cut into parts, the short ones
    reach only the first."""
    step = Step(5, [5000, 0, 129, 2047], [tokens, tokens, max(1, tokens // 2), tokens], 32)
    batch = step.batch(kq)
    c = kq.PagedCache(*(t.to(DEV) for t in ref.empty_cache(2, 1, 32, dim, F16)))
    assert kq.kq_attn_chunk_workspace(c.c, batch.of(step.M), group, window, sinks, tokens, step.max_len) > 0
    check_chunk(kq, step, group, 1, dim, F16, F16, window, sinks)


@pytest.mark.parametrize("max_tokens", [1, 5, 40, 1000])
@pytest.mark.parametrize("max_len", [1, 100, 5000, 1 << 30])
def test_chunk_expectations_change_the_speed_alone(kq, max_tokens, max_len):
    step = Step(3, [900, 0, 40, 2500, 64], [1, 100, 17, 33, 0], 64)
    check_chunk(kq, step, 8, 2, 128, BF16, BF16, max_tokens=max_tokens, max_len=max_len, types=(BF16,))
    check_chunk(kq, step, 8, 2, 128, BF16, BF16, 300, 7, max_tokens=max_tokens, max_len=max_len, types=(BF16,))


@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_chunk_few_keys(kq, qt, dim):
    """Two or three keys to a row, where the roundings of their weights do not average out; more heads
    to a key head than a block of 16 rows holds, and a number of them that is no power of 2."""
    check_chunk(kq, Step(7, [0, 1], [1, 140], 64), 8, 2, dim, qt, qt, 2, 1)
    check_chunk(kq, Step(8, [0, 1, 2], [2, 1, 1], 16), 100, 1, dim, qt, qt)
    check_chunk(kq, Step(9, [1, 0], [3, 30], 32), 72, 3, dim, qt, F8, 3, 0)


def test_chunk_many_sequences(kq):
    """More sequences than a wave looks at together, many of them without rows; single tokens among
    pieces of prompts."""
    rng = np.random.default_rng(0)
    new = rng.integers(0, 3, 300)
    new[::50] = 0
    step = Step(1, rng.integers(0, 90, 300), new, 16)
    check_chunk(kq, step, 4, 2, 64, F16, F16, types=(F16,))
    new[7] = 130
    step = Step(2, rng.integers(0, 90, 300), new, 16)
    check_chunk(kq, step, 4, 2, 64, F16, F16, 40, 3, types=(F16,))
    step = Step(2, np.zeros(130, int), [0] * 64 + [1] + [0] * 65, 16)
    check_chunk(kq, step, 4, 2, 64, F16, F16, types=(F16,))


def test_chunk_equals_tree(kq):
    """Up to 64 rows that see all before them: what attn_tree computes."""
    step = Step(4, [0, 77, 500], [64, 1, 30], 32)
    k, v = ref.fill_cache(step, 2, 128, BF16)
    q = up(ref.draw(step.rng, (step.M, 8, 128)).to(BF16))
    cache, batch = kq.PagedCache(up(k), up(v)), step.batch(kq)
    tree = kq.attn_tree(cache, batch, q, max_tokens=64, max_len=step.max_len, out_dtype=F32)
    got = kq.attn_chunk(cache, batch, q, max_tokens=64, max_len=step.max_len, out_dtype=F32)
    # each probability is rounded relative to another maximum: 2^-8 of |v| (under 5) each
    assert (tree - got).abs().max() <= 2 * 2.0 ** -8 * 5


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("qt,kvt,dim,group,tokens", [(BF16, BF16, 128, 1, 12), (F16, F16, 64, 4, 30), (BF16, F8, 128, 8, 60),
                                                     (F16, F8, 256, 2, 40), (BF16, BF16, 128, 4, 150), (F16, F16, 64, 2, 8),
                                                     (BF16, BF16, 256, 4, 60), (BF16, F8, 256, 3, 90)])
@pytest.mark.parametrize("window,longer", [(50, 0), (3100, 3300)], ids=["short", "long"])
def test_chunk_what_unseen_slots_hold_does_not_count(kq, bad, qt, kvt, dim, group, tokens, window, longer):
    """Slots with infinite or NaN keys and values: later tokens, slots before the window and between
    it and the sinks.  They reach the rows that see them and no other."""
    sinks = 3
    step = Step(9, [137 + longer, 0, 64, 300 + longer], [tokens, 5, max(1, tokens - 7), 1], 16)
    k, v = ref.fill_cache(step, 2, dim, kvt)
    kf, vf = k.float(), v.float()
    rotten = []
    for b, (L, n) in enumerate(zip(step.lens, step.new)):
        total = int(L + n)
        spots = [s for s in (5, total - 2, total // 2, total - window - 10) if 0 <= s < total]
        p, at = step.where(b, spots)
        vf[p, :, 3:dim:17, at] = bad
        kf[p[:1], :, at[:1]] = bad
        on = lref.seen(int(L), int(n), window, sinks)
        rotten.append(on[:, spots].any(-1))
    rotten = torch.cat(rotten)
    k, v = kf.to(kvt), vf.to(kvt)
    q = ref.draw(step.rng, (step.M, 2 * group, dim)).to(qt)
    clean_k, clean_v = (torch.where(torch.isfinite(t.float()), t.float(), 0.0).to(kvt) for t in (k, v))
    want, bound = lref.chunk(step, clean_k, clean_v, q, window, sinks, dim ** -0.5)
    clean = ~rotten
    assert clean.sum() >= 1 and rotten.sum() > 5
    tol = ref.rounded_bound(want, bound, qt)
    for most in (step.max_len, 40000):
        got = kq.attn_chunk(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q), window, sinks, max_tokens=tokens,
                            max_len=most).cpu().double()
        assert torch.isfinite(got[clean]).all()
        assert ((got - want).abs() <= tol)[clean].all()
        if kvt != F8 or math.isnan(bad):   # (8 bits have no infinities: clamped when stored)
            assert not torch.isfinite(got[rotten]).all(-1).any()


@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("tokens", [3, 100])
def test_chunk_scores_that_grow_and_dominate(kq, qt, tokens):
    step = Step(2, [900, 900], [tokens, 2], 64)
    for shape in ("rise", "fall", "spike"):
        k, v = ref.fill_cache(step, 1, 128, qt)
        kf = k.float()
        for b in range(2):
            n = int(step.lens[b] + step.new[b])
            p, at = step.where(b, np.arange(n))
            f = np.linspace(0, 4, n) if shape == "rise" else np.linspace(4, 0, n) if shape == "fall" else np.ones(n)
            if shape == "spike":
                f[n // 2] = 60.0
            kf[p, 0, at] = torch.from_numpy(f.astype(np.float32))[:, None] * (0.2 * ref.draw(step.rng, (n, 128)) + 0.5)
        for scale in (0.5, 0.088, -0.3, 0.0):
            check_chunk(kq, step, 4, 1, 128, qt, qt, k=kf.to(qt), v=v, scale=scale, types=(qt,))


@pytest.mark.parametrize("tokens", [1, 30, 200])
def test_chunk_bits_streams_and_graphs(kq, tokens):
    """The same bits every time, on other streams and replayed; two captured graphs and eager
    calls between them."""
    step = Step(8, [700, 33, 4000], [tokens, 1, max(1, tokens // 3)], 32)
    k, v = ref.fill_cache(step, 2, 128, BF16)
    q = up(ref.draw(step.rng, (step.M, 8, 128)).to(BF16))
    cache, batch = kq.PagedCache(up(k), up(v)), step.batch(kq)
    args = dict(window=0, max_tokens=tokens, max_len=step.max_len)
    first = kq.attn_chunk(cache, batch, q, **args)
    assert torch.equal(first, kq.attn_chunk(cache, batch, q, **args))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = kq.attn_chunk(cache, batch, q, stream=side, **args)
    raw = kq.attn_chunk(cache, batch, q, stream=side.cuda_stream, **args)
    torch.cuda.synchronize()
    assert torch.equal(first, other) and torch.equal(first, raw)
    outs, graphs = [torch.empty_like(first) for _ in range(2)], []
    for i, out in enumerate(outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kq.attn_chunk(cache, batch, q, out=out, **{**args, "window": 500 * i})
    for n in range(4):
        q.mul_(0.5)
        for i in ((0, 1), (1, 0))[n % 2]:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], kq.attn_chunk(cache, batch, q, **{**args, "window": 500 * i})), (n, i)


def test_chunk_rows_behind_the_last_sequence(kq):
    """A padded step: rows past offsets[n_seqs] are left as they were."""
    step = Step(6, [100, 7], [5, 40], 16)
    k, v = ref.fill_cache(step, 2, 64, F16)
    q = ref.draw(step.rng, (step.M + 19, 4, 64)).to(F16)
    out = torch.full_like(q, 3.0, device=DEV)
    kq.attn_chunk(kq.PagedCache(up(k), up(v)), step.batch(kq), up(q), out=out)
    assert (out[step.M:] == 3).all()
    want, bound = lref.chunk(step, k, v, q[:step.M], 0, 0, 64 ** -0.5)
    assert ((out[:step.M].cpu().double() - want).abs() <= ref.rounded_bound(want, bound, F16)).all()


def test_chunk_past_four_gigabytes(kq):
    """Pages at both ends of a cache of 4.5 GiB for keys and as much for values."""
    heads, dim, page = 8, 128, 64
    n_pages = (9 << 29) // (heads * dim * page * 2)
    step = Step(4, [200, 1000], [1, 70], page, n_pages=64)
    move = np.arange(64)
    move[::2] += n_pages - 64
    k0, v0 = ref.fill_cache(step, heads, dim, BF16)
    k = torch.zeros((n_pages, heads, page, dim), dtype=BF16, device=DEV)
    v = torch.zeros((n_pages, heads, dim, page), dtype=BF16, device=DEV)
    k[up(move)], v[up(move)] = up(k0), up(v0)
    q = ref.draw(step.rng, (step.M, 16, dim)).to(BF16)
    want, bound = lref.chunk(step, k0, v0, q, 0, 0, dim ** -0.5)
    step.pages = move[step.pages].astype(np.int32)
    for most in (1, 70):
        got = kq.attn_chunk(kq.PagedCache(k, v), step.batch(kq), up(q), max_tokens=most, max_len=step.max_len).cpu().double()
        assert ((got - want).abs() <= ref.rounded_bound(want, bound, BF16)).all()


def test_chunk_arrays_that_break_the_contract_stay_inside(kq):
    """Offsets, lengths and pages of nonsense: the call ends, and memory beside the output keeps
    its canaries."""
    heads, dim, page, M = 2, 64, 16, 12
    k, v = (t.to(DEV) for t in ref.empty_cache(5, heads, page, dim, F16, 0.5))
    q = torch.ones((M, 4, dim), dtype=F16, device=DEV)
    whole = torch.full((M + 16, 4, dim), 7.0, dtype=F16, device=DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    for off, lens, pages in (([0, 9, 3, 12], [-5, 1 << 30, 20], [[99, -4, 7]] * 3),
                             ([-7, 40, 1 << 30, -1], [2 ** 31 - 1, 5, -2 ** 31], [[-1, 2 ** 31 - 1, 0]] * 3)):
        for most in (1, 12, 200):
            for window in (0, 5):
                kq.attn_chunk(kq.PagedCache(k, v), kq.Batch(i32(off), i32(lens), i32(pages)), q, window, 3, max_tokens=most,
                              max_len=48, out=whole[8:8 + M])
                torch.cuda.synchronize()
                assert (whole[:8] == 7).all() and (whole[8 + M:] == 7).all()


@pytest.mark.parametrize("heads,group,dim,t", [(2, 2, 64, F16), (1, 16, 128, BF16), (4, 4, 256, F8)])
def test_chunk_arrays_that_break_the_contract_in_runs(kq, heads, group, dim, t):
    """The same where the work is cut into runs: with offsets that fall, two searches of them may find
    different sequences for a block, and blocks may be none at all."""
    page, M = 16, 900
    qt = BF16 if t == F8 else t
    k, v = (a.to(DEV) for a in ref.empty_cache(90, heads, page, dim, t, 0.5))
    q = torch.ones((M, heads * group, dim), dtype=qt, device=DEV)
    whole = torch.full((M + 16, heads * group, dim), 7.0, dtype=qt, device=DEV)
    rng = np.random.default_rng(11)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int64).astype(np.int32)).to(DEV)  # noqa: E731
    cache = kq.PagedCache(k, v)
    for n in (1, 3, 70):
        for offsets in (rng.integers(-50, M + 50, n + 1), rng.integers(0, M + 1, n + 1), np.full(n + 1, M), np.full(n + 1, -3),
                        np.sort(rng.integers(0, M + 1, n + 1))[::-1], np.where(np.arange(n + 1) % 2, M, 0)):
            batch = kq.Batch(i32(offsets), i32(rng.integers(-100, 1500, n)), i32(rng.integers(-10, 100, (n, 80))))
            for most in (1, 8, 60, M):
                for window, most_len in ((0, 20000), (300, 2000), (0, 1 << 20)):
                    kq.attn_chunk(cache, batch, q, window, 9, max_tokens=most, max_len=most_len, out=whole[8:8 + M])
                    torch.cuda.synchronize()
                    assert (whole[:8] == 7).all() and (whole[8 + M:] == 7).all()


# ----------------------------------------------------------------------- lora

def activations(kq, rng, M, K, act):
    a = kq.quantize_act(up(ref.draw(rng, (M, K))), act)
    qs, d, _ = kq.act_views(a, act, M, K)
    return a, qs.cpu(), d.cpu()


def check_lora(kq, M, N, K, rank, n, ids, t=BF16, act=1, scaled=True, based=True, pad=0, in_place=False, seed=0):
    rng = np.random.default_rng(seed + M + N + K + rank)
    a, qs, d = activations(kq, rng, M, K, act)
    A, B = ref.draw(rng, (n, rank, K), K ** -0.5).to(t), ref.draw(rng, (n, N, rank), rank ** -0.5).to(t)
    scale = torch.from_numpy(rng.uniform(0.5, 2, n).astype(np.float32)) if scaled else None
    base = ref.draw(rng, (M, N)) if based else None
    ids = torch.as_tensor(ids, dtype=torch.int32)
    want, bound = lref.lora(qs, d, 256 if act == 1 else 128, A, B, scale, ids, base)
    db = None if base is None else apart(base, pad)
    whole = torch.full((M, N + pad), 55.0, device=DEV)
    out = db if in_place else whole[:, :N]
    got = kq.lora(a, up(A), up(B), up(ids), None if scale is None else up(scale), db, act, out=out)
    torch.cuda.synchronize()
    got = got.cpu().double()
    off = (got - want).abs()
    assert (off <= bound).all(), (off / bound.clamp(min=1e-300)).max()
    if not in_place and pad:
        assert (whole[:, N:] == 55).all()
    fresh = kq.lora(a, up(A), up(B), up(ids), None if scale is None else up(scale), None if base is None else up(base), act)
    assert torch.equal(fresh.cpu().double(), got)
    return (off / bound.clamp(min=1e-300)).max().item()


@pytest.mark.parametrize("t", [BF16, F16], ids=str)
@pytest.mark.parametrize("act", [1, 2], ids=["q8_k", "q8_128"])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("M", [1, 5, 65, 200, 601])
def test_lora_types_and_ranks(kq, t, act, rank, M):
    n = 5
    ids = np.random.default_rng(M).integers(-1, n + 1, M)   # some outside at either end
    say("lora", t, act, rank, M, check_lora(kq, M, 193, 768, rank, n, ids, t, act, pad=3))


@pytest.mark.parametrize("N", [1, 31, 32, 33, 64, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("M", [3, 64, 65, 128, 131])
def test_lora_sizes(kq, N, M):
    """Rows sorted by request and not; odd numbers of rows and columns."""
    check_lora(kq, M, N, 256, 16, 3, np.arange(M) * 3 // M)
    check_lora(kq, M, N, 256, 64, 3, np.arange(M) * 3 // M)
    check_lora(kq, M, N, 256, 128, 7, np.arange(M) * 5 % 8 - 1)


@pytest.mark.parametrize("act,K", [(1, 256), (1, 512), (1, 2304), (1, 14336), (2, 128), (2, 640), (2, 5120)])
@pytest.mark.parametrize("M", [2, 257])
def test_lora_depths(kq, act, K, M):
    check_lora(kq, M, 100, K, 16, 2, np.arange(M) % 2, F16, act)


@pytest.mark.parametrize("M", [4, 515])
def test_lora_without(kq, M):
    for scaled in (False, True):
        for based in (False, True):
            check_lora(kq, M, 200, 512, 8, 3, np.arange(M) % 4, scaled=scaled, based=based)
    check_lora(kq, M, 200, 512, 8, 3, np.arange(M) % 4, in_place=True, pad=5)
    check_lora(kq, M, 200, 512, 8, 3, np.full(M, -1), in_place=True)
    check_lora(kq, M, 200, 512, 8, 3, np.full(M, -1))


def test_lora_each_row_its_own(kq):
    for M in (64, 300):
        check_lora(kq, M, 300, 512, 16, M, np.random.default_rng(1).permutation(M))


def test_lora_no_adapters(kq):
    M, N, K = 5, 40, 256
    a, _, _ = activations(kq, np.random.default_rng(0), M, K, 1)
    base = torch.randn(M, N, device=DEV)
    empty = torch.empty((0, 16, K), dtype=BF16, device=DEV), torch.empty((0, N, 16), dtype=BF16, device=DEV)
    ids = torch.zeros(M, dtype=torch.int32, device=DEV)
    assert torch.equal(kq.lora(a, *empty, ids, base=base), base)
    assert (kq.lora(a, *empty, ids) == 0).all()


@pytest.mark.parametrize("M", [6, 290])
def test_lora_odd_adapters_and_rows_stay_apart(kq, M):
    """Infinities and NaN in an adapter nobody else uses, and rows whose activations are NaN."""
    N, K, n = 150, 512, 4
    rng = np.random.default_rng(3)
    x, r = ref.draw(rng, (M, K)), None
    x[M - 1] = math.nan
    a = kq.norm_quantize(up(x))
    qs, d, _ = (None if v is None else v.cpu() for v in kq.act_views(a, 1, M, K))
    A, B = ref.draw(rng, (n, 16, K), K ** -0.5), ref.draw(rng, (n, N, 16), 0.25)
    A[1, 3, 5], B[2, 7, 1] = math.inf, math.nan
    A, B = A.to(BF16), B.to(BF16)
    ids = torch.arange(M, dtype=torch.int32) % n
    base = ref.draw(rng, (M, N))
    got = kq.lora(a, up(A), up(B), up(ids), base=up(base)).cpu().double()
    fine = ((ids == 0) | (ids == 3)) & (torch.arange(M) != M - 1)
    want, bound = lref.lora(qs[fine], d[fine], 256, A, B, None, ids[fine], base[fine])
    assert ((got[fine] - want).abs() <= bound).all()
    assert torch.isnan(got[M - 1]).all()
    assert not torch.isfinite(got[ids == 1]).any()
    assert torch.isnan(got[ids == 2][:, 7]).all() and torch.isfinite(got[(ids == 2) & (torch.arange(M) != M - 1)][:, 8:]).all()


@pytest.mark.parametrize("M", [7, 300])
def test_lora_bits_streams_and_graphs(kq, M):
    N, K, n = 500, 1024, 3
    rng = np.random.default_rng(5)
    a, _, _ = activations(kq, rng, M, K, 1)
    A, B = up(ref.draw(rng, (n, 16, K), 0.03).to(BF16)), up(ref.draw(rng, (n, N, 16), 0.25).to(BF16))
    ids, base = up((np.arange(M) % 4).astype(np.int32)), up(ref.draw(rng, (M, N)))
    first = kq.lora(a, A, B, ids, base=base)
    assert torch.equal(first, kq.lora(a, A, B, ids, base=base))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        other = kq.lora(a, A, B, ids, base=base, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first, other)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(first)
    with torch.cuda.graph(graph):
        kq.lora(a, A, B, ids, base=base, out=out)
    for _ in range(4):
        base.add_(1.0)
        B.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kq.lora(a, A, B, ids, base=base))


def test_lora_past_four_gigabytes(kq):
    """Adapters whose weights begin past 2^32 bytes, and 2^31 elements."""
    N, K, rank = 8192, 8192, 128
    n = (5 << 30) // (rank * K * 2)
    rng = np.random.default_rng(6)
    a, qs, d = activations(kq, rng, 70, K, 1)
    A = torch.zeros((n, rank, K), dtype=BF16, device=DEV)
    B = torch.zeros((n, N, rank), dtype=BF16, device=DEV)
    last = ref.draw(rng, (2, rank, K), 0.01).to(BF16), ref.draw(rng, (2, N, rank), 0.1).to(BF16)
    A[n - 2:], B[n - 2:] = up(last[0]), up(last[1])
    for M in (3, 70):
        ids = torch.arange(M, dtype=torch.int32) % 2
        buf = kq.quantize_act(up((qs[:M].double() * d[:M].double().repeat_interleave(256, 1)).float()))
        q2, d2, _ = kq.act_views(buf, 1, M, K)
        want, bound = lref.lora(q2.cpu(), d2.cpu(), 256, *last, None, ids, None)
        got = kq.lora(buf, A, B, up(ids + (n - 2))).cpu().double()
        assert ((got - want).abs() <= bound).all()


# -------------------------------------------------------------------- together

@pytest.mark.parametrize("act", [1, 2], ids=["q8_k", "q8_128"])
@pytest.mark.parametrize("max_len", [300, 40000])
def test_a_layer_captured(kq, act, max_len):
    """norm_quantize, a product, its adapters in place, rope_append and attn_chunk of a step with prompts
    and single tokens, captured twice (two activation formats and two cuts of the work) and replayed
    with other inputs: the eager calls' bits every time."""
    import datagen
    K, heads, dim = 512, 2, 64
    N = 4 * heads * dim
    step = Step(12, [250, 0, 33, 7], [1, 40, 7, 1], 32)
    M, fmt = step.M, kq.KQ_Q4_K if act == 1 else kq.KQ_TQ2
    W = up(datagen.make_weights(fmt, N, K, 5))
    x, r = up(ref.draw(step.rng, (M, K))), up(ref.draw(step.rng, (M, K)).to(BF16))
    total = torch.empty_like(r)
    A, B = up(ref.draw(step.rng, (3, 16, K), 0.05).to(BF16)), up(ref.draw(step.rng, (3, N, 16), 0.25).to(BF16))
    ids = up((np.arange(M) % 4 - 1).astype(np.int32))
    angle = np.arange(300)[:, None] / 100.0 ** (np.arange(dim // 2) / (dim // 2))
    rope = up(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    cache, batch = kq.PagedCache(*(up(t) for t in ref.fill_cache(step, heads, dim, BF16))), step.batch(kq)

    def layer(out=None):
        a = kq.norm_quantize(x, r, act_fmt=act, sum_out=total)
        qkv = kq.gemm(fmt, W, a, M, N, K)
        kq.lora(a, A, B, ids, base=qkv, act_fmt=act, out=qkv)
        q = kq.rope_append(cache, batch, qkv, 2 * heads, rope)
        return kq.attn_chunk(cache, batch, q, 100, 2, max_tokens=40, max_len=max_len, out=out)

    first = layer()
    assert torch.isfinite(first).all()
    outs, graphs = [torch.empty_like(first) for _ in range(2)], []
    for out in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer(out)
    for n in range(4):
        x.add_(0.125 * (n + 1)).mul_(-0.5)
        r.mul_(0.75)
        want = layer()
        kept = total.clone()
        total.zero_()
        for i in ((0, 1), (1, 0))[n % 2]:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(total, kept), n
        assert not torch.equal(want, first)


def test_counters(kq):
    kq.kq_layer_count_reset()
    check_norm(kq, 2, 256)
    check_lora(kq, 2, 32, 256, 8, 1, [0, 0])
    check_lora(kq, 700, 32, 256, 8, 1, [0] * 700)
    check_chunk(kq, Step(1, [5], [1], 16), 2, 1, 64, BF16, BF16, types=(BF16,), max_len=40)
    check_chunk(kq, Step(1, [5], [30], 16), 2, 1, 64, BF16, BF16, types=(BF16,), max_len=40)
    counts = kq.layer_counts()
    assert counts == {"norm_quantize": 1, "chunk_few": 1, "chunk_rows": 1, "lora_few": 2, "lora_tile": 2}
