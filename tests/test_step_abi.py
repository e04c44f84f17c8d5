"""CPU tests of the step operators' C ABI (paged cache, attention, log
probabilities): invalid arguments are refused with their status code before any
HIP call, sizes of workspaces, and the binding's own checks."""
from __future__ import annotations

import ctypes
import math
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20   # a fake, aligned "device address": never dereferenced on these paths


@pytest.fixture(scope="module")
def kq():
    import block_quantized_matmul_act_amd as kq
    if not os.path.exists(kq.LIB_PATH):
        from block_quantized_matmul_act_amd import build
        build.build()
    kq.lib()
    return kq


def cache(kq, **kw):
    f = dict(k=A, v=A, n_pages=10, type=kq.KQ_T_BF16, heads=2, dim=128, page=16, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return kq.kq_cache(*(f[n] for n, _ in kq.kq_cache._fields_))


def batch(kq, **kw):
    f = dict(offsets=A, lens=A, pages=A, n_seqs=3, n_tokens=5, max_pages=4)
    f.update(kw)
    return kq.kq_batch(*(f[n] for n, _ in kq.kq_batch._fields_))


def ref(d):
    return None if d is None else ctypes.addressof(d)


BAD_CACHES = [(dict(type=kind), "KQ_ERR_FMT") for kind in (0, 1, 5, -1)] + \
    [(dict(dim=d), "KQ_ERR_UNSUPPORTED") for d in (0, 32, 96, 512, -64)] + \
    [(dict(page=p), "KQ_ERR_UNSUPPORTED") for p in (0, 1, 8, 24, 512, -16)] + \
    [(dict(heads=h), "KQ_ERR_SHAPE") for h in (0, -1, 65536)] + \
    [(dict(n_pages=n), "KQ_ERR_SHAPE") for n in (-1, 0, 1 << 31)] + \
    [(dict(k_scale=s), "KQ_ERR_SHAPE") for s in (0.0, -1.0, math.inf, math.nan)] + \
    [(dict(v_scale=s), "KQ_ERR_SHAPE") for s in (0.0, math.nan)] + \
    [(dict(k=None), "KQ_ERR_NULL"), (dict(v=None), "KQ_ERR_NULL"), (dict(k=A + 8), "KQ_ERR_ALIGN"), (dict(v=A + 2), "KQ_ERR_ALIGN")]
BAD_BATCHES = [(dict(n_seqs=-1), "KQ_ERR_SHAPE"), (dict(n_tokens=-1), "KQ_ERR_SHAPE"), (dict(max_pages=-1), "KQ_ERR_SHAPE"),
               (dict(n_seqs=1 << 31), "KQ_ERR_SHAPE"), (dict(n_tokens=1 << 31), "KQ_ERR_SHAPE"), (dict(max_pages=0), "KQ_ERR_SHAPE"),
               (dict(offsets=None), "KQ_ERR_NULL"), (dict(lens=None), "KQ_ERR_NULL"), (dict(pages=None), "KQ_ERR_NULL"),
               (dict(offsets=A + 2), "KQ_ERR_ALIGN"), (dict(lens=A + 1), "KQ_ERR_ALIGN"), (dict(pages=A + 3), "KQ_ERR_ALIGN")]


def rope(kq, c=None, b=None, **kw):
    f = dict(x=A, ldx=1024, q_heads=4, q_norm=A, k_norm=A, eps=1e-6, rope=A, n_pos=100, rot=128, pairs=0, positions=A,
             q_type=kq.KQ_T_BF16, q=A)
    f.update(kw)
    return kq.lib().kq_rope_append(ref(c), ref(b), *f.values(), None)


def attn(kq, c=None, b=None, **kw):
    f = dict(q_type=kq.KQ_T_BF16, q=A, q_heads=4, mask=A, scale=0.1, max_tokens=4, max_len=64, out_type=kq.KQ_T_BF16,
             out=A, ws=A, ws_bytes=1 << 40)
    f.update(kw)
    return kq.lib().kq_attn_tree(ref(c), ref(b), *f.values(), None)


def keep(kq, c=None, b=None, n=1, path=A, counts=A):
    return kq.lib().kq_cache_keep(ref(c), n, ref(b), path, counts, None)


def logprobs(kq, **kw):
    f = dict(type=kq.KQ_T_F32, x=A, M=3, V=100, ldx=100, tokens=A, n_given=2, n_top=5, logprob=A, entropy=A, ids=A, tops=A,
             ws=A, ws_bytes=1 << 40)
    f.update(kw)
    return kq.lib().kq_logprobs(*f.values(), None)


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=str)
def test_bad_caches(kq, bad, code):
    c, b = cache(kq, **bad), batch(kq)
    for call in (rope, attn, keep):
        assert call(kq, c, b) == getattr(kq, code), call.__name__


@pytest.mark.parametrize("bad,code", BAD_BATCHES, ids=str)
def test_bad_batches(kq, bad, code):
    c, b = cache(kq), batch(kq, **bad)
    for call in (rope, attn, keep):
        assert call(kq, c, b) == getattr(kq, code), call.__name__


def test_no_descriptor(kq):
    for call in (rope, attn, keep):
        assert call(kq, None, batch(kq)) == kq.KQ_ERR_NULL
        assert call(kq, cache(kq), None) == kq.KQ_ERR_NULL


def test_no_rows_is_no_work(kq):
    for b in (batch(kq, n_tokens=0), batch(kq, n_seqs=0)):
        b.offsets = b.lens = b.pages = None
        c = cache(kq, k=None, v=None)
        assert rope(kq, c, b, x=None, q=None) == kq.KQ_OK
        assert attn(kq, c, b, q=None, out=None) == kq.KQ_OK
        assert keep(kq, c, b, path=None, counts=None) == kq.KQ_OK
    assert keep(kq, None, batch(kq), n=0) == kq.KQ_OK
    assert logprobs(kq, M=0, x=None) == kq.KQ_OK


@pytest.mark.parametrize("kw,code", [
    (dict(q_type=1), "KQ_ERR_FMT"), (dict(q_type=3), "KQ_ERR_FMT"), (dict(q_type=4), "KQ_ERR_FMT"),
    (dict(q_heads=0), "KQ_ERR_SHAPE"), (dict(q_heads=65536), "KQ_ERR_SHAPE"), (dict(rot=12), "KQ_ERR_SHAPE"),
    (dict(rot=136), "KQ_ERR_SHAPE"), (dict(rot=-8), "KQ_ERR_SHAPE"), (dict(n_pos=0), "KQ_ERR_SHAPE"), (dict(n_pos=-1), "KQ_ERR_SHAPE"),
    (dict(eps=-1.0), "KQ_ERR_SHAPE"), (dict(eps=math.nan), "KQ_ERR_SHAPE"), (dict(eps=math.inf), "KQ_ERR_SHAPE"),
    (dict(ldx=1020), "KQ_ERR_SHAPE"), (dict(ldx=1026), "KQ_ERR_SHAPE"), (dict(ldx=-1024), "KQ_ERR_SHAPE"),
    (dict(x=None), "KQ_ERR_NULL"), (dict(q=None), "KQ_ERR_NULL"), (dict(rope=None), "KQ_ERR_NULL"),
    (dict(x=A + 4), "KQ_ERR_ALIGN"), (dict(q=A + 8), "KQ_ERR_ALIGN"), (dict(rope=A + 4), "KQ_ERR_ALIGN"),
    (dict(q_norm=A + 4), "KQ_ERR_ALIGN"), (dict(k_norm=A + 8), "KQ_ERR_ALIGN"), (dict(positions=A + 2), "KQ_ERR_ALIGN")], ids=str)
def test_rope_refusals(kq, kw, code):
    assert rope(kq, cache(kq), batch(kq), **kw) == getattr(kq, code)


def test_rope_grid_limit(kq):
    assert rope(kq, cache(kq), batch(kq, n_tokens=(1 << 30) - 1)) == kq.KQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(q_type=1), "KQ_ERR_FMT"), (dict(q_type=3), "KQ_ERR_FMT"), (dict(out_type=3), "KQ_ERR_FMT"), (dict(out_type=0), "KQ_ERR_FMT"),
    (dict(q_heads=0), "KQ_ERR_SHAPE"), (dict(q_heads=3), "KQ_ERR_SHAPE"), (dict(q_heads=65536), "KQ_ERR_SHAPE"),
    (dict(scale=math.nan), "KQ_ERR_SHAPE"), (dict(scale=math.inf), "KQ_ERR_SHAPE"),
    (dict(max_tokens=65), "KQ_ERR_UNSUPPORTED"), (dict(max_tokens=-1), "KQ_ERR_SHAPE"), (dict(max_tokens=0), "KQ_ERR_SHAPE"),
    (dict(max_len=0), "KQ_ERR_SHAPE"), (dict(max_len=-1), "KQ_ERR_SHAPE"), (dict(max_len=(1 << 30) + 1), "KQ_ERR_SHAPE"),
    (dict(q=None), "KQ_ERR_NULL"), (dict(out=None), "KQ_ERR_NULL"), (dict(q=A + 2), "KQ_ERR_ALIGN"), (dict(out=A + 4), "KQ_ERR_ALIGN"),
    (dict(mask=A + 4), "KQ_ERR_ALIGN"), (dict(max_len=10000, ws=None), "KQ_ERR_NULL"),
    (dict(max_len=10000, ws=A + 8), "KQ_ERR_ALIGN"), (dict(max_len=10000, ws_bytes=100), "KQ_ERR_SHAPE")], ids=str)
def test_attn_refusals(kq, kw, code):
    assert attn(kq, cache(kq), batch(kq), **kw) == getattr(kq, code)


def test_attn_size_limits(kq):
    big = batch(kq, n_tokens=(1 << 31) // (4 * 128))
    assert attn(kq, cache(kq), big) == kq.KQ_ERR_UNSUPPORTED
    many = batch(kq, n_seqs=1 << 30)
    assert attn(kq, cache(kq, heads=4), many) == kq.KQ_ERR_UNSUPPORTED   # units past int32


def test_attn_workspace(kq):
    """Calls that cut nothing need none; the size is bounded however long the
    sequences, and falls with no argument."""
    c = cache(kq)
    size = lambda n, t, q, m: kq.kq_attn_tree_workspace(c, batch(kq, n_seqs=n, n_tokens=n * t), q, t, m)  # noqa: E731
    assert size(1, 1, 4, 1) == size(9, 1, 4, 128) == 0
    assert size(1, 1, 4, 100000) > 0
    for n in (1, 5, 64):
        for t in (1, 7, 64):
            last = 0
            for m in (1, 128, 129, 1000, 8191, 131072, 1 << 20):
                s = size(n, t, 16, m)
                assert last <= s <= 2 * 512 * 256 * (128 * 4 + 8) + 16 * n
                last = s
    for bad in (size(1, 65, 4, 10), size(-1, 1, 4, 10), size(1, 1, 5, 10), size(1, 1, 4, 0), size(1, 1, 4, 1 << 31)):
        assert bad == 0


def test_keep_refusals(kq):
    b = batch(kq)
    assert keep(kq, cache(kq), b, n=-1) == kq.KQ_ERR_SHAPE
    assert keep(kq, cache(kq), b, path=None) == kq.KQ_ERR_NULL
    assert keep(kq, cache(kq), b, counts=None) == kq.KQ_ERR_NULL
    assert keep(kq, cache(kq), b, path=A + 2) == kq.KQ_ERR_ALIGN
    assert keep(kq, cache(kq), b, counts=A + 2) == kq.KQ_ERR_ALIGN
    for other in (dict(type=kq.KQ_T_F8), dict(heads=3), dict(dim=64), dict(page=32), dict(n_pages=11)):
        two = (kq.kq_cache * 2)(cache(kq), cache(kq, **other))
        assert keep(kq, two, b, n=2) == kq.KQ_ERR_SHAPE, other
    two = (kq.kq_cache * 2)(cache(kq), cache(kq, v=None))
    assert keep(kq, two, b, n=2) == kq.KQ_ERR_NULL


@pytest.mark.parametrize("kw,code", [
    (dict(type=0), "KQ_ERR_FMT"), (dict(type=4), "KQ_ERR_FMT"), (dict(M=-1), "KQ_ERR_SHAPE"), (dict(V=-1), "KQ_ERR_SHAPE"),
    (dict(V=0, n_top=0), "KQ_ERR_SHAPE"), (dict(ldx=99), "KQ_ERR_SHAPE"), (dict(n_given=-1), "KQ_ERR_SHAPE"), (dict(n_top=-1), "KQ_ERR_SHAPE"),
    (dict(n_top=65), "KQ_ERR_UNSUPPORTED"), (dict(V=3, ldx=3, n_top=4), "KQ_ERR_SHAPE"), (dict(V=1 << 31, ldx=1 << 31), "KQ_ERR_SHAPE"),
    (dict(M=1 << 31), "KQ_ERR_SHAPE"), (dict(x=None), "KQ_ERR_NULL"), (dict(tokens=None), "KQ_ERR_NULL"), (dict(logprob=None), "KQ_ERR_NULL"),
    (dict(ids=None), "KQ_ERR_NULL"), (dict(tops=None), "KQ_ERR_NULL"), (dict(x=A + 2), "KQ_ERR_ALIGN"), (dict(type=2, x=A + 1), "KQ_ERR_ALIGN"),
    (dict(tokens=A + 1), "KQ_ERR_ALIGN"), (dict(logprob=A + 2), "KQ_ERR_ALIGN"), (dict(entropy=A + 2), "KQ_ERR_ALIGN"),
    (dict(ids=A + 2), "KQ_ERR_ALIGN"), (dict(tops=A + 2), "KQ_ERR_ALIGN"), (dict(V=100000, ldx=100000, ws=None), "KQ_ERR_NULL"),
    (dict(V=100000, ldx=100000, ws=A + 4), "KQ_ERR_ALIGN"), (dict(V=100000, ldx=100000, ws_bytes=10), "KQ_ERR_SHAPE")], ids=str)
def test_logprobs_refusals(kq, kw, code):
    assert logprobs(kq, **kw) == getattr(kq, code)


def test_logprobs_workspace(kq):
    assert kq.kq_logprobs_workspace(1, 1000, 20) == 0
    assert kq.kq_logprobs_workspace(1, 128256, 20) > kq.kq_logprobs_workspace(1, 128256, 0) > 0
    for bad in ((0, 10, 0), (-1, 10, 0), (1, 0, 0), (1, 10, 65), (1, 10, 11), (1, 1 << 31, 0)):
        assert kq.kq_logprobs_workspace(*bad) == 0


def test_binding_refuses_host_tensors(kq):
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(ValueError, match="device tensor"):
        kq.PagedCache(z(2, 1, 16, 64), z(2, 1, 64, 16))
    with pytest.raises(ValueError, match="n_pages"):
        kq.PagedCache(z(2, 16, 64), z(2, 64, 16))
    with pytest.raises(ValueError, match="device tensor"):
        kq.Batch(z(2, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        kq.logprobs(z(2, 10))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_argument_handling_under_sanitizers(tmp_path):
    """kq_step_api.cpp linked with recording stubs instead of the kernels' launchers
    (tests/host/step_driver.cpp), host code under AddressSanitizer and UBSan."""
    exe = str(tmp_path / "step_driver")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(ROOT, "tests", "host", "step_driver.cpp"),
                    os.path.join(ROOT, "block_quantized_matmul_act_amd", "csrc", "kq_step_api.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-4000:]


def test_step_variants_named_and_counted(kq):
    names = [kq.kq_step_variant_name(v) for v in range(kq.kq_num_step_variants())]
    assert names == ["rope_append", "attn_few", "attn_rows", "cache_keep", "logprobs_row", "logprobs_parts"]
    assert kq.kq_step_variant_name(len(names)) is None and kq.kq_step_variant_name(-1) is None
    assert kq.kq_step_count(-1) == kq.kq_step_count(len(names)) == 0
    kq.kq_step_count_reset()
    assert set(kq.step_counts().values()) == {0}
    assert not set(names) & set(kq.dispatch_counts())  # the products' counters are apart
