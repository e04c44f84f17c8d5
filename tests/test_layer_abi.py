"""CPU tests of the C ABI of the operators around the products of a layer
(norm_quantize, attn_chunk, lora): invalid arguments are refused with their status
code before any HIP call, sizes of workspaces, plans, and the binding's own checks."""
from __future__ import annotations

import math
import os
import shutil
import subprocess

import pytest

from test_step_abi import BAD_BATCHES, BAD_CACHES, A, ROOT, batch, cache, kq, ref  # noqa: F401


def norm(kq, **kw):
    f = dict(act=kq.KQ_ACT_Q8_K, x_type=kq.KQ_T_F32, x=A, ldx=512, r_type=kq.KQ_T_BF16, residual=A, ldr=512, sum=A, lds=512,
             weight=A, eps=1e-6, M=3, K=512, a_q8=A)
    f.update(kw)
    return kq.lib().kq_norm_quantize(*f.values(), None)


def chunk(kq, c=None, b=None, **kw):
    f = dict(q_type=kq.KQ_T_BF16, q=A, q_heads=4, window=0, sinks=0, scale=0.1, max_tokens=4, max_len=64,
             out_type=kq.KQ_T_BF16, out=A, ws=A, ws_bytes=1 << 40)
    f.update(kw)
    return kq.lib().kq_attn_chunk(ref(c), ref(b), *f.values(), None)


def lora(kq, **kw):
    f = dict(type=kq.KQ_T_BF16, rank=16, A=A, B=A, scale=A, n=3, act=kq.KQ_ACT_Q8_K, a_q8=A, M=5, N=100, K=512, ids=A,
             base=A, ldb=100, out=A + 4096, ldo=100, ws=A, ws_bytes=1 << 40)
    f.update(kw)
    return kq.lib().kq_lora(*f.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(act=0), "KQ_ERR_FMT"), (dict(act=3), "KQ_ERR_FMT"), (dict(x_type=0), "KQ_ERR_FMT"), (dict(x_type=4), "KQ_ERR_FMT"),
    (dict(r_type=0), "KQ_ERR_FMT"), (dict(r_type=4, sum=None), "KQ_ERR_FMT"), (dict(r_type=4, residual=None), "KQ_ERR_FMT"),
    (dict(M=-1), "KQ_ERR_SHAPE"), (dict(K=-256), "KQ_ERR_SHAPE"), (dict(K=384), "KQ_ERR_SHAPE"), (dict(act=2, K=192), "KQ_ERR_SHAPE"),
    (dict(M=1 << 31), "KQ_ERR_SHAPE"), (dict(eps=-1.0), "KQ_ERR_SHAPE"), (dict(eps=math.nan), "KQ_ERR_SHAPE"), (dict(eps=math.inf), "KQ_ERR_SHAPE"),
    (dict(ldx=508), "KQ_ERR_SHAPE"), (dict(ldx=514), "KQ_ERR_SHAPE"), (dict(ldr=516), "KQ_ERR_SHAPE"), (dict(lds=504), "KQ_ERR_SHAPE"),
    (dict(x_type=3, ldx=516), "KQ_ERR_SHAPE"), (dict(lds=520), "KQ_ERR_SHAPE"), (dict(ldx=1 << 41), "KQ_ERR_SHAPE"),
    (dict(K=65536 + 256, ldx=1 << 20, ldr=1 << 20, lds=1 << 20), "KQ_ERR_UNSUPPORTED"),
    (dict(x=None), "KQ_ERR_NULL"), (dict(a_q8=None), "KQ_ERR_NULL"), (dict(x=A + 4), "KQ_ERR_ALIGN"), (dict(residual=A + 8), "KQ_ERR_ALIGN"),
    (dict(sum=A + 2), "KQ_ERR_ALIGN"), (dict(weight=A + 4), "KQ_ERR_ALIGN"), (dict(a_q8=A + 1), "KQ_ERR_ALIGN")], ids=str)
def test_norm_refusals(kq, kw, code):  # noqa: F811
    assert norm(kq, **kw) == getattr(kq, code)


def test_norm_no_work(kq):  # noqa: F811
    assert norm(kq, M=0, x=None, a_q8=None) == kq.KQ_OK
    assert norm(kq, K=0, ldx=0, ldr=0, lds=0, x=None, a_q8=None) == kq.KQ_OK
    # neither a residual nor a sum: their type and strides are not looked at
    assert norm(kq, M=0, residual=None, sum=None, r_type=0, ldr=-1, lds=-1) == kq.KQ_OK


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=str)
def test_chunk_bad_caches(kq, bad, code):  # noqa: F811
    assert chunk(kq, cache(kq, **bad), batch(kq)) == getattr(kq, code)


@pytest.mark.parametrize("bad,code", BAD_BATCHES, ids=str)
def test_chunk_bad_batches(kq, bad, code):  # noqa: F811
    assert chunk(kq, cache(kq), batch(kq, **bad)) == getattr(kq, code)


@pytest.mark.parametrize("kw,code", [
    (dict(q_type=1), "KQ_ERR_FMT"), (dict(q_type=3), "KQ_ERR_FMT"), (dict(out_type=3), "KQ_ERR_FMT"), (dict(out_type=0), "KQ_ERR_FMT"),
    (dict(q_heads=0), "KQ_ERR_SHAPE"), (dict(q_heads=3), "KQ_ERR_SHAPE"), (dict(q_heads=65536), "KQ_ERR_SHAPE"),
    (dict(scale=math.nan), "KQ_ERR_SHAPE"), (dict(scale=math.inf), "KQ_ERR_SHAPE"),
    (dict(window=-1), "KQ_ERR_SHAPE"), (dict(window=(1 << 30) + 1), "KQ_ERR_SHAPE"), (dict(sinks=-1), "KQ_ERR_SHAPE"),
    (dict(sinks=1 << 31), "KQ_ERR_SHAPE"), (dict(max_tokens=-1), "KQ_ERR_SHAPE"), (dict(max_tokens=0), "KQ_ERR_SHAPE"),
    (dict(max_len=0), "KQ_ERR_SHAPE"), (dict(max_len=-1), "KQ_ERR_SHAPE"), (dict(max_len=(1 << 30) + 1), "KQ_ERR_SHAPE"),
    (dict(q=None), "KQ_ERR_NULL"), (dict(out=None), "KQ_ERR_NULL"), (dict(q=A + 2), "KQ_ERR_ALIGN"), (dict(out=A + 4), "KQ_ERR_ALIGN"),
    (dict(max_len=10000, ws=None), "KQ_ERR_NULL"), (dict(max_len=10000, ws=A + 8), "KQ_ERR_ALIGN"),
    (dict(max_len=10000, ws_bytes=100), "KQ_ERR_SHAPE")], ids=str)
def test_chunk_refusals(kq, kw, code):  # noqa: F811
    assert chunk(kq, cache(kq), batch(kq), **kw) == getattr(kq, code)


def test_chunk_no_work_and_no_descriptor(kq):  # noqa: F811
    for b in (batch(kq, n_tokens=0), batch(kq, n_seqs=0)):
        b.offsets = b.lens = b.pages = None
        assert chunk(kq, cache(kq, k=None, v=None), b, q=None, out=None) == kq.KQ_OK
    assert chunk(kq, None, batch(kq)) == kq.KQ_ERR_NULL
    assert chunk(kq, cache(kq), None) == kq.KQ_ERR_NULL


def test_chunk_size_limits(kq):  # noqa: F811
    assert chunk(kq, cache(kq), batch(kq, n_tokens=(1 << 31) // (4 * 128))) == kq.KQ_ERR_UNSUPPORTED
    assert chunk(kq, cache(kq, heads=4), batch(kq, n_seqs=1 << 30)) == kq.KQ_ERR_UNSUPPORTED


def test_chunk_workspace(kq):  # noqa: F811
    """None where every block is a workgroup's; bounded however long the sequences; 0 for bad arguments."""
    c = cache(kq, heads=8)
    size = lambda n, t, q, w, m: kq.kq_attn_chunk_workspace(c, batch(kq, n_seqs=n, n_tokens=n * t), q, w, 4, t, m)  # noqa: E731
    assert size(200, 1, 32, 0, 500) == size(1, 4096, 32, 0, 4096) == size(1, 1, 32, 0, 64) == size(1, 1, 32, 30, 1 << 20) == 0
    assert size(1, 1, 32, 0, 100000) > size(1, 1, 32, 0, 500) > 0
    for n in (1, 5, 64):
        for t in (1, 7, 64, 1000):
            for m in (1, 128, 1000, 131072, 1 << 30):
                for w in (0, 1, 5000):
                    # two slots to each of 256 workgroups of 256 rows (or 512 of 128) and the blocks' units
                    assert size(n, t, 16, w, m) <= 2 * 256 * 256 * (128 * 4 + 8) + 1025 * 4
    for bad in (size(-1, 1, 8, 0, 10), size(1, 1, 9, 0, 10), size(1, 1, 8, 0, 0), size(1, 1, 8, -1, 10), size(1, 0, 8, 0, 10)):
        assert bad == 0


@pytest.mark.parametrize("kw,code", [
    (dict(type=1), "KQ_ERR_FMT"), (dict(type=4), "KQ_ERR_FMT"), (dict(act=0), "KQ_ERR_FMT"),
    (dict(rank=0), "KQ_ERR_SHAPE"), (dict(rank=-8), "KQ_ERR_SHAPE"), (dict(rank=12), "KQ_ERR_UNSUPPORTED"), (dict(rank=256), "KQ_ERR_UNSUPPORTED"),
    (dict(n=-1), "KQ_ERR_SHAPE"), (dict(n=1 << 31), "KQ_ERR_SHAPE"), (dict(M=-1), "KQ_ERR_SHAPE"), (dict(N=-1), "KQ_ERR_SHAPE"),
    (dict(K=-256), "KQ_ERR_SHAPE"), (dict(K=384), "KQ_ERR_SHAPE"), (dict(N=1 << 31, ldo=1 << 31, ldb=1 << 31), "KQ_ERR_SHAPE"),
    (dict(n=1 << 30, N=1 << 20, ldo=1 << 20, ldb=1 << 20), "KQ_ERR_SHAPE"),
    (dict(ldo=99), "KQ_ERR_SHAPE"), (dict(ldb=99), "KQ_ERR_SHAPE"), (dict(ldo=1 << 41), "KQ_ERR_SHAPE"),
    (dict(base=A, out=A, ldb=100, ldo=101), "KQ_ERR_SHAPE"), (dict(M=65535 * 32 + 1), "KQ_ERR_UNSUPPORTED"),
    (dict(n=1, N=(1 << 31) - 256, ldo=1 << 31, ldb=1 << 31), "KQ_ERR_UNSUPPORTED"),
    (dict(A=None), "KQ_ERR_NULL"), (dict(B=None), "KQ_ERR_NULL"), (dict(a_q8=None), "KQ_ERR_NULL"), (dict(ids=None), "KQ_ERR_NULL"),
    (dict(out=None), "KQ_ERR_NULL"), (dict(ws=None), "KQ_ERR_NULL"), (dict(A=A + 8), "KQ_ERR_ALIGN"), (dict(B=A + 2), "KQ_ERR_ALIGN"),
    (dict(a_q8=A + 4), "KQ_ERR_ALIGN"), (dict(ids=A + 2), "KQ_ERR_ALIGN"), (dict(scale=A + 2), "KQ_ERR_ALIGN"),
    (dict(base=A + 1), "KQ_ERR_ALIGN"), (dict(out=A + 2), "KQ_ERR_ALIGN"), (dict(ws=A + 8), "KQ_ERR_ALIGN"),
    (dict(ws_bytes=5 * 16 * 4 - 1), "KQ_ERR_SHAPE")], ids=str)
def test_lora_refusals(kq, kw, code):  # noqa: F811
    assert lora(kq, **kw) == getattr(kq, code)


def test_lora_no_work(kq):  # noqa: F811
    none = dict(A=None, B=None, a_q8=None, ids=None, base=None, out=None, ws=None)
    assert lora(kq, M=0, **none) == kq.KQ_OK
    assert lora(kq, N=0, ldo=0, **none) == kq.KQ_OK
    assert kq.kq_lora_workspace(16, 5) == 320
    for bad in ((0, 5), (16, 0), (16, -1), (256, 5), (16, 1 << 31)):
        assert kq.kq_lora_workspace(*bad) == 0


def test_layer_variants_named_and_counted(kq):  # noqa: F811
    names = [kq.kq_layer_variant_name(v) for v in range(kq.kq_num_layer_variants())]
    assert names == ["norm_quantize", "chunk_few", "chunk_rows", "lora_few", "lora_tile"]
    assert kq.kq_layer_variant_name(len(names)) is None and kq.kq_layer_variant_name(-1) is None
    assert kq.kq_layer_count(-1) == kq.kq_layer_count(len(names)) == 0
    kq.kq_layer_count_reset()
    assert set(kq.layer_counts().values()) == {0}


def test_binding_refuses_host_tensors(kq):  # noqa: F811
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(ValueError, match="device tensor"):
        kq.norm_quantize(z(2, 256))
    with pytest.raises(ValueError, match="device tensor"):
        kq.lora(z(600, dtype=torch.uint8), z(1, 8, 256, dtype=torch.bfloat16), z(1, 4, 8, dtype=torch.bfloat16),
                z(2, dtype=torch.int32))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_argument_handling_under_sanitizers(tmp_path):
    """kq_layer_api.cpp linked with recording stubs instead of the kernels' launchers
    (tests/host/layer_driver.cpp), host code under AddressSanitizer and UBSan."""
    exe = str(tmp_path / "layer_driver")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(ROOT, "tests", "host", "layer_driver.cpp"),
                    os.path.join(ROOT, "block_quantized_matmul_act_amd", "csrc", "kq_layer_api.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-4000:]
