"""CPU tests of the operators around the products of a layer at the ends of their
ranges: sizes that the kernels' 32-bit counts do not hold, and buffers that act_views
takes."""
from __future__ import annotations

import pytest

from test_layer_abi import kq, lora  # noqa: F401


@pytest.mark.parametrize("act,K", [(1, (1 << 31) - 256), (2, (1 << 31) - 128), (1, (1 << 31) - 4096), (2, (1 << 31) - 4096)])
@pytest.mark.parametrize("M", [1, 600])
def test_lora_inputs_that_a_step_of_the_loops_would_overflow(kq, act, K, M):  # noqa: F811
    """The kernels go through K in steps of up to 4096 and count in 32 bits: the step past
    the last column has to stay in them."""
    assert lora(kq, rank=8, n=1, act=act, M=M, K=K) == kq.KQ_ERR_UNSUPPORTED
    assert lora(kq, rank=8, n=1, act=act, M=0, K=K) == kq.KQ_OK


@pytest.mark.parametrize("act,M,K", [(1, 5, 512), (1, 1, 256), (1, 64, 1280), (2, 3, 384), (2, 7, 128)])
@pytest.mark.parametrize("at", [0, 16])
def test_act_views_want_only_what_they_show(kq, act, M, K, at):  # noqa: F811
    """A buffer that ends with the last section that is viewed (without Q8_K's alpha, or the
    bytes that round a section's size up) is enough, one byte less is not."""
    torch = pytest.importorskip("torch")
    section = lambda s: kq.kq_act_section_offset(act, s, M, K)  # noqa: E731
    bs = 256 if act == 1 else 128
    end = section(kq.KQ_SEC_BSUMS) + 2 * M * (K // 16) if act == 1 else section(kq.KQ_SEC_D) + 4 * M * (K // bs)
    assert end < kq.kq_act_bytes(act, M, K)
    data = torch.arange(at + end + 9).remainder(251).to(torch.uint8)
    for size in (end, end + 1, end + 4):
        buf = data[at:at + size]
        qs, d, bsums = kq.act_views(buf, act, M, K)
        assert torch.equal(qs, buf[:M * K].view(torch.int8).view(M, K))
        from_d = buf[section(kq.KQ_SEC_D):][:4 * M * (K // bs)].clone().view(torch.int32).view(K // bs, M)
        assert d.shape == (M, K // bs) and torch.equal(d.t().contiguous().view(torch.int32), from_d)
        if act == 1:
            assert torch.equal(bsums, buf[section(kq.KQ_SEC_BSUMS):end].clone().view(torch.int16).view(M, K // 16))
        else:
            assert bsums is None
    with pytest.raises(ValueError):
        kq.act_views(data[at:at + end - 1], act, M, K)


@pytest.mark.parametrize("act,M,K", [(0, 4, 256), (3, 4, 128), (1, 4, 384), (1, 3, 100), (2, 4, 192), (2, -1, 128), (1, 0, 100)])
def test_act_views_refuse_what_is_no_buffer(kq, act, M, K):  # noqa: F811
    """An unknown format, or sizes that no buffer has, inside a longer tensor: an error, and no
    view of what lies around."""
    torch = pytest.importorskip("torch")
    whole = torch.zeros(1 << 14, dtype=torch.uint8)
    for buf in (whole, whole[256:], whole[4096:8192]):
        with pytest.raises(ValueError, match="act_views"):
            kq.act_views(buf, act, M, K)


def test_act_views_refuse_bytes_that_lie_apart(kq):  # noqa: F811
    """Columns of a wider tensor hold as many bytes, but not one after another."""
    torch = pytest.importorskip("torch")
    need = kq.kq_act_bytes(1, 2, 256)
    wide = torch.zeros((4, need), dtype=torch.uint8)
    for buf in (wide[:, :need // 2], wide[:, 0], wide.view(-1)[::2]):
        with pytest.raises(ValueError, match="act_views"):
            kq.act_views(buf, 1, 2, 256)
    assert kq.act_views(wide[1], 1, 2, 256)[0].shape == (2, 256)


@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("f16", [False, True], ids=["bf16", "f16"])
def test_the_bound_of_the_second_product_tells_24_bits_from_16(rank, f16):
    """What holds lora's second product on the GPU: with all three parts of t the plain form
    keeps to its bound, with two of them, or with B's first 8 bits in float16, it does not."""
    torch = pytest.importorskip("torch")
    import numpy as np

    import layer_edge_ref as eref
    rng = np.random.default_rng(rank)
    M, N, K, n, kind = 40, 150, 512, 3, torch.float16 if f16 else torch.bfloat16
    A, B, scale, ids, base, picked = eref.pick_case(rng, M, N, rank, K, n, kind, dense=False)
    qs, d = torch.from_numpy(rng.integers(-127, 128, (M, K)).astype(np.int8)), torch.from_numpy(rng.uniform(1e-3, 1e-1, (M, 2)).astype(np.float32))
    t = eref.picked_t(qs, d, 256, scale, ids, picked)
    x = qs.double() * d.double().repeat_interleave(256, 1)
    for i in range(n):   # (t is the adapter's first product)
        rows = ids == i
        want = (x[rows] @ A[i].double().t()) * float(scale[i])
        assert ((t[rows].double() - want).abs() <= 2.0 ** -23 * want.abs()).all()
    want, bound = eref.second(t, B, ids, base, dense=False)

    def off(t, B):
        return ((eref.second(t, B, ids, base, dense=False)[0] - want).abs() - bound).max().item()
    assert torch.equal(eref.parts(t, 3), t) and off(eref.parts(t, 3), B) <= 0
    assert off(eref.parts(t, 2), B) > 0 and off(eref.parts(t, 1), B) > 0
    if f16:
        assert off(t, B.to(torch.bfloat16).to(torch.float16)) > 0
