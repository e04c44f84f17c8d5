"""GPU tests of the operators around the products of a layer at the edges of their ranges:
the bits of lora's second product, workspaces that hold anything."""
from __future__ import annotations

import math

import numpy as np
import pytest

import layer_edge_ref as eref
import step_ref as ref
from step_ref import BF16, F16

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
