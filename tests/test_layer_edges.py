"""CPU tests of the operators around the products of a layer at the ends of their
ranges: sizes that the kernels' 32-bit counts do not hold."""
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
