"""CPU tests of the step operators at the edges of their ranges: what the host
can tell of a call is refused, whatever the arrays on the device hold."""
from __future__ import annotations

import pytest

from test_step_abi import A, attn, batch, cache, kq  # noqa: F401

torch = pytest.importorskip("torch")


class Tensor:
    """A device tensor as far as the binding looks at one: nothing is behind its
    address."""

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.on = dtype, torch.Size(shape), device
        self.is_cuda, self.device = True, torch.device("cpu")   # (where the binding allocates)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(torch.empty(self.shape, device="meta").stride())

    def get_device(self):
        return self.on

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


def step_args(kq, rows, seqs, device=0):  # noqa: F811
    t = lambda *a: Tensor(*a, device=device)  # noqa: E731
    i32, bf = torch.int32, torch.bfloat16
    c = kq.PagedCache(t(bf, 9, 2, 16, 64), t(bf, 9, 2, 64, 16))
    b = kq.Batch(t(i32, seqs + 1), t(i32, seqs), t(i32, seqs, 4))
    return c, b, t(torch.float32, rows, 8 * 64), t(bf, rows, 4, 64)


@pytest.mark.parametrize("seqs,tokens,bound", [(1, 65, 64), (3, 13, 4), (3, 1 << 20, 64), (2, 3, 1)])
def test_attn_more_rows_than_the_bound_allows(kq, seqs, tokens, bound):  # noqa: F811
    """Some sequence has more rows than max_tokens: refused, and no workspace."""
    s = batch(kq, n_seqs=seqs, n_tokens=tokens)
    assert attn(kq, cache(kq), s, max_tokens=bound) == kq.KQ_ERR_SHAPE
    assert kq.kq_attn_tree_workspace(cache(kq), s, 4, bound, 100000) == 0
    s.n_tokens = seqs * bound
    assert kq.kq_attn_tree_workspace(cache(kq), s, 4, bound, 100000) > 0


def test_rows_of_no_sequence(kq):  # noqa: F811
    """Nothing would compute them, and what comes back would be what lay in memory."""
    c, b, x, q = step_args(kq, 3, 0)
    with pytest.raises(ValueError, match="no sequence"):
        kq.rope_append(c, b, x, 4, out=q)
    with pytest.raises(ValueError, match="no sequence"):
        kq.attn_tree(c, b, q, out=q)
