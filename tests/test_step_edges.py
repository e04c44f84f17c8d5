"""CPU tests of the step operators at the edges of their ranges: what the host
can tell of a call is refused, whatever the arrays on the device hold."""
from __future__ import annotations

import contextlib
import os
import shutil
import subprocess
import types

import pytest

from test_step_abi import A, attn, batch, cache, keep, kq, logprobs, rope  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def test_rows_of_no_sequence(kq, devices):  # noqa: F811
    """Nothing would compute them, and what comes back would be what lay in memory."""
    c, b, x, q = step_args(kq, 3, 0)
    with pytest.raises(ValueError, match="no sequence"):
        kq.rope_append(c, b, x, 4, out=q)
    with pytest.raises(ValueError, match="no sequence"):
        kq.attn_tree(c, b, q, out=q)


@pytest.fixture
def devices(kq, monkeypatch):  # noqa: F811
    """Two devices of which 0 is current; the library notes which one is current
    when it is called, and whose stream it is given."""
    now, calls = [0], []
    kq._step_lib()

    @contextlib.contextmanager
    def switch(device):
        before, now[0] = now[0], device
        yield
        now[0] = before

    def call(*args):
        calls.append((now[0], args[-1]))
        return 0

    names = ("kq_rope_append", "kq_attn_tree", "kq_cache_keep", "kq_logprobs")
    spaces = ("kq_attn_tree_workspace", "kq_logprobs_workspace")
    fake = types.SimpleNamespace(**{n: call for n in names}, **{n: lambda *a: 0 for n in spaces})
    monkeypatch.setattr(kq, "_step", fake)
    monkeypatch.setattr(kq, "_current_device", lambda: now[0])
    monkeypatch.setattr(kq, "_current_stream", lambda device: 100 + device)
    monkeypatch.setattr(torch.cuda, "device", switch)
    return now, calls


def calls_on(kq, device):  # noqa: F811
    c, b, x, q = step_args(kq, 3, 3, device)
    i32 = lambda *n: Tensor(torch.int32, *n, device=device)  # noqa: E731
    logits = Tensor(torch.float32, 3, 50, device=device)
    return [lambda **kw: kq.rope_append(c, b, x, 4, out=q, **kw), lambda **kw: kq.attn_tree(c, b, q, out=q, **kw),
            lambda **kw: kq.cache_keep([c], b, i32(3), i32(3), **kw),
            lambda **kw: kq.logprobs(logits, i32(3, 2), n_top=1, **kw)]


@pytest.mark.parametrize("device", [0, 1])
def test_calls_run_on_their_tensors_device(kq, devices, device):  # noqa: F811
    now, seen = devices
    for call in calls_on(kq, device):
        call()
    assert seen == [(device, 100 + device)] * 4 and now == [0]


def test_stream_of_another_device(kq, devices):  # noqa: F811
    for call in calls_on(kq, 1):
        with pytest.raises(ValueError, match="stream of device 0"):
            call(stream=types.SimpleNamespace(device_index=0, cuda_stream=7))
    assert not devices[1]


def test_stream_with_host_tensors(kq):  # noqa: F811
    with pytest.raises(ValueError, match="device tensors"):
        kq.logprobs(torch.zeros(2, 10), stream=5)


def test_scales_that_leave_fp32(kq):  # noqa: F811
    """A cache scale without a finite inverse, a score scale that is infinite in
    the kernel's units: zeros would come out as NaN."""
    for bad in (dict(k_scale=1e-39), dict(v_scale=1e-39)):
        assert rope(kq, cache(kq, **bad), batch(kq)) == kq.KQ_ERR_SHAPE
    assert attn(kq, cache(kq), batch(kq), scale=3e38) == kq.KQ_ERR_SHAPE
    assert attn(kq, cache(kq, k_scale=1e20), batch(kq), scale=-1e19) == kq.KQ_ERR_SHAPE


def test_launches_past_the_grid(kq):  # noqa: F811
    """More workgroups of 256 threads than a launch can count threads for."""
    n = 1 << 24
    one = dict(heads=1, dim=64)
    assert logprobs(kq, M=n, V=64, ldx=64) == kq.KQ_ERR_UNSUPPORTED
    assert logprobs(kq, M=(1 << 31) - 1, V=1, ldx=1, n_top=0) == kq.KQ_ERR_UNSUPPORTED
    assert rope(kq, cache(kq, **one), batch(kq, n_tokens=4 * n, n_seqs=n), q_heads=1, rot=0) == kq.KQ_ERR_UNSUPPORTED
    assert keep(kq, cache(kq, **one), batch(kq, n_seqs=n)) == kq.KQ_ERR_UNSUPPORTED
    assert attn(kq, cache(kq, **one), batch(kq, n_seqs=n, n_tokens=n), q_heads=1, max_tokens=1, max_len=129) == kq.KQ_ERR_UNSUPPORTED


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_every_launch_that_is_let_through_fits_the_grid(tmp_path):
    """kq_step_api.cpp with stubs for the launchers (tests/host/step_grids.cpp):
    the workgroups of each launch at sizes around the limit."""
    exe = str(tmp_path / "step_grids")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", os.path.join(ROOT, "tests", "host", "step_grids.cpp"),
                    os.path.join(ROOT, "block_quantized_matmul_act_amd", "csrc", "kq_step_api.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-4000:]


def test_one_batch_with_other_row_counts(kq, devices, monkeypatch):  # noqa: F811
    """While a call is under way (in another thread, say) the same batch serves
    calls of other row counts: each has its own, to its end."""
    c, b, x, q = step_args(kq, 3, 3)
    _, _, more, q_more = step_args(kq, 5, 3)
    rows = []

    def n_tokens(at):
        return kq.kq_batch.from_address(at).n_tokens

    def append(cache, at, *a):
        outer = len(rows) == 0
        rows.append(n_tokens(at))
        if outer:
            kq.rope_append(c, b, more, 4, out=q_more)
            kq.attn_tree(c, b, q_more, out=q_more)
            kq.cache_keep([c], b, Tensor(torch.int32, 4), Tensor(torch.int32, 3))
            rows.append(n_tokens(at))
        return 0

    def attend(cache, at, *a):
        rows.append(n_tokens(at))
        return 0

    monkeypatch.setattr(kq._step, "kq_rope_append", append)
    monkeypatch.setattr(kq._step, "kq_attn_tree", attend)
    monkeypatch.setattr(kq._step, "kq_cache_keep", lambda caches, n, at, *a: rows.append(n_tokens(at)) or 0)
    kq.rope_append(c, b, x, 4, out=q)
    assert rows == [3, 5, 5, 4, 3]


def test_logprobs_of_fewer_than_no_alternatives(kq, devices):  # noqa: F811
    with pytest.raises(ValueError, match="n_top"):
        kq.logprobs(Tensor(torch.float32, 3, 50), n_top=-1)
    assert not devices[1]
