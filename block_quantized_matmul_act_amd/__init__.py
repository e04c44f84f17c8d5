"""Python binding of libkq (include/kq.h): block-quantized GEMM for MI355X.

Argument marshalling only.  Every step of the path runs in the HIP kernels of
libkq.so; there is no CPU fallback.  If the library is missing the first call
raises.  The kq_* functions mirror the C ABI one to one and accept torch
tensors (their data_ptr() is passed) or plain integer addresses.  `stream`
defaults to torch's current HIP stream.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkq.so")

KQ_Q4_K, KQ_Q6_K, KQ_TQ, KQ_TQ2 = 1, 2, 3, 4
KQ_ACT_Q8_K, KQ_ACT_Q8_128 = 1, 2
KQ_SEC_QS, KQ_SEC_D, KQ_SEC_BSUMS, KQ_SEC_ALPHA = 0, 1, 2, 3
KQ_OK = 0
KQ_DEBUG_UNPACK_MAX_BLOCKS = 1 << 24
KQ_GEMM_ID_MAX_EXPERTS = 1024
KQ_ERR_FMT, KQ_ERR_SHAPE, KQ_ERR_NULL, KQ_ERR_ALIGN, KQ_ERR_UNSUPPORTED, KQ_ERR_HIP = (
    -1, -2, -3, -4, -5, -6)
(KQ_CALIB_MFMA_I8, KQ_CALIB_MFMA_I8_TOGGLE, KQ_CALIB_VALU_F32, KQ_CALIB_MFMA_I8_VALU,
 KQ_CALIB_HBM_READ) = 0, 1, 2, 3, 4

KQ_T_F32, KQ_T_BF16, KQ_T_F16, KQ_T_F8 = 1, 2, 3, 4
KQ_ATTN_MAX_TOKENS = KQ_KEEP_MAX_TOKENS = KQ_LOGPROBS_MAX_TOP = 64

# Every symbol include/kq.h declares, with its ctypes signature.
_P, _I, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class kq_cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("n_pages", _I64), ("type", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("page", ctypes.c_int32), ("k_scale", _F), ("v_scale", _F)]


class kq_batch(ctypes.Structure):
    _fields_ = [("offsets", _P), ("lens", _P), ("pages", _P), ("n_seqs", _I64), ("n_tokens", _I64),
                ("max_pages", _I64)]


SIGNATURES = {
    "kq_weight_bytes": (_SZ, [_I, _I64, _I64]),
    "kq_act_bytes": (_SZ, [_I, _I64, _I64]),
    "kq_act_section_offset": (_I64, [_I, _I, _I64, _I64]),
    "kq_act_fmt_for": (_I, [_I]),
    "kq_quantize_act": (_I, [_I, _P, _I64, _I64, _P, _P]),
    "kq_gemm": (_I, [_I, _P, _P, _I64, _I64, _I64, _P, _P]),
    "kq_gemm_subsums": (_I, [_I, _P, _P, _I64, _I64, _I64, _P, _P]),
    "kq_debug_unpack": (_I, [_I, _P, _I64, _P, _P, _P]),
    "kq_gemm_id": (_I, [_I, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _I64, _P, _P]),
    "kq_num_variants": (_I, []),
    "kq_variant_name": (ctypes.c_char_p, [_I]),
    "kq_dispatch_count": (ctypes.c_uint64, [_I]),
    "kq_dispatch_reset": (None, []),
    "kq_num_step_variants": (_I, []),
    "kq_step_variant_name": (ctypes.c_char_p, [_I]),
    "kq_step_count": (ctypes.c_uint64, [_I]),
    "kq_step_count_reset": (None, []),
    "kq_select_variant": (_I, [_I, _I64, _I64, _I64]),
    "kq_calib_launch": (_I, [_I, _I, _P, _I64, ctypes.POINTER(ctypes.c_double), _P]),
    "kq_rope_append": (_I, [_P, _P, _P, _I64, _I64, _P, _P, _F, _P, _I64, _I64, _I, _P, _I, _P, _P]),
    "kq_attn_tree": (_I, [_P, _P, _I, _P, _I64, _P, _F, _I64, _I64, _I, _P, _P, _SZ, _P]),
    "kq_attn_tree_workspace": (_SZ, [_P, _P, _I64, _I64, _I64]),
    "kq_cache_keep": (_I, [_P, _I64, _P, _P, _P, _P]),
    "kq_logprobs": (_I, [_I, _P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "kq_logprobs_workspace": (_SZ, [_I64, _I64, _I64]),
    "kq_strerror": (ctypes.c_char_p, [_I]),
    "kq_version": (_I, []),
}


class KQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {kq_strerror(status)} (status {status})")
        self.status = status


_lib = None


def lib():
    """Load libkq.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(hipcc --offload-arch=gfx950); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> int:
    if status != KQ_OK:
        raise KQError(status, where)
    return status


def _need(t, nbytes, what, dtype=None):
    """Host-side check of a torch tensor argument before its address goes to the
    library (plain integer addresses are passed through unchecked): a
    contiguous device tensor of the right element type holding at least
    nbytes bytes.  Raises ValueError; nothing is launched."""
    if t is None or isinstance(t, int):
        return
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{what}: expected a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    if dtype is not None and str(t.dtype) != "torch." + dtype:
        raise ValueError(f"{what}: expected dtype {dtype}, got {t.dtype}")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{what}: {have} bytes, {nbytes} needed")


def _sub_block(fmt):
    return {KQ_Q4_K: 32, KQ_Q6_K: 16}.get(fmt, 128)


# ---------------------------------------------------------------- C ABI mirror

def kq_weight_bytes(fmt, N, K):
    return lib().kq_weight_bytes(fmt, N, K)


def kq_act_bytes(act_fmt, M, K):
    return lib().kq_act_bytes(act_fmt, M, K)


def kq_act_section_offset(act_fmt, section, M, K):
    return lib().kq_act_section_offset(act_fmt, section, M, K)


def kq_act_fmt_for(fmt):
    return lib().kq_act_fmt_for(fmt)


def kq_quantize_act(act_fmt, x, M, K, a_q8, stream=None):
    _need(x, 4 * max(M, 0) * max(K, 0), "kq_quantize_act x", "float32")
    _need(a_q8, kq_act_bytes(act_fmt, M, K), "kq_quantize_act a_q8")
    return _check(lib().kq_quantize_act(act_fmt, _ptr(x), M, K, _ptr(a_q8), _stream(stream)),
                  "kq_quantize_act")


def _need_gemm_inputs(fmt, W, a_q8, M, N, K, where, n_experts=1):
    _need(W, n_experts * kq_weight_bytes(fmt, N, K), where + " W")
    act = kq_act_fmt_for(fmt)
    if act > 0:
        _need(a_q8, kq_act_bytes(act, M, K), where + " a_q8")


def kq_gemm(fmt, W, a_q8, M, N, K, out, stream=None):
    _need_gemm_inputs(fmt, W, a_q8, M, N, K, "kq_gemm")
    _need(out, 4 * max(M, 0) * max(N, 0), "kq_gemm out", "float32")
    return _check(lib().kq_gemm(fmt, _ptr(W), _ptr(a_q8), M, N, K, _ptr(out), _stream(stream)),
                  "kq_gemm")


def kq_gemm_subsums(fmt, W, a_q8, M, N, K, sums, stream=None):
    _need_gemm_inputs(fmt, W, a_q8, M, N, K, "kq_gemm_subsums")
    _need(sums, 4 * max(M, 0) * max(N, 0) * max(K, 0) // _sub_block(fmt), "kq_gemm_subsums sums", "int32")
    return _check(lib().kq_gemm_subsums(fmt, _ptr(W), _ptr(a_q8), M, N, K, _ptr(sums),
                                        _stream(stream)), "kq_gemm_subsums")


def kq_num_variants():
    return lib().kq_num_variants()


def kq_variant_name(v):
    s = lib().kq_variant_name(v)
    return s.decode() if s else None


def kq_dispatch_count(v):
    return lib().kq_dispatch_count(v)


def kq_dispatch_reset():
    lib().kq_dispatch_reset()


def kq_select_variant(fmt, M, N, K):
    return lib().kq_select_variant(fmt, M, N, K)


def kq_debug_unpack(fmt, W, nblocks, q, scales, stream=None):
    return _check(lib().kq_debug_unpack(fmt, _ptr(W), nblocks, _ptr(q), _ptr(scales),
                                        _stream(stream)), "kq_debug_unpack")


def kq_gemm_id(fmt, W, n_experts, a_q8, M, N, K, expert_offsets, rows, R, out, stream=None):
    if 1 <= n_experts <= KQ_GEMM_ID_MAX_EXPERTS:
        _need_gemm_inputs(fmt, W, a_q8, M, N, K, "kq_gemm_id", n_experts)
        _need(expert_offsets, 4 * (n_experts + 1), "kq_gemm_id expert_offsets", "int32")
    _need(rows, 4 * max(R, 0), "kq_gemm_id rows", "int32")
    _need(out, 4 * max(R, 0) * max(N, 0), "kq_gemm_id out", "float32")
    return _check(lib().kq_gemm_id(fmt, _ptr(W), n_experts, _ptr(a_q8), M, N, K, _ptr(expert_offsets),
                                   _ptr(rows), R, _ptr(out), _stream(stream)), "kq_gemm_id")


def kq_calib_launch(kind, param=0, buf=None, nbytes=0, stream=None):
    """Launch one calibration kernel; returns the work it does (int8 ops, fp32
    flops or bytes)."""
    work = ctypes.c_double(0.0)
    _check(lib().kq_calib_launch(kind, param, _ptr(buf), nbytes, ctypes.byref(work), _stream(stream)),
           "kq_calib_launch")
    return work.value


def _ref(d):
    """A descriptor (kq_cache, kq_batch or an array of them) as an argument."""
    return None if d is None else ctypes.addressof(d)


def kq_rope_append(cache, batch, x, ldx, q_heads, q_norm, k_norm, eps, rope, n_pos, rot_dim, pairs, positions, q_type,
                   q, stream=None):
    return _check(lib().kq_rope_append(_ref(cache), _ref(batch), _ptr(x), ldx, q_heads, _ptr(q_norm), _ptr(k_norm), eps,
                                       _ptr(rope), n_pos, rot_dim, int(pairs), _ptr(positions), q_type, _ptr(q),
                                       _stream(stream)), "kq_rope_append")


def kq_attn_tree_workspace(cache, batch, q_heads, max_tokens, max_len):
    return lib().kq_attn_tree_workspace(_ref(cache), _ref(batch), q_heads, max_tokens, max_len)


def kq_attn_tree(cache, batch, q_type, q, q_heads, mask, scale, max_tokens, max_len, out_type, out, workspace,
                 workspace_bytes, stream=None):
    return _check(lib().kq_attn_tree(_ref(cache), _ref(batch), q_type, _ptr(q), q_heads, _ptr(mask), scale, max_tokens,
                                     max_len, out_type, _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)),
                  "kq_attn_tree")


def kq_cache_keep(caches, n_caches, batch, path, counts, stream=None):
    return _check(lib().kq_cache_keep(_ref(caches), n_caches, _ref(batch), _ptr(path), _ptr(counts), _stream(stream)),
                  "kq_cache_keep")


def kq_logprobs_workspace(M, V, n_top):
    return lib().kq_logprobs_workspace(M, V, n_top)


def kq_logprobs(type, logits, M, V, ldx, tokens, n_given, n_top, logprob, entropy, top_ids, top_logprobs, workspace,
                workspace_bytes, stream=None):
    return _check(lib().kq_logprobs(type, _ptr(logits), M, V, ldx, _ptr(tokens), n_given, n_top, _ptr(logprob),
                                    _ptr(entropy), _ptr(top_ids), _ptr(top_logprobs), _ptr(workspace), workspace_bytes,
                                    _stream(stream)), "kq_logprobs")


def kq_num_step_variants():
    return lib().kq_num_step_variants()


def kq_step_variant_name(v):
    s = lib().kq_step_variant_name(v)
    return s.decode() if s else None


def kq_step_count(v):
    return lib().kq_step_count(v)


def kq_step_count_reset():
    lib().kq_step_count_reset()


def kq_strerror(status):
    return lib().kq_strerror(status).decode()


def kq_version():
    return lib().kq_version()


# ------------------------------------------------- torch conveniences (allocation)

def step_counts() -> dict:
    return {kq_step_variant_name(v): kq_step_count(v) for v in range(kq_num_step_variants())}


def dispatch_counts() -> dict:
    return {kq_variant_name(v): kq_dispatch_count(v) for v in range(kq_num_variants())}


def quantize_act(x, act_fmt=KQ_ACT_Q8_K, stream=None):
    """fp32 [M][K] device tensor -> uint8 device tensor holding the activation buffer."""
    import torch
    M, K = x.shape
    a_q8 = torch.empty(kq_act_bytes(act_fmt, M, K), dtype=torch.uint8, device=x.device)
    kq_quantize_act(act_fmt, x, M, K, a_q8, stream)
    return a_q8


def act_views(a_q8, act_fmt, M, K):
    """(qs int8 [M][K], d fp32 [M][K/bs], bsums int16 [M][K/16] or None) views of a
    buffer.  d is stored block-major ([K/bs][M]); the view is its transpose."""
    import torch
    bs = 256 if act_fmt == KQ_ACT_Q8_K else 128
    od = kq_act_section_offset(act_fmt, KQ_SEC_D, M, K)
    qs = a_q8[:M * K].view(torch.int8).view(M, K)
    d = a_q8[od:od + M * (K // bs) * 4].view(torch.float32).view(K // bs, M).t()
    bsums = None
    if act_fmt == KQ_ACT_Q8_K:
        ob = kq_act_section_offset(act_fmt, KQ_SEC_BSUMS, M, K)
        bsums = a_q8[ob:ob + M * (K // 16) * 2].view(torch.int16).view(M, K // 16)
    return qs, d, bsums


def alpha_view(a_q8, M, K):
    """The Q8_K alpha section as int16 bit patterns of bf16 values, [K/256][2][M][8]."""
    import torch
    oa = kq_act_section_offset(KQ_ACT_Q8_K, KQ_SEC_ALPHA, M, K)
    n = (K // 256) * 2 * M * 8
    return a_q8[oa:oa + 2 * n].view(torch.int16).view(K // 256, 2, M, 8)


def gemm(fmt, W, a_q8, M, N, K, out=None, stream=None):
    """out fp32 [M][N] = W x A (device tensors)."""
    import torch
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=a_q8.device)
    kq_gemm(fmt, W, a_q8, M, N, K, out, stream)
    return out


def debug_unpack(fmt, W, nblocks, stream=None):
    """Decode nblocks weight blocks (uint8 device tensor) with the tile kernel's
    loaders: (q int8 [nblocks][QK], scales int32 [nblocks][16] or None)."""
    import torch
    ternary = fmt in (KQ_TQ, KQ_TQ2)
    qk = 128 if ternary else 256
    q = torch.empty((nblocks, qk), dtype=torch.int8, device=W.device)
    scales = None if ternary else torch.empty((nblocks, 16), dtype=torch.int32, device=W.device)
    kq_debug_unpack(fmt, W, nblocks, q, scales, stream)
    return q, scales


def gemm_id(fmt, W, n_experts, a_q8, M, N, K, expert_offsets, rows, out=None, stream=None):
    """out fp32 [R][N]: routed row r = expert e's weights x token rows[r]
    (expert_offsets int32 [n_experts + 1], rows int32 [R]; device tensors)."""
    import torch
    R = rows.numel()
    if out is None:
        out = torch.empty((R, N), dtype=torch.float32, device=a_q8.device)
    kq_gemm_id(fmt, W, n_experts, a_q8, M, N, K, expert_offsets, rows, R, out, stream)
    return out


# ------------------------------- the step between two products (cache, attention, answer)
#
# These calls are a few microseconds of GPU work where one token is decoded, so
# their checks are written to cost little: a tensor that is as it should be takes
# one test each of device, type, shape and layout, and the message is worked out
# only for one that is not.

_addressof = ctypes.addressof
_types = _current_stream = _current_device = _step = _torch = None


def _step_lib():
    """The library's entry points of the step, torch and its types, once."""
    global _types, _current_stream, _current_device, _step, _torch
    import torch
    _torch = torch
    _types = {torch.float32: KQ_T_F32, torch.bfloat16: KQ_T_BF16, torch.float16: KQ_T_F16,
              torch.float8_e4m3fn: KQ_T_F8}
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _step = lib()
    return _step


def _refuse(t, dtype, shape, device, where):
    """Raise what is wrong with a tensor argument (None in a shape: any size)."""
    if not t.is_cuda:
        raise ValueError(f"{where}: expected a device tensor")
    if t.get_device() != device:
        raise ValueError(f"{where}: expected a tensor on device {device}, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{where}: expected dtype {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(n is not None and n != h for n, h in zip(shape, t.shape)):
        raise ValueError(f"{where}: expected shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{where}: expected a contiguous tensor")


def _tensor(t, dtype, shape, device, where):
    """The address of a tensor argument after its checks."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, shape, device, where)


def _rows(t, n, device, where):
    """(address, row stride) of a [rows][n] tensor whose rows may lie apart."""
    if device < 0:
        raise ValueError(f"{where}: expected a device tensor")
    if t.dim() != 2 or (n is not None and t.shape[1] != n):
        raise ValueError(f"{where}: expected shape (None, {n}), got {tuple(t.shape)}")
    rows, n = t.shape
    ld, one = t.stride()
    if rows <= 1:
        ld = max(n, 1)
    if one != 1 and n > 1:
        raise ValueError(f"{where}: expected rows of neighbouring elements")
    if ld < n:
        raise ValueError(f"{where}: rows overlap (stride {ld}, {n} elements)")
    return t.data_ptr(), ld


def _type(dtype, where):
    kind = (_types or _step_lib() and _types).get(dtype)
    if kind is None:
        raise ValueError(f"{where}: element type {dtype} not taken")
    return kind


def _on(stream, device):
    """A context in which the tensors' device is the current one (kernels go to the
    current device, and a handle of 0 is its default stream), and a stream, if one
    is given (a torch stream or a raw handle), torch's current one there: what is
    allocated in it belongs to that stream, so neither the results nor the workspace
    can be handed to other work that it overtakes."""
    torch = _torch
    if device < 0:
        raise ValueError("expected device tensors")
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    if stream.device_index != device:
        raise ValueError(f"a stream of device {stream.device_index} for tensors on device {device}")
    return torch.cuda.stream(stream)


class PagedCache:
    """Keys [n_pages][heads][page][dim] and values [n_pages][heads][dim][page]
    of one layer (bfloat16, float16 or float8_e4m3fn device tensors); what is
    stored times k_scale / v_scale is the key / value."""
    __slots__ = ("k", "v", "dtype", "device", "c", "at")

    def __init__(self, k, v, k_scale=1.0, v_scale=1.0):
        if k.dim() != 4:
            raise ValueError(f"PagedCache k: expected [n_pages][heads][page][dim], got {tuple(k.shape)}")
        n, heads, page, dim = shape = k.shape
        self.k, self.v, self.dtype = k, v, k.dtype
        self.device = device = k.get_device()
        pk, pv = k.data_ptr(), v.data_ptr()
        if device < 0 or not k.is_contiguous():
            _refuse(k, k.dtype, shape, device, "PagedCache k")
        if v.dtype is not k.dtype or v.shape != (n, heads, dim, page) or v.get_device() != device or not v.is_contiguous():
            _refuse(v, k.dtype, (n, heads, dim, page), device, "PagedCache v")
        self.c = c = kq_cache(pk, pv, n, _type(k.dtype, "PagedCache k"), heads, dim, page, k_scale, v_scale)
        self.at = ctypes.addressof(c)


class Batch:
    """The sequences of one step (int32 device tensors): offsets [n_seqs + 1] of
    their token rows, lens [n_seqs] tokens already cached, pages [n_seqs][max_pages]."""
    __slots__ = ("offsets", "lens", "pages", "device", "c", "_last", "_spare")

    def __init__(self, offsets, lens, pages):
        if _torch is None:
            _step_lib()
        i32 = _torch.int32
        n = lens.shape[0]
        wide = pages.shape[-1]
        self.offsets, self.lens, self.pages = offsets, lens, pages
        self.device = device = lens.get_device()
        if not (device >= 0 and offsets.dtype is i32 and lens.dtype is i32 and pages.dtype is i32 and lens.dim() == 1
                and offsets.shape == (n + 1,) and pages.shape == (n, wide) and offsets.get_device() == device
                and pages.get_device() == device and offsets.is_contiguous() and lens.is_contiguous()
                and pages.is_contiguous()):
            _tensor(offsets, i32, (n + 1,), device, "Batch offsets")
            _tensor(lens, i32, (n,), device, "Batch lens")
            _tensor(pages, i32, (n, wide), device, "Batch pages")
            raise ValueError("Batch: expected device tensors")
        self.c = c = kq_batch(offsets.data_ptr(), lens.data_ptr(), pages.data_ptr(), n, 0, wide)
        self._last, self._spare = None, [c]

    def of(self, n_tokens):
        """The descriptor of a step of n_tokens rows.  Calls with any number of rows (in
        other threads, too) share this object, so a descriptor that a call may hold is
        not changed: the first call takes the one that is there, others make one."""
        c = self._last
        if c is None or c.n_tokens != n_tokens:
            try:
                c = self._spare.pop()
                c.n_tokens = n_tokens
            except IndexError:
                b = self.c
                c = kq_batch(b.offsets, b.lens, b.pages, b.n_seqs, n_tokens, b.max_pages)
            self._last = c
        return c


def _together(device, cache, batch, rows, where):
    if cache.device != device or batch.device != device:
        raise ValueError(f"{where}: tensors on devices {device}, {cache.device} and {batch.device}")
    if rows and not batch.c.n_seqs:
        raise ValueError(f"{where}: {rows} rows of no sequence")


def rope_append(cache, batch, x, q_heads, rope=None, positions=None, q_norm=None, k_norm=None, eps=1e-6, pairs=False,
                q_dtype=None, out=None, stream=None):
    """Split x [n_tokens][(q_heads + 2 heads) dim] (float32): q normed, rotated and
    returned as [n_tokens][q_heads][dim] (q_dtype: the cache's, bfloat16 for an
    8-bit cache); k normed and rotated, and v, stored in the cache's slots of the
    rows.  rope: float32 [n_pos][rot_dim], the cosines and then the sines."""
    torch, device = _torch, x.get_device()
    if stream is not None or (device >= 0 and device != _current_device()):
        with _on(stream, device):
            return rope_append(cache, batch, x, q_heads, rope, positions, q_norm, k_norm, eps, pairs, q_dtype, out)
    f32, c = torch.float32, cache.c
    heads, dim = c.heads, c.dim
    px, ldx = _rows(x, (q_heads + 2 * heads) * dim, device, "rope_append x")
    if x.dtype is not f32:
        _refuse(x, f32, x.shape, device, "rope_append x")
    M = x.shape[0]
    _together(device, cache, batch, M, "rope_append")
    if out is None:
        if q_dtype is None:
            q_dtype = torch.bfloat16 if c.type == KQ_T_F8 else cache.dtype
        out = torch.empty((M, q_heads, dim), dtype=q_dtype, device=x.device)
        pq = out.data_ptr()
    else:
        q_dtype = q_dtype or out.dtype
        pq = _tensor(out, q_dtype, (M, q_heads, dim), device, "rope_append out")
    pr, n_pos, rot = None, 0, 0
    if rope is not None:
        n_pos, rot = rope.shape if rope.dim() == 2 else (None, None)
        pr = _tensor(rope, f32, (n_pos, rot), device, "rope_append rope")
    pqn = None if q_norm is None else _tensor(q_norm, f32, (dim,), device, "rope_append q_norm")
    pkn = None if k_norm is None else _tensor(k_norm, f32, (dim,), device, "rope_append k_norm")
    pp = None if positions is None else _tensor(positions, torch.int32, (M,), device, "rope_append positions")
    rows = batch.of(M)
    _check((_step or _step_lib()).kq_rope_append(cache.at, _addressof(rows), px, ldx, q_heads, pqn, pkn, eps, pr, n_pos, rot,
                                                 1 if pairs else 0, pp, _type(q_dtype, "rope_append out"), pq,
                                                 _current_stream(device)), "kq_rope_append")
    return out


def attn_tree(cache, batch, q, mask=None, scale=None, max_tokens=KQ_ATTN_MAX_TOKENS, max_len=None, out_dtype=None,
              out=None, stream=None):
    """Attention of q [n_tokens][q_heads][dim] over the cache, each row over its
    sequence's cached tokens and those of its new rows that its bits in mask
    name (int64 [n_tokens], bit j: the j-th new row; None: the rows up to its
    own).  max_tokens / max_len: upper bounds of a sequence's new rows (past it:
    refused where the host can tell, else NaN) and of its whole length (default: what
    the pages hold).  A longer prompt, appended whole, attends as several sequences
    over its page row, the i-th with 64 i more cached tokens and the next 64 rows.
    out_dtype: q's or float32."""
    torch, device = _torch, q.get_device()
    if stream is not None or (device >= 0 and device != _current_device()):
        with _on(stream, device):
            return attn_tree(cache, batch, q, mask, scale, max_tokens, max_len, out_dtype, out)
    c, q_dtype = cache.c, q.dtype
    dim = c.dim
    if device < 0 or q.dim() != 3 or q.shape[2] != dim or not q.is_contiguous():
        _refuse(q, q_dtype, (None, None, dim), device, "attn_tree q")
    M, heads, _ = shape = q.shape
    _together(device, cache, batch, M, "attn_tree")
    if out is None:
        out = torch.empty_like(q) if out_dtype is None else torch.empty(shape, dtype=out_dtype, device=q.device)
        po = out.data_ptr()
    else:
        po = _tensor(out, out_dtype or out.dtype, shape, device, "attn_tree out")
    pm = None if mask is None else _tensor(mask, torch.int64, (M,), device, "attn_tree mask")
    if max_len is None:
        max_len = batch.c.max_pages * c.page
    if scale is None:
        scale = dim ** -0.5
    rows = batch.of(M)
    at = _addressof(rows)
    step = _step or _step_lib()
    need = step.kq_attn_tree_workspace(cache.at, at, heads, max_tokens, max_len)
    work = pw = None
    if need:
        work = torch.empty(need, dtype=torch.uint8, device=q.device)
        pw = work.data_ptr()
    _check(step.kq_attn_tree(cache.at, at, _type(q_dtype, "attn_tree q"), q.data_ptr(), heads, pm, scale, max_tokens,
                             max_len, _type(out.dtype, "attn_tree out"), po, pw, need, _current_stream(device)),
           "kq_attn_tree")
    return out


def cache_keep(caches, batch, path, counts, stream=None):
    """Keep an accepted branch in every cache of a list (one per layer): slot
    lens[b] + j takes what slot lens[b] + path[offsets[b] + j] held, j < counts[b]
    (int32 [n_tokens] and [n_seqs])."""
    i32, device, n = _torch.int32, path.get_device(), len(caches)
    if stream is not None or (device >= 0 and device != _current_device()):
        with _on(stream, device):
            return cache_keep(caches, batch, path, counts)
    if device < 0 or path.dim() != 1:
        _refuse(path, i32, (None,), device, "cache_keep path")
    pp = _tensor(path, i32, path.shape, device, "cache_keep path")
    pc = _tensor(counts, i32, (batch.c.n_seqs,), device, "cache_keep counts")
    for c in caches:
        if c.device != device:
            _together(device, c, batch, 0, "cache_keep")
    if batch.device != device:
        raise ValueError(f"cache_keep: tensors on devices {device} and {batch.device}")
    rows = batch.of(path.shape[0])
    if n == 1:
        at = caches[0].at
    else:
        every = (kq_cache * n)(*[c.c for c in caches])
        at = ctypes.addressof(every)
    step = _step or _step_lib()
    _check(step.kq_cache_keep(at, n, _addressof(rows), pp, pc, _current_stream(device)), "kq_cache_keep")


class LogProbs:
    """What logprobs() found: logprob [M][n_given], entropy [M], top_ids and
    top_logprobs [M][n_top] (None where not asked for)."""
    __slots__ = ("logprob", "entropy", "top_ids", "top_logprobs")


def logprobs(logits, tokens=None, n_top=0, entropy=True, stream=None):
    """Log probabilities of tokens [M][n_given] (int32) under logits [M][V]
    (float32, bfloat16 or float16; rows may lie apart), the entropy of each row,
    and the n_top largest logits' indices and log probabilities."""
    if _torch is None:
        _step_lib()
    torch, device = _torch, logits.get_device()
    if stream is not None or (device >= 0 and device != _current_device()):
        with _on(stream, device):
            return logprobs(logits, tokens, n_top, entropy)
    px, ldx = _rows(logits, None, device, "logprobs logits")
    M, V = logits.shape
    kind, dev = _type(logits.dtype, "logprobs logits"), logits.device
    step = _step or _step_lib()
    given, pt = 0, None
    if tokens is not None:
        given = tokens.shape[-1]
        pt = _tensor(tokens, torch.int32, (M, given), device, "logprobs tokens")
    n_top = int(n_top)
    if n_top < 0:
        raise ValueError(f"logprobs n_top: {n_top}")
    # one allocation: the floats [M][n_given], [M], [M][n_top], the ids, the workspace
    lens = (M * given, M if entropy else 0, M * n_top)
    need = step.kq_logprobs_workspace(M, V, n_top)
    floats = lens[0] + lens[1] + lens[2]
    at = (floats + lens[2] + 3) // 4 * 4
    block = torch.empty(at + (need + 3) // 4, dtype=torch.float32, device=dev)
    p = block.data_ptr()
    r = LogProbs()
    r.logprob = r.entropy = r.top_ids = r.top_logprobs = None
    p_given = p_entropy = p_ids = p_tops = None
    if tokens is not None:
        r.logprob, p_given = block.as_strided((M, given), (given, 1), 0), p
    if entropy:
        r.entropy, p_entropy = block.as_strided((M,), (1,), lens[0]), p + 4 * lens[0]
    if n_top:
        r.top_logprobs, p_tops = block.as_strided((M, n_top), (n_top, 1), lens[0] + lens[1]), p + 4 * (lens[0] + lens[1])
        r.top_ids, p_ids = block.view(torch.int32).as_strided((M, n_top), (n_top, 1), floats), p + 4 * floats
    _check(step.kq_logprobs(kind, px, M, V, ldx, pt, given, n_top, p_given, p_entropy, p_ids, p_tops,
                            p + 4 * at if need else None, need, _current_stream(device)), "kq_logprobs")
    return r
