"""W4A16 fused MoE layer for MI355X (gfx950), and operators for rows grouped by expert: Python binding of the C ABI.

Every function here has the name of an entry point in include/w4a16_moe.h and
does argument marshalling only: torch tensors supply device memory and the
current HIP stream; all computation runs in the library's HIP kernels. A
non-OK status raises W4A16Error.
"""
from __future__ import annotations

import ctypes

from ._lib import LIB_PATH, Shape, load

__all__ = [
    "W4A16Error", "Shape", "LIB_PATH", "load", "make_shape", "w4a16_status_string", "w4a16_packed_bytes",
    "w4a16_repack", "moe_align_capacity", "moe_align_workspace_bytes", "w4a16_choose_block_m", "moe_align",
    "moe_route_align", "moe_align_filtered", "moe_align_split", "w4a16_moe_routed_workspace_bytes", "w4a16_moe_routed_split",
    "w4a16_moe_routed_forward", "w4a16_moe_routed_forward_noalloc", "NOALLOC_SCRATCH_BYTES",
    "w4a16_moe_contiguous_workspace_bytes", "w4a16_moe_contiguous_forward",
    "w4a16_moe_masked_block_m", "w4a16_moe_masked_workspace_bytes", "w4a16_moe_masked_forward",
    "w4a16_moe_stage_workspace_bytes", "w4a16_moe_prepare_x", "w4a16_moe_prepare_h",
    "w4a16_moe_workspace_bytes", "w4a16_moe_forward", "w4a16_moe_gate_up", "w4a16_moe_down",
    "w4a16_moe_combine", "align_buffers",
    "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
    "mxfp4_quantize", "mxfp4_silu_mul_quantize", "mxfp4_dequantize", "mxfp4_packed_bytes", "mxfp4_repack",
    "mxfp4_moe_gemm",
    "moe_grouped_gemm", "moe_grouped_gemm_wgrad_workspace_bytes", "moe_grouped_gemm_wgrad",
    "mxfp8_quantize", "mxfp8_dequantize", "mxfp8_silu_mul", "mxfp8_silu_mul_backward",
]

OK = 0


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {w4a16_status_string(status)} (status {status})")


def make_shape(num_experts: int, hidden: int, intermediate: int, group_size: int = 32) -> Shape:
    return Shape(num_experts, hidden, intermediate, group_size)


def _p(t):
    """Device pointer of a tensor (None -> NULL)."""
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, where: str):
    if status != OK:
        raise W4A16Error(status, where)


def w4a16_status_string(status: int) -> str:
    return load().w4a16_status_string(status).decode()


def w4a16_packed_bytes(shape: Shape) -> tuple[int, int]:
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().w4a16_packed_bytes(ctypes.byref(shape), ctypes.byref(a), ctypes.byref(b)), "w4a16_packed_bytes")
    return a.value, b.value


def w4a16_repack(shape: Shape, w13_q, w13_s, w2_q, w2_s, w13_packed, w2_packed, stream=None):
    _check(load().w4a16_repack(ctypes.byref(shape), _p(w13_q), _p(w13_s), _p(w2_q), _p(w2_s), _p(w13_packed),
                               _p(w2_packed), _stream(stream)), "w4a16_repack")


def moe_align_capacity(T: int, topk: int, num_experts: int, block_m: int) -> int:
    return load().moe_align_capacity(T, topk, num_experts, block_m)


def moe_align_workspace_bytes(T: int, topk: int, num_experts: int, block_m: int) -> int:
    return load().moe_align_workspace_bytes(T, topk, num_experts, block_m)


def w4a16_choose_block_m(T: int, topk: int, num_experts_local: int, num_experts_global: int) -> int:
    return load().w4a16_choose_block_m(T, topk, num_experts_local, num_experts_global)


def moe_align(topk_ids, num_experts: int, block_m: int, sorted_token_ids, expert_ids, num_tokens_post_padded,
              expert_counts=None, workspace=None, stream=None):
    T, topk = topk_ids.shape
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().moe_align(_p(topk_ids), T, topk, num_experts, block_m, _p(sorted_token_ids),
                            sorted_token_ids.numel(), _p(expert_ids), _p(num_tokens_post_padded),
                            _p(expert_counts), _p(workspace), nbytes, _stream(stream)), "moe_align")


def moe_route_align(logits, topk: int, num_experts: int, block_m: int, topk_ids, topk_weights, sorted_token_ids,
                    expert_ids, num_tokens_post_padded, bias=None, expert_counts=None, workspace=None, stream=None):
    T, Eg = logits.shape
    _check(load().moe_route_align(_p(logits), _p(bias), T, Eg, topk, num_experts, block_m, _p(topk_ids),
                                  _p(topk_weights), _p(sorted_token_ids), sorted_token_ids.numel(), _p(expert_ids),
                                  _p(num_tokens_post_padded), _p(expert_counts), _p(workspace), _nbytes(workspace),
                                  _stream(stream)), "moe_route_align")


def w4a16_moe_contiguous_workspace_bytes(shape: Shape, M: int) -> int:
    return load().w4a16_moe_contiguous_workspace_bytes(ctypes.byref(shape), M)


def w4a16_moe_contiguous_forward(shape: Shape, x, m_indices, w13_packed, w2_packed, out, workspace, stream=None):
    M = x.shape[0]
    _check(load().w4a16_moe_contiguous_forward(ctypes.byref(shape), _p(x), M, _p(m_indices), _p(w13_packed),
                                               _p(w2_packed), _p(out), _p(workspace), _nbytes(workspace),
                                               _stream(stream)), "w4a16_moe_contiguous_forward")


def w4a16_moe_masked_block_m(max_m: int, expected_m: int) -> int:
    return load().w4a16_moe_masked_block_m(max_m, expected_m)


def w4a16_moe_masked_workspace_bytes(shape: Shape, max_m: int, block_m: int) -> int:
    return load().w4a16_moe_masked_workspace_bytes(ctypes.byref(shape), max_m, block_m)


def w4a16_moe_masked_forward(shape: Shape, x, masked_m, block_m: int, w13_packed, w2_packed, out, workspace,
                             stream=None):
    max_m = x.shape[1]
    _check(load().w4a16_moe_masked_forward(ctypes.byref(shape), _p(x), max_m, _p(masked_m), block_m,
                                           _p(w13_packed), _p(w2_packed), _p(out), _p(workspace),
                                           _nbytes(workspace), _stream(stream)), "w4a16_moe_masked_forward")


def moe_align_filtered(topk_ids, num_experts: int, block_m: int, min_count: int, max_count: int, sorted_token_ids,
                       expert_ids, num_tokens_post_padded, expert_counts=None, workspace=None, stream=None):
    T, topk = topk_ids.shape
    _check(load().moe_align_filtered(_p(topk_ids), T, topk, num_experts, block_m, min_count, max_count,
                                     _p(sorted_token_ids), sorted_token_ids.numel(), _p(expert_ids),
                                     _p(num_tokens_post_padded), _p(expert_counts), _p(workspace), _nbytes(workspace),
                                     _stream(stream)), "moe_align_filtered")


def moe_align_split(topk_ids, num_experts: int, split_count: int, heavy_block_m: int, heavy_capacity: int,
                    heavy_expert_ids, heavy_num_tokens_post_padded, light_block_m: int, light_expert_ids,
                    light_num_tokens_post_padded, sorted_token_ids, workspace=None, stream=None):
    """Heavy and light alignments in one pass; sorted_token_ids holds the heavy set's
    heavy_capacity ids, then the light set's (the rest of the tensor)."""
    T, topk = topk_ids.shape
    light_capacity = sorted_token_ids.numel() - heavy_capacity
    _check(load().moe_align_split(_p(topk_ids), T, topk, num_experts, split_count, heavy_block_m, heavy_capacity,
                                  _p(heavy_expert_ids), _p(heavy_num_tokens_post_padded), light_block_m,
                                  light_capacity, _p(light_expert_ids), _p(light_num_tokens_post_padded),
                                  _p(sorted_token_ids), _p(workspace), _nbytes(workspace), _stream(stream)),
           "moe_align_split")


def w4a16_moe_routed_workspace_bytes(shape: Shape, T: int, topk: int, num_experts_global: int) -> int:
    return load().w4a16_moe_routed_workspace_bytes(ctypes.byref(shape), T, topk, num_experts_global)


def w4a16_moe_routed_split(shape: Shape, T: int, topk: int, num_experts_global: int) -> int:
    return load().w4a16_moe_routed_split(ctypes.byref(shape), T, topk, num_experts_global)


def w4a16_moe_routed_forward(shape: Shape, x, topk_ids, topk_weights, num_experts_global: int, w13_packed, w2_packed,
                             out, workspace, stream=None):
    T, topk = topk_ids.shape
    _check(load().w4a16_moe_routed_forward(ctypes.byref(shape), _p(x), T, topk, num_experts_global, _p(topk_ids),
                                           _p(topk_weights), _p(w13_packed), _p(w2_packed), _p(out), _p(workspace),
                                           _nbytes(workspace), _stream(stream)), "w4a16_moe_routed_forward")


# W4A16_NOALLOC_SCRATCH_BYTES of include/w4a16_moe.h
NOALLOC_SCRATCH_BYTES = 64 << 20


def w4a16_moe_routed_forward_noalloc(shape: Shape, x, topk_ids, topk_weights, num_experts_global: int, w13_packed,
                                     w2_packed, out, stream=None):
    T, topk = topk_ids.shape
    _check(load().w4a16_moe_routed_forward_noalloc(ctypes.byref(shape), _p(x), T, topk, num_experts_global,
                                                   _p(topk_ids), _p(topk_weights), _p(w13_packed), _p(w2_packed),
                                                   _p(out), _stream(stream)), "w4a16_moe_routed_forward_noalloc")


def w4a16_moe_workspace_bytes(shape: Shape, T: int, topk: int, block_m: int) -> int:
    return load().w4a16_moe_workspace_bytes(ctypes.byref(shape), T, topk, block_m)


def w4a16_moe_forward(shape: Shape, x, topk_ids, topk_weights, sorted_token_ids, expert_ids, num_tokens_post_padded,
                      block_m: int, w13_packed, w2_packed, out, workspace, stream=None):
    T, topk = topk_ids.shape
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().w4a16_moe_forward(ctypes.byref(shape), _p(x), T, topk, _p(topk_ids), _p(topk_weights),
                                    _p(sorted_token_ids), sorted_token_ids.numel(), _p(expert_ids),
                                    _p(num_tokens_post_padded), block_m, _p(w13_packed), _p(w2_packed), _p(out),
                                    _p(workspace), nbytes, _stream(stream)), "w4a16_moe_forward")


def w4a16_moe_stage_workspace_bytes(shape: Shape, T: int, topk: int, block_m: int) -> int:
    return load().w4a16_moe_stage_workspace_bytes(ctypes.byref(shape), T, topk, block_m)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def w4a16_moe_prepare_x(shape: Shape, x, topk_ids, block_m: int, workspace=None, stream=None):
    T, topk = topk_ids.shape
    _check(load().w4a16_moe_prepare_x(ctypes.byref(shape), _p(x), T, topk, _p(topk_ids), block_m, _p(workspace),
                                      _nbytes(workspace), _stream(stream)), "w4a16_moe_prepare_x")


def w4a16_moe_gate_up(shape: Shape, x, T: int, topk: int, sorted_token_ids, expert_ids, num_tokens_post_padded,
                      block_m: int, w13_packed, h, workspace=None, stream=None):
    _check(load().w4a16_moe_gate_up(ctypes.byref(shape), _p(x), T, topk, _p(sorted_token_ids),
                                    sorted_token_ids.numel(), _p(expert_ids), _p(num_tokens_post_padded), block_m,
                                    _p(w13_packed), _p(h), _p(workspace), _nbytes(workspace), _stream(stream)),
           "w4a16_moe_gate_up")


def w4a16_moe_prepare_h(shape: Shape, T: int, topk: int, h, sorted_token_ids, num_tokens_post_padded, block_m: int,
                        workspace=None, stream=None):
    _check(load().w4a16_moe_prepare_h(ctypes.byref(shape), T, topk, _p(h), _p(sorted_token_ids),
                                      sorted_token_ids.numel(), _p(num_tokens_post_padded), block_m, _p(workspace),
                                      _nbytes(workspace), _stream(stream)), "w4a16_moe_prepare_h")


def w4a16_moe_down(shape: Shape, T: int, topk: int, h, sorted_token_ids, expert_ids, num_tokens_post_padded,
                   block_m: int, w2_packed, y, workspace=None, stream=None):
    _check(load().w4a16_moe_down(ctypes.byref(shape), T, topk, _p(h), _p(sorted_token_ids), sorted_token_ids.numel(),
                                 _p(expert_ids), _p(num_tokens_post_padded), block_m, _p(w2_packed), _p(y),
                                 _p(workspace), _nbytes(workspace), _stream(stream)), "w4a16_moe_down")


def w4a16_moe_combine(shape: Shape, topk_ids, topk_weights, y, out, stream=None):
    T, topk = topk_ids.shape
    _check(load().w4a16_moe_combine(ctypes.byref(shape), T, topk, _p(topk_ids), _p(topk_weights), _p(y), _p(out),
                                    _stream(stream)), "w4a16_moe_combine")


# ---------------------------------------------------------------------------
# Rows sorted by expert and back; 4-bit floating point. These take torch's own
# bfloat16, float16 and float32 tensors (int16 and uint16 count as bf16 bits, as
# everywhere in this package) and refuse, with the status the C ABI would give,
# what a pointer alone cannot show: another device than the current one, strides
# that are not the contiguous ones, a type or shape that does not fit.
# ---------------------------------------------------------------------------

INVALID_ARG, UNSUPPORTED, CAPACITY = 1, 2, 3
_codes = {}  # torch dtype -> w4a16_dtype
_torch = None
_current = None  # device index -> handle of torch's current stream there


def _t():
    """torch, imported at the first call that needs it."""
    global _torch, _current
    if _torch is None:
        import torch

        # without the Stream object that torch.cuda.current_stream makes: 2.8 us less a call
        _current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)

        _codes.update({torch.bfloat16: 0, torch.int16: 0, torch.uint16: 0, torch.float16: 1, torch.float32: 2})
        _torch = torch
    return _torch


def _refuse(where: str, what: str, status: int = INVALID_ARG):
    raise W4A16Error(status, f"{where}: {what}")


def _sizes(where: str, *sizes: int):
    """The C ABI's sizes are int32, and ctypes would pass the low 32 bits of a larger one. Callers look at all of
    theirs at once first (0.07 us instead of 0.23)."""
    if max(sizes) > 0x7FFFFFFF:
        _refuse(where, "a size is past 32 bits", UNSUPPORTED)
    if min(sizes) < -0x80000000:
        _refuse(where, "a size is negative")


def _dtype(t, where: str) -> int:
    _t()
    code = _codes.get(t.dtype)
    if code is None:
        _refuse(where, f"{t.dtype} rows", UNSUPPORTED)
    return code


def _launch(fn, where: str, args, tensors, stream):
    """Check that every tensor is contiguous and on the current device, then call the C ABI on the stream."""
    cuda = _t().cuda
    try:
        here = cuda.current_device()
    except (RuntimeError, AssertionError):  # no GPU: no tensor is on it
        here = None
    for t in tensors:
        if t is not None:
            if t.get_device() != here:
                _refuse(where, f"a tensor is on {t.device}, not on the current GPU")
            if not t.is_contiguous():
                _refuse(where, "a tensor is not contiguous")
    if stream is not None and stream.device_index != here:
        _refuse(where, f"the stream is of GPU {stream.device_index}, not of the current one")
    status = fn(*args, _current(here) if stream is None else stream.cuda_stream)
    if status != OK:
        raise W4A16Error(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _int32(where: str, *tensors):
    int32 = _t().int32
    for t in tensors:
        if t is not None and t.dtype is not int32:
            _refuse(where, "indexes and counts are int32")


def _count(where: str, t):
    """A row count on the device: one int32 (an empty tensor's null pointer would mean that there is none)."""
    if t is not None and (t.dtype is not _t().int32 or t.numel() < 1):
        _refuse(where, "a row count is one int32")


def _fp32(where: str, *tensors):
    float32 = _t().float32
    for t in tensors:
        if t is not None and t.dtype is not float32:
            _refuse(where, "weights are float32")


def moe_permute(x, sorted_token_ids, num_tokens_post_padded, topk: int, xp, slot_rows, stream=None):
    name = "moe_permute"
    T, H = x.shape
    capacity = sorted_token_ids.numel()
    if slot_rows.shape != (T, topk):
        _refuse(name, "slot_rows is not [T, topk]")
    rows, width = xp.shape
    if width != H or xp.dtype is not x.dtype:
        _refuse(name, "xp is not [rows, hidden] of x's type")
    if rows < capacity:
        _refuse(name, "xp has fewer rows than sorted_token_ids", CAPACITY)
    if (T | topk | H | capacity) >> 31:
        _sizes(name, T, topk, H, capacity)
    _int32(name, sorted_token_ids, slot_rows)
    _count(name, num_tokens_post_padded)
    _launch(load().moe_permute, name,
            (x.data_ptr(), _dtype(x, name), T, topk, H, sorted_token_ids.data_ptr(), capacity,
             num_tokens_post_padded.data_ptr(), xp.data_ptr(), slot_rows.data_ptr()),
            (x, sorted_token_ids, num_tokens_post_padded, xp, slot_rows), stream)


def moe_permute_backward(dxp, slot_rows, dx, stream=None):
    name = "moe_permute_backward"
    rows, H = dxp.shape
    T, topk = slot_rows.shape
    if dx.shape != (T, H) or dx.dtype is not dxp.dtype:
        _refuse(name, "dx is not [T, hidden] of dxp's type")
    if (rows | T | topk | H) >> 31:
        _sizes(name, rows, T, topk, H)
    _int32(name, slot_rows)
    _launch(load().moe_permute_backward, name,
            (dxp.data_ptr(), _dtype(dxp, name), rows, T, topk, H, slot_rows.data_ptr(), dx.data_ptr()),
            (dxp, slot_rows, dx), stream)


def moe_unpermute(y, slot_rows, out, topk_weights=None, stream=None):
    name = "moe_unpermute"
    rows, H = y.shape
    T, topk = slot_rows.shape
    if out.shape != (T, H):
        _refuse(name, "out is not [T, hidden]")
    if topk_weights is not None and topk_weights.shape != (T, topk):
        _refuse(name, "topk_weights is not [T, topk]")
    if (rows | T | topk | H) >> 31:
        _sizes(name, rows, T, topk, H)
    _int32(name, slot_rows)
    _fp32(name, topk_weights)
    _launch(load().moe_unpermute, name,
            (y.data_ptr(), _dtype(y, name), rows, T, topk, H, slot_rows.data_ptr(), _ptr(topk_weights),
             out.data_ptr(), _dtype(out, name)),
            (y, slot_rows, topk_weights, out), stream)


def moe_unpermute_backward(dout, y, slot_rows, topk_weights, sorted_token_ids, num_tokens_post_padded, dy, dweights,
                           stream=None):
    """dy or dweights may be None (not wanted), and y where dweights is; topk_weights None means weights of 1."""
    name = "moe_unpermute_backward"
    given = y if y is not None else dy
    if given is None:
        _refuse(name, "neither y nor dy")
    rows, H = given.shape
    T, topk = slot_rows.shape
    if dout.shape != (T, H):
        _refuse(name, "dout is not [T, hidden]")
    if dy is not None and (dy.shape != given.shape or dy.dtype is not given.dtype):
        _refuse(name, "dy is not like y")
    if dy is not None and (sorted_token_ids is None or num_tokens_post_padded is None):
        _refuse(name, "dy needs sorted_token_ids and num_tokens_post_padded")
    if dweights is not None and (y is None or dweights.shape != (T, topk)):
        _refuse(name, "dweights is not [T, topk], or y is missing")
    if topk_weights is not None and topk_weights.shape != (T, topk):
        _refuse(name, "topk_weights is not [T, topk]")
    _int32(name, slot_rows, sorted_token_ids)
    _count(name, num_tokens_post_padded)
    _fp32(name, topk_weights, dweights)
    capacity = 0 if sorted_token_ids is None else sorted_token_ids.numel()
    if (rows | T | topk | H | capacity) >> 31:
        _sizes(name, rows, T, topk, H, capacity)
    _launch(load().moe_unpermute_backward, name,
            (dout.data_ptr(), _dtype(dout, name), _ptr(y), _dtype(given, name), rows, T, topk, H,
             slot_rows.data_ptr(), _ptr(topk_weights), _ptr(sorted_token_ids), capacity,
             _ptr(num_tokens_post_padded), _ptr(dy), _ptr(dweights)),
            (dout, y, slot_rows, topk_weights, sorted_token_ids, num_tokens_post_padded, dy, dweights), stream)


def _fp4_buffers(name: str, rows: int, K: int, q, s, num_rows):
    uint8 = _t().uint8
    if K % 32:
        _refuse(name, "rows are not a multiple of 32 long", UNSUPPORTED)
    if (rows | K) >> 31:
        _sizes(name, rows, K)
    if q.shape != (rows, K // 2) or s.shape != (rows, K // 32):
        _refuse(name, "codes and scales are not [rows, K / 2] and [rows, K / 32]")
    if q.dtype is not uint8 or s.dtype is not uint8:
        _refuse(name, "codes and scales are uint8")
    _count(name, num_rows)


def mxfp4_quantize(x, q, s, num_rows=None, stream=None):
    name = "mxfp4_quantize"
    rows, K = x.shape
    _fp4_buffers(name, rows, K, q, s, num_rows)
    _launch(load().mxfp4_quantize, name,
            (x.data_ptr(), _dtype(x, name), rows, K, _ptr(num_rows), q.data_ptr(), s.data_ptr()),
            (x, q, s, num_rows), stream)


def mxfp4_silu_mul_quantize(gu, q, s, num_rows=None, stream=None):
    name = "mxfp4_silu_mul_quantize"
    rows, two_i = gu.shape
    if two_i % 2:
        _refuse(name, "gu is not [rows, 2 I]")
    _fp4_buffers(name, rows, two_i // 2, q, s, num_rows)
    _launch(load().mxfp4_silu_mul_quantize, name,
            (gu.data_ptr(), _dtype(gu, name), rows, two_i // 2, _ptr(num_rows), q.data_ptr(), s.data_ptr()),
            (gu, q, s, num_rows), stream)


def mxfp4_dequantize(q, s, out, num_rows=None, stream=None):
    name = "mxfp4_dequantize"
    rows, K = out.shape
    _fp4_buffers(name, rows, K, q, s, num_rows)
    _launch(load().mxfp4_dequantize, name,
            (q.data_ptr(), s.data_ptr(), rows, K, _ptr(num_rows), out.data_ptr(), _dtype(out, name)),
            (q, s, out, num_rows), stream)


def mxfp4_packed_bytes(num_experts: int, N: int, K: int) -> int:
    if (num_experts | N | K) >> 31:
        _sizes("mxfp4_packed_bytes", num_experts, N, K)
    n = ctypes.c_size_t(0)
    _check(load().mxfp4_packed_bytes(num_experts, N, K, ctypes.byref(n)), "mxfp4_packed_bytes")
    return n.value


def mxfp4_repack(w_q, w_s, packed, stream=None):
    name = "mxfp4_repack"
    uint8 = _t().uint8
    E, N, half = w_q.shape
    need = mxfp4_packed_bytes(E, N, 2 * half)
    if w_s.shape != (E, N, half // 16) or w_q.dtype is not uint8 or w_s.dtype is not uint8:
        _refuse(name, "w_q and w_s are not uint8 [E, N, K / 2] and [E, N, K / 32]")
    if _nbytes(packed) < need:
        _refuse(name, "packed is smaller than mxfp4_packed_bytes")
    _launch(load().mxfp4_repack, name, (E, N, 2 * half, w_q.data_ptr(), w_s.data_ptr(), packed.data_ptr()),
            (w_q, w_s, packed), stream)


def mxfp4_moe_gemm(a_q, a_s, T: int, topk: int, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m: int,
                   num_experts: int, packed, out, gather: bool = False, stream=None):
    """gather: A holds token rows [T, K] (gate_up), read through sorted_token_ids; else aligned rows (down)."""
    name = "mxfp4_moe_gemm"
    rows, half = a_q.shape
    out_rows, N = out.shape
    K = 2 * half
    capacity = sorted_token_ids.numel()
    if (T | topk | capacity | block_m) >> 31:
        _sizes(name, T, topk, capacity, block_m)
    _fp4_buffers(name, rows, K, a_q, a_s, None)
    if out_rows < capacity:
        _refuse(name, "out has fewer rows than sorted_token_ids", CAPACITY)
    if block_m > 0 and expert_ids.numel() < capacity // block_m:
        _refuse(name, "expert_ids has too few blocks")
    if _nbytes(packed) < mxfp4_packed_bytes(num_experts, N, K):
        _refuse(name, "packed is smaller than mxfp4_packed_bytes")
    _int32(name, sorted_token_ids, expert_ids)
    _count(name, num_tokens_post_padded)
    _launch(load().mxfp4_moe_gemm, name,
            (num_experts, N, K, a_q.data_ptr(), a_s.data_ptr(), rows, 1 if gather else 0, T, topk,
             sorted_token_ids.data_ptr(), capacity, expert_ids.data_ptr(), num_tokens_post_padded.data_ptr(), block_m,
             packed.data_ptr(), out.data_ptr(), _dtype(out, name)),
            (a_q, a_s, sorted_token_ids, expert_ids, num_tokens_post_padded, packed, out), stream)


def moe_grouped_gemm(a, T: int, topk: int, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m: int, w, out,
                     gather: bool = False, transposed: bool = False, stream=None):
    """gather: a holds token rows, read through sorted_token_ids. transposed: w is [E, K, N], for the rows' gradient."""
    name = "moe_grouped_gemm"
    rows, K = a.shape
    out_rows, N = out.shape
    E = w.shape[0]
    capacity = sorted_token_ids.numel()
    if w.shape != ((E, K, N) if transposed else (E, N, K)):
        _refuse(name, "w is not [E, K, N]" if transposed else "w is not [E, N, K]")
    if w.dtype is not a.dtype:
        _refuse(name, "w is not of a's type")
    if out_rows < capacity:
        _refuse(name, "out has fewer rows than sorted_token_ids", CAPACITY)
    if block_m > 0 and expert_ids.numel() < capacity // block_m:
        _refuse(name, "expert_ids has too few blocks")
    if (T | topk | capacity | block_m | rows | E | K | N) >> 31:
        _sizes(name, T, topk, capacity, block_m, rows, E, K, N)
    _int32(name, sorted_token_ids, expert_ids)
    _count(name, num_tokens_post_padded)
    _launch(load().moe_grouped_gemm, name,
            (E, N, K, a.data_ptr(), _dtype(a, name), rows, 1 if gather else 0, T, topk, sorted_token_ids.data_ptr(),
             capacity, expert_ids.data_ptr(), num_tokens_post_padded.data_ptr(), block_m, w.data_ptr(),
             1 if transposed else 0, out.data_ptr(), _dtype(out, name)),
            (a, sorted_token_ids, expert_ids, num_tokens_post_padded, w, out), stream)


def moe_grouped_gemm_wgrad_workspace_bytes(num_experts: int, N: int, K: int, capacity: int) -> int:
    if (num_experts | N | K | capacity) >> 31:
        _sizes("moe_grouped_gemm_wgrad_workspace_bytes", num_experts, N, K, capacity)
    return load().moe_grouped_gemm_wgrad_workspace_bytes(num_experts, N, K, capacity)


def moe_grouped_gemm_wgrad(dout, a, T: int, topk: int, sorted_token_ids, expert_ids, num_tokens_post_padded,
                           block_m: int, dw, gather: bool = False, accumulate: bool = False, workspace=None,
                           stream=None):
    """accumulate: the gradient is added to what dw holds."""
    name = "moe_grouped_gemm_wgrad"
    E, N, K = dw.shape
    rows, width = a.shape
    capacity = sorted_token_ids.numel()
    if width != K or dout.dim() != 2 or dout.shape[1] != N:
        _refuse(name, "a and dout are not [rows, K] and [rows, N] of dw's [E, N, K]")
    if dout.dtype is not a.dtype:
        _refuse(name, "dout is not of a's type")
    if dout.shape[0] < capacity:
        _refuse(name, "dout has fewer rows than sorted_token_ids", CAPACITY)
    if block_m > 0 and expert_ids.numel() < capacity // block_m:
        _refuse(name, "expert_ids has too few blocks")
    if (T | topk | capacity | block_m | rows | E | K | N) >> 31:
        _sizes(name, T, topk, capacity, block_m, rows, E, K, N)
    _int32(name, sorted_token_ids, expert_ids)
    _count(name, num_tokens_post_padded)
    _launch(load().moe_grouped_gemm_wgrad, name,
            (E, N, K, dout.data_ptr(), a.data_ptr(), _dtype(a, name), rows, 1 if gather else 0, T, topk,
             sorted_token_ids.data_ptr(), capacity, expert_ids.data_ptr(), num_tokens_post_padded.data_ptr(), block_m,
             dw.data_ptr(), _dtype(dw, name), 1 if accumulate else 0, _ptr(workspace), _nbytes(workspace)),
            (dout, a, sorted_token_ids, expert_ids, num_tokens_post_padded, dw, workspace), stream)


def _fp8_buffers(name: str, rows: int, K: int, q, s, num_rows):
    uint8 = _t().uint8
    if K % 32:
        _refuse(name, "rows are not a multiple of 32 long", UNSUPPORTED)
    if (rows | K) >> 31:
        _sizes(name, rows, K)
    if q.shape != (rows, K) or s.shape != (rows, K // 32):
        _refuse(name, "codes and scales are not [rows, K] and [rows, K / 32]")
    if q.dtype is not uint8 or s.dtype is not uint8:
        _refuse(name, "codes and scales are uint8")
    _count(name, num_rows)


def mxfp8_quantize(x, q, s, num_rows=None, stream=None):
    name = "mxfp8_quantize"
    rows, K = x.shape
    _fp8_buffers(name, rows, K, q, s, num_rows)
    _launch(load().mxfp8_quantize, name,
            (x.data_ptr(), _dtype(x, name), rows, K, _ptr(num_rows), q.data_ptr(), s.data_ptr()),
            (x, q, s, num_rows), stream)


def mxfp8_dequantize(q, s, out, num_rows=None, stream=None):
    name = "mxfp8_dequantize"
    rows, K = out.shape
    _fp8_buffers(name, rows, K, q, s, num_rows)
    _launch(load().mxfp8_dequantize, name,
            (q.data_ptr(), s.data_ptr(), rows, K, _ptr(num_rows), out.data_ptr(), _dtype(out, name)),
            (q, s, out, num_rows), stream)


def mxfp8_silu_mul(gu, h, q, s, num_rows=None, stream=None):
    """gu [rows, 2 I] -> h [rows, I], and gu in 8 bits (q [rows, 2 I], s [rows, I / 16]) for the backward pass."""
    name = "mxfp8_silu_mul"
    rows, I = h.shape
    if gu.shape != (rows, 2 * I) or gu.dtype is not h.dtype:
        _refuse(name, "gu is not [rows, 2 I] of h's type")
    if I % 32:
        _refuse(name, "rows are not a multiple of 32 long", UNSUPPORTED)
    _fp8_buffers(name, rows, 2 * I, q, s, num_rows)
    _launch(load().mxfp8_silu_mul, name,
            (gu.data_ptr(), _dtype(gu, name), rows, I, _ptr(num_rows), h.data_ptr(), q.data_ptr(), s.data_ptr()),
            (gu, h, q, s, num_rows), stream)


def mxfp8_silu_mul_backward(q, s, dh, dgu, h=None, num_rows=None, stream=None):
    name = "mxfp8_silu_mul_backward"
    rows, I = dh.shape
    if dgu.shape != (rows, 2 * I) or dgu.dtype is not dh.dtype:
        _refuse(name, "dgu is not [rows, 2 I] of dh's type")
    if h is not None and (h.shape != dh.shape or h.dtype is not dh.dtype):
        _refuse(name, "h is not like dh")
    if I % 32:
        _refuse(name, "rows are not a multiple of 32 long", UNSUPPORTED)
    _fp8_buffers(name, rows, 2 * I, q, s, num_rows)
    _launch(load().mxfp8_silu_mul_backward, name,
            (q.data_ptr(), s.data_ptr(), dh.data_ptr(), _dtype(dh, name), rows, I, _ptr(num_rows), dgu.data_ptr(),
             _ptr(h)),
            (q, s, dh, dgu, h, num_rows), stream)


def align_buffers(T: int, topk: int, num_experts: int, block_m: int, device="cuda"):
    """Allocate (torch) the alignment outputs and workspace for one call."""
    import torch

    cap = moe_align_capacity(T, topk, num_experts, block_m)
    if cap == 0 and T * topk + num_experts * (block_m - 1) != 0:
        raise W4A16Error(2, "moe_align_capacity")
    nblk = (cap + block_m - 1) // block_m
    ws = moe_align_workspace_bytes(T, topk, num_experts, block_m)
    return dict(
        sorted_token_ids=torch.empty(max(cap, 1), dtype=torch.int32, device=device)[:cap],
        expert_ids=torch.empty(max(nblk, 1), dtype=torch.int32, device=device)[:nblk],
        num_tokens_post_padded=torch.empty(1, dtype=torch.int32, device=device),
        expert_counts=torch.empty(num_experts, dtype=torch.int32, device=device),
        workspace=torch.empty(max(ws, 1), dtype=torch.uint8, device=device) if ws else None,
    )
