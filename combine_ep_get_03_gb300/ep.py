"""ctypes binding of ``libep_gb300.so`` -- the C ABI in ``include/ep.h``.

Argument marshalling only: every function takes torch tensors (or None for a
NULL pointer), checks dtype / device / contiguity, and passes raw device
pointers and the current CUDA stream to the library call of the same name.
All computation happens in the library's CUDA kernels; if the library is
missing this module raises instead of computing anything itself.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep_gb300.so")

EP_OK, EP_ERR_INVALID_ARG, EP_ERR_CUDA, EP_ERR_CAPACITY, EP_ERR_BAD_EXPERT, EP_ERR_TIMEOUT, EP_ERR_STATE = range(7)
EP_BF16, EP_FP8_E4M3 = 0, 1
EP_LAYOUT_RANK_MAJOR, EP_LAYOUT_LOW_LATENCY, EP_LAYOUT_EXPERT_MAJOR = 0, 1, 2
EP_LOGITS_FP32, EP_LOGITS_BF16 = 0, 1
EP_GATE_SOFTMAX, EP_GATE_SIGMOID = 0, 1
EP_REAL_FP32, EP_REAL_BF16 = 0, 1

_lock = threading.Lock()
_lib = None


class EPError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: {status_str(status)} ({status})")
        self.status = status


# ep_groups_t, ep_fp8_rows_t and ep_block_norm_t of include/ep.h, as the bytes of one struct
_GROUPS = struct.Struct("@PPiqqP")
_FP8_ROWS = struct.Struct("@PPqq")
_BLOCK_NORM = struct.Struct("@PPPPiiiiiff4x")


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -m combine_ep_get_03_gb300.build); there is no fallback path")
            L = ctypes.CDLL(LIB_PATH)
            P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
            L.ep_handle_create.argtypes = [I, I, I, I, I, ctypes.POINTER(P)]
            L.ep_handle_destroy.argtypes = [P]
            L.ep_get_dispatch_layout.argtypes = [P, P, I, P, P, P, P]
            L.ep_get_num_recv.argtypes = [P, P, P, P, P]
            L.ep_dispatch.argtypes = [P, P, P, I, P, P, I64, P, P, P, I, P]
            L.ep_combine.argtypes = [P, P, I64, P, I, P]
            L.ep_combine_ex.argtypes = [P, I, P, P, I64, P, P, P, I, P]
            L.ep_handle_set_topk_idx_bits.argtypes = [P, I]
            L.ep_handle_topk_idx_bits.argtypes = [P]
            L.ep_handle_topk_idx_bits.restype = I
            L.ep_em_layout_and_dispatch.argtypes = [P, P, I, P, P, I, I, P, P, I64, I64, P, P, I, P]
            L.ep_em_dispatch.argtypes = [P, P, P, I, P, P, I64, I64, P, P, I, P]
            L.ep_em_get_layout.argtypes = [P, P, P, P]
            L.ep_em_combine.argtypes = [P, P, I64, P, I, P]
            L.ep_em_combine_weighted.argtypes = [P, P, I64, P, P, I, P]
            L.ep_em_combine_weighted_backward.argtypes = [P, P, P, I64, P, I, P, P, I64, P, I, P]
            L.ep_em_get_groups.argtypes = [P, P, P, P]
            L.ep_em_combine_weights.argtypes = [P, P, I64, P, P]
            L.ep_get_buffer_size_hint.argtypes = [I, I, I, I, I, I, I, I, P, P]
            L.ep_layout_and_dispatch.argtypes = [P, P, I, P, P, I, P, P, I64, P, P, P, I, P]
            L.ep_low_latency_dispatch.argtypes = [P, P, P, I, I, P, P, P, P, I, P]
            L.ep_low_latency_combine.argtypes = [P, P, P, P, I, P]
            L.ep_get_device_status.argtypes = [P, P]
            L.ep_check_wait_timeout.argtypes = [P, P]
            L.ep_get_dispatch_layout_noalloc.argtypes = [I, I, I, P, I, P, P, P, P, P, P, P, P, P, P]
            F32 = ctypes.c_float
            GP, RP = ctypes.c_char_p, ctypes.c_char_p
            L.ep_gate_workspace_bytes.argtypes = [I, P]
            L.ep_gate_forward.argtypes = [P, I, I64, P, I, I, I, I, I, I, F32, P, I, P, P, P, P, P, I, P]
            L.ep_gate_backward.argtypes = [P, I, I64, P, I, I, I, I, F32, P, I, P, P, P, P, I64, I, P]
            L.ep_grouped_matmul.argtypes = [GP, RP, P, P, I, I, P, I, P]
            L.ep_grouped_matmul_swiglu.argtypes = [GP, RP, P, P, I, I, P, RP, RP, I, P]
            L.ep_grouped_matmul_w4.argtypes = [GP, RP, P, P, I, I, P, I, P]
            L.ep_grouped_matmul_w4_swiglu.argtypes = [GP, RP, P, P, I, I, P, RP, I, P]
            L.ep_grouped_swiglu_backward.argtypes = [GP, P, RP, P, I, RP, P, I, P]
            L.ep_grouped_weight_grad.argtypes = [GP, RP, I, RP, I, P, I, P]
            L.ep_block_norm_forward.argtypes = [GP, P, P, P, P, P, I, P]
            L.ep_block_norm_workspace_bytes.argtypes = [I, P]
            L.ep_block_norm_backward.argtypes = [GP, P, P, P, P, P, P, P, P, P, P, P, I, P]
            L.ep_status_str.argtypes = [I]
            L.ep_status_str.restype = ctypes.c_char_p
            for n in ("ep_handle_create", "ep_handle_destroy", "ep_get_dispatch_layout", "ep_get_num_recv",
                      "ep_dispatch", "ep_combine", "ep_layout_and_dispatch", "ep_low_latency_dispatch",
                      "ep_low_latency_combine", "ep_combine_ex", "ep_handle_set_topk_idx_bits",
                      "ep_em_layout_and_dispatch", "ep_em_dispatch", "ep_em_get_layout", "ep_em_combine",
                      "ep_get_buffer_size_hint", "ep_em_get_groups", "ep_em_combine_weights", "ep_em_combine_weighted",
                      "ep_em_combine_weighted_backward", "ep_gate_workspace_bytes", "ep_gate_forward", "ep_gate_backward",
                      "ep_grouped_matmul", "ep_grouped_matmul_swiglu", "ep_grouped_swiglu_backward",
                      "ep_grouped_weight_grad", "ep_grouped_matmul_w4", "ep_grouped_matmul_w4_swiglu",
                      "ep_block_norm_forward", "ep_block_norm_workspace_bytes", "ep_block_norm_backward",
                      "ep_get_device_status", "ep_check_wait_timeout", "ep_get_dispatch_layout_noalloc"):
                getattr(L, n).restype = I
            _lib = L
    return _lib


def status_str(s: int) -> str:
    return lib().ep_status_str(int(s)).decode()


ep_status_str = status_str


def _check(status: int, call: str) -> int:
    if status != EP_OK:
        raise EPError(status, call)
    return status


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        # the current stream's handle without building a Stream object (a few
        # microseconds a call, which the low-latency calls notice)
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t, dtypes=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.data_ptr()


_FP8_BYTES = (torch.uint8, torch.float8_e4m3fn)


def _ids_ptr(h, topk_idx):
    """topk_idx must have the width the handle reads (int64 or int32)."""
    bits = lib().ep_handle_topk_idx_bits(h)
    return _ptr(topk_idx, (torch.int32,) if bits == 32 else (torch.int64,), "topk_idx")


# ------------------------------------------------------------------ calls

def ep_handle_create(num_ranks: int, num_experts: int, num_topk: int, hidden: int,
                     max_tokens_per_rank: int) -> int:
    h = ctypes.c_void_p()
    _check(lib().ep_handle_create(num_ranks, num_experts, num_topk, hidden, max_tokens_per_rank,
                                  ctypes.byref(h)), "ep_handle_create")
    return h.value


def ep_handle_set_topk_idx_bits(h: int, bits: int) -> None:
    _check(lib().ep_handle_set_topk_idx_bits(h, int(bits)), "ep_handle_set_topk_idx_bits")


def ep_handle_topk_idx_bits(h: int) -> int:
    return int(lib().ep_handle_topk_idx_bits(h))


def ep_handle_destroy(h: int) -> None:
    _check(lib().ep_handle_destroy(h), "ep_handle_destroy")


def ep_get_dispatch_layout(h, topk_idx, num_tokens_per_rank=None, num_tokens_per_expert=None,
                           is_token_in_rank=None, stream=None) -> None:
    T = topk_idx.shape[0]
    _check(lib().ep_get_dispatch_layout(
        h, _ids_ptr(h, topk_idx), T,
        _ptr(num_tokens_per_rank, (torch.int32,), "num_tokens_per_rank"),
        _ptr(num_tokens_per_expert, (torch.int32,), "num_tokens_per_expert"),
        _ptr(is_token_in_rank, (torch.bool, torch.uint8), "is_token_in_rank"),
        _stream(stream)), "ep_get_dispatch_layout")


def ep_get_num_recv(h, num_ranks: int, num_experts: int, stream=None, check: bool = True):
    """-> (num_recv_tokens_per_rank [R], num_recv_tokens_per_expert [E],
    rank_offset [R+1]) as numpy int32, plus the latched device status."""
    a = np.zeros(num_ranks, np.int32)
    b = np.zeros(num_experts, np.int32)
    c = np.zeros(num_ranks + 1, np.int32)
    st = lib().ep_get_num_recv(h, a.ctypes.data, b.ctypes.data, c.ctypes.data, _stream(stream))
    if check:
        _check(st, "ep_get_num_recv")
    return a, b, c, st


def ep_dispatch(h, x, topk_weights, dtype: int, recv_x, recv_scales=None, recv_src_idx=None,
                recv_topk_idx=None, recv_topk_weights=None, num_sms: int = 0, stream=None) -> None:
    fp8 = dtype == EP_FP8_E4M3
    cap = recv_x.shape[0] if recv_x is not None else 0
    _check(lib().ep_dispatch(
        h, _ptr(x, (torch.bfloat16,), "x"), _ptr(topk_weights, (torch.float32,), "topk_weights"), int(dtype),
        _ptr(recv_x, _FP8_BYTES if fp8 else (torch.bfloat16,), "recv_x"),
        _ptr(recv_scales, (torch.float32,), "recv_scales") if fp8 else None, cap,
        _ptr(recv_src_idx, (torch.int32,), "recv_src_idx"),
        _ptr(recv_topk_idx, (torch.int32,), "recv_topk_idx"),
        _ptr(recv_topk_weights, (torch.float32,), "recv_topk_weights"),
        int(num_sms), _stream(stream)), "ep_dispatch")


def ep_layout_and_dispatch(h, topk_idx, x, topk_weights, dtype: int, recv_x, recv_scales=None, recv_src_idx=None,
                           recv_topk_idx=None, recv_topk_weights=None, num_sms: int = 0, stream=None) -> None:
    fp8 = dtype == EP_FP8_E4M3
    cap = recv_x.shape[0] if recv_x is not None else 0
    _check(lib().ep_layout_and_dispatch(
        h, _ids_ptr(h, topk_idx), topk_idx.shape[0], _ptr(x, (torch.bfloat16,), "x"),
        _ptr(topk_weights, (torch.float32,), "topk_weights"), int(dtype),
        _ptr(recv_x, _FP8_BYTES if fp8 else (torch.bfloat16,), "recv_x"),
        _ptr(recv_scales, (torch.float32,), "recv_scales") if fp8 else None, cap,
        _ptr(recv_src_idx, (torch.int32,), "recv_src_idx"),
        _ptr(recv_topk_idx, (torch.int32,), "recv_topk_idx"),
        _ptr(recv_topk_weights, (torch.float32,), "recv_topk_weights"),
        int(num_sms), _stream(stream)), "ep_layout_and_dispatch")


def ep_combine(h, y, out, num_sms: int = 0, stream=None) -> None:
    _check(lib().ep_combine(h, _ptr(y, (torch.bfloat16,), "y"), y.shape[0],
                            _ptr(out, (torch.bfloat16,), "out"), int(num_sms), _stream(stream)), "ep_combine")


def ep_combine_ex(h, y, out, y_scales=None, recv_topk_weights=None, combined_topk_weights=None, num_sms: int = 0,
                  stream=None) -> None:
    """y bf16 [rows, H], or e4m3 bytes [rows, H] with fp32 y_scales [rows, H/128]."""
    fp8 = y_scales is not None
    _check(lib().ep_combine_ex(
        h, EP_FP8_E4M3 if fp8 else EP_BF16, _ptr(y, _FP8_BYTES if fp8 else (torch.bfloat16,), "y"),
        _ptr(y_scales, (torch.float32,), "y_scales"), y.shape[0],
        _ptr(recv_topk_weights, (torch.float32,), "recv_topk_weights"), _ptr(out, (torch.bfloat16,), "out"),
        _ptr(combined_topk_weights, (torch.float32,), "combined_topk_weights"), int(num_sms), _stream(stream)),
        "ep_combine_ex")


def ep_low_latency_dispatch(h, x, topk_idx, dtype: int, recv_x, recv_scales=None, recv_src_info=None,
                            recv_count=None, num_sms: int = 0, stream=None) -> None:
    fp8 = dtype == EP_FP8_E4M3
    _check(lib().ep_low_latency_dispatch(
        h, _ptr(x, (torch.bfloat16,), "x"), _ids_ptr(h, topk_idx), topk_idx.shape[0],
        int(dtype), _ptr(recv_x, _FP8_BYTES if fp8 else (torch.bfloat16,), "recv_x"),
        _ptr(recv_scales, (torch.float32,), "recv_scales") if fp8 else None,
        _ptr(recv_src_info, (torch.int32,), "recv_src_info"), _ptr(recv_count, (torch.int32,), "recv_count"),
        int(num_sms), _stream(stream)), "ep_low_latency_dispatch")


def ep_low_latency_combine(h, y, topk_weights, out, num_sms: int = 0, stream=None) -> None:
    _check(lib().ep_low_latency_combine(
        h, _ptr(y, (torch.bfloat16,), "y"), _ptr(topk_weights, (torch.float32,), "topk_weights"),
        _ptr(out, (torch.bfloat16,), "out"), int(num_sms), _stream(stream)), "ep_low_latency_combine")


def _em_out(h, dtype, topk_weights, recv_x, recv_scales, recv_src_idx, recv_weights):
    fp8 = dtype == EP_FP8_E4M3
    cap = recv_x.shape[0] if recv_x is not None else 0
    if fp8 and recv_scales is not None and (recv_scales.dim() != 2 or recv_scales.stride(1) != 1):
        raise ValueError("recv_scales must be a contiguous [H/128, scales_ld] tensor")
    ld = recv_scales.shape[1] if (fp8 and recv_scales is not None) else 0
    return (_ptr(topk_weights, (torch.float32,), "topk_weights"), int(dtype),
            _ptr(recv_x, _FP8_BYTES if fp8 else (torch.bfloat16,), "recv_x"),
            _ptr(recv_scales, (torch.float32,), "recv_scales") if fp8 else None, ld, cap,
            _ptr(recv_src_idx, (torch.int32,), "recv_src_idx"), _ptr(recv_weights, (torch.float32,), "recv_weights"))


def ep_em_layout_and_dispatch(h, topk_idx, x, topk_weights, dtype: int, expert_alignment: int, recv_x,
                              recv_scales=None, recv_src_idx=None, recv_weights=None, num_sms: int = 0,
                              stream=None) -> None:
    w, dt, rx, rs, ld, cap, si, rw = _em_out(h, dtype, topk_weights, recv_x, recv_scales, recv_src_idx, recv_weights)
    _check(lib().ep_em_layout_and_dispatch(h, _ids_ptr(h, topk_idx), topk_idx.shape[0],
                                           _ptr(x, (torch.bfloat16,), "x"), w, dt, int(expert_alignment), rx, rs,
                                           ld, cap, si, rw, int(num_sms), _stream(stream)),
           "ep_em_layout_and_dispatch")


def ep_em_dispatch(h, x, topk_weights, dtype: int, recv_x, recv_scales=None, recv_src_idx=None, recv_weights=None,
                   num_sms: int = 0, stream=None) -> None:
    w, dt, rx, rs, ld, cap, si, rw = _em_out(h, dtype, topk_weights, recv_x, recv_scales, recv_src_idx, recv_weights)
    _check(lib().ep_em_dispatch(h, _ptr(x, (torch.bfloat16,), "x"), w, dt, rx, rs, ld, cap, si, rw, int(num_sms),
                                _stream(stream)), "ep_em_dispatch")


def ep_em_get_layout(h, num_experts: int, stream=None, check: bool = True):
    """-> (num_recv_tokens_per_expert [E], expert_offset [E+1]) numpy int32, status."""
    a = np.zeros(num_experts, np.int32)
    b = np.zeros(num_experts + 1, np.int32)
    st = lib().ep_em_get_layout(h, a.ctypes.data, b.ctypes.data, _stream(stream))
    if check:
        _check(st, "ep_em_get_layout")
    return a, b, st


def ep_em_combine(h, y, out, num_sms: int = 0, stream=None) -> None:
    _check(lib().ep_em_combine(h, _ptr(y, (torch.bfloat16,), "y"), y.shape[0], _ptr(out, (torch.bfloat16,), "out"),
                               int(num_sms), _stream(stream)), "ep_em_combine")


def ep_em_combine_weighted(h, y, topk_weights, out, num_sms: int = 0, stream=None) -> None:
    """out[t] = the sum of topk_weights[t, j] y[row of (t, j)] over the unmasked entries."""
    _check(lib().ep_em_combine_weighted(h, _ptr(y, (torch.bfloat16,), "y"), y.shape[0],
                                        _ptr(topk_weights, (torch.float32,), "topk_weights"),
                                        _ptr(out, (torch.bfloat16,), "out"), int(num_sms), _stream(stream)),
           "ep_em_combine_weighted")


def ep_em_combine_weighted_backward(h, grad_out, y, topk_weights, dtype: int, grad_y=None, grad_y_scales=None,
                                    grad_topk_weights=None, num_sms: int = 0, stream=None) -> None:
    """Gradients of ep_em_combine_weighted: of the rows (bf16, or e4m3 with
    scales [H/128, scales_ld]) and of the weights; either may be None."""
    fp8 = dtype == EP_FP8_E4M3
    like = grad_y if grad_y is not None else y
    if like is None:
        raise ValueError("grad_y or y is required")
    if y is not None and y.shape != like.shape:
        raise ValueError(f"y is {list(y.shape)}, grad_y {list(like.shape)}")
    if fp8 and grad_y is not None and (grad_y_scales is None or grad_y_scales.dim() != 2):
        raise ValueError("grad_y_scales must be a contiguous [H/128, scales_ld] tensor")
    _check(lib().ep_em_combine_weighted_backward(
        h, _ptr(grad_out, (torch.bfloat16,), "grad_out"), _ptr(y, (torch.bfloat16,), "y"), like.shape[0],
        _ptr(topk_weights, (torch.float32,), "topk_weights"), int(dtype),
        _ptr(grad_y, _FP8_BYTES if fp8 else (torch.bfloat16,), "grad_y"),
        _ptr(grad_y_scales, (torch.float32,), "grad_y_scales") if fp8 else None,
        grad_y_scales.shape[1] if fp8 and grad_y_scales is not None else 0,
        _ptr(grad_topk_weights, (torch.float32,), "grad_topk_weights"), int(num_sms), _stream(stream)),
        "ep_em_combine_weighted_backward")


def ep_em_get_groups(h, group_offset=None, group_count=None, stream=None) -> None:
    """Copy the last expert-major layout's group offsets [E+1] and counts [E]
    to device tensors, without synchronising."""
    _check(lib().ep_em_get_groups(h, _ptr(group_offset, (torch.int32,), "group_offset"),
                                  _ptr(group_count, (torch.int32,), "group_count"), _stream(stream)),
           "ep_em_get_groups")


def ep_em_combine_weights(h, row_weights, topk_weights, stream=None) -> None:
    """topk_weights [T, k] = the value of each entry's expert-major row, 0 where masked."""
    _check(lib().ep_em_combine_weights(h, _ptr(row_weights, (torch.float32,), "row_weights"), row_weights.numel(),
                                       _ptr(topk_weights, (torch.float32,), "topk_weights"), _stream(stream)),
           "ep_em_combine_weights")


def ep_get_buffer_size_hint(num_ranks, num_experts, num_topk, hidden, max_tokens_per_rank, dtype: int,
                            layout: int, expert_alignment: int = 1):
    """-> (rows, bytes): the largest receive buffers any routing can need."""
    rows, nbytes = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().ep_get_buffer_size_hint(num_ranks, num_experts, num_topk, hidden, max_tokens_per_rank, int(dtype),
                                         int(layout), int(expert_alignment), ctypes.byref(rows),
                                         ctypes.byref(nbytes)), "ep_get_buffer_size_hint")
    return rows.value, nbytes.value


def ep_get_device_status(h, stream=None) -> int:
    """Synchronise, then return and clear the latched device status."""
    return lib().ep_get_device_status(h, _stream(stream))


def ep_check_wait_timeout(h, stream=None) -> None:
    """Enqueue the bounded-wait self-check (waits that cannot complete give
    up and latch EP_ERR_TIMEOUT; read it with ep_get_device_status)."""
    _check(lib().ep_check_wait_timeout(h, _stream(stream)), "ep_check_wait_timeout")


def ep_get_dispatch_layout_noalloc(num_ranks, num_experts, num_topk, topk_idx, num_recv_tokens_per_rank,
                                   num_recv_tokens_per_expert, rank_offset, token_dest, topk_idx32,
                                   num_tokens_per_rank=None, num_tokens_per_expert=None, is_token_in_rank=None,
                                   device_status=None, stream=None) -> None:
    """The handle-free, allocation-free layout: every output is a caller tensor
    (see include/ep.h for shapes); the scan state lives in the library."""
    R, E, k = num_ranks, num_experts, num_topk
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2 or topk_idx.shape[1] != k:
        raise ValueError(f"topk_idx must be a [T, {k}] tensor (num_topk columns)")
    T = topk_idx.shape[0]
    kmax = min(k, R)
    for t, n, name in ((num_recv_tokens_per_rank, R, "num_recv_tokens_per_rank"),
                       (num_recv_tokens_per_expert, E, "num_recv_tokens_per_expert"),
                       (rank_offset, R + 1, "rank_offset"), (token_dest, T * kmax * 2, "token_dest"),
                       (topk_idx32, T * k, "topk_idx32"), (num_tokens_per_rank, R * R, "num_tokens_per_rank"),
                       (num_tokens_per_expert, R * E, "num_tokens_per_expert"),
                       (is_token_in_rank, T * R, "is_token_in_rank"), (device_status, 1, "device_status")):
        if t is not None and t.numel() < n:
            raise ValueError(f"{name} holds {t.numel()} elements, the call needs {n}")
    _check(lib().ep_get_dispatch_layout_noalloc(
        R, E, k, _ptr(topk_idx, (torch.int64,), "topk_idx"), T,
        _ptr(num_tokens_per_rank, (torch.int32,), "num_tokens_per_rank"),
        _ptr(num_tokens_per_expert, (torch.int32,), "num_tokens_per_expert"),
        _ptr(is_token_in_rank, (torch.bool, torch.uint8), "is_token_in_rank"),
        _ptr(num_recv_tokens_per_rank, (torch.int32,), "num_recv_tokens_per_rank"),
        _ptr(num_recv_tokens_per_expert, (torch.int32,), "num_recv_tokens_per_expert"),
        _ptr(rank_offset, (torch.int32,), "rank_offset"), _ptr(token_dest, (torch.int32,), "token_dest"),
        _ptr(topk_idx32, (torch.int32,), "topk_idx32"), _ptr(device_status, (torch.int32,), "device_status"),
        _stream(stream)), "ep_get_dispatch_layout_noalloc")


# ------------------------------------------------------- gate and experts
#
# Row buffers are either expert-major ([rows, width], with group_offset) or
# low latency ([E, M, width], group_offset None); FP8 scales follow as the
# dispatches leave them: [width/128, ld >= rows] or [E, M, width/128].

# These calls are short, so their checks are written for few attribute reads.

_F32, _I32, _BF16 = (torch.float32,), (torch.int32,), (torch.bfloat16,)
_U8 = (torch.uint8,)
_IDS, _MASK = (torch.int64, torch.int32), (torch.bool, torch.uint8)


def _dev_ptr(t, dtypes, name, dev):
    """Device pointer of a contiguous tensor on the current device."""
    try:
        if t.get_device() == dev and t.dtype in dtypes and t.is_contiguous():  # a CPU tensor's device is -1
            return t.data_ptr()
    except AttributeError:  # not a tensor: refused below
        pass
    p = _ptr(t, dtypes, name)
    if p is None:
        raise ValueError(f"{name} is required")
    raise ValueError(f"{name} must be on the current device (cuda:{dev}), got {t.device}")


def _vector(t, n, dtypes, name, dev):
    p = _dev_ptr(t, dtypes, name, dev)
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {n}")
    return p


def _optional(t, n, dtypes, name, dev):
    return None if t is None else _vector(t, n, dtypes, name, dev)


# `lay` below is the layout of a call's row buffers, (dimensions, first
# dimension, M or 0), as _groups finds it in the first of them.

def _groups(rows_like, group_count, group_offset, device_status, name, dev):
    """ep_groups_t of a row buffer, its number of groups, rows and layout."""
    if not isinstance(rows_like, torch.Tensor):
        raise ValueError(f"{name} must be a [rows, width] or [E, M, width] tensor")
    shape = rows_like.shape
    nd = len(shape)
    cp = _dev_ptr(group_count, _I32, "group_count", dev)
    E = group_count.numel()
    if nd == 2:
        if group_offset is None:
            raise ValueError("expert-major rows need group_offset: the first row of each group")
        op, rows, per = _vector(group_offset, E, _I32, "group_offset", dev), shape[0], 0
    elif nd == 3:
        if group_offset is not None:
            raise ValueError("low-latency rows [E, M, width] take no group_offset")
        if shape[0] != E:
            raise ValueError(f"{name} holds {shape[0]} groups, group_count {E}")
        op, per = 0, shape[1]
        rows = E * per
    else:
        raise ValueError(f"{name} must be [rows, width] or [E, M, width], got {list(shape)}")
    st = 0 if device_status is None else _vector(device_status, 1, _I32, "device_status", dev)
    return _GROUPS.pack(cp, op, E, rows, per, st), E, rows, (nd, shape[0], per)


def _width(shape, lay, name):
    """Width of a row buffer that must have the call's layout."""
    nd, first, per = lay
    if len(shape) != nd or shape[0] != first or (nd == 3 and shape[1] != per) or shape[-1] == 0:
        lead = [first] if nd == 2 else [first, per]
        raise ValueError(f"{name} must be [{', '.join(map(str, lead))}, width], got {list(shape)}")
    return shape[-1]


def _fp8_rows(data, scales, lay, name, dev):
    """ep_fp8_rows_t of a row buffer with its scales, and its width."""
    p = _dev_ptr(data, _FP8_BYTES, name, dev)
    width = _width(data.shape, lay, name)
    if width & 127:
        raise ValueError(f"{name}'s width must be a multiple of 128, got {width}")
    sp = _dev_ptr(scales, _F32, f"{name}_scales", dev)
    g, have = width >> 7, scales.shape
    nd, first, per = lay
    if nd == 2:
        if len(have) != 2 or have[0] != g or have[1] < first:
            raise ValueError(f"{name}_scales must be [{g}, ld >= {first}] for expert-major rows, got {list(have)}")
        return _FP8_ROWS.pack(p, sp, 1, have[1]), width
    if have != (first, per, g):
        raise ValueError(f"{name}_scales must be {[first, per, g]} for low-latency rows, got {list(have)}")
    return _FP8_ROWS.pack(p, sp, g, 1), width


def _bf16_rows(t, lay, name, dev):
    return _dev_ptr(t, _BF16, name, dev), _width(t.shape, lay, name)


def _expert_weights(w, w_scales, E, N, K, dev):
    wp, sp = _dev_ptr(w, _FP8_BYTES, "w", dev), _dev_ptr(w_scales, _F32, "w_scales", dev)
    if w.shape != (E, N, K):
        raise ValueError(f"w must be [{E}, {N}, {K}], got {list(w.shape)}")
    if w_scales.shape != (E, (N + 127) >> 7, K >> 7):
        raise ValueError(f"w_scales must be [{E}, {(N + 127) >> 7}, {K >> 7}], got {list(w_scales.shape)}")
    return wp, sp


def _stream_on(stream, dev):
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def ep_gate_workspace_bytes(num_experts: int) -> int:
    n = ctypes.c_int64()
    _check(lib().ep_gate_workspace_bytes(num_experts, ctypes.byref(n)), "ep_gate_workspace_bytes")
    return n.value


def _logits(t, name, dev):
    """Pointer, type, row stride and shape of [T, E] logits; rows may be strided."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device (cuda:{dev})")
    dtype, shape = t.dtype, t.shape
    kind = EP_LOGITS_FP32 if dtype is torch.float32 else EP_LOGITS_BF16
    if len(shape) != 2 or (kind == EP_LOGITS_BF16 and dtype is not torch.bfloat16):
        raise ValueError(f"{name} must be [T, E] fp32 or bf16")
    T, E = shape
    ld, step = t.stride()
    if T <= 1:
        ld = max(E, 1)
    if (step != 1 and E > 1 and T > 0) or ld < E:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), kind, ld, T, E


def _topk(topk_idx, T, dev):
    p = _dev_ptr(topk_idx, _IDS, "topk_idx", dev)
    shape = topk_idx.shape
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"topk_idx must be [{T}, k], got {list(shape)}")
    return p, 64 if topk_idx.dtype is torch.int64 else 32, shape[1]


def ep_gate_forward(logits, topk_idx, topk_weights, expert_count, expert_prob, loss, workspace,
                    score: int = EP_GATE_SOFTMAX, num_groups: int = 1, topk_groups: int = 1, loss_coef: float = 0.0,
                    token_mask=None, num_sms: int = 0, stream=None) -> None:
    """Top-k routing of logits [T, E] (rows may be strided): fills topk_idx
    [T, k], topk_weights [T, k], expert_count [E + 1], expert_prob [E] and
    loss [1].  workspace: ep_gate_workspace_bytes(E) zeroed bytes, reusable."""
    dev = torch.cuda.current_device()
    lp, lt, ld, T, E = _logits(logits, "logits", dev)
    ip, bits, k = _topk(topk_idx, T, dev)
    if not isinstance(workspace, torch.Tensor) or workspace.numel() * workspace.element_size() < 16 + 12 * E:
        raise ValueError(f"workspace must be a tensor of at least {16 + 12 * E} zeroed bytes")
    _check(lib().ep_gate_forward(
        lp, lt, ld, _optional(token_mask, T, _MASK, "token_mask", dev), T, E, k, num_groups, topk_groups, score,
        loss_coef, ip, bits, _vector(topk_weights, T * k, _F32, "topk_weights", dev),
        _vector(expert_count, E + 1, _I32, "expert_count", dev), _vector(expert_prob, E, _F32, "expert_prob", dev),
        _vector(loss, 1, _F32, "loss", dev), _dev_ptr(workspace, (workspace.dtype,), "workspace", dev), num_sms,
        _stream_on(stream, dev)), "ep_gate_forward")


def ep_gate_backward(logits, topk_idx, expert_count, grad_topk_weights, grad_loss, grad_logits,
                     score: int = EP_GATE_SOFTMAX, loss_coef: float = 0.0, token_mask=None, num_sms: int = 0,
                     stream=None) -> None:
    """Gradient with respect to the logits from those of topk_weights [T, k]
    and loss [1] (either may be None)."""
    dev = torch.cuda.current_device()
    lp, lt, ld, T, E = _logits(logits, "logits", dev)
    ip, bits, k = _topk(topk_idx, T, dev)
    gp, gt, gld, gT, gE = _logits(grad_logits, "grad_logits", dev)
    if gt != lt or gT != T or gE != E:
        raise ValueError("grad_logits must have the logits' shape and dtype")
    _check(lib().ep_gate_backward(
        lp, lt, ld, _optional(token_mask, T, _MASK, "token_mask", dev), T, E, k, score, loss_coef, ip, bits,
        _vector(expert_count, E + 1, _I32, "expert_count", dev),
        _optional(grad_topk_weights, T * k, _F32, "grad_topk_weights", dev),
        _optional(grad_loss, 1, _F32, "grad_loss", dev), gp, gld, num_sms, _stream_on(stream, dev)), "ep_gate_backward")


def ep_grouped_matmul(x, x_scales, w, w_scales, out, group_count, group_offset=None, device_status=None,
                      num_sms: int = 0, stream=None) -> None:
    """out = x @ w[e].T for the rows of every group: e4m3 x and w [E, N, K]
    with 128-channel and 128 x 128 scales, bf16 out."""
    dev = torch.cuda.current_device()
    g, E, _, lay = _groups(x, group_count, group_offset, device_status, "x", dev)
    xr, K = _fp8_rows(x, x_scales, lay, "x", dev)
    op, N = _bf16_rows(out, lay, "out", dev)
    wp, sp = _expert_weights(w, w_scales, E, N, K, dev)
    _check(lib().ep_grouped_matmul(g, xr, wp, sp, N, K, op, num_sms, _stream_on(stream, dev)), "ep_grouped_matmul")


def ep_grouped_matmul_swiglu(x, x_scales, w, w_scales, act, act_scales, group_count, group_offset=None,
                             row_weights=None, pre=None, pre_scales=None, device_status=None, num_sms: int = 0,
                             stream=None) -> None:
    """act = row_weights * silu(gate) * up in e4m3 with scales, where (gate, up)
    = x @ w[e].T, w [E, 2F, K]; pre (optional) keeps (gate, up) in e4m3."""
    dev = torch.cuda.current_device()
    g, E, rows, lay = _groups(x, group_count, group_offset, device_status, "x", dev)
    xr, K = _fp8_rows(x, x_scales, lay, "x", dev)
    ar, F = _fp8_rows(act, act_scales, lay, "act", dev)
    pr = None
    if pre is not None:
        pr, two = _fp8_rows(pre, pre_scales, lay, "pre", dev)
        if two != 2 * F:
            raise ValueError(f"pre must be {2 * F} wide, got {two}")
    wp, sp = _expert_weights(w, w_scales, E, 2 * F, K, dev)
    _check(lib().ep_grouped_matmul_swiglu(g, xr, wp, sp, F, K, _optional(row_weights, rows, _F32, "row_weights", dev),
                                          ar, pr, num_sms, _stream_on(stream, dev)), "ep_grouped_matmul_swiglu")


def _expert_weights4(w, w_scales, E, N, K, dev):
    wp, sp = _dev_ptr(w, _U8, "w", dev), _dev_ptr(w_scales, _U8, "w_scales", dev)
    if w.shape != (E, N, K >> 1):
        raise ValueError(f"w must be [{E}, {N}, {K >> 1}] for 4-bit codes, got {list(w.shape)}")
    if w_scales.shape != (E, (N + 127) >> 7, K >> 7, 512):
        raise ValueError(f"w_scales must be [{E}, {(N + 127) >> 7}, {K >> 7}, 512], got {list(w_scales.shape)}")
    return wp, sp


def ep_grouped_matmul_w4(x, x_scales, w, w_scales, out, group_count, group_offset=None, device_status=None,
                         num_sms: int = 0, stream=None) -> None:
    """out = x @ w[e].T for the rows of every group: e4m3 x with 128-channel
    scales, w [E, N, K/2] bytes of two e2m1 codes with an exponent for every 32
    channels, w_scales [E, ceil(N/128), K/128, 512] bytes; bf16 out."""
    dev = torch.cuda.current_device()
    g, E, _, lay = _groups(x, group_count, group_offset, device_status, "x", dev)
    xr, K = _fp8_rows(x, x_scales, lay, "x", dev)
    op, N = _bf16_rows(out, lay, "out", dev)
    wp, sp = _expert_weights4(w, w_scales, E, N, K, dev)
    _check(lib().ep_grouped_matmul_w4(g, xr, wp, sp, N, K, op, num_sms, _stream_on(stream, dev)), "ep_grouped_matmul_w4")


def ep_grouped_matmul_w4_swiglu(x, x_scales, w, w_scales, act, act_scales, group_count, group_offset=None,
                                row_weights=None, device_status=None, num_sms: int = 0, stream=None) -> None:
    """act = row_weights * silu(gate) * up in e4m3 with scales, where (gate, up)
    = x @ w[e].T, w [E, 2F, K/2] 4-bit codes with their exponents."""
    dev = torch.cuda.current_device()
    g, E, rows, lay = _groups(x, group_count, group_offset, device_status, "x", dev)
    xr, K = _fp8_rows(x, x_scales, lay, "x", dev)
    ar, F = _fp8_rows(act, act_scales, lay, "act", dev)
    wp, sp = _expert_weights4(w, w_scales, E, 2 * F, K, dev)
    _check(lib().ep_grouped_matmul_w4_swiglu(g, xr, wp, sp, F, K, _optional(row_weights, rows, _F32, "row_weights", dev),
                                             ar, num_sms, _stream_on(stream, dev)), "ep_grouped_matmul_w4_swiglu")


def ep_grouped_swiglu_backward(grad_act, pre, pre_scales, grad_pre, grad_pre_scales, group_count, group_offset=None,
                               row_weights=None, grad_row_weights=None, device_status=None, num_sms: int = 0,
                               stream=None) -> None:
    """Gradient of the pre-activations (e4m3 with scales) and of the row
    weights, from grad_act (bf16) and the 8-bit pre-activations.  128 channels
    whose largest gradient is below 1e-4 lose bits: scale the loss up first."""
    dev = torch.cuda.current_device()
    g, _, rows, lay = _groups(grad_act, group_count, group_offset, device_status, "grad_act", dev)
    dp, F = _bf16_rows(grad_act, lay, "grad_act", dev)
    pr, two = _fp8_rows(pre, pre_scales, lay, "pre", dev)
    gr, two_out = _fp8_rows(grad_pre, grad_pre_scales, lay, "grad_pre", dev)
    if two != 2 * F or two_out != 2 * F:
        raise ValueError(f"pre and grad_pre must be {2 * F} wide, got {two} and {two_out}")
    _check(lib().ep_grouped_swiglu_backward(
        g, dp, pr, _optional(row_weights, rows, _F32, "row_weights", dev), F, gr,
        _optional(grad_row_weights, rows, _F32, "grad_row_weights", dev), num_sms, _stream_on(stream, dev)),
        "ep_grouped_swiglu_backward")


def ep_grouped_weight_grad(grad_out, grad_out_scales, x, x_scales, grad_w, group_count, group_offset=None,
                           device_status=None, num_sms: int = 0, stream=None) -> None:
    """grad_w[e] = grad_out.T @ x over the rows of group e, both e4m3 with
    scales; bf16 [E, N, K]."""
    dev = torch.cuda.current_device()
    g, E, _, lay = _groups(x, group_count, group_offset, device_status, "x", dev)
    yr, N = _fp8_rows(grad_out, grad_out_scales, lay, "grad_out", dev)
    xr, K = _fp8_rows(x, x_scales, lay, "x", dev)
    gp = _dev_ptr(grad_w, _BF16, "grad_w", dev)
    if grad_w.shape != (E, N, K):
        raise ValueError(f"grad_w must be [{E}, {N}, {K}], got {list(grad_w.shape)}")
    _check(lib().ep_grouped_weight_grad(g, yr, N, xr, K, gp, num_sms, _stream_on(stream, dev)), "ep_grouped_weight_grad")


# ------------------------------------------------ the norms around a block

_REALS = (torch.float32, torch.bfloat16)
_BF = torch.bfloat16


def _shaped(t, shape, dtype, name, dev):
    """Device pointer of a contiguous tensor of a shape and dtype, NULL for None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor: refused below
        pass
    _dev_ptr(t, (dtype,), name, dev)
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _block_norm(like, name, post_weight, pre_weight, gate, token_mask, eps, residual_scale, dev):
    """ep_block_norm_t of a call on tensors like [T, H] `like`, its shape and
    dtype, whether the gate comes per token."""
    if not isinstance(like, torch.Tensor) or like.dim() != 2 or like.dtype not in _REALS:
        raise ValueError(f"{name} must be a [T, H] fp32 or bf16 tensor")
    shape, dtype = like.shape, like.dtype
    T, H = shape
    per_token = gate is not None and gate.dim() == 2
    first = post_weight if post_weight is not None else pre_weight if pre_weight is not None else gate
    kind = torch.float32 if first is None or per_token and first is gate else first.dtype
    if kind not in _REALS:
        raise ValueError(f"weights must be fp32 or bf16, got {kind}")
    row = (H,)
    post = _shaped(post_weight, row, kind, "post_weight", dev)
    pre = _shaped(pre_weight, row, kind, "pre_weight", dev)
    g = _shaped(gate, shape, _BF, "gate", dev) if per_token else _shaped(gate, row, kind, "gate", dev)
    mask = 0 if token_mask is None else _vector(token_mask, T, _MASK, "token_mask", dev)
    return _BLOCK_NORM.pack(post or 0, pre or 0, g or 0, mask, T, H, per_token, dtype is _BF, kind is _BF, eps,
                            residual_scale), shape, dtype, per_token


def ep_block_norm_forward(residual, y, new_residual, x, rstd=None, post_weight=None, pre_weight=None, gate=None,
                          eps: float = 1e-6, residual_scale: float = 1.0, token_mask=None, num_sms: int = 0,
                          stream=None) -> None:
    """new_residual = residual + residual_scale * gate * (norm(y) * post_weight)
    and x = norm(new_residual) * pre_weight, norm(v) = v / sqrt(mean(v^2) + eps).

    residual and new_residual [T, H] fp32 or bf16 (they may be one tensor); y
    and x [T, H] bf16; weights [H] fp32 or bf16, all of one dtype; gate [H], or
    [T, H] bf16.  post_weight, gate and pre_weight (with x) may be None; y None:
    no block behind, x is the norm of residual.  rstd [2, T] fp32 keeps what the
    backward pass needs."""
    dev = torch.cuda.current_device()
    n, shape, dtype, _ = _block_norm(residual, "residual", post_weight, pre_weight, gate, token_mask, eps, residual_scale,
                                     dev)
    if (x is None) != (pre_weight is None):
        raise ValueError("x and pre_weight come together")
    if y is None:
        if post_weight is not None or gate is not None or new_residual is not None:
            raise ValueError("post_weight, gate and new_residual need y")
        if x is None:
            raise ValueError("y or x is required")
    elif new_residual is None:
        raise ValueError("new_residual is required")
    _check(lib().ep_block_norm_forward(
        n, _shaped(residual, shape, dtype, "residual", dev), _shaped(y, shape, _BF, "y", dev),
        _shaped(new_residual, shape, dtype, "new_residual", dev), _shaped(x, shape, _BF, "x", dev),
        None if rstd is None else _vector(rstd, 2 * shape[0], _F32, "rstd", dev), num_sms, _stream_on(stream, dev)),
        "ep_block_norm_forward")


def ep_block_norm_workspace_bytes(hidden: int) -> int:
    n = ctypes.c_int64()
    _check(lib().ep_block_norm_workspace_bytes(hidden, ctypes.byref(n)), "ep_block_norm_workspace_bytes")
    return n.value


def ep_block_norm_backward(new_residual, y, rstd, grad_new_residual, grad_x, grad_residual, grad_y, workspace,
                           post_weight=None, pre_weight=None, gate=None, grad_post_weight=None, grad_pre_weight=None,
                           grad_gate=None, residual_scale: float = 1.0, token_mask=None, num_sms: int = 0,
                           stream=None) -> None:
    """Gradients of ep_block_norm_forward from those of new_residual and x
    (either may be None), on what it left: new_residual, rstd, and its y.

    grad_residual [T, H] has the residual's dtype (and may be
    grad_new_residual); grad_y [T, H] bf16; grad_post_weight, grad_pre_weight
    and grad_gate [H] fp32 (grad_gate [T, H] bf16 for a gate per token); each
    may be None.  workspace: ep_block_norm_workspace_bytes(H) bytes."""
    dev = torch.cuda.current_device()
    like = new_residual if new_residual is not None else grad_residual if grad_residual is not None else grad_new_residual
    n, shape, dtype, per_token = _block_norm(like, "new_residual", post_weight, pre_weight, gate, token_mask, 0.0,
                                             residual_scale, dev)
    T, H = shape
    row, f32 = (H,), torch.float32
    if workspace is not None and (not isinstance(workspace, torch.Tensor) or
                                  workspace.numel() * workspace.element_size() < 2048 * H):
        raise ValueError(f"workspace must be a tensor of at least {2048 * H} bytes")
    _check(lib().ep_block_norm_backward(
        n, _shaped(new_residual, shape, dtype, "new_residual", dev), _shaped(y, shape, _BF, "y", dev),
        None if rstd is None else _vector(rstd, 2 * T, _F32, "rstd", dev),
        _shaped(grad_new_residual, shape, dtype, "grad_new_residual", dev), _shaped(grad_x, shape, _BF, "grad_x", dev),
        _shaped(grad_residual, shape, dtype, "grad_residual", dev), _shaped(grad_y, shape, _BF, "grad_y", dev),
        _shaped(grad_gate, shape, _BF, "grad_gate", dev) if per_token else _shaped(grad_gate, row, f32, "grad_gate", dev),
        _shaped(grad_post_weight, row, f32, "grad_post_weight", dev),
        _shaped(grad_pre_weight, row, f32, "grad_pre_weight", dev),
        None if workspace is None else _dev_ptr(workspace, (workspace.dtype,), "workspace", dev), num_sms,
        _stream_on(stream, dev)), "ep_block_norm_backward")


class Handle:
    """Owns one ep_handle_t; methods call the ABI functions of the same name
    after checking that every buffer is large enough for the call."""

    def __init__(self, num_ranks, num_experts, num_topk, hidden, max_tokens_per_rank):
        self.R, self.E, self.k, self.H = num_ranks, num_experts, num_topk, hidden
        self.max_tokens_per_rank = max_tokens_per_rank
        self.T = None      # tokens of the last layout
        self.T_ll = None   # tokens of the last low-latency dispatch
        self.T_em = None   # tokens of the last expert-major layout
        self.em_layouts = 0  # expert-major layouts so far: tells whether the last one is still a caller's own
        self.em_captured = False  # ... unless a graph that makes one was replayed, which nothing here sees
        self.ptr = ep_handle_create(num_ranks, num_experts, num_topk, hidden, max_tokens_per_rank)

    @property
    def topk_idx_bits(self) -> int:
        return ep_handle_topk_idx_bits(self.ptr)

    def set_topk_idx_bits(self, bits: int) -> None:
        ep_handle_set_topk_idx_bits(self.ptr, bits)

    @property
    def M(self) -> int:
        """Rows per expert in the low-latency receive buffer."""
        return self.R * self.max_tokens_per_rank

    @property
    def G(self) -> int:
        return self.H // 128

    def close(self):
        if getattr(self, "ptr", None):
            ep_handle_destroy(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @staticmethod
    def _need(t, n, name):
        if t is not None and t.numel() < n:
            raise ValueError(f"{name} holds {t.numel()} elements, the call needs {n}")

    def get_dispatch_layout(self, topk_idx, num_tokens_per_rank=None, num_tokens_per_expert=None,
                            is_token_in_rank=None, stream=None):
        T = topk_idx.shape[0]
        if topk_idx.dim() != 2 or topk_idx.shape[1] != self.k:
            raise ValueError(f"topk_idx must be [T, {self.k}]")
        self._need(num_tokens_per_rank, self.R * self.R, "num_tokens_per_rank")
        self._need(num_tokens_per_expert, self.R * self.E, "num_tokens_per_expert")
        self._need(is_token_in_rank, T * self.R, "is_token_in_rank")
        ep_get_dispatch_layout(self.ptr, topk_idx, num_tokens_per_rank, num_tokens_per_expert,
                               is_token_in_rank, stream)
        self.T = T

    def get_num_recv(self, stream=None, check=True):
        return ep_get_num_recv(self.ptr, self.R, self.E, stream=stream, check=check)

    def dispatch(self, x, topk_weights, dtype, recv_x, recv_scales=None, recv_src_idx=None,
                 recv_topk_idx=None, recv_topk_weights=None, num_sms=0, stream=None):
        if self.T is None:
            raise RuntimeError("dispatch before any layout on this handle")
        cap = recv_x.shape[0]
        if recv_x.dim() != 2 or recv_x.shape[1] != self.H:
            raise ValueError(f"recv_x must be [cap, {self.H}]")
        self._need(x, self.T * self.H, "x")
        self._need(topk_weights, self.T * self.k, "topk_weights")
        if dtype == EP_FP8_E4M3:
            if recv_scales is None:
                raise ValueError("FP8 dispatch needs recv_scales")
            self._need(recv_scales, cap * self.G, "recv_scales")
        self._need(recv_src_idx, cap, "recv_src_idx")
        self._need(recv_topk_idx, cap * self.k, "recv_topk_idx")
        self._need(recv_topk_weights, cap * self.k, "recv_topk_weights")
        ep_dispatch(self.ptr, x, topk_weights, dtype, recv_x, recv_scales, recv_src_idx, recv_topk_idx,
                    recv_topk_weights, num_sms, stream)

    def layout_and_dispatch(self, topk_idx, x, topk_weights, dtype, recv_x, recv_scales=None, recv_src_idx=None,
                            recv_topk_idx=None, recv_topk_weights=None, num_sms=0, stream=None):
        T = topk_idx.shape[0]
        if topk_idx.dim() != 2 or topk_idx.shape[1] != self.k:
            raise ValueError(f"topk_idx must be [T, {self.k}]")
        cap = recv_x.shape[0]
        if recv_x.dim() != 2 or recv_x.shape[1] != self.H:
            raise ValueError(f"recv_x must be [cap, {self.H}]")
        self._need(x, T * self.H, "x")
        self._need(topk_weights, T * self.k, "topk_weights")
        if dtype == EP_FP8_E4M3:
            if recv_scales is None:
                raise ValueError("FP8 dispatch needs recv_scales")
            self._need(recv_scales, cap * self.G, "recv_scales")
        self._need(recv_src_idx, cap, "recv_src_idx")
        self._need(recv_topk_idx, cap * self.k, "recv_topk_idx")
        self._need(recv_topk_weights, cap * self.k, "recv_topk_weights")
        ep_layout_and_dispatch(self.ptr, topk_idx, x, topk_weights, dtype, recv_x, recv_scales, recv_src_idx,
                               recv_topk_idx, recv_topk_weights, num_sms, stream)
        self.T = T

    def combine(self, y, out, num_sms=0, stream=None):
        if self.T is None:
            raise RuntimeError("combine before any layout on this handle")
        if y.dim() != 2 or y.shape[1] != self.H:
            raise ValueError(f"y must be [rows, {self.H}]")
        self._need(out, self.T * self.H, "out")
        ep_combine(self.ptr, y, out, num_sms, stream)

    def combine_ex(self, y, out, y_scales=None, recv_topk_weights=None, combined_topk_weights=None, num_sms=0,
                   stream=None):
        if self.T is None:
            raise RuntimeError("combine before any layout on this handle")
        if y.dim() != 2 or y.shape[1] != self.H:
            raise ValueError(f"y must be [rows, {self.H}]")
        rows = y.shape[0]
        self._need(out, self.T * self.H, "out")
        self._need(y_scales, rows * self.G, "y_scales")
        self._need(recv_topk_weights, rows * self.k, "recv_topk_weights")
        self._need(combined_topk_weights, self.T * self.k, "combined_topk_weights")
        ep_combine_ex(self.ptr, y, out, y_scales, recv_topk_weights, combined_topk_weights, num_sms, stream)

    def low_latency_dispatch(self, x, topk_idx, dtype, recv_x, recv_scales=None, recv_src_info=None,
                             recv_count=None, num_sms=0, stream=None):
        T = topk_idx.shape[0]
        if topk_idx.dim() != 2 or topk_idx.shape[1] != self.k:
            raise ValueError(f"topk_idx must be [T, {self.k}]")
        rows = self.E * self.M
        self._need(x, T * self.H, "x")
        if recv_x.numel() < rows * self.H:
            raise ValueError(f"recv_x must hold [E, M, H] = [{self.E}, {self.M}, {self.H}]")
        if dtype == EP_FP8_E4M3:
            if recv_scales is None:
                raise ValueError("FP8 dispatch needs recv_scales")
            self._need(recv_scales, rows * self.G, "recv_scales")
        self._need(recv_src_info, rows, "recv_src_info")
        self._need(recv_count, self.E, "recv_count")
        ep_low_latency_dispatch(self.ptr, x, topk_idx, dtype, recv_x, recv_scales, recv_src_info, recv_count,
                                num_sms, stream)
        self.T_ll = T

    def low_latency_combine(self, y, topk_weights, out, num_sms=0, stream=None):
        if self.T_ll is None:
            raise RuntimeError("low-latency combine before any low-latency dispatch")
        if y.numel() < self.E * self.M * self.H:
            raise ValueError(f"y must hold [E, M, H] = [{self.E}, {self.M}, {self.H}]")
        self._need(topk_weights, self.T_ll * self.k, "topk_weights")
        self._need(out, self.T_ll * self.H, "out")
        ep_low_latency_combine(self.ptr, y, topk_weights, out, num_sms, stream)

    # -------------------------------------------------------- expert-major

    def _em_need(self, T, topk_weights, dtype, recv_x, recv_scales, recv_src_idx, recv_weights):
        if recv_x.dim() != 2 or recv_x.shape[1] != self.H:
            raise ValueError(f"recv_x must be [cap, {self.H}]")
        cap = recv_x.shape[0]
        self._need(topk_weights, T * self.k, "topk_weights")
        if dtype == EP_FP8_E4M3:
            if recv_scales is None or recv_scales.dim() != 2 or recv_scales.shape[0] != self.G:
                raise ValueError(f"FP8 dispatch needs recv_scales [{self.G}, scales_ld]")
            if recv_scales.shape[1] < cap:
                raise ValueError("scales_ld must be >= the capacity rows")
        self._need(recv_src_idx, cap, "recv_src_idx")
        self._need(recv_weights, cap, "recv_weights")

    def em_layout_and_dispatch(self, topk_idx, x, topk_weights, dtype, expert_alignment, recv_x, recv_scales=None,
                               recv_src_idx=None, recv_weights=None, num_sms=0, stream=None):
        T = topk_idx.shape[0]
        if topk_idx.dim() != 2 or topk_idx.shape[1] != self.k:
            raise ValueError(f"topk_idx must be [T, {self.k}]")
        self._need(x, T * self.H, "x")
        self._em_need(T, topk_weights, dtype, recv_x, recv_scales, recv_src_idx, recv_weights)
        ep_em_layout_and_dispatch(self.ptr, topk_idx, x, topk_weights, dtype, expert_alignment, recv_x, recv_scales,
                                  recv_src_idx, recv_weights, num_sms, stream)
        self.T_em = T
        self.em_layouts += 1
        self.em_captured = self.em_captured or torch.cuda.is_current_stream_capturing()

    def em_dispatch(self, x, topk_weights, dtype, recv_x, recv_scales=None, recv_src_idx=None, recv_weights=None,
                    num_sms=0, stream=None):
        if self.T_em is None:
            raise RuntimeError("expert-major dispatch before any expert-major layout")
        self._need(x, self.T_em * self.H, "x")
        self._em_need(self.T_em, topk_weights, dtype, recv_x, recv_scales, recv_src_idx, recv_weights)
        ep_em_dispatch(self.ptr, x, topk_weights, dtype, recv_x, recv_scales, recv_src_idx, recv_weights, num_sms,
                       stream)

    def em_get_layout(self, stream=None, check=True):
        return ep_em_get_layout(self.ptr, self.E, stream=stream, check=check)

    def em_combine(self, y, out, num_sms=0, stream=None):
        if self.T_em is None:
            raise RuntimeError("expert-major combine before any expert-major layout")
        if y.dim() != 2 or y.shape[1] != self.H:
            raise ValueError(f"y must be [rows, {self.H}]")
        self._need(out, self.T_em * self.H, "out")
        ep_em_combine(self.ptr, y, out, num_sms, stream)

    def em_combine_weighted(self, y, topk_weights, out, num_sms=0, stream=None):
        if self.T_em is None:
            raise RuntimeError("expert-major combine before any expert-major layout")
        if y.dim() != 2 or y.shape[1] != self.H:
            raise ValueError(f"y must be [rows, {self.H}]")
        self._need(topk_weights, self.T_em * self.k, "topk_weights")
        self._need(out, self.T_em * self.H, "out")
        ep_em_combine_weighted(self.ptr, y, topk_weights, out, num_sms, stream)

    def em_combine_weighted_backward(self, grad_out, y, topk_weights, dtype, grad_y=None, grad_y_scales=None,
                                     grad_topk_weights=None, num_sms=0, stream=None):
        if self.T_em is None:
            raise RuntimeError("expert-major combine before any expert-major layout")
        rows = None
        for t, name in ((y, "y"), (grad_y, "grad_y")):
            if t is None:
                continue
            if t.dim() != 2 or t.shape[1] != self.H:
                raise ValueError(f"{name} must be [rows, {self.H}]")
            if rows is not None and t.shape[0] != rows:
                raise ValueError(f"y has {rows} rows, grad_y {t.shape[0]}")
            rows = t.shape[0]
        self._need(grad_out, self.T_em * self.H, "grad_out")
        self._need(topk_weights, self.T_em * self.k, "topk_weights")
        self._need(grad_topk_weights, self.T_em * self.k, "grad_topk_weights")
        if dtype == EP_FP8_E4M3 and grad_y is not None:
            if grad_y_scales is None or grad_y_scales.dim() != 2 or grad_y_scales.shape[0] != self.G:
                raise ValueError(f"e4m3 rows need grad_y_scales [{self.G}, scales_ld]")
            if grad_y_scales.shape[1] < rows:
                raise ValueError("scales_ld must be >= the rows")
        ep_em_combine_weighted_backward(self.ptr, grad_out, y, topk_weights, dtype, grad_y, grad_y_scales,
                                        grad_topk_weights, num_sms, stream)

    def em_get_groups(self, group_offset=None, group_count=None, stream=None):
        self._need(group_offset, self.E + 1, "group_offset")
        self._need(group_count, self.E, "group_count")
        ep_em_get_groups(self.ptr, group_offset, group_count, stream)

    def em_combine_weights(self, row_weights, topk_weights, stream=None):
        if self.T_em is None:
            raise RuntimeError("expert-major combine before any expert-major layout")
        self._need(topk_weights, self.T_em * self.k, "topk_weights")
        ep_em_combine_weights(self.ptr, row_weights, topk_weights, stream)

    def get_device_status(self, stream=None):
        return ep_get_device_status(self.ptr, stream)

    def check_wait_timeout(self, stream=None):
        ep_check_wait_timeout(self.ptr, stream)
