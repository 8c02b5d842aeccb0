"""Thin Python binding over the libmoedc C ABI.

Argument marshalling only: torch tensors supply device pointers and the
current CUDA stream; every step of layout / dispatch / combine runs in the
library's CUDA kernels.  There is no CPU fallback: if libmoedc.so is missing
or cannot load, every call raises.

Functions named moedc_* mirror the C entry points one to one (caller-owned
outputs, nothing allocated).  layout / dispatch / combine / layout_dispatch
are conveniences that allocate their outputs with torch first.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

from . import build as _build

OK = 0
ERR_ARG = 1
ERR_CAPACITY = 2
ERR_EXPERT_RANGE = 3
ERR_CUDA = 4
ERR_TIMEOUT = 5
ERR_UNIMPLEMENTED = 6

BF16 = 0
FP8_E4M3 = 1
F16 = 2                     # F16 and F32: router, sorted rows, 4-bit products
F32 = 3
SCALES_COL_MAJOR = 0x100    # OR into FP8_E4M3: scales stored [E, H/128, cap]
SCALES_PER_TOKEN = 0x200    # OR into FP8_E4M3: one scale per row, scales [E, cap]
TOKEN_SCALE_MAX_H = 32768   # MOEDC_TOKEN_SCALE_MAX_H

GATE_SOFTMAX = 0
GATE_SIGMOID = 1
GATE_NORMALIZE = 0x10       # OR into either: weights renormalised over the chosen experts
GATE_BIAS_SCORE = 0x100     # OR into either: the choice by score + bias instead of logit + bias
SWIGLU = 1                  # MOEDC_SWIGLU

EXPORTED = ("moedc_api_version", "moedc_strerror", "moedc_layout_workspace_bytes",
            "moedc_layout", "moedc_dispatch", "moedc_combine", "moedc_layout_dispatch",
            "moedc_layout_static_scratch", "moedc_dequant_e4m3", "moedc_rank_layout",
            "moedc_rank_dispatch", "moedc_rank_combine", "moedc_combine_e4m3",
            "moedc_gate", "moedc_gate_grad", "moedc_sort_rows", "moedc_sort_workspace_bytes",
           "moedc_sort", "moedc_unsort", "moedc_unsort_grad", "moedc_matvec_int4",
           "moedc_matvec_int4_workspace_bytes", "moedc_layout_dispatch_workspace_bytes", "moedc_test_set_wait_extra")

STATIC_SCRATCH_BYTES = 1 << 20   # MOEDC_STATIC_SCRATCH_BYTES

_lib = None


class MoedcError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} (status {code})")


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libmoedc.so (built in-tree by __graft_entry__.build()).  Raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libmoedc.so not found at {p}: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(p)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L, F = ctypes.c_int64, ctypes.c_float
    lib.moedc_api_version.argtypes = []
    lib.moedc_api_version.restype = I
    lib.moedc_strerror.argtypes = [I]
    lib.moedc_strerror.restype = ctypes.c_char_p
    lib.moedc_layout_workspace_bytes.argtypes = [I, I, I, I]
    lib.moedc_layout_workspace_bytes.restype = Z
    lib.moedc_layout_dispatch_workspace_bytes.argtypes = [I, I, I, I]
    lib.moedc_layout_dispatch_workspace_bytes.restype = Z
    lib.moedc_layout.argtypes = [P, I, I, I, I, I, P, P, P, P, P, Z, P, P]
    lib.moedc_layout.restype = I
    lib.moedc_dispatch.argtypes = [P, I, I, P, P, P, I, I, I, I, P, P, P, P, P]
    lib.moedc_dispatch.restype = I
    lib.moedc_combine.argtypes = [P, I, I, I, P, P, P, I, I, P, P, P]
    lib.moedc_combine.restype = I
    lib.moedc_layout_dispatch.argtypes = [P, P, I, I, I, I, I, I, I, P, P, P, P, P, P, P, P, Z,
                                          P, P]
    lib.moedc_layout_dispatch.restype = I
    lib.moedc_layout_static_scratch.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P]
    lib.moedc_layout_static_scratch.restype = I
    lib.moedc_dequant_e4m3.argtypes = [P, P, I, P, I, I, I, P, P]
    lib.moedc_dequant_e4m3.restype = I
    lib.moedc_rank_layout.argtypes = [P, I, I, I, P, P, P]
    lib.moedc_rank_layout.restype = I
    lib.moedc_rank_dispatch.argtypes = [P, I, I, P, P, I, I, I, P, P, P, P]
    lib.moedc_rank_dispatch.restype = I
    lib.moedc_rank_combine.argtypes = [P, I, I, I, P, I, P, P]
    lib.moedc_rank_combine.restype = I
    lib.moedc_combine_e4m3.argtypes = [P, P, I, I, I, I, P, P, P, I, I, P, P, P]
    lib.moedc_combine_e4m3.restype = I
    lib.moedc_gate.argtypes = [P, L, I, I, I, I, P, I, F, P, P, P]
    lib.moedc_gate.restype = I
    lib.moedc_gate_grad.argtypes = [P, L, I, I, I, I, P, I, F, P, P, P, P]
    lib.moedc_gate_grad.restype = I
    lib.moedc_sort_rows.argtypes = [I, I, I, I]
    lib.moedc_sort_rows.restype = Z
    lib.moedc_sort_workspace_bytes.argtypes = [I, I, I]
    lib.moedc_sort_workspace_bytes.restype = Z
    lib.moedc_sort.argtypes = [P, L, I, I, I, P, I, I, I, I, P, P, P, P, P, P, Z, P, P]
    lib.moedc_sort.restype = I
    lib.moedc_unsort.argtypes = [P, I, I, I, P, P, I, I, P, P]
    lib.moedc_unsort.restype = I
    lib.moedc_unsort_grad.argtypes = [P, L, P, I, I, I, I, P, P, P, I, P, P, P]
    lib.moedc_unsort_grad.restype = I
    lib.moedc_matvec_int4.argtypes = [P, L, I, I, I, P, P, I, P, I, I, I, I, P, P, P, I, I, P, P,
                                      Z, P, P]
    lib.moedc_matvec_int4.restype = I
    lib.moedc_matvec_int4_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.moedc_matvec_int4_workspace_bytes.restype = Z
    lib.moedc_test_set_wait_extra.argtypes = [ctypes.c_uint]
    lib.moedc_test_set_wait_extra.restype = None
    if path is None:
        _lib = lib
    return lib


def strerror(code: int) -> str:
    try:
        return load().moedc_strerror(int(code)).decode()
    except Exception:  # the library itself is missing
        return f"status {code}"


def _p(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object, which takes
# longer (2.9 us) than the rest of a small call's marshalling.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream: torch.cuda.Stream | None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def _check(code: int, where: str) -> None:
    if code != OK:
        raise MoedcError(code, where)


# ------------------------------------------------------------ raw entry points


def moedc_layout_workspace_bytes(T: int, K: int, E: int, R: int) -> int:
    return int(load().moedc_layout_workspace_bytes(T, K, E, R))


def moedc_layout_dispatch_workspace_bytes(T: int, K: int, E: int, R: int) -> int:
    return int(load().moedc_layout_dispatch_workspace_bytes(T, K, E, R))


def moedc_layout(topk_idx, T, K, E, R, cap, num_tokens_per_expert, num_tokens_per_rank,
                 is_token_in_rank, slot, workspace, workspace_bytes, dev_status,
                 stream=None) -> int:
    return load().moedc_layout(_p(topk_idx), T, K, E, R, cap, _p(num_tokens_per_expert),
                               _p(num_tokens_per_rank), _p(is_token_in_rank), _p(slot),
                               _p(workspace), workspace_bytes, _p(dev_status), _stream(stream))


def moedc_layout_static_scratch(topk_idx, T, K, E, R, cap, num_tokens_per_expert,
                                num_tokens_per_rank, is_token_in_rank, slot, dev_status,
                                stream=None) -> int:
    """moedc_layout without a workspace: for callers that cannot allocate
    device memory, the library's own fixed-size device array serves as
    scratch.  Calls that overlap on the GPU race on that array."""
    return load().moedc_layout_static_scratch(
        _p(topk_idx), T, K, E, R, cap, _p(num_tokens_per_expert), _p(num_tokens_per_rank),
        _p(is_token_in_rank), _p(slot), _p(dev_status), _stream(stream))


def moedc_dispatch(x, T, H, topk_idx, slot, num_tokens_per_expert, K, E, cap, out_dtype, recv,
                   scales, src_idx, dev_status, stream=None) -> int:
    return load().moedc_dispatch(_p(x), T, H, _p(topk_idx), _p(slot), _p(num_tokens_per_expert),
                                 K, E, cap, out_dtype, _p(recv), _p(scales), _p(src_idx),
                                 _p(dev_status), _stream(stream))


def moedc_combine(expert_out, E, cap, H, topk_idx, slot, topk_weights, T, K, y, dev_status,
                  stream=None) -> int:
    return load().moedc_combine(_p(expert_out), E, cap, H, _p(topk_idx), _p(slot),
                                _p(topk_weights), T, K, _p(y), _p(dev_status), _stream(stream))


def moedc_layout_dispatch(x, topk_idx, T, H, K, E, R, cap, out_dtype, num_tokens_per_expert,
                          num_tokens_per_rank, is_token_in_rank, slot, recv, scales, src_idx,
                          workspace, workspace_bytes, dev_status, stream=None) -> int:
    return load().moedc_layout_dispatch(
        _p(x), _p(topk_idx), T, H, K, E, R, cap, out_dtype, _p(num_tokens_per_expert),
        _p(num_tokens_per_rank), _p(is_token_in_rank), _p(slot), _p(recv), _p(scales),
        _p(src_idx), _p(workspace), workspace_bytes, _p(dev_status), _stream(stream))


def moedc_dequant_e4m3(recv, scales, scale_layout, num_tokens_per_expert, E, cap, H, out,
                       stream=None) -> int:
    return load().moedc_dequant_e4m3(_p(recv), _p(scales), scale_layout,
                                     _p(num_tokens_per_expert), E, cap, H, _p(out),
                                     _stream(stream))


def moedc_combine_e4m3(expert_out, expert_scales, scale_layout, E, cap, H, topk_idx, slot,
                       topk_weights, T, K, y, dev_status, stream=None) -> int:
    return load().moedc_combine_e4m3(_p(expert_out), _p(expert_scales), scale_layout, E, cap, H,
                                     _p(topk_idx), _p(slot), _p(topk_weights), T, K, _p(y),
                                     _p(dev_status), _stream(stream))


def moedc_rank_layout(is_token_in_rank, T, R, cap_rank, rank_slot, dev_status, stream=None) -> int:
    return load().moedc_rank_layout(_p(is_token_in_rank), T, R, cap_rank, _p(rank_slot),
                                    _p(dev_status), _stream(stream))


def moedc_rank_dispatch(x, T, H, rank_slot, num_tokens_per_rank, R, cap_rank, out_dtype,
                        recv_rank, scales_rank, rank_src_idx, stream=None) -> int:
    return load().moedc_rank_dispatch(_p(x), T, H, _p(rank_slot), _p(num_tokens_per_rank), R,
                                      cap_rank, out_dtype, _p(recv_rank), _p(scales_rank),
                                      _p(rank_src_idx), _stream(stream))


def moedc_rank_combine(rank_out, R, cap_rank, H, rank_slot, T, y, stream=None) -> int:
    return load().moedc_rank_combine(_p(rank_out), R, cap_rank, H, _p(rank_slot), T, _p(y),
                                     _stream(stream))


def moedc_gate(logits, ld_logits, dtype, T, E, K, bias, flags, scale, topk_idx, topk_weights,
               stream=None) -> int:
    return load().moedc_gate(_p(logits), ld_logits, dtype, T, E, K, _p(bias), flags, scale,
                             _p(topk_idx), _p(topk_weights), _stream(stream))


def moedc_gate_grad(logits, ld_logits, dtype, T, E, K, bias, flags, scale, topk_idx, dweights,
                    dlogits, stream=None) -> int:
    return load().moedc_gate_grad(_p(logits), ld_logits, dtype, T, E, K, _p(bias), flags, scale,
                                  _p(topk_idx), _p(dweights), _p(dlogits), _stream(stream))


def moedc_sort_rows(T: int, K: int, E: int, align: int) -> int:
    return int(load().moedc_sort_rows(T, K, E, align))


def moedc_sort_workspace_bytes(T: int, K: int, E: int) -> int:
    return int(load().moedc_sort_workspace_bytes(T, K, E))


def moedc_sort(x, ldx, dtype, T, H, topk_idx, K, E, align, rows, sorted, row, src, offsets,
               counts, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return load().moedc_sort(_p(x), ldx, dtype, T, H, _p(topk_idx), K, E, align, rows,
                             _p(sorted), _p(row), _p(src), _p(offsets), _p(counts),
                             _p(workspace), workspace_bytes, _p(dev_status), _stream(stream))


def moedc_unsort(sorted, dtype, rows, H, row, topk_weights, T, K, y, stream=None) -> int:
    return load().moedc_unsort(_p(sorted), dtype, rows, H, _p(row), _p(topk_weights), T, K, _p(y),
                               _stream(stream))


def moedc_unsort_grad(dy, lddy, sorted, dtype, T, H, K, row, src, topk_weights, rows, dsorted,
                      dweights, stream=None) -> int:
    return load().moedc_unsort_grad(_p(dy), lddy, _p(sorted), dtype, T, H, K, _p(row), _p(src),
                                    _p(topk_weights), rows, _p(dsorted), _p(dweights),
                                    _stream(stream))


def moedc_matvec_int4_workspace_bytes(x_rows: int, Kd: int, E: int, N: int, flags: int,
                                      rows: int) -> int:
    return int(load().moedc_matvec_int4_workspace_bytes(x_rows, Kd, E, N, flags, rows))


def moedc_matvec_int4(x, ldx, dtype, x_rows, Kd, wq, scales, scale_dtype, zeros, group, E, N,
                      flags, offsets, counts, src, top_k, rows, out, workspace, workspace_bytes,
                      dev_status, stream=None) -> int:
    return load().moedc_matvec_int4(_p(x), ldx, dtype, x_rows, Kd, _p(wq), _p(scales),
                                    scale_dtype, _p(zeros), group, E, N, flags, _p(offsets),
                                    _p(counts), _p(src), top_k, rows, _p(out), _p(workspace),
                                    workspace_bytes, _p(dev_status), _stream(stream))


# ---------------------------------------------------------------- conveniences


@dataclass
class Layout:
    num_tokens_per_expert: torch.Tensor   # int32 [E]
    num_tokens_per_rank: torch.Tensor     # int32 [R]
    is_token_in_rank: torch.Tensor        # uint8 [T, R]
    slot: torch.Tensor                    # int32 [T, K]
    status: torch.Tensor                  # int32 [1] (device)


def _dev_i32(n, device):
    return torch.empty(n, dtype=torch.int32, device=device)


def _need(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def layout_workspace(T: int, K: int, E: int, R: int, device) -> torch.Tensor | None:
    n = moedc_layout_workspace_bytes(T, K, E, R)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device) if n else None


def layout_dispatch_workspace(T: int, K: int, E: int, R: int, device) -> torch.Tensor | None:
    """Workspace that lets moedc_layout_dispatch run as one launch at any T
    (uninitialised memory is fine; do not share it between concurrent calls)."""
    n = moedc_layout_dispatch_workspace_bytes(T, K, E, R)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device) if n else None


def layout(topk_idx: torch.Tensor, E: int, R: int, cap: int,
           workspace: torch.Tensor | None = None, status: torch.Tensor | None = None) -> Layout:
    _need(topk_idx, torch.int32, "topk_idx")
    T, K = topk_idx.shape
    dev = topk_idx.device
    out = Layout(_dev_i32(E, dev), _dev_i32(R, dev),
                 torch.empty((T, R), dtype=torch.uint8, device=dev), _dev_i32((T, K), dev),
                 status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = layout_workspace(T, K, E, R, dev)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(moedc_layout(topk_idx, T, K, E, R, cap, out.num_tokens_per_expert,
                        out.num_tokens_per_rank, out.is_token_in_rank, out.slot, workspace, wsb,
                        out.status), "moedc_layout")
    return out


def alloc_recv(E: int, cap: int, H: int, out_dtype: int, device):
    """recv [E,cap,H] (bf16, or e4m3 as torch.float8_e4m3fn), scales [E,cap,H/128]
    ([E,H/128,cap] with SCALES_COL_MAJOR, [E,cap] with SCALES_PER_TOKEN; fp32,
    e4m3 only) and src_idx [E,cap]."""
    if out_dtype & ~(SCALES_COL_MAJOR | SCALES_PER_TOKEN) == FP8_E4M3:
        recv = torch.empty((E, cap, H), dtype=torch.float8_e4m3fn, device=device)
        shape = ((E, cap) if out_dtype & SCALES_PER_TOKEN
                 else (E, H // 128, cap) if out_dtype & SCALES_COL_MAJOR else (E, cap, H // 128))
        scales = torch.empty(shape, dtype=torch.float32, device=device)
    else:
        recv = torch.empty((E, cap, H), dtype=torch.bfloat16, device=device)
        scales = None
    return recv, scales, torch.empty((E, cap), dtype=torch.int32, device=device)


def dispatch(x: torch.Tensor, topk_idx: torch.Tensor, lay: Layout, E: int, cap: int,
             out_dtype: int, out=None):
    """Returns (recv, scales or None, src_idx)."""
    _need(x, torch.bfloat16, "x")
    _need(topk_idx, torch.int32, "topk_idx")
    T, H = x.shape
    K = topk_idx.shape[1]
    recv, scales, src_idx = out if out is not None else alloc_recv(E, cap, H, out_dtype, x.device)
    _check(moedc_dispatch(x, T, H, topk_idx, lay.slot, lay.num_tokens_per_expert, K, E, cap,
                          out_dtype, recv, scales, src_idx, lay.status), "moedc_dispatch")
    return recv, scales, src_idx


def combine(expert_out: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
            topk_weights: torch.Tensor, status: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    _need(expert_out, torch.bfloat16, "expert_out")
    _need(topk_weights, torch.float32, "topk_weights")
    E, cap, H = expert_out.shape
    T, K = topk_idx.shape
    y = out if out is not None else torch.empty((T, H), dtype=torch.bfloat16,
                                                device=expert_out.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=expert_out.device)
    _check(moedc_combine(expert_out, E, cap, H, topk_idx, slot, topk_weights, T, K, y, status),
           "moedc_combine")
    return y


def layout_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, E: int, R: int, cap: int,
                    out_dtype: int, workspace: torch.Tensor | None = None):
    """Returns (Layout, recv, scales or None, src_idx)."""
    _need(x, torch.bfloat16, "x")
    _need(topk_idx, torch.int32, "topk_idx")
    T, H = x.shape
    K = topk_idx.shape[1]
    dev = x.device
    lay = Layout(_dev_i32(E, dev), _dev_i32(R, dev),
                 torch.empty((T, R), dtype=torch.uint8, device=dev), _dev_i32((T, K), dev),
                 torch.zeros(1, dtype=torch.int32, device=dev))
    recv, scales, src_idx = alloc_recv(E, cap, H, out_dtype, dev)
    if workspace is None:
        workspace = layout_dispatch_workspace(T, K, E, R, dev)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(moedc_layout_dispatch(x, topk_idx, T, H, K, E, R, cap, out_dtype,
                                 lay.num_tokens_per_expert, lay.num_tokens_per_rank,
                                 lay.is_token_in_rank, lay.slot, recv, scales, src_idx, workspace,
                                 wsb, lay.status), "moedc_layout_dispatch")
    return lay, recv, scales, src_idx


def dequant_e4m3(recv: torch.Tensor, scales: torch.Tensor, num_tokens_per_expert: torch.Tensor,
                 out: torch.Tensor | None = None, scale_layout: int = 0) -> torch.Tensor:
    """bf16 [E, cap, H] view of an e4m3 receive buffer (filled rows only)."""
    E, cap, H = recv.shape
    if out is None:
        out = torch.zeros((E, cap, H), dtype=torch.bfloat16, device=recv.device)
    _check(moedc_dequant_e4m3(recv, scales, scale_layout, num_tokens_per_expert, E, cap, H, out),
           "moedc_dequant_e4m3")
    return out


def combine_e4m3(expert_out: torch.Tensor, expert_scales: torch.Tensor, topk_idx: torch.Tensor,
                 slot: torch.Tensor, topk_weights: torch.Tensor, scale_layout: int = 0,
                 status: torch.Tensor | None = None) -> torch.Tensor:
    """Combine from e4m3 expert outputs [E, cap, H] with fp32 scales in the
    given scale_layout (0, SCALES_COL_MAJOR or SCALES_PER_TOKEN)."""
    _need(topk_weights, torch.float32, "topk_weights")
    E, cap, H = expert_out.shape
    T, K = topk_idx.shape
    y = torch.empty((T, H), dtype=torch.bfloat16, device=expert_out.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=expert_out.device)
    _check(moedc_combine_e4m3(expert_out, expert_scales, scale_layout, E, cap, H, topk_idx, slot,
                              topk_weights, T, K, y, status), "moedc_combine_e4m3")
    return y


def rank_layout(lay: Layout, cap_rank: int) -> torch.Tensor:
    """rank_slot [T, R] from a Layout (raises on argument errors)."""
    T, R = lay.is_token_in_rank.shape
    rank_slot = torch.empty((T, R), dtype=torch.int32, device=lay.slot.device)
    _check(moedc_rank_layout(lay.is_token_in_rank, T, R, cap_rank, rank_slot, lay.status),
           "moedc_rank_layout")
    return rank_slot


def rank_dispatch(x: torch.Tensor, rank_slot: torch.Tensor, lay: Layout, cap_rank: int,
                  out_dtype: int):
    """Returns (recv_rank [R, cap_rank, H], scales_rank or None, rank_src_idx [R, cap_rank])."""
    _need(x, torch.bfloat16, "x")
    T, H = x.shape
    R = rank_slot.shape[1]
    recv, scales, src = alloc_recv(R, cap_rank, H, out_dtype, x.device)
    _check(moedc_rank_dispatch(x, T, H, rank_slot, lay.num_tokens_per_rank, R, cap_rank,
                               out_dtype, recv, scales, src), "moedc_rank_dispatch")
    return recv, scales, src


def rank_combine(rank_out: torch.Tensor, rank_slot: torch.Tensor) -> torch.Tensor:
    _need(rank_out, torch.bfloat16, "rank_out")
    R, cap_rank, H = rank_out.shape
    T = rank_slot.shape[0]
    y = torch.empty((T, H), dtype=torch.bfloat16, device=rank_out.device)
    _check(moedc_rank_combine(rank_out, R, cap_rank, H, rank_slot, T, y), "moedc_rank_combine")
    return y


# ------------------------------------------ router, sorted rows, 4-bit products

_LM_DTYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}


def _lm_dtype(t: torch.Tensor, name: str) -> int:
    d = _LM_DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, not {t.dtype}")
    return d


def _need_rows(t: torch.Tensor, name: str) -> int:
    """A 2-D CUDA tensor whose rows are contiguous; returns its row stride."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA matrix with contiguous rows")
    if t.is_contiguous():
        return t.shape[1]
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be a CUDA matrix with contiguous rows")
    ld = t.stride(0)
    if ld < t.shape[1]:
        if t.shape[0] > 1:
            raise ValueError(f"{name} must not repeat or overlap its rows")
        ld = t.shape[1]
    return ld


def _need_shape(t: torch.Tensor, shape, name: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def gate(logits: torch.Tensor, K: int, bias: torch.Tensor | None = None,
         flags: int = GATE_SOFTMAX | GATE_NORMALIZE, scale: float = 1.0, out=None):
    """Top-k router: (topk_idx int32 [T, K], topk_weights fp32 [T, K]) from
    logits [T, E].  bias [E] moves the choice alone: it is added to the logits, or,
    with GATE_BIAS_SCORE (auxiliary-loss-free balancing), to the scores.  `out`
    takes an earlier call's result to write into."""
    ld = _need_rows(logits, "logits")
    dtype = _lm_dtype(logits, "logits")
    T, E = logits.shape
    if bias is not None:
        _need(bias, torch.float32, "bias")
        _need_shape(bias, (E,), "bias")
    if out is None:
        out = (_dev_i32((T, K), logits.device),
               torch.empty((T, K), dtype=torch.float32, device=logits.device))
    idx, w = out
    _need(idx, torch.int32, "out[0]")
    _need(w, torch.float32, "out[1]")
    _need_shape(idx, (T, K), "out[0]")
    _need_shape(w, (T, K), "out[1]")
    _check((_lib or load()).moedc_gate(logits.data_ptr(), ld, dtype, T, E, K, _p(bias), flags,
                                       scale, idx.data_ptr(), w.data_ptr(), _stream(None)),
           "moedc_gate")
    return out


def gate_grad(logits: torch.Tensor, topk_idx: torch.Tensor, dweights: torch.Tensor,
              bias: torch.Tensor | None = None, flags: int = GATE_SOFTMAX | GATE_NORMALIZE,
              scale: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """dlogits [T, E] of gate() with the same arguments, from dweights [T, K]."""
    ld = _need_rows(logits, "logits")
    dtype = _lm_dtype(logits, "logits")
    _need(topk_idx, torch.int32, "topk_idx")
    _need(dweights, torch.float32, "dweights")
    T, E = logits.shape
    K = topk_idx.shape[1]
    _need_shape(topk_idx, (T, K), "topk_idx")
    _need_shape(dweights, (T, K), "dweights")
    if bias is not None:
        _need(bias, torch.float32, "bias")
        _need_shape(bias, (E,), "bias")
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _need(out, logits.dtype, "out")
    _need_shape(out, (T, E), "out")
    _check((_lib or load()).moedc_gate_grad(logits.data_ptr(), ld, dtype, T, E, K, _p(bias), flags,
                                            scale, topk_idx.data_ptr(), dweights.data_ptr(),
                                            out.data_ptr(), _stream(None)), "moedc_gate_grad")
    return out


@dataclass
class Sorted:
    rows: torch.Tensor | None     # [R, H], x's dtype (None: maps only)
    row: torch.Tensor             # int32 [T, K]
    src: torch.Tensor             # int32 [R]
    offsets: torch.Tensor         # int32 [E + 1]
    counts: torch.Tensor          # int32 [E]
    status: torch.Tensor          # int32 [1] (device)
    workspace: torch.Tensor


def sort(x: torch.Tensor | None, topk_idx: torch.Tensor, E: int, align: int = 1,
         status: torch.Tensor | None = None, out: Sorted | None = None,
         rows: int | None = None) -> Sorted:
    """Token rows sorted by expert (x None: the maps alone).  `rows` sets the
    packed buffer's rows (default: as many as any routing of this shape
    needs); `out` takes an earlier call's result of the same shapes to write
    into, its workspace included."""
    _need(topk_idx, torch.int32, "topk_idx")
    T, K = topk_idx.shape
    H, ld, dtype = 1, 1, BF16
    if x is not None:
        ld = _need_rows(x, "x")
        dtype = _lm_dtype(x, "x")
        H = x.shape[1]
        _need_shape(x, (T, H), "x")
    dev = topk_idx.device
    if out is None:
        if rows is None:
            rows = moedc_sort_rows(T, K, E, align)
            if rows == 0 and T > 0:
                raise MoedcError(ERR_ARG, "moedc_sort_rows")
        ws = moedc_sort_workspace_bytes(T, K, E)
        out = Sorted(torch.empty((rows, H), dtype=x.dtype, device=dev) if x is not None else None,
                     _dev_i32((T, K), dev), _dev_i32(rows, dev), _dev_i32(E + 1, dev),
                     _dev_i32(E, dev),
                     status if status is not None
                     else torch.zeros(1, dtype=torch.int32, device=dev),
                     torch.empty(ws, dtype=torch.uint8, device=dev))
    else:
        if status is not None:
            out.status = status
        n = out.src.shape[0]
        if rows is not None and rows != n:
            raise ValueError(f"out holds {n} rows, not {rows}")
        rows = n
        if (x is None) != (out.rows is None):
            raise ValueError("out must hold rows exactly when x is given")
        if x is not None:
            _need(out.rows, x.dtype, "out.rows")
            _need_shape(out.rows, (rows, H), "out.rows")
        _need(out.row, torch.int32, "out.row")
        _need_shape(out.row, (T, K), "out.row")
        _need(out.src, torch.int32, "out.src")
        _need(out.offsets, torch.int32, "out.offsets")
        _need_shape(out.offsets, (E + 1,), "out.offsets")
        _need(out.counts, torch.int32, "out.counts")
        _need_shape(out.counts, (E,), "out.counts")
        _need(out.workspace, torch.uint8, "out.workspace")
    _need(out.status, torch.int32, "status")
    _check((_lib or load()).moedc_sort(_p(x), ld, dtype, T, H, topk_idx.data_ptr(), K, E, align,
                                       rows, _p(out.rows), out.row.data_ptr(),
                                       out.src.data_ptr(), out.offsets.data_ptr(),
                                       out.counts.data_ptr(), out.workspace.data_ptr(),
                                       out.workspace.numel(), out.status.data_ptr(),
                                       _stream(None)), "moedc_sort")
    return out


def unsort(rows: torch.Tensor, row: torch.Tensor, topk_weights: torch.Tensor | None = None,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """y [T, H]: each token's packed rows summed with their weights (None: 1)."""
    dtype = _lm_dtype(rows, "rows")
    _need(rows, rows.dtype, "rows")
    _need(row, torch.int32, "row")
    R, H = rows.shape
    T, K = row.shape
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights")
        _need_shape(topk_weights, (T, K), "topk_weights")
    if out is None:
        out = torch.empty((T, H), dtype=rows.dtype, device=rows.device)
    _need(out, rows.dtype, "out")
    _need_shape(out, (T, H), "out")
    _check((_lib or load()).moedc_unsort(rows.data_ptr(), dtype, R, H, row.data_ptr(),
                                         _p(topk_weights), T, K, out.data_ptr(), _stream(None)),
           "moedc_unsort")
    return out


def sort_grad(drows: torch.Tensor, row: torch.Tensor,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """dx [T, H] of sort(): the gradients of a token's packed rows, summed."""
    return unsort(drows, row, None, out)


def unsort_grad(dy: torch.Tensor, rows: torch.Tensor | None, row: torch.Tensor,
                src: torch.Tensor, topk_weights: torch.Tensor, out=None):
    """(drows [R, H], dweights fp32 [T, K]) of unsort(); rows None: drows alone,
    dweights None."""
    ld = _need_rows(dy, "dy")
    dtype = _lm_dtype(dy, "dy")
    _need(row, torch.int32, "row")
    _need(src, torch.int32, "src")
    _need(topk_weights, torch.float32, "topk_weights")
    T, H = dy.shape
    K = row.shape[1]
    R = src.shape[0]
    _need_shape(row, (T, K), "row")
    _need_shape(topk_weights, (T, K), "topk_weights")
    if rows is not None:
        _need(rows, dy.dtype, "rows")
        _need_shape(rows, (R, H), "rows")
    if out is None:
        out = (torch.empty((R, H), dtype=dy.dtype, device=dy.device),
               torch.empty((T, K), dtype=torch.float32, device=dy.device)
               if rows is not None else None)
    drows, dw = out
    _need(drows, dy.dtype, "out[0]")
    _need_shape(drows, (R, H), "out[0]")
    if dw is not None:
        _need(dw, torch.float32, "out[1]")
        _need_shape(dw, (T, K), "out[1]")
    _check((_lib or load()).moedc_unsort_grad(dy.data_ptr(), ld, _p(rows), dtype, T, H, K,
                                              row.data_ptr(), src.data_ptr(),
                                              topk_weights.data_ptr(), R, drows.data_ptr(),
                                              _p(dw), _stream(None)), "moedc_unsort_grad")
    return out


# a question of sizes alone; asking the library takes 0.8 us of a call's 10
@functools.lru_cache(maxsize=1024)
def _matvec_int4_bytes(x_rows: int, Kd: int, E: int, N: int, flags: int, rows: int) -> int:
    return load().moedc_matvec_int4_workspace_bytes(x_rows, Kd, E, N, flags, rows)


def matvec_int4(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor,
                zeros: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                counts: torch.Tensor | None = None, src: torch.Tensor | None = None,
                top_k: int = 1, swiglu: bool = False, status: torch.Tensor | None = None,
                out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """out [R, N]: packed expert rows times 4-bit weights wq uint8 [E, N, Kd/2]
    ([N, Kd/2]: one linear layer) with scales [E, N, Kd/group]; swiglu: 2N
    weight rows, silu(gate) * up.  offsets and counts from sort(); src and
    top_k read x in token order.  status (int32 [1], for instance sort()'s) takes
    data errors; without one the call waits for its kernels and raises them.
    workspace: moedc_matvec_int4_workspace_bytes bytes, allocated here when None
    and needed."""
    ld = _need_rows(x, "x")
    dtype = _lm_dtype(x, "x")
    if wq.dim() == 2:
        wq, scales = wq[None], scales[None]
        zeros = None if zeros is None else zeros[None]
    _need(wq, torch.uint8, "wq")
    _need(scales, scales.dtype, "scales")
    E, wn, half = wq.shape
    Kd = 2 * half
    if x.shape[1] != Kd:
        raise ValueError(f"x must have {Kd} channels, not {x.shape[1]}")
    groups = scales.shape[-1]
    if scales.shape != (E, wn, groups) or Kd % max(1, groups):
        raise ValueError(f"scales must have shape [{E}, {wn}, {Kd} / group]")
    if zeros is not None:
        _need(zeros, torch.uint8, "zeros")
        _need_shape(zeros, scales.shape, "zeros")
    if swiglu and wn % 2:
        raise ValueError("swiglu needs an even number of weight rows")
    N = wn // 2 if swiglu else wn
    if offsets is not None:
        _need(offsets, torch.int32, "offsets")
        _need_shape(offsets, (E + 1,), "offsets")
    if counts is not None:
        _need(counts, torch.int32, "counts")
        _need_shape(counts, (E,), "counts")
    if src is not None:
        _need(src, torch.int32, "src")
    R = src.shape[0] if src is not None else x.shape[0]
    if out is None:
        out = torch.empty((R, N), dtype=x.dtype, device=x.device)
    _need(out, x.dtype, "out")
    _need_shape(out, (R, N), "out")
    wait = status is None
    if wait:
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("status must be given while a graph is captured")
        status = torch.zeros(1, dtype=torch.int32, device=x.device)
    else:
        _need(status, torch.int32, "status")
    lib = _lib or load()
    flags = SWIGLU if swiglu else 0
    xr = x.shape[0]
    if workspace is None:
        n = _matvec_int4_bytes(xr, Kd, E, N, flags, R)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    else:
        _need(workspace, torch.uint8, "workspace")
    _check(lib.moedc_matvec_int4(x.data_ptr(), ld, dtype, xr, Kd, wq.data_ptr(),
                                 scales.data_ptr(), _lm_dtype(scales, "scales"), _p(zeros),
                                 Kd // max(1, groups), E, N, flags, _p(offsets), _p(counts),
                                 _p(src), top_k, R, out.data_ptr(), _p(workspace),
                                 0 if workspace is None else workspace.numel(),
                                 status.data_ptr(), _stream(None)), "moedc_matvec_int4")
    if wait:
        _check(int(status), "moedc_matvec_int4")
    return out
