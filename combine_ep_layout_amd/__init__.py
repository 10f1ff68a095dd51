"""Python binding of libep_layout.so: MoE expert-parallel dispatch/combine on
one MI355X (gfx950).

Argument marshalling only: every step of layout, dispatch and combine, of the
router, the experts' feed-forward (batches through the pool, a few tokens in one
call) and the optimisers runs in the library's HIP kernels (_ep_torch.so, host
code, checks lists of tensors).  PyTorch provides device memory and streams; the
library is loaded after torch so that both share torch's HIP runtime.  Import
fails loudly when the library has not been built
(``python combine_ep_layout_amd/build.py``).

The names follow the C ABI in include/ep_layout.h (ep_handle_create,
ep_layout, ep_dispatch, ep_combine, ...); ``EpHandle`` bundles them.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Tuple

import numpy as np
import torch

try:
    from . import _ep_torch
except ImportError as e:
    raise ImportError("combine_ep_layout_amd/_ep_torch.so is missing or does not fit this torch: build it with "
                      f"'python combine_ep_layout_amd/build.py' ({e})") from e

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libep_layout.so")

EP_OK = 0
EP_ERR_INVALID_ARGUMENT = 1
EP_ERR_UNSUPPORTED = 2
EP_ERR_OUT_OF_MEMORY = 3
EP_ERR_HANDLE_STATE = 4
EP_ERR_BAD_ROUTING = 5
EP_ERR_TIMEOUT = 6
EP_ERR_HIP = 7

EP_DISPATCH_FP8 = 1 << 0
EP_DISPATCH_TILE_READY = 1 << 1
EP_DISPATCH_BORROW = 1 << 2
EP_CONSUME_GATHER = 1 << 3
EP_SCALE_F32 = 1 << 4
EP_SCALE_ROUND = 1 << 5
EP_SCALE_MN_MAJOR = 1 << 6
EP_CONSUME_SIGNAL_DONE = 1 << 7
EP_CONSUME_STAMPS = 1 << 8

EP_GRAD_F32 = 1 << 9
EP_GRAD_ACCUMULATE = 1 << 10

EP_ROUTE_BF16 = 1 << 11
EP_ROUTE_SIGMOID = 1 << 12
EP_ROUTE_NORMALIZE = 1 << 13
EP_ADAMW_PARAM_BF16 = 1 << 14
EP_ADAMW_GRAD_BF16 = 1 << 15
EP_ADAMW_STATE_8BIT = 1 << 16
EP_MOE_MXFP4 = 1 << 17
EP_MXFP4_BF16 = 1 << 18
EP_MUON_PARAM_BF16 = 1 << 19
EP_MUON_GRAD_BF16 = 1 << 20
EP_MUON_NESTEROV = 1 << 21

# scores of the router by name: flags
SCORES = {"softmax": 0, "sigmoid": EP_ROUTE_SIGMOID}

# activations of the experts' feed-forward by name
ACTIVATIONS = {"silu": 0, "gelu": 1}

# scale flavours by name: flags, element dtype
SCALE_KINDS = {
    "ue8m0": (0, torch.uint8),
    "f32": (EP_SCALE_F32, torch.float32),
    "pow2_f32": (EP_SCALE_F32 | EP_SCALE_ROUND, torch.float32),
}

ARRAYS = {
    "expert_counts": (0, torch.int32),
    "expert_pool_block_offset": (1, torch.int32),
    "num_tiles": (2, torch.int32),
    "tile_expert": (3, torch.int32),
    "pool_arrival_target": (4, torch.int32),
    "pool_arrival_count": (5, torch.int32),
    "tile_ready": (6, torch.int32),
    "slot_to_pool_row": (7, torch.int32),
    "pool_recv_token": (8, torch.int32),
    "topk_weights": (9, torch.float32),
    "y_done_per_token": (10, torch.int32),
    "tile_stamp": (11, torch.int64),
}

EXPORTS = [
    "ep_handle_create", "ep_handle_destroy", "ep_pool_capacity_rows", "ep_max_tiles",
    "ep_num_tokens", "ep_layout", "ep_dispatch", "ep_combine", "ep_handle_get_view",
    "ep_array_bytes", "ep_copy_array", "ep_counts_to_host", "ep_handle_sync_status",
    "ep_tile_consume", "ep_status_string", "ep_borrow_release", "ep_combine_backward",
    "ep_dispatch_backward", "ep_combine_gated", "ep_fp8_cast_back", "ep_scale_ld",
    "ep_layout_noalloc", "ep_set_density_hint", "ep_layout_density", "ep_layout_dispatch",
    "ep_expert_ffn", "ep_expert_ffn_backward", "ep_route", "ep_route_backward", "ep_adamw",
    "ep_moe_tokens", "ep_mxfp4_quantize", "ep_mxfp4_cast_back",
    "ep_muon_workspace_bytes", "ep_muon", "ep_orthogonalize",
]

EP_DENSITY_AUTO = 0
EP_DENSITY_SPARSE = 1
EP_DENSITY_DENSE = 2


class EpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.ep_status_string(status).decode()} (status {status})")


class _Config(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("block_m", ctypes.c_int32)]


class _AdamwConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("step_dev", ctypes.c_void_p), ("grad_scale_dev", ctypes.c_void_p),
                ("grad_scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


class _MoeTokensArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("num_tokens", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("activation", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("scale", ctypes.c_float), ("logits", ctypes.c_void_p), ("logits_ld", ctypes.c_int64),
                ("bias", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p), ("topk_weights", ctypes.c_void_p),
                ("w_gate_up", ctypes.c_void_p), ("gate_up_scales", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("down_scales", ctypes.c_void_p), ("act", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class _MuonConfig(ctypes.Structure):
    _fields_ = [(k, ctypes.c_double) for k in ("lr", "momentum", "weight_decay", "scale", "eps", "a", "b", "c")] + \
               [("steps", ctypes.c_int32), ("flags", ctypes.c_uint32)]


# ep_muon_tensor, one row of an array
_MUON_TENSOR = np.dtype([(k, np.uint64) for k in ("param", "grad", "momentum", "copy")] +
                        [("batch", np.int64), ("rows", np.int32), ("cols", np.int32)])

# ep_adamw_tensor, one row of an array
_ADAMW_TENSOR = np.dtype([(k, np.uint64) for k in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                                   "exp_avg_sq_scale", "copy")] + [("n", np.int64)])


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          f"'python combine_ep_layout_amd/build.py' (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, U32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_int64
    st = ctypes.c_int
    sig = {
        "ep_handle_create": (st, [ctypes.POINTER(_Config), ctypes.POINTER(P)]),
        "ep_handle_destroy": (st, [P]),
        "ep_pool_capacity_rows": (I64, [P]),
        "ep_max_tiles": (I32, [P]),
        "ep_num_tokens": (I32, [P]),
        "ep_layout": (st, [P, P, P, I32, P, ctypes.POINTER(U32)]),
        "ep_dispatch": (st, [P, P, I32, P, P, U32, P, ctypes.POINTER(U32)]),
        "ep_layout_dispatch": (st, [P, P, P, I32, P, I32, P, P, U32, P, ctypes.POINTER(U32),
                                    ctypes.POINTER(U32)]),
        "ep_combine": (st, [P, U32, P, I32, P, P]),
        "ep_handle_get_view": (st, [P, P]),
        "ep_array_bytes": (I64, [P, ctypes.c_int]),
        "ep_copy_array": (st, [P, ctypes.c_int, P, I64, P]),
        "ep_counts_to_host": (st, [P, P, P, P]),
        "ep_handle_sync_status": (st, [P, P]),
        "ep_tile_consume": (st, [P, U32, P, P, I32, U32, P, I32, U32, P]),
        "ep_status_string": (ctypes.c_char_p, [st]),
        "ep_borrow_release": (st, [P, P]),
        "ep_combine_backward": (st, [P, U32, P, P, I32, P, P, P]),
        "ep_dispatch_backward": (st, [P, U32, P, I32, P, P]),
        "ep_combine_gated": (st, [P, U32, P, I32, P, U32, U32, P]),
        "ep_fp8_cast_back": (st, [P, P, U32, I64, I64, I32, P, P]),
        "ep_scale_ld": (I64, [P]),
        "ep_layout_noalloc": (st, [P, I32, I32, I32, I32, I64, P, P, P, P, P, P, P, P, P]),
        "ep_expert_ffn": (st, [P, U32, P, I32, P, P, I32, I32, P, P, P, P]),
        "ep_expert_ffn_backward": (st, [P, U32, P, P, I32, P, P, I32, I32, P, P, U32, P, P, P, P, P]),
        "ep_route": (st, [P, I64, I32, I32, I32, U32, P, ctypes.c_float, P, P, P]),
        "ep_route_backward": (st, [P, I64, I32, I32, I32, U32, ctypes.c_float, P, P, P, I64, P]),
        "ep_adamw": (st, [P, I32, ctypes.POINTER(_AdamwConfig), P]),
        "ep_moe_tokens": (st, [ctypes.POINTER(_MoeTokensArgs), P]),
        "ep_mxfp4_quantize": (st, [P, I64, U32, P, P, P]),
        "ep_mxfp4_cast_back": (st, [P, P, I64, P, P]),
        "ep_muon_workspace_bytes": (I64, [P, I32]),
        "ep_muon": (st, [P, I32, ctypes.POINTER(_MuonConfig), P, I64, P]),
        "ep_orthogonalize": (st, [P, I64, I32, I32, I32, ctypes.POINTER(ctypes.c_double), ctypes.c_double, U32, P, I64,
                                  P, P]),
        "ep_set_density_hint": (st, [P, I32]),
        "ep_layout_density": (I32, [P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    # the raw handle: torch.cuda.current_stream() makes a Stream object for 2.7 us
    if stream is None:
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(stream, shape, dtype, device: torch.device) -> torch.Tensor:
    """Memory that a call makes, out of the pool of the stream that the call runs on:
    a block of the current stream's pool may still be in use by work that is queued
    there, which the call's stream does not wait for."""
    if stream is None or stream == torch.cuda.current_stream(device):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _used_on(stream, *tensors) -> None:
    """Tensors that a call on another stream than the current one hands out or was
    given: their memory is not handed out again before both streams are past their
    use (a stream that the memory belongs to already is no matter)."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                current = torch.cuda.current_stream(t.device)
                if stream != current:
                    t.record_stream(stream)
                    t.record_stream(current)


def _check(status: int, where: str):
    if status != EP_OK:
        raise EpError(status, where)


def _require(t: torch.Tensor, dtype, name: str, device: torch.device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


# --------------------------------------------------- functions of the C ABI --

def ep_handle_create(max_tokens: int, top_k: int, num_experts: int, block_m: int) -> ctypes.c_void_p:
    cfg = _Config(max_tokens, top_k, num_experts, block_m)
    h = ctypes.c_void_p()
    _check(_lib.ep_handle_create(ctypes.byref(cfg), ctypes.byref(h)), "ep_handle_create")
    return h


def ep_handle_destroy(h) -> None:
    _check(_lib.ep_handle_destroy(h), "ep_handle_destroy")


def ep_layout(h, topk_idx: torch.Tensor, topk_weights: torch.Tensor, stream=None) -> int:
    epoch = ctypes.c_uint32()
    T = topk_idx.shape[0]
    _check(_lib.ep_layout(h, _ptr(topk_idx), _ptr(topk_weights), T, _stream(stream),
                          ctypes.byref(epoch)), "ep_layout")
    return epoch.value


def ep_dispatch(h, x: torch.Tensor, pool: torch.Tensor, pool_scales: Optional[torch.Tensor],
                flags: int, stream=None) -> int:
    seq = ctypes.c_uint32()
    _check(_lib.ep_dispatch(h, _ptr(x), x.shape[1], _ptr(pool), _ptr(pool_scales), flags,
                            _stream(stream), ctypes.byref(seq)), "ep_dispatch")
    return seq.value


def ep_layout_dispatch(h, topk_idx: torch.Tensor, topk_weights: torch.Tensor, x: torch.Tensor,
                       pool: torch.Tensor, pool_scales: Optional[torch.Tensor], flags: int,
                       stream=None) -> tuple:
    epoch = ctypes.c_uint32()
    seq = ctypes.c_uint32()
    _check(_lib.ep_layout_dispatch(h, _ptr(topk_idx), _ptr(topk_weights), topk_idx.shape[0], _ptr(x),
                                   x.shape[1], _ptr(pool), _ptr(pool_scales), flags, _stream(stream),
                                   ctypes.byref(epoch), ctypes.byref(seq)), "ep_layout_dispatch")
    return epoch.value, seq.value


def ep_combine(h, epoch: int, expert_out: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    _check(_lib.ep_combine(h, epoch, _ptr(expert_out), expert_out.shape[1], _ptr(y),
                           _stream(stream)), "ep_combine")


def ep_combine_gated(h, epoch: int, expert_out: torch.Tensor, y: torch.Tensor, round: int,
                     spin_limit_us: int, stream=None) -> None:
    _check(_lib.ep_combine_gated(h, epoch, _ptr(expert_out), expert_out.shape[1], _ptr(y), round,
                                 spin_limit_us, _stream(stream)), "ep_combine_gated")


def ep_fp8_cast_back(q: torch.Tensor, scales: torch.Tensor, flags: int, rows: int, scale_ld: int,
                     out: torch.Tensor, stream=None) -> None:
    _check(_lib.ep_fp8_cast_back(_ptr(q), _ptr(scales), flags, rows, scale_ld, q.shape[1], _ptr(out),
                                 _stream(stream)), "ep_fp8_cast_back")


def scale_shape(rows: int, hidden: int, kind: str, mn_major: bool, ld: Optional[int] = None):
    """Shape and dtype of a scale array for `rows` pool rows."""
    _, dtype = SCALE_KINDS[kind]
    G = hidden // 128
    if not mn_major:
        return (rows, G), dtype
    ld = rows if ld is None else ld
    if kind == "ue8m0":
        return ((G + 3) // 4, ld), torch.int32      # packed words
    return (G, ld), dtype


def scale_flags(kind: str, mn_major: bool) -> int:
    return SCALE_KINDS[kind][0] | (EP_SCALE_MN_MAJOR if mn_major else 0)


def cast_back(q: torch.Tensor, scales: torch.Tensor, kind: str = "ue8m0", mn_major: bool = False,
              rows: Optional[int] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """per_token_cast_back: bf16 [rows, H] from e4m3fn codes and their scales."""
    if q.dtype != torch.uint8 or not q.is_contiguous() or q.dim() != 2:
        raise TypeError("q must be a contiguous uint8 [rows, hidden] tensor")
    rows = q.shape[0] if rows is None else int(rows)
    H = q.shape[1]
    if rows > q.shape[0]:
        raise ValueError("rows exceeds q")
    shape, dtype = scale_shape(rows, H, kind, mn_major, scales.shape[1] if mn_major else None)
    if mn_major:      # [groups or words, ld >= rows]
        ok = scales.dim() == 2 and scales.shape[0] == shape[0] and scales.shape[1] >= rows
    else:             # [>= rows, groups]
        ok = scales.dim() == 2 and scales.shape[0] >= rows and scales.shape[1] == shape[1]
    if scales.dtype != dtype or not scales.is_contiguous() or not ok:
        raise ValueError(f"scales must be {dtype} {shape}")
    if out is None:
        out = _empty(stream, (rows, H), torch.bfloat16, q.device)
    if out.dtype != torch.bfloat16 or not out.is_contiguous() or out.shape[0] < rows or out.shape[1] != H:
        raise ValueError("out must be bf16 [rows, hidden]")
    ld = scales.shape[1] if mn_major else 0
    ep_fp8_cast_back(q, scales, scale_flags(kind, mn_major), rows, ld, out, stream)
    _used_on(stream, out)
    return out


def ep_tile_consume(h, seq: int, pool: torch.Tensor, pool_scales: Optional[torch.Tensor],
                    hidden: int, flags: int, out: torch.Tensor, workgroups: int,
                    spin_limit_us: int, stream=None) -> None:
    _check(_lib.ep_tile_consume(h, seq, _ptr(pool), _ptr(pool_scales), hidden, flags, _ptr(out),
                                workgroups, spin_limit_us, _stream(stream)), "ep_tile_consume")


def ep_combine_backward(h, epoch: int, grad_y: torch.Tensor, expert_out: torch.Tensor,
                        grad_expert_out: torch.Tensor, grad_weights: torch.Tensor,
                        stream=None) -> None:
    _check(_lib.ep_combine_backward(h, epoch, _ptr(grad_y), _ptr(expert_out), grad_y.shape[1],
                                    _ptr(grad_expert_out), _ptr(grad_weights), _stream(stream)),
           "ep_combine_backward")


def ep_dispatch_backward(h, epoch: int, grad_pool: torch.Tensor, grad_x: torch.Tensor,
                         stream=None) -> None:
    _check(_lib.ep_dispatch_backward(h, epoch, _ptr(grad_pool), grad_pool.shape[1], _ptr(grad_x),
                                     _stream(stream)), "ep_dispatch_backward")


def ep_expert_ffn(h, epoch: int, pool: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                  activation: int, act: torch.Tensor, gate_up: Optional[torch.Tensor], out: torch.Tensor,
                  stream=None) -> None:
    _check(_lib.ep_expert_ffn(h, epoch, _ptr(pool), pool.shape[1], _ptr(w_gate_up), _ptr(w_down),
                              w_down.shape[2], activation, _ptr(act), _ptr(gate_up), _ptr(out),
                              _stream(stream)), "ep_expert_ffn")


def ep_expert_ffn_backward(h, epoch: int, grad_out: torch.Tensor, pool: torch.Tensor,
                           w_gate_up: torch.Tensor, w_down: torch.Tensor, activation: int,
                           act: torch.Tensor, gate_up: torch.Tensor, flags: int,
                           grad_gate_up: torch.Tensor, grad_pool: Optional[torch.Tensor],
                           grad_w_gate_up: Optional[torch.Tensor], grad_w_down: Optional[torch.Tensor],
                           stream=None) -> None:
    _check(_lib.ep_expert_ffn_backward(h, epoch, _ptr(grad_out), _ptr(pool), pool.shape[1], _ptr(w_gate_up),
                                       _ptr(w_down), w_down.shape[2], activation, _ptr(act), _ptr(gate_up),
                                       flags, _ptr(grad_gate_up), _ptr(grad_pool), _ptr(grad_w_gate_up),
                                       _ptr(grad_w_down), _stream(stream)), "ep_expert_ffn_backward")


def ep_borrow_release(h, consumer_stream=None) -> None:
    _check(_lib.ep_borrow_release(h, _stream(consumer_stream)), "ep_borrow_release")


def ep_handle_sync_status(h, stream=None) -> int:
    return int(_lib.ep_handle_sync_status(h, _stream(stream)))


def _route_args(logits: torch.Tensor, score: str, normalize: bool) -> int:
    """Checks a router's logits; returns the call's flags."""
    dtype = logits.dtype
    if dtype is torch.float32:
        flags = 0
    elif dtype is torch.bfloat16:
        flags = EP_ROUTE_BF16
    else:
        raise TypeError(f"logits must be float32 or bfloat16, got {dtype}")
    if not logits.is_cuda:
        raise ValueError(f"logits must be on a GPU, got {logits.device}")
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    if logits.dim() != 2 or not _plain_rows(logits):
        raise ValueError("logits must be [num_tokens, num_experts] with contiguous rows that do not overlap")
    return flags | SCORES[score] | (EP_ROUTE_NORMALIZE if normalize else 0)


def _plain_rows(t: torch.Tensor) -> bool:
    return t.is_contiguous() or ((t.shape[1] == 1 or t.stride(1) == 1) and _row_stride(t) >= t.shape[1])


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
          normalize: bool = True, scale: float = 1.0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The router: (topk_idx int32, topk_weights fp32), both [num_tokens, top_k],
    from logits [num_tokens, num_experts] (fp32 or bf16, rows may be strided).

    score "softmax" or "sigmoid"; bias [num_experts] is added to sigmoid scores
    for the choice alone; normalize divides a token's weights by their sum.
    Equal scores: the lowest expert first.  -inf closes an expert; slots without
    an expert get -1 and weight 0 (masked for layout())."""
    flags = _route_args(logits, score, normalize)
    device = logits.device
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return route(logits, top_k, score, bias, normalize, scale, stream)
    T, E = logits.shape
    if bias is not None:
        _require(bias, torch.float32, "bias", device)
        if tuple(bias.shape) != (E,):
            raise ValueError(f"bias must be [{E}]")
    idx = _empty(stream, (T, top_k), torch.int32, device)
    w = _empty(stream, (T, top_k), torch.float32, device)
    _check(_lib.ep_route(logits.data_ptr(), _row_stride(logits), T, E, top_k, flags,
                         None if bias is None else bias.data_ptr(), scale, idx.data_ptr(), w.data_ptr(),
                         _stream(stream)), "ep_route")
    _used_on(stream, idx, w)
    return idx, w


def route_backward(logits: torch.Tensor, topk_idx: torch.Tensor, grad_weights: torch.Tensor,
                   score: str = "softmax", normalize: bool = True, scale: float = 1.0,
                   grad_logits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Backward of route: the logits' gradient, in their type, from that of the
    weights (combine_backward()'s grad_weights)."""
    flags = _route_args(logits, score, normalize)
    device = logits.device
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return route_backward(logits, topk_idx, grad_weights, score, normalize, scale, grad_logits, stream)
    T, E = logits.shape
    _require(topk_idx, torch.int32, "topk_idx", device)
    _require(grad_weights, torch.float32, "grad_weights", device)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T or grad_weights.shape != topk_idx.shape:
        raise ValueError("topk_idx / grad_weights must both be [num_tokens, top_k]")
    if grad_logits is None:
        grad_logits = _empty(stream, (T, E), logits.dtype, device)
    elif grad_logits.dtype != logits.dtype or grad_logits.device != device or grad_logits.shape != logits.shape or \
            not _plain_rows(grad_logits):
        raise ValueError("grad_logits must be like logits")
    _check(_lib.ep_route_backward(logits.data_ptr(), _row_stride(logits), T, E, topk_idx.shape[1], flags, scale,
                                  topk_idx.data_ptr(), grad_weights.data_ptr(), grad_logits.data_ptr(),
                                  _row_stride(grad_logits), _stream(stream)), "ep_route_backward")
    _used_on(stream, grad_logits)
    return grad_logits


class Mxfp4(NamedTuple):
    """Values [..., n] as 4-bit codes with an exponent byte for each 32 of them."""
    codes: torch.Tensor         # uint8 [..., n / 2]
    scales: torch.Tensor        # uint8 [..., n / 32]


def mxfp4_quantize(values: torch.Tensor, out: Optional[Mxfp4] = None, stream=None) -> Mxfp4:
    """Values (float32 or bfloat16, the last dimension a multiple of 32) as e2m1 codes,
    two a byte with the lower index in the lower half, and one exponent byte for each
    32: the least power of two under which none is larger than 6.  Values go to the
    nearest code, ties to the even one; a block with an infinity or a NaN reads as NaN."""
    if values.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"values must be float32 or bfloat16, got {values.dtype}")
    device = values.device
    if device.type != "cuda":
        raise ValueError(f"values must be on a GPU, got {device}")
    if not values.is_contiguous() or values.dim() < 1 or values.shape[-1] % 32 != 0:
        raise ValueError("values must be contiguous, their last dimension a multiple of 32")
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return mxfp4_quantize(values, out, stream)
    lead, n = tuple(values.shape[:-1]), values.shape[-1]
    if out is None:
        out = Mxfp4(_empty(stream, (*lead, n // 2), torch.uint8, device), _empty(stream, (*lead, n // 32), torch.uint8, device))
    _check_mxfp4(out, (*lead, n), "out", device)
    _check(_lib.ep_mxfp4_quantize(_ptr(values), values.numel(), EP_MXFP4_BF16 if values.dtype == torch.bfloat16 else 0,
                                  _ptr(out.codes), _ptr(out.scales), _stream(stream)), "ep_mxfp4_quantize")
    _used_on(stream, *out)
    return Mxfp4(*out)


def mxfp4_cast_back(q: Mxfp4, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The bf16 values that codes and scales stand for (what expert_ffn takes, for
    batches that moe_tokens is not for)."""
    codes, scales = q
    device = codes.device
    if device.type != "cuda":
        raise ValueError(f"codes must be on a GPU, got {device}")
    if codes.dim() < 1:
        raise ValueError("codes must have at least one dimension")
    shape = (*codes.shape[:-1], codes.shape[-1] * 2)
    _check_mxfp4(q, shape, "q", device)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return mxfp4_cast_back(q, out, stream)
    if out is None:
        out = _empty(stream, shape, torch.bfloat16, device)
    _require(out, torch.bfloat16, "out", device)
    if tuple(out.shape) != shape:
        raise ValueError(f"out must be {list(shape)}")
    _check(_lib.ep_mxfp4_cast_back(_ptr(codes), _ptr(scales), out.numel(), _ptr(out), _stream(stream)), "ep_mxfp4_cast_back")
    _used_on(stream, out)
    return out


def _check_mxfp4(q, shape, name: str, device: torch.device) -> None:
    """Codes and scales of values of this shape."""
    codes, scales = q
    _require(codes, torch.uint8, f"{name}.codes", device)
    _require(scales, torch.uint8, f"{name}.scales", device)
    lead, n = tuple(shape[:-1]), shape[-1]
    if n % 32 != 0 or tuple(codes.shape) != (*lead, n // 2) or tuple(scales.shape) != (*lead, n // 32):
        raise ValueError(f"{name} must be the codes and scales of {list(shape)} values, the last a multiple of 32")


def moe_tokens(x: torch.Tensor, w_gate_up, w_down, logits: Optional[torch.Tensor] = None, top_k: Optional[int] = None,
               score: str = "softmax", bias: Optional[torch.Tensor] = None, normalize: bool = True, scale: float = 1.0,
               topk_idx: Optional[torch.Tensor] = None, topk_weights: Optional[torch.Tensor] = None,
               activation: str = "silu", y: Optional[torch.Tensor] = None, stream=None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """A whole layer for up to 64 tokens, without a handle: (y, topk_idx, topk_weights),
    y [num_tokens, hidden] bf16.

    x [num_tokens, hidden] bf16, rows may be strided.  The experts' weights are those of
    EpHandle.expert_ffn, w_gate_up [num_experts, 2 * inter, hidden] and w_down
    [num_experts, hidden, inter] in bf16, or both Mxfp4 of these shapes.  With logits
    and top_k the choice is route()'s (score, bias, normalize and scale as there);
    otherwise topk_idx int32 and topk_weights float32 [num_tokens, top_k] make it, and
    an index outside [0, num_experts) is masked.  Where experts have more than some 20
    tokens each, layout_dispatch and expert_ffn are faster."""
    four = isinstance(w_gate_up, tuple)
    if four != isinstance(w_down, tuple):
        raise TypeError("w_gate_up and w_down must both be bfloat16 tensors or both Mxfp4")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"x must be {torch.bfloat16}, got {x.dtype}")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"x must be on a GPU, got {device}")
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return moe_tokens(x, w_gate_up, w_down, logits, top_k, score, bias, normalize, scale, topk_idx, topk_weights,
                              activation, y, stream)
    if x.dim() != 2 or not _plain_rows(x):
        raise ValueError("x must be [num_tokens, hidden] with contiguous rows that do not overlap")
    T, H = x.shape
    down = w_down[0] if four else w_down
    if down.dim() != 3 or down.shape[1] != H:
        raise ValueError(f"w_down must be [num_experts, {H}, inter]")
    E, I = down.shape[0], down.shape[2] * (2 if four else 1)
    for w, shape, name in ((w_gate_up, (E, 2 * I, H), "w_gate_up"), (w_down, (E, H, I), "w_down")):
        if four:
            _check_mxfp4(w, shape, name, device)
        else:
            _require(w, torch.bfloat16, name, device)
            if tuple(w.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}")
    a = _MoeTokensArgs(x=x.data_ptr(), x_ld=_row_stride(x), num_tokens=T, hidden=H, inter=I, num_experts=E,
                       activation=ACTIVATIONS[activation], scale=scale, flags=EP_MOE_MXFP4 if four else 0)
    if logits is not None:
        if topk_idx is not None or topk_weights is not None or top_k is None:
            raise ValueError("give logits with top_k, or topk_idx with topk_weights")
        a.flags |= _route_args(logits, score, normalize)
        if logits.device != device or tuple(logits.shape) != (T, E):
            raise ValueError(f"logits must be [{T}, {E}] on {device}")
        a.logits, a.logits_ld = logits.data_ptr(), _row_stride(logits)
        if bias is not None:
            _require(bias, torch.float32, "bias", device)
            if tuple(bias.shape) != (E,):
                raise ValueError(f"bias must be [{E}]")
            a.bias = bias.data_ptr()
        topk_idx = _empty(stream, (T, top_k), torch.int32, device)
        topk_weights = _empty(stream, (T, top_k), torch.float32, device)
    elif topk_idx is None or topk_weights is None or bias is not None:
        raise ValueError("give logits with top_k, or topk_idx with topk_weights and no bias")
    else:
        _require(topk_idx, torch.int32, "topk_idx", device)
        _require(topk_weights, torch.float32, "topk_weights", device)
        if topk_idx.dim() != 2 or topk_idx.shape[0] != T or topk_weights.shape != topk_idx.shape or \
                top_k not in (None, topk_idx.shape[1]):
            raise ValueError("topk_idx / topk_weights must both be [num_tokens, top_k]")
    a.top_k = K = topk_idx.shape[1]
    a.topk_idx, a.topk_weights = topk_idx.data_ptr(), topk_weights.data_ptr()
    if four:
        a.w_gate_up, a.gate_up_scales = w_gate_up[0].data_ptr(), w_gate_up[1].data_ptr()
        a.w_down, a.down_scales = w_down[0].data_ptr(), w_down[1].data_ptr()
    else:
        a.w_gate_up, a.w_down = w_gate_up.data_ptr(), w_down.data_ptr()
    act = _empty(stream, (T * K, I), torch.bfloat16, device)
    if y is None:
        y = _empty(stream, (T, H), torch.bfloat16, device)
    else:
        _require(y, torch.bfloat16, "y", device)
        if tuple(y.shape) != (T, H):
            raise ValueError(f"y must be [{T}, {H}]")
    a.act, a.y = act.data_ptr(), y.data_ptr()
    _check(_lib.ep_moe_tokens(ctypes.byref(a), _stream(stream)), "ep_moe_tokens")
    _used_on(stream, y, topk_idx, topk_weights)
    return y, topk_idx, topk_weights


_GATHER_ERRORS = {1: (ValueError, "must have as many tensors as params"), 2: (TypeError, "must hold dense tensors"),
                  3: (TypeError, "must be {dtype}"), 4: (ValueError, "must be on {device}"),
                  5: (ValueError, "must be contiguous"),
                  6: (ValueError, "has another number of values than its parameter needs")}


def _gather(table: np.ndarray, key: str, tensors, dtype, device: torch.device, per: int = 1) -> None:
    """Checks one kind of the step's tensors and puts their addresses into the
    table's column (per 0: their lengths into the column n)."""
    base, offset = table.ctypes.data, table.dtype.fields[key][1]
    if per == 0:
        sizes = np.empty(len(table), np.int64)
    else:
        sizes = np.ascontiguousarray(table["n"])
    wrong, which = _ep_torch.gather(tensors, dtype, device.index, sizes.ctypes.data, len(table), per, base + offset,
                                    table.itemsize)
    if wrong:
        kind, text = _GATHER_ERRORS[wrong]
        raise kind(f"{key}s, tensor {which}: " + text.format(dtype=dtype, device=device))
    if per == 0:
        table["n"] = sizes


def adamw(params, grads, exp_avgs, exp_avg_sqs, step, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
          eps: float = 1e-8, weight_decay: float = 1e-2, exp_avg_scales=None, exp_avg_sq_scales=None, copies=None,
          grad_scale=1.0, stream=None) -> None:
    """One AdamW step over lists of tensors, in place.

    params float32 or bfloat16, grads float32 or bfloat16 (each list of one
    type); exp_avgs and exp_avg_sqs float32, or uint8 with exp_avg_scales and
    exp_avg_sq_scales (float32, one for each 128 values): e4m3fn codes of the
    first moment and of the root of the second, which cast_back's "f32" flavour
    reads.  copies: bfloat16 tensors that receive the updated float32
    parameters.  step: the step's number from 1, or an int64 tensor on the GPU
    that holds it when the step runs (for graphs); grad_scale: a number or a
    float32 tensor on the GPU that the gradients are multiplied by."""
    n = len(params)
    if n == 0:
        return
    device, eight = params[0].device, exp_avg_scales is not None
    if eight != (exp_avg_sq_scales is not None):
        raise ValueError("8-bit states need exp_avg_scales and exp_avg_sq_scales")
    if device.type != "cuda":
        raise ValueError(f"params must be on a GPU, got {device}")
    p_dtype, g_dtype = params[0].dtype, grads[0].dtype if len(grads) else None
    for dtype, name in ((p_dtype, "params"), (g_dtype, "grads")):
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    state = torch.uint8 if eight else torch.float32
    t = np.zeros(n, _ADAMW_TENSOR)
    _gather(t, "param", params, p_dtype, device, per=0)
    _gather(t, "grad", grads, g_dtype, device)
    _gather(t, "exp_avg", exp_avgs, state, device)
    _gather(t, "exp_avg_sq", exp_avg_sqs, state, device)
    if eight:
        _gather(t, "exp_avg_scale", exp_avg_scales, torch.float32, device, per=128)
        _gather(t, "exp_avg_sq_scale", exp_avg_sq_scales, torch.float32, device, per=128)
    if copies is not None:
        _gather(t, "copy", copies, torch.bfloat16, device)
    cfg = _AdamwConfig(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay, grad_scale=1.0)
    cfg.flags = (EP_ADAMW_PARAM_BF16 if p_dtype == torch.bfloat16 else 0) | \
        (EP_ADAMW_GRAD_BF16 if g_dtype == torch.bfloat16 else 0) | (EP_ADAMW_STATE_8BIT if eight else 0)
    if isinstance(step, torch.Tensor):
        _require(step, torch.int64, "step", device)
        if step.numel() != 1:
            raise ValueError("step must hold one number")
        cfg.step_dev = step.data_ptr()
    else:
        cfg.step = int(step)
    if isinstance(grad_scale, torch.Tensor):
        _require(grad_scale, torch.float32, "grad_scale", device)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must hold one number")
        cfg.grad_scale_dev = grad_scale.data_ptr()
    else:
        cfg.grad_scale = float(grad_scale)
    with torch.cuda.device(device):
        _check(_lib.ep_adamw(t.ctypes.data_as(ctypes.c_void_p), n, ctypes.byref(cfg), _stream(stream)), "ep_adamw")


NEWTON_SCHULZ = (3.4445, -4.775, 2.0315)


def _muon_workspace(table: np.ndarray, workspace: Optional[torch.Tensor], stream, device: torch.device) -> torch.Tensor:
    """The given workspace, or one of the size that is of use."""
    if workspace is not None:
        _require(workspace, torch.uint8, "workspace", device)
        return workspace
    need = int(_lib.ep_muon_workspace_bytes(table.ctypes.data_as(ctypes.c_void_p), len(table)))
    if need < 0:
        raise EpError(EP_ERR_UNSUPPORTED, "ep_muon_workspace_bytes")
    return _empty(stream, (need,), torch.uint8, device)


def orthogonalize(x: torch.Tensor, steps: int = 5, coefficients=NEWTON_SCHULZ, eps: float = 1e-7,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """x [..., rows, cols] (float32 or bfloat16) orthogonalised, matrix by matrix, in bf16:
    `steps` times X = a X + (b G + c G G) X with G = X X^T (on the shorter side) and
    coefficients (a, b, c), from X = x / (|x| + eps).

    workspace: a uint8 tensor to use (made when not given; with less than it would
    be, fewer matrices go through at once)."""
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"x must be on a GPU, got {device}")
    if x.dim() < 2 or not x.is_contiguous():
        raise ValueError("x must be contiguous [..., rows, cols]")
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return orthogonalize(x, steps, coefficients, eps, out, workspace, stream)
    rows, cols = x.shape[-2:]
    batch = x.numel() // (rows * cols) if rows and cols else 0
    if out is None:
        out = _empty(stream, tuple(x.shape), torch.bfloat16, device)
    _require(out, torch.bfloat16, "out", device)
    if out.shape != x.shape:
        raise ValueError(f"out must be {list(x.shape)}")
    table = np.zeros(1, _MUON_TENSOR)
    table["batch"], table["rows"], table["cols"] = batch, rows, cols
    workspace = _muon_workspace(table, workspace, stream, device)
    abc = (ctypes.c_double * 3)(*coefficients)
    _check(_lib.ep_orthogonalize(_ptr(x), batch, rows, cols, steps, abc, eps,
                                 EP_MUON_GRAD_BF16 if x.dtype == torch.bfloat16 else 0, _ptr(workspace),
                                 workspace.numel(), _ptr(out), _stream(stream)), "ep_orthogonalize")
    _used_on(stream, out)
    return out


def muon(params, grads, momenta, lr: float = 1e-3, momentum: float = 0.95, weight_decay: float = 1e-2,
         nesterov: bool = True, steps: int = 5, coefficients=NEWTON_SCHULZ, eps: float = 1e-7,
         scale: Optional[float] = None, copies=None, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """One step over lists of tensors of matrices [..., rows, cols], in place, whose update
    is orthogonalised matrix by matrix (orthogonalize): the momentum is
    momentum * m + (1 - momentum) * g, the update X of it (nesterov: of its mix with g),
    and p = p (1 - lr weight_decay) - lr scale X.

    params float32 or bfloat16, grads float32 or bfloat16 (each list of one type),
    momenta float32; copies: bfloat16 tensors that receive the updated float32
    parameters.  scale None: 0.2 sqrt(max(rows, cols)), which makes the update as
    large as adamw's.  The experts' gate and up matrices count as two when
    w_gate_up is given as w_gate_up.view(2 * num_experts, inter, hidden).
    workspace: a uint8 tensor to use, as for orthogonalize."""
    n = len(params)
    if n == 0:
        return
    device = params[0].device
    if device.type != "cuda":
        raise ValueError(f"params must be on a GPU, got {device}")
    p_dtype, g_dtype = params[0].dtype, grads[0].dtype if len(grads) else None
    for dtype, name in ((p_dtype, "params"), (g_dtype, "grads")):
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    if scale is not None and not scale > 0:
        raise ValueError("scale must be above zero")
    lists = [("param", params, p_dtype), ("grad", grads, g_dtype), ("momentum", momenta, torch.float32)]
    if copies is not None:
        lists.append(("copy", copies, torch.bfloat16))
    t = np.zeros(n, [*_MUON_TENSOR.descr, ("n", np.int64)])
    for i, (key, tensors, dtype) in enumerate(lists):
        _gather(t, key, tensors, dtype, device, per=1 if i else 0)
    for i, p in enumerate(params):
        if p.dim() < 2 or any(other[i].shape != p.shape for _, other, _ in lists[1:]):
            raise ValueError(f"tensor {i}: params, grads, momenta and copies must have one shape [..., rows, cols]")
        rows, cols = p.shape[-2:]
        t[i]["rows"], t[i]["cols"] = rows, cols
        t[i]["batch"] = p.numel() // (rows * cols) if rows and cols else 0
    table = np.empty(n, _MUON_TENSOR)
    for key in _MUON_TENSOR.names:
        table[key] = t[key]
    cfg = _MuonConfig(lr=lr, momentum=momentum, weight_decay=weight_decay, scale=scale or 0.0, eps=eps, a=coefficients[0],
                      b=coefficients[1], c=coefficients[2], steps=steps)
    cfg.flags = (EP_MUON_PARAM_BF16 if p_dtype == torch.bfloat16 else 0) | \
        (EP_MUON_GRAD_BF16 if g_dtype == torch.bfloat16 else 0) | (EP_MUON_NESTEROV if nesterov else 0)
    with torch.cuda.device(device):
        workspace = _muon_workspace(table, workspace, stream, device)
        _check(_lib.ep_muon(table.ctypes.data_as(ctypes.c_void_p), n, ctypes.byref(cfg), _ptr(workspace), workspace.numel(),
                            _stream(stream)), "ep_muon")


# ------------------------------------------------------------- convenience --

class FfnSaved(NamedTuple):
    """What expert_ffn(save=True) keeps for expert_ffn_backward."""
    act: torch.Tensor           # bf16 [capacity_rows, inter]
    gate_up: torch.Tensor       # fp32 [capacity_rows, 2 * inter]


class EpHandle:
    """One layout's metadata on the current device (owns an ep_handle)."""

    def __init__(self, max_tokens: int, top_k: int, num_experts: int, block_m: int):
        self.max_tokens, self.top_k = int(max_tokens), int(top_k)
        self.num_experts, self.block_m = int(num_experts), int(block_m)
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._h = ep_handle_create(max_tokens, top_k, num_experts, block_m)
        self.capacity_rows = int(_lib.ep_pool_capacity_rows(self._h))
        self.max_tiles = int(_lib.ep_max_tiles(self._h))
        self.scale_ld = int(_lib.ep_scale_ld(self._h))

    @property
    def raw(self):
        return self._h

    @property
    def num_tokens(self) -> int:
        return int(_lib.ep_num_tokens(self._h))

    def close(self):
        if self._h is not None and self._h.value:
            ep_handle_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def layout(self, topk_idx: torch.Tensor, topk_weights: torch.Tensor, stream=None) -> int:
        _require(topk_idx, torch.int32, "topk_idx", self.device)
        _require(topk_weights, torch.float32, "topk_weights", self.device)
        if topk_idx.dim() != 2 or topk_idx.shape[1] != self.top_k or topk_weights.shape != topk_idx.shape:
            raise ValueError("topk_idx / topk_weights must both be [num_tokens, top_k]")
        return ep_layout(self._h, topk_idx, topk_weights, stream)

    def scale_shape(self, hidden: int, kind: str = "ue8m0", mn_major: bool = False):
        return scale_shape(self.capacity_rows, hidden, kind, mn_major, self.scale_ld)

    def new_pool(self, hidden: int, fp8: bool = False, scale_kind: str = "ue8m0",
                 mn_major: bool = False) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        if fp8:
            shape, dtype = self.scale_shape(hidden, scale_kind, mn_major)
            return (torch.empty(self.capacity_rows, hidden, dtype=torch.uint8, device=self.device),
                    torch.empty(shape, dtype=dtype, device=self.device))
        return torch.empty(self.capacity_rows, hidden, dtype=torch.bfloat16, device=self.device), None

    def dispatch(self, x: torch.Tensor, pool: torch.Tensor, pool_scales: Optional[torch.Tensor] = None,
                 fp8: bool = False, tile_ready: bool = False, stream=None,
                 scale_kind: str = "ue8m0", mn_major: bool = False) -> int:
        _require(x, torch.bfloat16, "x", self.device)
        if x.dim() != 2 or x.shape[0] != self.num_tokens:
            raise ValueError("x must be [num_tokens of the layout, hidden]")
        H = x.shape[1]
        if pool.shape[0] < self.capacity_rows or pool.shape[1] != H:
            raise ValueError(f"pool must be at least [{self.capacity_rows}, {H}]")
        _require(pool, torch.uint8 if fp8 else torch.bfloat16, "pool", self.device)
        if fp8:
            shape, dtype = self.scale_shape(H, scale_kind, mn_major)
            if pool_scales is None or tuple(pool_scales.shape) != shape:
                raise ValueError(f"pool_scales must be {shape}")
            _require(pool_scales, dtype, "pool_scales", self.device)
        elif scale_kind != "ue8m0" or mn_major:
            raise ValueError("scale flavours apply to FP8 dispatch only")
        flags = (EP_DISPATCH_FP8 | scale_flags(scale_kind, mn_major) if fp8 else 0) | \
                (EP_DISPATCH_TILE_READY if tile_ready else 0)
        return ep_dispatch(self._h, x, pool, pool_scales if fp8 else None, flags, stream)

    def layout_dispatch(self, topk_idx: torch.Tensor, topk_weights: torch.Tensor, x: torch.Tensor,
                        pool: torch.Tensor, pool_scales: Optional[torch.Tensor] = None, fp8: bool = False,
                        stream=None, scale_kind: str = "ue8m0", mn_major: bool = False) -> tuple:
        """layout() and dispatch() in one call (one kernel launch for batches
        of at most 2048 slots); returns (epoch, dispatch sequence number)."""
        _require(topk_idx, torch.int32, "topk_idx", self.device)
        _require(topk_weights, torch.float32, "topk_weights", self.device)
        if topk_idx.dim() != 2 or topk_idx.shape[1] != self.top_k or topk_weights.shape != topk_idx.shape:
            raise ValueError("topk_idx / topk_weights must both be [num_tokens, top_k]")
        _require(x, torch.bfloat16, "x", self.device)
        if x.dim() != 2 or x.shape[0] != topk_idx.shape[0]:
            raise ValueError("x must be [num_tokens, hidden]")
        H = x.shape[1]
        if pool.shape[0] < self.capacity_rows or pool.shape[1] != H:
            raise ValueError(f"pool must be at least [{self.capacity_rows}, {H}]")
        _require(pool, torch.uint8 if fp8 else torch.bfloat16, "pool", self.device)
        if fp8:
            shape, dtype = self.scale_shape(H, scale_kind, mn_major)
            if pool_scales is None or tuple(pool_scales.shape) != shape:
                raise ValueError(f"pool_scales must be {shape}")
            _require(pool_scales, dtype, "pool_scales", self.device)
        elif scale_kind != "ue8m0" or mn_major:
            raise ValueError("scale flavours apply to FP8 dispatch only")
        flags = EP_DISPATCH_FP8 | scale_flags(scale_kind, mn_major) if fp8 else 0
        return ep_layout_dispatch(self._h, topk_idx, topk_weights, x, pool, pool_scales if fp8 else None,
                                  flags, stream)

    def combine_backward(self, epoch: int, grad_y: torch.Tensor, expert_out: torch.Tensor,
                         grad_expert_out: Optional[torch.Tensor] = None, stream=None):
        """Returns (grad_expert_out [capacity_rows, H] bf16, grad_weights [T, K] fp32)."""
        _require(grad_y, torch.bfloat16, "grad_y", self.device)
        _require(expert_out, torch.bfloat16, "expert_out", self.device)
        H = grad_y.shape[1]
        if grad_y.shape[0] != self.num_tokens or expert_out.shape[0] < self.capacity_rows \
                or expert_out.shape[1] != H:
            raise ValueError("grad_y must be [num_tokens, H], expert_out [capacity_rows, H]")
        if grad_expert_out is None:
            grad_expert_out = _empty(stream, (self.capacity_rows, H), torch.bfloat16, self.device)
        _require(grad_expert_out, torch.bfloat16, "grad_expert_out", self.device)
        if grad_expert_out.shape[0] < self.capacity_rows or grad_expert_out.shape[1] != H:
            raise ValueError("grad_expert_out must be at least [capacity_rows, H]")
        grad_w = _empty(stream, (self.num_tokens, self.top_k), torch.float32, self.device)
        ep_combine_backward(self._h, epoch, grad_y, expert_out, grad_expert_out, grad_w, stream)
        _used_on(stream, grad_expert_out, grad_w)
        return grad_expert_out, grad_w

    def dispatch_backward(self, epoch: int, grad_pool: torch.Tensor,
                          grad_x: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        _require(grad_pool, torch.bfloat16, "grad_pool", self.device)
        H = grad_pool.shape[1]
        if grad_pool.shape[0] < self.capacity_rows:
            raise ValueError("grad_pool must have at least capacity_rows rows")
        if grad_x is None:
            grad_x = _empty(stream, (self.num_tokens, H), torch.bfloat16, self.device)
        _require(grad_x, torch.bfloat16, "grad_x", self.device)
        if grad_x.shape != (self.num_tokens, H):
            raise ValueError("grad_x must be [num_tokens, H]")
        ep_dispatch_backward(self._h, epoch, grad_pool, grad_x, stream)
        _used_on(stream, grad_x)
        return grad_x

    def _check_rows(self, t: torch.Tensor, width: int, dtype, name: str) -> None:
        _require(t, dtype, name, self.device)
        if t.dim() != 2 or t.shape[0] < self.capacity_rows or t.shape[1] != width:
            raise ValueError(f"{name} must be at least [{self.capacity_rows}, {width}]")

    def _check_experts(self, pool: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                       activation: str) -> Tuple[int, int]:
        """(hidden, inter) of a feed-forward's operands."""
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        _require(w_gate_up, torch.bfloat16, "w_gate_up", self.device)
        _require(w_down, torch.bfloat16, "w_down", self.device)
        E = self.num_experts
        if w_down.dim() != 3 or w_down.shape[0] != E:
            raise ValueError(f"w_down must be [{E}, hidden, inter]")
        H, I = int(w_down.shape[1]), int(w_down.shape[2])
        if tuple(w_gate_up.shape) != (E, 2 * I, H):
            raise ValueError(f"w_gate_up must be [{E}, {2 * I}, {H}]")
        self._check_rows(pool, H, torch.bfloat16, "pool")
        return H, I

    def expert_ffn(self, epoch: int, pool: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                   activation: str = "silu", out: Optional[torch.Tensor] = None,
                   act: Optional[torch.Tensor] = None, gate_up: Optional[torch.Tensor] = None,
                   save: bool = False, stream=None):
        """The experts' gated feed-forward over the dispatched pool:
        out = (act(x Wg^T) * (x Wu^T)) Wd^T per real row, bf16
        [capacity_rows, hidden], combine()'s expert_out.

        w_gate_up is [num_experts, 2 * inter, hidden] (gate rows, then up rows),
        w_down [num_experts, hidden, inter], both bf16.  With save=True returns
        (out, FfnSaved) for expert_ffn_backward; act and gate_up are the buffers
        to use for it (made when not given; act also without save, as the
        call's workspace).  out may be the pool itself without save only: the
        backward pass reads the pool."""
        H, I = self._check_experts(pool, w_gate_up, w_down, activation)
        cap = self.capacity_rows
        if gate_up is not None and not save:
            raise ValueError("gate_up is written with save=True only")
        workspace = act is None and not save
        if out is None:
            out = _empty(stream, (cap, H), torch.bfloat16, self.device)
        if act is None:
            act = _empty(stream, (cap, I), torch.bfloat16, self.device)
        if save and gate_up is None:
            gate_up = _empty(stream, (cap, 2 * I), torch.float32, self.device)
        self._check_rows(out, H, torch.bfloat16, "out")
        self._check_rows(act, I, torch.bfloat16, "act")
        if save:
            self._check_rows(gate_up, 2 * I, torch.float32, "gate_up")
        ep_expert_ffn(self._h, epoch, pool, w_gate_up, w_down, ACTIVATIONS[activation], act, gate_up, out, stream)
        _used_on(stream, out, None if workspace else act, gate_up)
        return (out, FfnSaved(act, gate_up)) if save else out

    def expert_ffn_backward(self, epoch: int, grad_out: torch.Tensor, pool: torch.Tensor,
                            w_gate_up: torch.Tensor, w_down: torch.Tensor, saved: FfnSaved,
                            activation: str = "silu", grad_pool: Optional[torch.Tensor] = None,
                            grad_w_gate_up: Optional[torch.Tensor] = None,
                            grad_w_down: Optional[torch.Tensor] = None, accumulate: bool = False,
                            grad_gate_up: Optional[torch.Tensor] = None, stream=None):
        """Backward of expert_ffn: returns (grad_pool, grad_w_gate_up,
        grad_w_down) for grad_out, combine_backward()'s grad_expert_out.

        The weight gradients are bf16 or float32, as the buffers given (bf16
        when none is); accumulate=True adds to float32 buffers.  grad_gate_up
        is the workspace, bf16 [capacity_rows, 2 * inter] (made when not given)."""
        H, I = self._check_experts(pool, w_gate_up, w_down, activation)
        E = self.num_experts
        self._check_rows(grad_out, H, torch.bfloat16, "grad_out")
        self._check_rows(saved.act, I, torch.bfloat16, "saved.act")
        self._check_rows(saved.gate_up, 2 * I, torch.float32, "saved.gate_up")
        given = [g for g in (grad_w_gate_up, grad_w_down) if g is not None]
        dtype = given[0].dtype if given else torch.bfloat16
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"weight gradients must be bfloat16 or float32, got {dtype}")
        if accumulate and (len(given) < 2 or dtype != torch.float32):
            raise ValueError("accumulate needs both weight gradients, in float32")
        workspace = grad_gate_up is None
        if grad_pool is None:
            grad_pool = _empty(stream, (self.capacity_rows, H), torch.bfloat16, self.device)
        if grad_w_gate_up is None:
            grad_w_gate_up = _empty(stream, (E, 2 * I, H), dtype, self.device)
        if grad_w_down is None:
            grad_w_down = _empty(stream, (E, H, I), dtype, self.device)
        if grad_gate_up is None:
            grad_gate_up = _empty(stream, (self.capacity_rows, 2 * I), torch.bfloat16, self.device)
        self._check_rows(grad_pool, H, torch.bfloat16, "grad_pool")
        self._check_rows(grad_gate_up, 2 * I, torch.bfloat16, "grad_gate_up")
        for g, shape, name in ((grad_w_gate_up, (E, 2 * I, H), "grad_w_gate_up"),
                               (grad_w_down, (E, H, I), "grad_w_down")):
            _require(g, dtype, name, self.device)
            if tuple(g.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}")
        flags = (EP_GRAD_F32 if dtype == torch.float32 else 0) | (EP_GRAD_ACCUMULATE if accumulate else 0)
        ep_expert_ffn_backward(self._h, epoch, grad_out, pool, w_gate_up, w_down, ACTIVATIONS[activation],
                               saved.act, saved.gate_up, flags, grad_gate_up, grad_pool, grad_w_gate_up,
                               grad_w_down, stream)
        _used_on(stream, grad_pool, None if workspace else grad_gate_up, grad_w_gate_up, grad_w_down)
        return grad_pool, grad_w_gate_up, grad_w_down

    def borrow(self, x: torch.Tensor, stream=None) -> int:
        """Dispatch without a copy: lend x through the row map
        (pool_recv_token).  Holds the handle's lease until release()."""
        _require(x, torch.bfloat16, "x", self.device)
        if x.dim() != 2 or x.shape[0] != self.num_tokens:
            raise ValueError("x must be [num_tokens of the layout, hidden]")
        return ep_dispatch(self._h, x, None, None, EP_DISPATCH_BORROW, stream)

    def release(self, consumer_stream=None) -> None:
        ep_borrow_release(self._h, consumer_stream)

    def combine(self, epoch: int, expert_out: torch.Tensor, y: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        _require(expert_out, torch.bfloat16, "expert_out", self.device)
        H = expert_out.shape[1]
        if expert_out.shape[0] < self.capacity_rows:
            raise ValueError(f"expert_out must have at least {self.capacity_rows} rows")
        if y is None:
            y = _empty(stream, (max(self.num_tokens, 0), H), torch.bfloat16, self.device)
        _require(y, torch.bfloat16, "y", self.device)
        if y.shape != (self.num_tokens, H):
            raise ValueError("y must be [num_tokens of the layout, hidden]")
        ep_combine(self._h, epoch, expert_out, y, stream)
        _used_on(stream, y)
        return y

    def combine_gated(self, epoch: int, expert_out: torch.Tensor, round: int = 1,
                      y: Optional[torch.Tensor] = None, spin_limit_us: int = 2_000_000,
                      stream=None) -> torch.Tensor:
        """combine behind the per-token gate: token t waits until
        y_done_per_token[t] >= round * (its unmasked slots)."""
        _require(expert_out, torch.bfloat16, "expert_out", self.device)
        H = expert_out.shape[1]
        if expert_out.shape[0] < self.capacity_rows:
            raise ValueError(f"expert_out must have at least {self.capacity_rows} rows")
        if y is None:
            y = _empty(stream, (max(self.num_tokens, 0), H), torch.bfloat16, self.device)
        _require(y, torch.bfloat16, "y", self.device)
        if y.shape != (self.num_tokens, H):
            raise ValueError("y must be [num_tokens of the layout, hidden]")
        ep_combine_gated(self._h, epoch, expert_out, y, round, spin_limit_us, stream)
        _used_on(stream, y)
        return y

    def tile_consume(self, seq: int, pool: torch.Tensor, pool_scales: Optional[torch.Tensor],
                     hidden: int, out: torch.Tensor, fp8: bool = False, workgroups: int = 32,
                     spin_limit_us: int = 2_000_000, stream=None, gather: bool = False,
                     signal_done: bool = False, scale_kind: str = "ue8m0",
                     mn_major: bool = False, stamps: bool = False) -> None:
        _require(out, torch.bfloat16, "out", self.device)
        if out.shape[0] < self.capacity_rows or out.shape[1] != hidden:
            raise ValueError("out must be at least [capacity_rows, hidden]")
        if gather:
            # pool is the borrowed slab x [num_tokens, hidden]
            _require(pool, torch.bfloat16, "slab", self.device)
            if pool.shape != (self.num_tokens, hidden):
                raise ValueError("the gathered slab must be [num_tokens, hidden]")
        elif pool.shape[0] < self.capacity_rows:
            raise ValueError("pool must have at least capacity_rows rows")
        if not fp8 and (scale_kind != "ue8m0" or mn_major):
            raise ValueError("scale flavours apply to FP8 pools only")
        flags = (EP_DISPATCH_FP8 | scale_flags(scale_kind, mn_major) if fp8 else 0) | \
                (EP_CONSUME_GATHER if gather else 0) | (EP_CONSUME_SIGNAL_DONE if signal_done else 0) | \
                (EP_CONSUME_STAMPS if stamps else 0)
        ep_tile_consume(self._h, seq, pool, pool_scales if fp8 else None, hidden, flags, out,
                        workgroups, spin_limit_us, stream)

    def array(self, name: str, stream=None) -> torch.Tensor:
        """Device copy of one metadata array (see ARRAYS)."""
        which, dtype = ARRAYS[name]
        nbytes = int(_lib.ep_array_bytes(self._h, which))
        out = _empty(stream, (nbytes // dtype.itemsize,), dtype, self.device)
        _check(_lib.ep_copy_array(self._h, which, _ptr(out), nbytes, _stream(stream)), "ep_copy_array")
        _used_on(stream, out)
        return out

    def counts_to_host(self, stream=None) -> Tuple[np.ndarray, int]:
        counts = np.empty(self.num_experts, np.int32)
        nt = np.zeros(1, np.int32)
        _check(_lib.ep_counts_to_host(self._h, counts.ctypes.data_as(ctypes.c_void_p),
                                      nt.ctypes.data_as(ctypes.c_void_p), _stream(stream)),
               "ep_counts_to_host")
        return counts, int(nt[0])

    def set_density_hint(self, hint: int) -> None:
        """EP_DENSITY_AUTO / _SPARSE / _DENSE: launch shape of the combine calls (forward
        and both backward calls) and of the bf16 dispatch of at least 64 MiB of x."""
        _check(_lib.ep_set_density_hint(self._h, int(hint)), "ep_set_density_hint")

    def layout_density(self, stream=None) -> int:
        """The density the current layout reported (EP_DENSITY_SPARSE / _DENSE)."""
        return int(_lib.ep_layout_density(self._h, _stream(stream)))

    def sync_status(self, stream=None) -> int:
        return ep_handle_sync_status(self._h, stream)
