"""Python binding of the MI355X fused MoE forward library (libmoe_hip.so).

Argument marshalling only: tensors are checked (device, dtype, shape,
contiguity), their device pointers and torch's current HIP stream are passed
to the C ABI declared in include/moe.h, and a non-OK status is raised as
RuntimeError. Every computation runs in the library's HIP kernels; torch
provides device memory and the stream. Calls are asynchronous on the current
stream, exactly like the C entry points.

If the library has not been built, every call raises RuntimeError; there is
no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

import torch

__all__ = [
    "MOE_DTYPE_F32", "MOE_DTYPE_BF16", "GATE_UP_SWIGLU", "DOWN", "NUM_EVENTS",
    "lib", "library_path", "status_str",
    "route", "slot_map", "permute", "permute_noalloc", "permute_workspace_size",
    "grouped_gemm", "combine",
    "forward", "forward_workspace_size", "ForwardConfig",
    "a2a_dispatch", "a2a_dispatch_workspace_size", "a2a_combine",
    "rms_norm", "balance_loss", "balance_loss_workspace_size", "route_backward",
    "MXFP4", "quantize_mxfp4", "dequantize_mxfp4", "grouped_gemm_mxfp4",
    "layer_norm", "layer_norm_backward", "rms_norm_backward", "norm_backward_workspace_size",
    "combine_backward", "permute_backward", "swiglu", "grouped_gemm_backward",
    "grouped_gemm_weight_grad", "grouped_gemm_weight_grad_workspace_size",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_HIP_LIBRARY selects another build of the same library (the tests use it
# for a host-sanitized build); it must exist like the default one.
_LIB_FILE = os.environ.get("MOE_HIP_LIBRARY") or os.path.join(_HERE, "libmoe_hip.so")

MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_FP8_E4M3 = 2
MOE_DTYPE_MXFP4 = 3
GATE_UP_SWIGLU = 0
DOWN = 1
NUM_EVENTS = 6
MAX_EXPERTS = 1024
MAX_TOPK = 32
MAX_SLOTS = 1024

# ForwardConfig dtype of the 4-bit expert path (a name for it where torch has no such type)
MXFP4 = getattr(torch, "float4_e2m1fn_x2", "float4_e2m1fn_x2")
_DT = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16,
       torch.float8_e4m3fn: MOE_DTYPE_FP8_E4M3, MXFP4: MOE_DTYPE_MXFP4}
MX_GROUP = 32  # weights that share one scale byte
FP8 = torch.float8_e4m3fn  # ForwardConfig dtype of the FP8 expert path
_CODES = (torch.uint8, torch.float8_e4m3fn)  # tensors holding E4M3 codes
_TORCH_DT = {MOE_DTYPE_F32: torch.float32, MOE_DTYPE_BF16: torch.bfloat16}

_p = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t


class _Config(ctypes.Structure):
    _fields_ = [("T_max", _i), ("T", _i), ("H", _i), ("I", _i), ("E_global", _i), ("K", _i),
                ("renormalize", _i), ("ep_size", _i), ("ep_rank", _i), ("S", _i),
                ("dtype", _i), ("out_dtype", _i), ("accumulate", _i),
                ("num_expert_group", _i), ("topk_group", _i), ("routing_on_input", _i),
                ("a1_scale", ctypes.c_float), ("a2_scale", ctypes.c_float),
                ("gemm_blocks", _i), ("x_codes", _i)]


class _ForwardArgs(ctypes.Structure):
    _fields_ = [("x", _p), ("logits", _p), ("topk_ids", _p), ("topk_w", _p),
                ("w_gate_up", _p), ("w_down", _p), ("rep_off", _p), ("rep_slots", _p),
                ("out", _p), ("events", _p * NUM_EVENTS), ("shared_out", _p),
                ("w_gate_up_scale", _p), ("w_down_scale", _p),
                ("w_gate_up_e8m0", _p), ("w_down_e8m0", _p)]


_SIGS = {
    "moe_status_str": (ctypes.c_char_p, [_i]),
    "moe_route": (_i, [_p, _i, _i, _i, _i, _p, _p, _p]),
    "moe_route_grouped": (_i, [_p, _i, _i, _i, _i, _i, _i, _p, _p, _p]),
    "moe_slot_map": (_i, [_p, _p, _i, _i, _i, _i, _i, _p, _p, _i, _p, _p, _p, _p]),
    "moe_permute_workspace_size": (_sz, [_i, _i, _i]),
    "moe_permute": (_i, [_p, _i, _i, _i, _i, _p, _p, _i, _p, _p, _p, _p, _p, _sz, _p]),
    "moe_permute_scaled": (_i, [_p, _i, _i, _i, _i, _p, _p, _i, _p, _p, _p, _p, _p, _p, _sz,
                                _p]),
    "moe_permute_noalloc": (_i, [_p, _i, _i, _i, _i, _p, _p, _i, _p, _p, _p, _p, _p]),
    "moe_grouped_gemm": (_i, [_i, _i, _p, _p, _i, _i, _p, _i, _i, _p, _p]),
    "moe_combine": (_i, [_p, _i, _p, _p, _i, _i, _i, _p, _i, _i, _p]),
    "moe_combine_shared": (_i, [_p, _i, _p, _p, _i, _i, _i, _p, _i, _p, _i, _i, _p]),
    "moe_forward_workspace_size": (_sz, [ctypes.POINTER(_Config)]),
    "moe_forward": (_i, [ctypes.POINTER(_Config), ctypes.POINTER(_ForwardArgs), _p, _sz, _p]),
    "moe_a2a_dispatch_workspace_size": (_sz, [_i, _i, _i]),
    "moe_a2a_dispatch": (_i, [_p, _i, _i, _i, _i, _p, _p, _i, _i, _i, _p, _p, _p, _p, _p, _p,
                              _p, _sz, _p]),
    "moe_a2a_combine": (_i, [_p, _i, _p, _i, _i, _i, _p, _i, _p]),
    "moe_quantize_fp8": (_i, [_p, _i, ctypes.c_int64, ctypes.c_float, _p, _p]),
    "moe_grouped_gemm_fp8": (_i, [_i, _p, ctypes.c_float, _p, _i, _i, _p, _p, _i, _i, _p,
                                  ctypes.c_float, _p]),
    "moe_quantize_mxfp4": (_i, [_p, _i, ctypes.c_int64, _p, _p, _p]),
    "moe_dequantize_mxfp4": (_i, [_p, _p, ctypes.c_int64, _p, _i, _p]),
    "moe_grouped_gemm_mxfp4": (_i, [_i, _p, _p, _i, _i, _p, _p, _i, _i, _p, _i, _p]),
    "moe_rms_norm": (_i, [_p, _p, _p, _i, _i, _i, ctypes.c_float, _p, _p, _p, ctypes.c_float, _p]),
    "moe_balance_loss_workspace_size": (_sz, [_i, _i, _i]),
    "moe_balance_loss": (_i, [_p, _p, _p, _i, _i, _i, ctypes.c_float, _p, _p, _p, _p, _sz, _p]),
    "moe_layer_norm": (_i, [_p, _p, _p, _p, _i, _i, _i, ctypes.c_float, _p, _p, _p,
                            ctypes.c_float, _p]),
    "moe_norm_backward_workspace_size": (_sz, [_i, _i]),
    "moe_rms_norm_backward": (_i, [_p, _p, _p, _p, _i, _i, _i, ctypes.c_float, _p, _p, _p, _sz,
                                   _p]),
    "moe_layer_norm_backward": (_i, [_p, _p, _p, _p, _i, _i, _i, ctypes.c_float, _p, _p, _p, _p,
                                     _sz, _p]),
    "moe_combine_backward": (_i, [_p, _i, _p, _i, _p, _p, _i, _i, _i, _p, _p, _p]),
    "moe_permute_backward": (_i, [_p, _i, _p, _p, _p, _i, _i, _i, _p, _i, _i, _p, _p]),
    "moe_swiglu": (_i, [_p, _i, _p, _i, _i, _i, _p, _p]),
    "moe_grouped_gemm_backward": (_i, [_i, _i, _p, _p, _i, _i, _p, _i, _i, _p, _p, _p]),
    "moe_grouped_gemm_weight_grad_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "moe_grouped_gemm_weight_grad": (_i, [_i, _p, _p, _p, _i, _i, _i, _i, _p, _i, _i, _p, _sz,
                                          _p]),
    "moe_route_backward": (_i, [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, ctypes.c_float, _p, _p]),
}
EXPORTED_SYMBOLS = tuple(_SIGS)

_lib = None


def library_path() -> str:
    return _LIB_FILE


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_FILE):
            raise RuntimeError(
                f"{_LIB_FILE} is missing: build it with `python -m moe_expert_dispatch_amd.build`; "
                "there is no non-HIP fallback")
        so = ctypes.CDLL(_LIB_FILE)
        for name, (res, args) in _SIGS.items():
            fn = getattr(so, name)
            fn.restype = res
            fn.argtypes = args
        _lib = so
    return _lib


def status_str(code: int) -> str:
    return lib().moe_status_str(code).decode()


def _check(code: int, what: str) -> None:
    if code != 0:
        raise RuntimeError(f"{what}: {status_str(code)}")


# The current stream's handle by device index: torch.cuda.current_stream() builds an object for
# it, which took longer than a small kernel runs (about 2 us of a 12 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        ok = dtype if isinstance(dtype, tuple) else (dtype,)
        if t.dtype not in ok:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {ok}")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


_WIDE = 1 << 31


def _fits(what: str, *sizes: int) -> None:
    """Sizes that an int of the C ABI holds: ctypes keeps the low 32 bits of a larger one."""
    most = max(sizes, default=0)
    if most >= _WIDE:
        raise ValueError(f"{what}: a size of {most} does not fit 32 bits")


def _size(what: str, *sizes: int) -> int:
    """A workspace size."""
    if max(sizes) >= _WIDE:
        _fits(what, *sizes)
    return getattr(_lib or lib(), what)(*sizes)


def _empty(shape, dtype, like: torch.Tensor) -> torch.Tensor:
    return like.new_empty(shape, dtype=dtype)


def _launch(what: str, like: torch.Tensor, others: Sequence[Optional[torch.Tensor]], *args) -> None:
    """Calls entry point `what` with args and the current stream of like's device, which is made
    the current device for the call; the other tensors have to be on it too. Rows that 32 bits do
    not hold are like's (sizes that are not the callers look at)."""
    if like.numel() >= _WIDE:
        _fits(what, *(a for a, kind in zip(args, _SIGS[what][1]) if kind is _i))
    dev = like.get_device()
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError(f"tensors on {like.device} and {o.device}: one device is needed")
    fn = getattr(_lib or lib(), what)
    if _current_device() == dev:
        code = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _raw_stream(dev))
    if code != 0:
        _check(code, what)


# ---------------------------------------------------------------- stages
def route(logits: torch.Tensor, K: int, renormalize: bool,
          ids: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
          num_groups: int = 0, topk_groups: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """moe_route (or moe_route_grouped when num_groups > 0):
    logits [T, E] f32 -> (ids [T, K] int32, w [T, K] f32)."""
    _dev(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    ids = _empty((T, K), torch.int32, logits) if ids is None else _dev(ids, "ids", torch.int32, (T, K))
    w = _empty((T, K), torch.float32, logits) if w is None else _dev(w, "w", torch.float32, (T, K))
    if num_groups:
        _launch("moe_route_grouped", logits, (ids, w), _ptr(logits), T, E, K,
                int(bool(renormalize)), num_groups, topk_groups, _ptr(ids), _ptr(w))
    else:
        _launch("moe_route", logits, (ids, w), _ptr(logits), T, E, K, int(bool(renormalize)),
                _ptr(ids), _ptr(w))
    return ids, w


def slot_map(ids: torch.Tensor, w: torch.Tensor, E_global: int, ep_size: int = 1,
             ep_rank: int = 0, rep_off: Optional[torch.Tensor] = None,
             rep_slots: Optional[torch.Tensor] = None, S: Optional[int] = None
             ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """moe_slot_map -> (slot [T,K] int32, w_masked [T,K] f32, mask [T,K] uint8)."""
    _dev(ids, "ids", torch.int32)
    if ids.dim() != 2:
        raise ValueError("ids must be [T, K]")
    T, K = ids.shape
    _dev(w, "w", torch.float32, (T, K))
    if rep_off is not None:
        _dev(rep_off, "rep_off", torch.int32)
        _dev(rep_slots, "rep_slots", torch.int32)
        S = rep_slots.numel() if S is None else S
    elif S is None:
        S = E_global // max(ep_size, 1)
    slot = _empty((T, K), torch.int32, ids)
    wm = _empty((T, K), torch.float32, ids)
    mask = _empty((T, K), torch.uint8, ids)
    _launch("moe_slot_map", ids, (w, rep_off, rep_slots), _ptr(ids), _ptr(w), T, K, E_global,
            ep_size, ep_rank, _ptr(rep_off), _ptr(rep_slots), S, _ptr(slot), _ptr(wm), _ptr(mask))
    return slot, wm, mask


def permute_workspace_size(T: int, K: int, S: int) -> int:
    return _size("moe_permute_workspace_size", T, K, S)


def permute(x: torch.Tensor, slot: torch.Tensor, mask: torch.Tensor, S: int,
            gather: bool = True, ws: Optional[torch.Tensor] = None,
            pair_w: Optional[torch.Tensor] = None):
    """moe_permute -> (offsets [S+1], sorted_pairs [T*K], pair_row [T*K], x_perm [T*K, H] or None).

    Only rows [0, offsets[S]) of x_perm and sorted_pairs are written. With
    pair_w [T, K] f32 (moe_permute_scaled) each row is pair_w[p] * x[p / K]."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    _dev(slot, "slot", torch.int32)
    T, K = slot.shape
    _dev(mask, "mask", torch.uint8, (T, K))
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T matching slot")
    H = x.shape[1]
    offsets = _empty((S + 1,), torch.int32, x)
    sorted_pairs = _empty((T * K,), torch.int32, x)
    pair_row = _empty((T * K,), torch.int32, x)
    x_perm = _empty((T * K, H), x.dtype, x) if gather else None
    need = permute_workspace_size(T, K, S)
    ws = _empty((max(need, 1),), torch.uint8, x) if ws is None else _dev(ws, "ws")
    if pair_w is not None:
        _dev(pair_w, "pair_w", torch.float32, (T, K))
        if x_perm is None:
            raise ValueError("pair_w needs the row gather")
        _launch("moe_permute_scaled", x, (slot, mask, pair_w, ws), _ptr(x), _DT[x.dtype], T, H, K,
                _ptr(slot), _ptr(mask), S, _ptr(pair_w), _ptr(offsets), _ptr(sorted_pairs),
                _ptr(pair_row), _ptr(x_perm), _ptr(ws), ws.numel() * ws.element_size())
    else:
        _launch("moe_permute", x, (slot, mask, ws), _ptr(x), _DT[x.dtype], T, H, K, _ptr(slot),
                _ptr(mask), S, _ptr(offsets), _ptr(sorted_pairs), _ptr(pair_row), _ptr(x_perm),
                _ptr(ws), ws.numel() * ws.element_size())
    return offsets, sorted_pairs, pair_row, x_perm


def permute_noalloc(x: torch.Tensor, slot: torch.Tensor, mask: torch.Tensor, S: int,
                    gather: bool = True, out=None):
    """moe_permute_noalloc: moe_permute with the library's static histogram
    memory (no workspace). `out` may pass preallocated (offsets, sorted_pairs,
    pair_row, x_perm) so that the call itself allocates nothing."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    _dev(slot, "slot", torch.int32)
    T, K = slot.shape
    _dev(mask, "mask", torch.uint8, (T, K))
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T matching slot")
    H = x.shape[1]
    if out is None:
        out = (_empty((S + 1,), torch.int32, x), _empty((T * K,), torch.int32, x),
               _empty((T * K,), torch.int32, x),
               _empty((T * K, H), x.dtype, x) if gather else None)
    offsets, sorted_pairs, pair_row, x_perm = out
    _dev(offsets, "offsets", torch.int32, (S + 1,))
    _dev(sorted_pairs, "sorted_pairs", torch.int32, (T * K,))
    _dev(pair_row, "pair_row", torch.int32, (T * K,))
    if x_perm is not None:
        _dev(x_perm, "x_perm", x.dtype, (T * K, H))
    _launch("moe_permute_noalloc", x, (slot, mask, offsets, sorted_pairs, pair_row, x_perm),
            _ptr(x), _DT[x.dtype], T, H, K, _ptr(slot), _ptr(mask), S, _ptr(offsets),
            _ptr(sorted_pairs), _ptr(pair_row), _ptr(x_perm))
    return offsets, sorted_pairs, pair_row, x_perm


def grouped_gemm(op: int, a: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor,
                 c: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_gemm. op GATE_UP_SWIGLU: a [rows, H], w [S, 2I, H] -> c [rows, I];
    op DOWN: a [rows, I], w [S, H, I] -> c [rows, H]."""
    _dev(a, "a", (torch.float32, torch.bfloat16))
    _dev(w, "w", a.dtype)
    _dev(offsets, "offsets", torch.int32)
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError("a must be 2-D and w 3-D")
    S = w.shape[0]
    if offsets.numel() != S + 1:
        raise ValueError("offsets must have S + 1 entries")
    rows = a.shape[0]
    if op == GATE_UP_SWIGLU:
        H = a.shape[1]
        I = w.shape[1] // 2
        if w.shape[2] != H or w.shape[1] != 2 * I:
            raise ValueError("w must be [S, 2I, H]")
        N = I
    elif op == DOWN:
        I = a.shape[1]
        H = w.shape[1]
        if w.shape[2] != I:
            raise ValueError("w must be [S, H, I]")
        N = H
    else:
        raise ValueError("op must be GATE_UP_SWIGLU or DOWN")
    c = _empty((rows, N), a.dtype, a) if c is None else _dev(c, "c", a.dtype, (rows, N))
    _launch("moe_grouped_gemm", a, (offsets, w, c), op, _DT[a.dtype], _ptr(a), _ptr(offsets), S,
            rows, _ptr(w), H, I, _ptr(c))
    return c


def quantize_fp8(x: torch.Tensor, scale: float, q: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_quantize_fp8: E4M3 codes (uint8, shape of x) of x (bf16 or f32) / scale."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    q = _empty(tuple(x.shape), torch.uint8, x) if q is None else _dev(q, "q", _CODES, x.shape)
    _launch("moe_quantize_fp8", x, (q,), _ptr(x), _DT[x.dtype], x.numel(), float(scale), _ptr(q))
    return q


def grouped_gemm_fp8(op: int, a: torch.Tensor, a_scale: float, offsets: torch.Tensor,
                     w: torch.Tensor, w_scale: torch.Tensor, c_scale: float = 1.0,
                     c: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_gemm_fp8. Codes a [rows, H] / [rows, I] and w (as grouped_gemm),
    f32 w_scale [S]. GATE_UP_SWIGLU -> codes [rows, I] quantized with c_scale;
    DOWN -> bf16 [rows, H]."""
    _dev(a, "a", _CODES)
    _dev(w, "w", _CODES)
    _dev(offsets, "offsets", torch.int32)
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError("a must be 2-D and w 3-D")
    S = w.shape[0]
    _dev(w_scale, "w_scale", torch.float32, (S,))
    if offsets.numel() != S + 1:
        raise ValueError("offsets must have S + 1 entries")
    rows = a.shape[0]
    if op == GATE_UP_SWIGLU:
        H, I = a.shape[1], w.shape[1] // 2
        if w.shape[2] != H or w.shape[1] != 2 * I:
            raise ValueError("w must be [S, 2I, H]")
        shape, cdt = (rows, I), _CODES
    elif op == DOWN:
        I, H = a.shape[1], w.shape[1]
        if w.shape[2] != I:
            raise ValueError("w must be [S, H, I]")
        shape, cdt = (rows, H), torch.bfloat16
    else:
        raise ValueError("op must be GATE_UP_SWIGLU or DOWN")
    if c is None:
        c = _empty(shape, torch.uint8 if op == GATE_UP_SWIGLU else torch.bfloat16, a)
    else:
        _dev(c, "c", cdt, shape)
    _launch("moe_grouped_gemm_fp8", a, (offsets, w, w_scale, c), op, _ptr(a), float(a_scale),
            _ptr(offsets), S, rows, _ptr(w), _ptr(w_scale), H, I, _ptr(c), float(c_scale))
    return c


def _mx_shape(w: torch.Tensor, name: str) -> Tuple[int, ...]:
    if w.dim() < 1 or w.shape[-1] % MX_GROUP != 0:
        raise ValueError(f"{name}: the last size must be a multiple of {MX_GROUP}, "
                         f"got {tuple(w.shape)}")
    return tuple(w.shape[:-1])


def quantize_mxfp4(w: torch.Tensor, codes: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """moe_quantize_mxfp4: w [..., K] (bf16 or f32, K % 32 == 0) -> (codes [..., K/2] uint8,
    scale [..., K/32] uint8)."""
    _dev(w, "w", (torch.float32, torch.bfloat16))
    lead, K = _mx_shape(w, "w"), w.shape[-1]
    codes = (_empty((*lead, K // 2), torch.uint8, w) if codes is None
             else _dev(codes, "codes", torch.uint8, (*lead, K // 2)))
    scale = (_empty((*lead, K // MX_GROUP), torch.uint8, w) if scale is None
             else _dev(scale, "scale", torch.uint8, (*lead, K // MX_GROUP)))
    _launch("moe_quantize_mxfp4", w, (codes, scale), w.data_ptr(), _DT[w.dtype], w.numel(),
            codes.data_ptr(), scale.data_ptr())
    return codes, scale


def dequantize_mxfp4(codes: torch.Tensor, scale: torch.Tensor,
                     dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_dequantize_mxfp4: the weights [..., K] (bf16 or f32) that codes [..., K/2] and
    scale [..., K/32] stand for."""
    _dev(codes, "codes", torch.uint8)
    if codes.dim() < 1 or (2 * codes.shape[-1]) % MX_GROUP != 0:
        raise ValueError(f"codes must be whole groups of {MX_GROUP // 2} bytes a row")
    lead, K = tuple(codes.shape[:-1]), 2 * codes.shape[-1]
    _dev(scale, "scale", torch.uint8, (*lead, K // MX_GROUP))
    if out is None:
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"dtype {dtype}, expected torch.float32 or torch.bfloat16")
        out = _empty((*lead, K), dtype, codes)
    else:
        _dev(out, "out", (torch.float32, torch.bfloat16), (*lead, K))
    _launch("moe_dequantize_mxfp4", codes, (scale, out), codes.data_ptr(), scale.data_ptr(),
            out.numel(), out.data_ptr(), _DT[out.dtype])
    return out


def grouped_gemm_mxfp4(op: int, a: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor,
                       w_scale: torch.Tensor, c: Optional[torch.Tensor] = None,
                       c_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """moe_grouped_gemm_mxfp4. GATE_UP_SWIGLU: a bf16 [rows, H], w codes [S, 2I, H/2], w_scale
    [S, 2I, H/32] -> bf16 [rows, I]. DOWN: a bf16 [rows, I], w [S, H, I/2], w_scale
    [S, H, I/32] -> [rows, H] of c_dtype (bf16 or f32)."""
    _dev(a, "a", torch.bfloat16)
    _dev(w, "w", torch.uint8)
    _dev(offsets, "offsets", torch.int32)
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError("a must be 2-D and w 3-D")
    S, N, half = w.shape
    rows, Kd = a.shape
    if offsets.numel() != S + 1:
        raise ValueError("offsets must have S + 1 entries")
    if 2 * half != Kd:
        raise ValueError(f"w rows hold {2 * half} codes, a rows {Kd} values")
    if op == GATE_UP_SWIGLU:
        if N % 2:
            raise ValueError("w must be [S, 2I, H/2]")
        H, I, cols, kinds = Kd, N // 2, N // 2, (torch.bfloat16,)
    elif op == DOWN:
        H, I, cols, kinds = N, Kd, N, (torch.bfloat16, torch.float32)
    else:
        raise ValueError("op must be GATE_UP_SWIGLU or DOWN")
    _dev(w_scale, "w_scale", torch.uint8, (S, N, Kd // MX_GROUP))
    if c is None:
        if c_dtype not in kinds:
            raise TypeError(f"c_dtype {c_dtype}, expected one of {kinds}")
        c = _empty((rows, cols), c_dtype, a)
    else:
        _dev(c, "c", kinds, (rows, cols))
    _launch("moe_grouped_gemm_mxfp4", a, (offsets, w, w_scale, c), op, a.data_ptr(),
            offsets.data_ptr(), S, rows, w.data_ptr(), w_scale.data_ptr(), H, I, c.data_ptr(),
            _DT[c.dtype])
    return c


# ---------------------------------------------------------------- before the layer
def rms_norm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, q_scale: Optional[float] = None,
             y: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
             q: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """moe_rms_norm -> (y [T, H], residual_out [T, H] or None, q codes [T, H] uint8 or None).

    x [T, H], gamma [H] and residual [T, H] of one dtype (bf16 or f32). residual_out is x +
    residual (only with a residual; pass x or residual itself to update it in place), q the E4M3
    codes of the norm at q_scale (only with a q_scale)."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    _dev(gamma, "gamma", x.dtype, (H,))
    if residual is not None:
        _dev(residual, "residual", x.dtype, (T, H))
        residual_out = (torch.empty_like(x) if residual_out is None
                        else _dev(residual_out, "residual_out", x.dtype, (T, H)))
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if q_scale is not None:
        q = (torch.empty_like(x, dtype=torch.uint8) if q is None else _dev(q, "q", _CODES, (T, H)))
    elif q is not None:
        raise ValueError("q needs a q_scale")
    y = torch.empty_like(x) if y is None else _dev(y, "y", x.dtype, (T, H))
    _launch("moe_rms_norm", x, (gamma, residual, residual_out, y, q), x.data_ptr(),
            _ptr(residual), gamma.data_ptr(), _DT[x.dtype], T, H, eps, _ptr(residual_out),
            y.data_ptr(), _ptr(q), 0.0 if q_scale is None else q_scale)
    return y, residual_out, q


def layer_norm(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
               q_scale: Optional[float] = None, y: Optional[torch.Tensor] = None,
               residual_out: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """moe_layer_norm -> (y [T, H], residual_out [T, H] or None, q codes [T, H] uint8 or None).

    As rms_norm, with the mean taken out and beta [H] (None: 0) added."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    _dev(gamma, "gamma", x.dtype, (H,))
    if beta is not None:
        _dev(beta, "beta", x.dtype, (H,))
    if residual is not None:
        _dev(residual, "residual", x.dtype, (T, H))
        residual_out = (torch.empty_like(x) if residual_out is None
                        else _dev(residual_out, "residual_out", x.dtype, (T, H)))
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if q_scale is not None:
        q = (torch.empty_like(x, dtype=torch.uint8) if q is None else _dev(q, "q", _CODES, (T, H)))
    elif q is not None:
        raise ValueError("q needs a q_scale")
    y = torch.empty_like(x) if y is None else _dev(y, "y", x.dtype, (T, H))
    _launch("moe_layer_norm", x, (gamma, beta, residual, residual_out, y, q), x.data_ptr(),
            _ptr(residual), gamma.data_ptr(), _ptr(beta), _DT[x.dtype], T, H, eps,
            _ptr(residual_out), y.data_ptr(), _ptr(q), 0.0 if q_scale is None else q_scale)
    return y, residual_out, q


def norm_backward_workspace_size(T: int, H: int) -> int:
    return _size("moe_norm_backward_workspace_size", T, H)


def _norm_backward(what, dy, x, gamma, eps, dresidual, dx, sums, ws):
    """dx and the sums over the rows: f32 [H] each, given or None."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    dt, shape = x.dtype, x.shape
    T, H = shape
    _dev(dy, "dy", dt, shape)
    _dev(gamma, "gamma", dt, (H,))
    if dresidual is not None:
        _dev(dresidual, "dresidual", dt, shape)
    dx = torch.empty_like(x) if dx is None else _dev(dx, "dx", dt, shape)
    # like gamma and by one number: a third of the time that a new shape takes torch
    sums = [torch.empty_like(gamma, dtype=torch.float32) if s is None
            else _dev(s, "dgamma and dbeta", torch.float32, (H,)) for s in sums]
    if ws is None:
        need = norm_backward_workspace_size(T, H)
        ws = x.new_empty(need, dtype=torch.uint8) if need else None
    else:
        _dev(ws, "ws")
    _launch(what, x, (dy, gamma, dresidual, dx, *sums, ws), dy.data_ptr(), x.data_ptr(),
            gamma.data_ptr(), _ptr(dresidual), _DT[dt], T, H, eps, dx.data_ptr(),
            *[s.data_ptr() for s in sums], _ptr(ws),
            0 if ws is None else ws.numel() * ws.element_size())
    return (dx, *sums)


def rms_norm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                      dresidual: Optional[torch.Tensor] = None,
                      dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """moe_rms_norm_backward -> (dx [T, H], dgamma [H] f32).

    dy is the gradient of rms_norm's y; x its input, or its residual_out where it added a
    residual, whose gradient dresidual is then added (dx is the gradient of both addends). dx may
    be dy, x or dresidual itself."""
    return _norm_backward("moe_rms_norm_backward", dy, x, gamma, eps, dresidual, dx, (dgamma,), ws)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5,
                        dresidual: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                        dbeta: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """moe_layer_norm_backward -> (dx [T, H], dgamma [H] f32, dbeta [H] f32); arguments as
    rms_norm_backward."""
    return _norm_backward("moe_layer_norm_backward", dy, x, gamma, eps, dresidual, dx,
                          (dgamma, dbeta), ws)


# ---------------------------------------------------------------- the router's training step
def _router_inputs(logits, ids, token_mask) -> Tuple[int, int, int]:
    _dev(logits, "logits", torch.float32)
    _dev(ids, "ids", torch.int32)
    if logits.dim() != 2 or ids.dim() != 2 or ids.shape[0] != logits.shape[0]:
        raise ValueError("logits must be [T, E] and ids [T, K]")
    T, E = logits.shape
    if token_mask is not None:
        _dev(token_mask, "token_mask", (torch.uint8, torch.bool), (T,))
    return T, E, ids.shape[1]


def balance_loss_workspace_size(T: int, E: int, K: int) -> int:
    return _size("moe_balance_loss_workspace_size", T, E, K)


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, coef: float,
                 token_mask: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """moe_balance_loss: logits [T, E] f32, ids [T, K] int32, token_mask [T] (uint8 or bool, 0 =
    padding) -> (loss f32 scalar, counts [E+1] int32 with the number of valid tokens last,
    prob [E] f32)."""
    T, E, K = _router_inputs(logits, ids, token_mask)
    counts = _empty((E + 1,), torch.int32, logits)
    prob = _empty((E,), torch.float32, logits)
    loss = _empty((), torch.float32, logits)
    if ws is None:
        ws = _empty((max(balance_loss_workspace_size(T, E, K), 1),), torch.uint8, logits)
    else:
        _dev(ws, "ws")
    _launch("moe_balance_loss", logits, (ids, token_mask, ws), logits.data_ptr(),
            ids.data_ptr(), _ptr(token_mask), T, E, K, coef, counts.data_ptr(), prob.data_ptr(),
            loss.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return loss, counts, prob


def route_backward(logits: torch.Tensor, ids: torch.Tensor, dw: Optional[torch.Tensor],
                   renormalize: bool, counts: Optional[torch.Tensor] = None, coef: float = 0.0,
                   dloss: Optional[torch.Tensor] = None,
                   token_mask: Optional[torch.Tensor] = None,
                   dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_route_backward: dlogits [T, E] f32 of the routing weights' gradient dw [T, K] f32
    (None: no such term) plus that of balance_loss, whose counts and coef are given (counts
    None: no such term), times dloss (one f32 on the device, None: 1)."""
    T, E, K = _router_inputs(logits, ids, token_mask)
    if dw is not None:
        _dev(dw, "dw", torch.float32, (T, K))
    if counts is not None:
        _dev(counts, "counts", torch.int32, (E + 1,))
    if dloss is not None:
        _dev(dloss, "dloss", torch.float32)
        if dloss.numel() != 1:
            raise ValueError("dloss must hold one value")
    dlogits = (torch.empty_like(logits) if dlogits is None
               else _dev(dlogits, "dlogits", torch.float32, (T, E)))
    _launch("moe_route_backward", logits, (ids, dw, counts, dloss, token_mask, dlogits),
            logits.data_ptr(), ids.data_ptr(), _ptr(dw), _ptr(token_mask), _ptr(counts),
            _ptr(dloss), T, E, K, 1 if renormalize else 0, coef, dlogits.data_ptr())
    return dlogits


def combine(y: torch.Tensor, pair_row: torch.Tensor, w_masked: Optional[torch.Tensor], K: int,
            out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
            accumulate: bool = False, shared: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_combine: out[t] (+)= sum_k w_masked[t,k] * y[pair_row[t,k]].
    w_masked None (unit weights) or shared [T, H] (added before the rounding)
    use moe_combine_shared."""
    _dev(y, "y", (torch.float32, torch.bfloat16))
    _dev(pair_row, "pair_row", torch.int32)
    P = pair_row.numel()
    if w_masked is not None:
        _dev(w_masked, "w_masked", torch.float32)
        if w_masked.numel() != P:
            raise ValueError("pair_row / w_masked must hold T*K entries")
    if P % K != 0:
        raise ValueError("pair_row must hold T*K entries")
    _fits("pair_row", P)
    T = P // K
    H = y.shape[1]
    if out is None:
        out = _empty((T, H), out_dtype or y.dtype, y)
        if accumulate:
            out.zero_()
    else:
        _dev(out, "out", (torch.float32, torch.bfloat16), (T, H))
    if w_masked is None or shared is not None:
        sdt = MOE_DTYPE_BF16
        if shared is not None:
            _dev(shared, "shared", (torch.float32, torch.bfloat16), (T, H))
            sdt = _DT[shared.dtype]
        _launch("moe_combine_shared", y, (pair_row, w_masked, shared, out), _ptr(y), _DT[y.dtype],
                _ptr(pair_row), _ptr(w_masked), T, K, H, _ptr(shared), sdt, _ptr(out),
                _DT[out.dtype], int(bool(accumulate)))
    else:
        _launch("moe_combine", y, (pair_row, w_masked, out), _ptr(y), _DT[y.dtype], _ptr(pair_row),
                _ptr(w_masked), T, K, H, _ptr(out), _DT[out.dtype], int(bool(accumulate)))
    return out


# ---------------------------------------------------------------- the layer's training step
def _pair_rows(pair_row, K: int) -> int:
    _dev(pair_row, "pair_row", torch.int32)
    P = pair_row.numel()
    if K < 1 or P % K != 0:
        raise ValueError("pair_row must hold T*K entries")
    if P >= _WIDE:
        _fits("pair_row", P)
    return P // K


def combine_backward(dout: torch.Tensor, y: Optional[torch.Tensor], pair_row: torch.Tensor,
                     w_masked: Optional[torch.Tensor], K: int,
                     dy: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """moe_combine_backward -> (dy [rows, H] of y's dtype, dw [T, K] f32).

    dout [T, H] is the gradient of combine's out, y [rows, H] the rows that it summed. dw is None
    without weights, where y may be None too (a dy is needed then). Rows of dy that no pair has
    are not written."""
    T = _pair_rows(pair_row, K)
    _dev(dout, "dout", (torch.float32, torch.bfloat16))
    if dout.dim() != 2 or dout.shape[0] != T:
        raise ValueError("dout must be [T, H] with T*K entries in pair_row")
    H = dout.shape[1]
    for t, name in ((y, "y"), (dy, "dy")):
        if t is not None:
            _dev(t, name, (torch.float32, torch.bfloat16))
            if t.dim() != 2 or t.shape[1] != H:
                raise ValueError(f"{name} must be [rows, H]")
    if y is not None:
        dy = torch.empty_like(y) if dy is None else _dev(dy, "dy", y.dtype, tuple(y.shape))
    elif dy is None:
        raise ValueError("dy is needed where there is no y")
    if w_masked is not None:
        _dev(w_masked, "w_masked", torch.float32)
        if w_masked.numel() != T * K:
            raise ValueError("w_masked must hold T*K entries")
        if y is None:
            raise ValueError("the weights' gradient needs y")
        if dw is not None:
            _dev(dw, "dw", torch.float32, (T, K))
        elif w_masked.shape == (T, K):
            dw = torch.empty_like(w_masked)
        else:
            dw = _empty((T, K), torch.float32, dout)
    elif dw is not None:
        raise ValueError("dw needs w_masked")
    if dy.shape[0] == 0:  # a share without pairs: an empty tensor has no address to pass
        return dy, None if dw is None else dw.zero_()
    _launch("moe_combine_backward", dout, (y, pair_row, w_masked, dy, dw), dout.data_ptr(),
            _DT[dout.dtype], _ptr(y), _DT[dy.dtype], pair_row.data_ptr(), _ptr(w_masked), T, K, H,
            dy.data_ptr(), _ptr(dw))
    return dy, dw


def permute_backward(dx_perm: torch.Tensor, pair_row: torch.Tensor, K: int,
                     pair_w: Optional[torch.Tensor] = None, x: Optional[torch.Tensor] = None,
                     dx: Optional[torch.Tensor] = None, dx_dtype: Optional[torch.dtype] = None,
                     accumulate: bool = False, dpair_w: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """moe_permute_backward -> (dx [T, H], dpair_w [T, K] f32 or None).

    dx_perm [rows, H] is the gradient of permute's rows. With pair_w [T, K] (rows that carry
    their weight) and x [T, H] dpair_w is the weights' gradient; without x it is None. accumulate
    adds to dx, which must be given."""
    T = _pair_rows(pair_row, K)
    _dev(dx_perm, "dx_perm", (torch.float32, torch.bfloat16))
    if dx_perm.dim() != 2:
        raise ValueError("dx_perm must be [rows, H]")
    H = dx_perm.shape[1]
    if pair_w is not None:
        _dev(pair_w, "pair_w", torch.float32)
        if pair_w.numel() != T * K:
            raise ValueError("pair_w must hold T*K entries")
    if x is not None:
        if pair_w is None:
            raise ValueError("the weights' gradient needs pair_w")
        _dev(x, "x", dx_perm.dtype, (T, H))
        dpair_w = (_empty((T, K), torch.float32, dx_perm) if dpair_w is None
                   else _dev(dpair_w, "dpair_w", torch.float32, (T, K)))
    elif dpair_w is not None:
        raise ValueError("dpair_w needs x")
    if dx is None:
        if accumulate:
            raise ValueError("accumulate needs dx")
        if dx_dtype not in (None, torch.float32, torch.bfloat16):
            raise TypeError(f"dx_dtype {dx_dtype}, expected torch.float32 or torch.bfloat16")
        dx = _empty((T, H), dx_dtype or dx_perm.dtype, dx_perm)
    else:
        _dev(dx, "dx", (torch.float32, torch.bfloat16), (T, H))
    if dx_perm.shape[0] == 0:
        return dx if accumulate else dx.zero_(), None if dpair_w is None else dpair_w.zero_()
    _launch("moe_permute_backward", dx_perm, (pair_row, pair_w, x, dx, dpair_w),
            dx_perm.data_ptr(), _DT[dx_perm.dtype], pair_row.data_ptr(), _ptr(pair_w), _ptr(x), T,
            K, H, dx.data_ptr(), _DT[dx.dtype], 1 if accumulate else 0, _ptr(dpair_w))
    return dx, dpair_w


def _slots(offsets) -> int:
    _dev(offsets, "offsets", torch.int32)
    n = offsets.numel()
    if offsets.dim() != 1 or n < 2:
        raise ValueError("offsets must have S + 1 entries")
    if n >= _WIDE:
        _fits("offsets", n)
    return n - 1


def swiglu(h: torch.Tensor, offsets: torch.Tensor, act: Optional[torch.Tensor] = None
           ) -> torch.Tensor:
    """moe_swiglu: h [rows, 2I] (gate, up) -> act [rows, I]; rows before offsets[0] and behind
    offsets[S] are not written. h is grouped_gemm(DOWN, x_perm, offsets, w_gate_up)."""
    _dev(h, "h", (torch.float32, torch.bfloat16))
    S = _slots(offsets)
    if h.dim() != 2 or h.shape[1] % 2:
        raise ValueError("h must be [rows, 2I]")
    rows, I = h.shape[0], h.shape[1] // 2
    act = (_empty((rows, I), h.dtype, h) if act is None
           else _dev(act, "act", h.dtype, (rows, I)))
    _launch("moe_swiglu", h, (offsets, act), h.data_ptr(), _DT[h.dtype], offsets.data_ptr(), S,
            rows, I, act.data_ptr())
    return act


def grouped_gemm_backward(op: int, dc: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor,
                          h: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None
                          ) -> torch.Tensor:
    """moe_grouped_gemm_backward, the rows' gradient. GATE_UP_SWIGLU: dc [rows, 2I] (gradient of
    h), w [S, 2I, H] -> [rows, H]. DOWN: dc [rows, H], w [S, H, I] -> [rows, I], or with h
    [rows, 2I] (swiglu's input) -> its gradient [rows, 2I]. Rows before offsets[0] and behind
    offsets[S] are not written."""
    _dev(dc, "dc", (torch.float32, torch.bfloat16))
    _dev(w, "w", dc.dtype)
    S = _slots(offsets)
    if dc.dim() != 2 or w.dim() != 3 or w.shape[0] != S or w.shape[1] != dc.shape[1]:
        raise ValueError("dc must be [rows, N] and w [S, N, K] with S + 1 offsets")
    rows = dc.shape[0]
    if op == GATE_UP_SWIGLU:
        if w.shape[1] % 2:
            raise ValueError("w must be [S, 2I, H]")
        if h is not None:
            raise ValueError("h belongs to DOWN")
        H, I, cols = w.shape[2], w.shape[1] // 2, w.shape[2]
    elif op == DOWN:
        H, I = w.shape[1], w.shape[2]
        cols = I if h is None else 2 * I
    else:
        raise ValueError("op must be GATE_UP_SWIGLU or DOWN")
    if h is not None:
        _dev(h, "h", dc.dtype, (rows, cols))
    out = (_empty((rows, cols), dc.dtype, dc) if out is None
           else _dev(out, "out", dc.dtype, (rows, cols)))
    _launch("moe_grouped_gemm_backward", dc, (offsets, w, h, out), op, _DT[dc.dtype],
            dc.data_ptr(), offsets.data_ptr(), S, rows, w.data_ptr(), H, I, _ptr(h),
            out.data_ptr())
    return out


def grouped_gemm_weight_grad_workspace_size(dtype: torch.dtype, S: int, rows: int, N: int, K: int
                                            ) -> int:
    return _size("moe_grouped_gemm_weight_grad_workspace_size", _DT[dtype], S, rows, N, K)


def grouped_gemm_weight_grad(dc: torch.Tensor, a: torch.Tensor, offsets: torch.Tensor,
                             dw: Optional[torch.Tensor] = None,
                             dw_dtype: torch.dtype = torch.float32, accumulate: bool = False,
                             ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_gemm_weight_grad: dw [S, N, K] (f32 or bf16) of dc [rows, N] and a [rows, K],
    zeros for slots without rows. accumulate adds to dw, which must be given. Tiles and splits are
    chosen by the buffers' rows: where the rows in use are known on the host, dc[:used] and
    a[:used] take the forms that suit them."""
    _dev(dc, "dc", (torch.float32, torch.bfloat16))
    _dev(a, "a", dc.dtype)
    S = _slots(offsets)
    if dc.dim() != 2 or a.dim() != 2 or a.shape[0] != dc.shape[0]:
        raise ValueError("dc must be [rows, N] and a [rows, K]")
    rows, N, Kd = dc.shape[0], dc.shape[1], a.shape[1]
    if Kd >= _WIDE:
        _fits("a", Kd)
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        if dw_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"dw_dtype {dw_dtype}, expected torch.float32 or torch.bfloat16")
        dw = _empty((S, N, Kd), dw_dtype, dc)
    else:
        _dev(dw, "dw", (torch.float32, torch.bfloat16), (S, N, Kd))
    if ws is None:
        need = grouped_gemm_weight_grad_workspace_size(dc.dtype, S, rows, N, Kd)
        ws = _empty((need,), torch.uint8, dc) if need else None
    else:
        _dev(ws, "ws")
    _launch("moe_grouped_gemm_weight_grad", dc, (a, offsets, dw, ws), _DT[dc.dtype],
            dc.data_ptr(), a.data_ptr(), offsets.data_ptr(), S, rows, N, Kd, dw.data_ptr(),
            _DT[dw.dtype], 1 if accumulate else 0, _ptr(ws),
            0 if ws is None else ws.numel() * ws.element_size())
    return dw


# ---------------------------------------------------------------- fused
class ForwardConfig:
    """Plain mirror of moe_config_t."""

    def __init__(self, T: int, H: int, I: int, E_global: int, K: int, renormalize: bool,
                 S: int, dtype: torch.dtype, out_dtype: Optional[torch.dtype] = None,
                 ep_size: int = 1, ep_rank: int = 0, accumulate: bool = False,
                 T_max: Optional[int] = None, num_expert_group: int = 0, topk_group: int = 0,
                 routing_on_input: bool = False, a1_scale: float = 1.0, a2_scale: float = 1.0,
                 gemm_blocks: int = 0, x_codes: bool = False):
        self.T, self.H, self.I, self.E_global, self.K = T, H, I, E_global, K
        self.renormalize, self.S, self.dtype = bool(renormalize), S, dtype
        # FP8 and MXFP4: x, shared_out and the default out are bf16
        self.out_dtype = out_dtype or (torch.bfloat16 if dtype in (FP8, MXFP4) else dtype)
        self.a1_scale, self.a2_scale = float(a1_scale), float(a2_scale)
        self.ep_size, self.ep_rank, self.accumulate = ep_size, ep_rank, bool(accumulate)
        self.T_max = T if T_max is None else T_max
        self.num_expert_group, self.topk_group = num_expert_group, topk_group
        self.routing_on_input = bool(routing_on_input)
        self.gemm_blocks = int(gemm_blocks)  # 0: one persistent GEMM block per compute unit
        self.x_codes = bool(x_codes)  # FP8: x holds E4M3 codes at a1_scale (rms_norm's q)
        _fits("ForwardConfig", self.T_max, T, H, I, E_global, K, S)

    def c_struct(self) -> _Config:
        return _Config(self.T_max, self.T, self.H, self.I, self.E_global, self.K,
                       int(self.renormalize), self.ep_size, self.ep_rank, self.S,
                       _DT[self.dtype], _DT[self.out_dtype], int(self.accumulate),
                       self.num_expert_group, self.topk_group, int(self.routing_on_input),
                       self.a1_scale, self.a2_scale, self.gemm_blocks, int(self.x_codes))


def _workspace_size(c: _Config) -> int:
    n = int(lib().moe_forward_workspace_size(ctypes.byref(c)))
    if n == 0:
        raise RuntimeError("moe_forward_workspace_size: invalid configuration")
    return n


def forward_workspace_size(cfg: ForwardConfig) -> int:
    return _workspace_size(cfg.c_struct())


_NO_EVENTS = (_p * NUM_EVENTS)()


def forward(cfg: ForwardConfig, x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
            logits: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
            topk_w: Optional[torch.Tensor] = None, rep_off: Optional[torch.Tensor] = None,
            rep_slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            ws: Optional[torch.Tensor] = None, events: Optional[Sequence[int]] = None,
            shared_out: Optional[torch.Tensor] = None,
            w_gate_up_scale: Optional[torch.Tensor] = None,
            w_down_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_forward. Pass logits [T, E_global] f32, or topk_ids [T, K] int32 and
    topk_w [T, K] f32. Weights are per slot: w_gate_up [S, 2I, H], w_down [S, H, I].
    `events`: up to NUM_EVENTS raw hipEvent_t handles (0 = skip) recorded at the
    stage boundaries. cfg.dtype FP8: x is bf16, the weights are E4M3 codes
    (uint8 or float8_e4m3fn) with f32 per-slot scales w_gate_up_scale,
    w_down_scale [S]; with cfg.x_codes x holds codes too (rms_norm's q).
    cfg.dtype MXFP4: x is bf16, the weights are codes [S, 2I, H/2], [S, H, I/2]
    and scales [S, 2I, H/32], [S, H, I/32], all uint8 (quantize_mxfp4)."""
    T, H, I, S = cfg.T, cfg.H, cfg.I, cfg.S
    if T >= _WIDE:  # set behind the constructor's look at it
        _fits("forward", T)
    fp8, mx = cfg.dtype == FP8, cfg.dtype == MXFP4
    xdt = torch.bfloat16 if fp8 or mx else cfg.dtype
    wdt = _CODES if fp8 else torch.uint8 if mx else cfg.dtype
    pack = 2 if mx else 1  # weights in an element
    _dev(x, "x", _CODES if fp8 and cfg.x_codes else xdt, (T, H))
    _dev(w_gate_up, "w_gate_up", wdt, (S, 2 * I, H // pack))
    _dev(w_down, "w_down", wdt, (S, H, I // pack))
    if mx:
        _dev(w_gate_up_scale, "w_gate_up_scale", torch.uint8, (S, 2 * I, H // MX_GROUP))
        _dev(w_down_scale, "w_down_scale", torch.uint8, (S, H, I // MX_GROUP))
    if fp8:
        _dev(w_gate_up_scale, "w_gate_up_scale", torch.float32, (S,))
        _dev(w_down_scale, "w_down_scale", torch.float32, (S,))
    if logits is not None:
        _dev(logits, "logits", torch.float32, (T, cfg.E_global))
    else:
        _dev(topk_ids, "topk_ids", torch.int32, (T, cfg.K))
        _dev(topk_w, "topk_w", torch.float32, (T, cfg.K))
    if rep_off is not None:
        _dev(rep_off, "rep_off", torch.int32, (cfg.E_global // cfg.ep_size + 1,))
        _dev(rep_slots, "rep_slots", torch.int32, (S,))
    if out is None:
        out = _empty((T, H), cfg.out_dtype, x)
        if cfg.accumulate:
            out.zero_()
    else:
        _dev(out, "out", cfg.out_dtype, (T, H))
    c = cfg.c_struct()
    need = _workspace_size(c)
    ws = _empty((need,), torch.uint8, x) if ws is None else _dev(ws, "ws")
    ev = _NO_EVENTS
    if events is not None:
        ev = (_p * NUM_EVENTS)()
        for i, e in enumerate(list(events)[:NUM_EVENTS]):
            ev[i] = e or 0
    if shared_out is not None:
        _dev(shared_out, "shared_out", xdt, (T, H))
    args = _ForwardArgs(_ptr(x), _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _ptr(w_gate_up),
                        _ptr(w_down), _ptr(rep_off), _ptr(rep_slots), _ptr(out), ev,
                        _ptr(shared_out), None if mx else _ptr(w_gate_up_scale),
                        None if mx else _ptr(w_down_scale),
                        _ptr(w_gate_up_scale) if mx else None,
                        _ptr(w_down_scale) if mx else None)
    _launch("moe_forward", x, (w_gate_up, w_down, logits, topk_ids, topk_w, rep_off, rep_slots, out,
                               ws, shared_out, w_gate_up_scale, w_down_scale),
            ctypes.byref(c), ctypes.byref(args), ws.data_ptr(), ws.numel() * ws.element_size())
    return out


# ---------------------------------------------------------------- all-to-all
def a2a_dispatch_workspace_size(T: int, ep_size: int, cap: int) -> int:
    return _size("moe_a2a_dispatch_workspace_size", T, ep_size, cap)


def a2a_dispatch(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, E_global: int,
                 ep_size: int, cap: Optional[int] = None, ws: Optional[torch.Tensor] = None):
    """moe_a2a_dispatch -> (offsets [ep+1], token_pos [T, ep], send_token [ep*cap],
    send_x [ep*cap, H], send_ids [ep*cap, K], send_w [ep*cap, K]).

    Rank r's block is rows [r*cap, (r+1)*cap); cap defaults to T."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    _dev(topk_ids, "topk_ids", torch.int32)
    T, K = topk_ids.shape
    _dev(topk_w, "topk_w", torch.float32, (T, K))
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T matching topk_ids")
    H = x.shape[1]
    cap = T if cap is None else cap
    _fits("cap", cap)
    offsets = _empty((ep_size + 1,), torch.int32, x)
    token_pos = _empty((T, ep_size), torch.int32, x)
    send_token = _empty((ep_size * cap,), torch.int32, x)
    send_x = _empty((ep_size * cap, H), x.dtype, x)
    send_ids = _empty((ep_size * cap, K), torch.int32, x)
    send_w = _empty((ep_size * cap, K), torch.float32, x)
    need = a2a_dispatch_workspace_size(T, ep_size, cap)
    ws = _empty((max(need, 1),), torch.uint8, x) if ws is None else _dev(ws, "ws")
    _launch("moe_a2a_dispatch", x, (topk_ids, topk_w, ws), _ptr(x), _DT[x.dtype], T, H, K,
            _ptr(topk_ids), _ptr(topk_w), E_global, ep_size, cap, _ptr(offsets), _ptr(token_pos),
            _ptr(send_token), _ptr(send_x), _ptr(send_ids), _ptr(send_w), _ptr(ws),
            ws.numel() * ws.element_size())
    return offsets, token_pos, send_token, send_x, send_ids, send_w


def a2a_combine(partial: torch.Tensor, token_pos: torch.Tensor,
                out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """moe_a2a_combine: out[t] = sum over ranks r (ascending) with
    token_pos[t, r] >= 0 of partial[token_pos[t, r]]."""
    _dev(partial, "partial", (torch.float32, torch.bfloat16))
    _dev(token_pos, "token_pos", torch.int32)
    T, ep_size = token_pos.shape
    H = partial.shape[1]
    out = _empty((T, H), out_dtype or partial.dtype, partial)
    _fits("token_pos", T)
    _launch("moe_a2a_combine", partial, (token_pos,), _ptr(partial), _DT[partial.dtype],
            _ptr(token_pos), T, ep_size, H, _ptr(out), _DT[out.dtype])
    return out
