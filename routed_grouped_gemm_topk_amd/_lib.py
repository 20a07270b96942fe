"""ctypes binding of libmoe.so: argument marshalling only.

Every function mirrors one ``extern "C"`` entry point of include/moe.h under the
same name.  Tensors are torch tensors on the current HIP device; the binding
checks dtype, shape, device and contiguity, then passes raw pointers and the
current stream.  All arithmetic happens in the HIP kernels behind the C ABI.
If libmoe.so is missing, loading raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_NULL = -1
MOE_ERR_SHAPE = -2
MOE_ERR_DTYPE = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_LAUNCH = -5
MOE_ERR_DEVICE = -6
MOE_ERR_ALIGN = -7

MOE_F32, MOE_BF16, MOE_E4M3, MOE_MXFP4 = 0, 1, 2, 3
_DT_NAME = {"f32": MOE_F32, "bf16": MOE_BF16, "e4m3": MOE_E4M3, "mxfp4": MOE_MXFP4}
_TORCH_DT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_E4M3: torch.float8_e4m3fn}

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
_SCORE = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_ACT_NONE, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH = 0, 1, 2, 3
_ACT = {"none": MOE_ACT_NONE, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU,
        "gelu_tanh": MOE_ACT_GELU_TANH}
MOE_NT, MOE_NN, MOE_TN = 0, 1, 2
_LAYOUT = {"nt": MOE_NT, "nn": MOE_NN, "tn": MOE_TN}

EXPORTS = ["moe_status_str", "moe_validate", "moe_pick_block_m", "moe_block_m_for", "moe_max_padded_slots",
           "moe_max_tiles", "moe_workspace_bytes", "moe_route", "moe_route_align", "moe_align",
           "moe_quantize_rows_e4m3", "moe_grouped_gemm_up", "moe_grouped_gemm_up_mxfp4",
           "moe_grouped_gemm_down", "moe_gemm_workspace_bytes",
           "moe_combine", "moe_forward", "moe_scratch_max_bytes", "moe_forward_scratch",
           "moe_permute", "moe_unpermute", "moe_unpermute_bwd", "moe_route_bwd",
           "moe_quantize_cols_e4m3", "moe_gemm_e4m3", "moe_grouped_gemm_e4m3",
           "moe_router_validate", "moe_route_scored", "moe_route_scored_bwd", "moe_rms_norm",
           "moe_rms_norm_bwd", "moe_rms_norm_bwd_workspace_bytes", "moe_gemm_bf16", "moe_act_bwd",
           "moe_act_bwd_workspace_bytes"]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} ({status})")


class Problem(ctypes.Structure):
    """Mirror of ``moe_problem``."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("block_m", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32)]

    def __repr__(self):
        return ("Problem(T=%d, H=%d, I=%d, E=%d, top_k=%d, block_m=%d, dtype=%d, w_dtype=%d)"
                % (self.T, self.H, self.I, self.E, self.top_k, self.block_m, self.dtype, self.w_dtype))


def make_problem(T, H, I, E, top_k, dtype="bf16", w_dtype=None, block_m=0) -> Problem:
    dt = _DT_NAME[dtype] if isinstance(dtype, str) else int(dtype)
    wdt = dt if w_dtype is None else (_DT_NAME[w_dtype] if isinstance(w_dtype, str) else int(w_dtype))
    return Problem(int(T), int(H), int(I), int(E), int(top_k), int(block_m), dt, wdt)


class Router(ctypes.Structure):
    """Mirror of ``moe_router``."""
    _fields_ = [("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __repr__(self):
        return ("Router(score=%d, renormalize=%d, n_groups=%d, topk_groups=%d, group_top=%d, scale=%g)"
                % (self.score, self.renormalize, self.n_groups, self.topk_groups, self.group_top,
                   self.scale))


def make_router(score="softmax", renormalize=True, n_groups=1, topk_groups=None, group_top=1,
                scale=1.0) -> Router:
    """How route_scored chooses and weighs experts; topk_groups None: all groups."""
    sc = _SCORE[score] if isinstance(score, str) else int(score)
    kept = n_groups if topk_groups is None else topk_groups
    return Router(sc, 1 if renormalize else 0, int(n_groups), int(kept), int(group_top),
                  float(scale))


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmoe.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"libmoe.so not found at {p}; build it with "
                          "`python -m routed_grouped_gemm_topk_amd.build` (needs hipcc)")
    lib = ctypes.CDLL(p)
    P = ctypes.POINTER(Problem)
    Q = ctypes.POINTER(Router)
    vp = ctypes.c_void_p
    i32 = ctypes.c_int32
    f32 = ctypes.c_float
    size = ctypes.c_size_t
    sig = {
        "moe_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_validate": (ctypes.c_int, [P]),
        "moe_pick_block_m": (i32, [P]),
        "moe_block_m_for": (i32, [ctypes.c_double, i32, i32]),
        "moe_max_padded_slots": (ctypes.c_int64, [P]),
        "moe_max_tiles": (ctypes.c_int64, [P]),
        "moe_workspace_bytes": (ctypes.c_int64, [P]),
        "moe_align": (ctypes.c_int, [P] + [vp] * 8 + [vp]),
        "moe_route": (ctypes.c_int, [P, vp, ctypes.c_int, vp, vp, vp]),
        "moe_route_align": (ctypes.c_int, [P, vp, ctypes.c_int] + [vp] * 9 + [vp]),
        "moe_quantize_rows_e4m3": (ctypes.c_int, [P, vp, vp, vp, vp]),
        "moe_grouped_gemm_up": (ctypes.c_int, [P] + [vp] * 11 + [ctypes.c_size_t, vp]),
        "moe_grouped_gemm_up_mxfp4": (ctypes.c_int, [P] + [vp] * 5 + [ctypes.c_float] * 2
                                      + [vp] * 6 + [vp]),
        "moe_grouped_gemm_down": (ctypes.c_int, [P] + [vp] * 11 + [ctypes.c_size_t, vp]),
        "moe_gemm_workspace_bytes": (ctypes.c_int64, [P]),
        "moe_combine": (ctypes.c_int, [P, vp, vp, vp, vp]),
        "moe_forward": (ctypes.c_int, [P] + [vp] * 9 + [ctypes.c_size_t, vp]),
        "moe_scratch_max_bytes": (ctypes.c_int64, []),
        "moe_forward_scratch": (ctypes.c_int, [P] + [vp] * 9 + [vp]),
        "moe_permute": (ctypes.c_int, [P, i32] + [vp] * 7 + [vp]),
        "moe_unpermute": (ctypes.c_int, [P, i32] + [vp] * 4 + [vp]),
        "moe_unpermute_bwd": (ctypes.c_int, [P, i32] + [vp] * 8 + [vp]),
        "moe_route_bwd": (ctypes.c_int, [P, vp, ctypes.c_int] + [vp] * 3 + [vp]),
        "moe_quantize_cols_e4m3": (ctypes.c_int, [i32] * 2 + [vp] * 3 + [vp]),
        "moe_gemm_e4m3": (ctypes.c_int, [i32] * 3 + [vp] * 4 + [i32, vp, i32, vp]),
        "moe_grouped_gemm_e4m3": (ctypes.c_int, [P, i32, i32] + [vp] * 9 + [i32, vp]),
        "moe_router_validate": (ctypes.c_int, [P, Q]),
        "moe_route_scored": (ctypes.c_int, [P, Q, vp, i32] + [vp] * 3 + [vp]),
        "moe_route_scored_bwd": (ctypes.c_int, [P, Q, vp, i32] + [vp] * 3 + [vp]),
        "moe_rms_norm": (ctypes.c_int, [i32] * 3 + [vp] * 3 + [f32] + [vp] * 5 + [vp]),
        "moe_rms_norm_bwd": (ctypes.c_int, [i32] * 3 + [vp] * 8 + [size, vp]),
        "moe_rms_norm_bwd_workspace_bytes": (ctypes.c_int64, [i32, i32]),
        "moe_gemm_bf16": (ctypes.c_int, [i32] * 4 + [vp] * 3 + [i32] + [vp] * 3 + [i32, vp]),
        "moe_act_bwd": (ctypes.c_int, [i32] * 3 + [vp] * 5 + [size, vp]),
        "moe_act_bwd_workspace_bytes": (ctypes.c_int64, [i32, i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


# ---------------------------------------------------------------------------------------------
# host-only queries
# ---------------------------------------------------------------------------------------------
def status_str(status: int) -> str:
    return load().moe_status_str(int(status)).decode()


def moe_validate(p: Problem) -> int:
    return load().moe_validate(ctypes.byref(p))


def _checked(v: int, where: str) -> int:
    if v < 0:
        raise MoeError(int(v), where)
    return int(v)


def moe_pick_block_m(p: Problem) -> int:
    return _checked(load().moe_pick_block_m(ctypes.byref(p)), "moe_pick_block_m")


def moe_block_m_for(slots_per_expert: float, dtype="bf16", w_dtype=None) -> int:
    dt = _DT_NAME[dtype] if isinstance(dtype, str) else int(dtype)
    wdt = dt if w_dtype is None else (_DT_NAME[w_dtype] if isinstance(w_dtype, str) else int(w_dtype))
    return _checked(load().moe_block_m_for(float(slots_per_expert), dt, wdt), "moe_block_m_for")


def moe_max_padded_slots(p: Problem) -> int:
    return _checked(load().moe_max_padded_slots(ctypes.byref(p)), "moe_max_padded_slots")


def moe_max_tiles(p: Problem) -> int:
    return _checked(load().moe_max_tiles(ctypes.byref(p)), "moe_max_tiles")


def moe_workspace_bytes(p: Problem) -> int:
    return _checked(load().moe_workspace_bytes(ctypes.byref(p)), "moe_workspace_bytes")


def moe_gemm_workspace_bytes(p: Problem) -> int:
    return _checked(load().moe_gemm_workspace_bytes(ctypes.byref(p)), "moe_gemm_workspace_bytes")


# ---------------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------------
def _stream(stream) -> Optional[int]:
    if stream is None:
        # the handle alone: building a torch.cuda.Stream around it costs 3 us per call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, numel=None, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a device tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _act_dtype(p: Problem):
    return torch.uint8 if p.w_dtype == MOE_E4M3 else _TORCH_DT[p.dtype]


def _w_dtype(p: Problem):
    return (torch.float8_e4m3fn, torch.uint8) if p.w_dtype == MOE_E4M3 else _TORCH_DT[p.w_dtype]


# ---------------------------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------------------------
def moe_align(p: Problem, topk_ids, counts, offsets, sorted_slots, slot_row, tiles, num_tiles,
              n_invalid, stream=None) -> None:
    N = p.T * p.top_k
    rows = moe_max_padded_slots(p)
    mt = moe_max_tiles(p)
    i32 = torch.int32
    args = [_ptr(topk_ids, "topk_ids", i32, N), _ptr(counts, "counts", i32, p.E),
            _ptr(offsets, "offsets", i32, p.E + 1), _ptr(sorted_slots, "sorted_slots", i32, rows),
            _ptr(slot_row, "slot_row", i32, N), _ptr(tiles, "tiles", i32, 2 * mt),
            _ptr(num_tiles, "num_tiles", i32, 1), _ptr(n_invalid, "n_invalid", i32, 1)]
    _checked(load().moe_align(ctypes.byref(p), *args, _stream(stream)), "moe_align")


def moe_route(p: Problem, logits, renormalize: bool, topk_ids, topk_weights, stream=None) -> None:
    N = p.T * p.top_k
    args = [_ptr(logits, "logits", torch.float32, p.T * p.E), ctypes.c_int(1 if renormalize else 0),
            _ptr(topk_ids, "topk_ids", torch.int32, N), _ptr(topk_weights, "topk_weights", torch.float32, N)]
    _checked(load().moe_route(ctypes.byref(p), *args, _stream(stream)), "moe_route")


def moe_route_align(p: Problem, logits, renormalize: bool, topk_ids, topk_weights, counts, offsets,
                    sorted_slots, slot_row, tiles, num_tiles, n_invalid, stream=None) -> None:
    N = p.T * p.top_k
    rows = moe_max_padded_slots(p)
    mt = moe_max_tiles(p)
    i32 = torch.int32
    args = [_ptr(logits, "logits", torch.float32, p.T * p.E), ctypes.c_int(1 if renormalize else 0),
            _ptr(topk_ids, "topk_ids", i32, N), _ptr(topk_weights, "topk_weights", torch.float32, N),
            _ptr(counts, "counts", i32, p.E), _ptr(offsets, "offsets", i32, p.E + 1),
            _ptr(sorted_slots, "sorted_slots", i32, rows), _ptr(slot_row, "slot_row", i32, N),
            _ptr(tiles, "tiles", i32, 2 * mt), _ptr(num_tiles, "num_tiles", i32, 1),
            _ptr(n_invalid, "n_invalid", i32, 1)]
    _checked(load().moe_route_align(ctypes.byref(p), *args, _stream(stream)), "moe_route_align")


def moe_quantize_rows_e4m3(p: Problem, x, xq, scales, stream=None) -> None:
    args = [_ptr(x, "x", torch.bfloat16, p.T * p.H),
            _ptr(xq, "xq", (torch.uint8, torch.float8_e4m3fn), p.T * p.H),
            _ptr(scales, "scales", torch.float32, p.T * p.H // 128)]
    _checked(load().moe_quantize_rows_e4m3(ctypes.byref(p), *args, _stream(stream)),
             "moe_quantize_rows_e4m3")


def moe_grouped_gemm_up(p: Problem, x, x_scales, w13, w13_scales, sorted_slots, offsets, tiles,
                        num_tiles, act, act_scales, workspace=None, stream=None) -> None:
    rows = moe_max_padded_slots(p)
    fp8 = p.w_dtype == MOE_E4M3
    xdt = (torch.uint8, torch.float8_e4m3fn) if fp8 else _TORCH_DT[p.dtype]
    args = [_ptr(x, "x", xdt, p.T * p.H),
            _ptr(x_scales, "x_scales", torch.float32, p.T * p.H // 128),
            _ptr(w13, "w13", _w_dtype(p), p.E * 2 * p.I * p.H),
            _ptr(w13_scales, "w13_scales", torch.float32, p.E * (2 * p.I // 128) * (p.H // 128)),
            _ptr(sorted_slots, "sorted_slots", torch.int32, rows),
            _ptr(offsets, "offsets", torch.int32, p.E + 1),
            _ptr(tiles, "tiles", torch.int32, 2 * moe_max_tiles(p)),
            _ptr(num_tiles, "num_tiles", torch.int32, 1),
            _ptr(act, "act", (_act_dtype(p), torch.float8_e4m3fn) if fp8 else _act_dtype(p), rows * p.I),
            _ptr(act_scales, "act_scales", torch.float32, rows * p.I // 128),
            _ptr(workspace, "workspace", torch.uint8),
            0 if workspace is None else workspace.numel() * workspace.element_size()]
    _checked(load().moe_grouped_gemm_up(ctypes.byref(p), *args, _stream(stream)),
             "moe_grouped_gemm_up")


def moe_grouped_gemm_up_mxfp4(p: Problem, x, x_scale, w13, w13_scales, bias, alpha: float,
                              limit: float, out_scale, sorted_slots, offsets, tiles, num_tiles,
                              act, stream=None) -> None:
    rows = moe_max_padded_slots(p)
    u8 = (torch.uint8, torch.float8_e4m3fn)
    args = [_ptr(x, "x", u8, p.T * p.H),
            _ptr(x_scale, "x_scale", torch.float32, 1),
            _ptr(w13, "w13", torch.uint8, p.E * 2 * p.I * p.H // 2),
            _ptr(w13_scales, "w13_scales", torch.uint8, p.E * (p.H // 32) * 2 * p.I),
            _ptr(bias, "bias", torch.float32, p.E * 2 * p.I),
            ctypes.c_float(alpha), ctypes.c_float(limit),
            _ptr(out_scale, "out_scale", torch.float32, 1),
            _ptr(sorted_slots, "sorted_slots", torch.int32, rows),
            _ptr(offsets, "offsets", torch.int32, p.E + 1),
            _ptr(tiles, "tiles", torch.int32, 2 * moe_max_tiles(p)),
            _ptr(num_tiles, "num_tiles", torch.int32, 1),
            _ptr(act, "act", u8, rows * p.I)]
    _checked(load().moe_grouped_gemm_up_mxfp4(ctypes.byref(p), *args, _stream(stream)),
             "moe_grouped_gemm_up_mxfp4")


def moe_grouped_gemm_down(p: Problem, act, act_scales, w2, w2_scales, topk_weights, sorted_slots,
                          offsets, tiles, num_tiles, slot_out, workspace=None, stream=None) -> None:
    rows = moe_max_padded_slots(p)
    fp8 = p.w_dtype == MOE_E4M3
    args = [_ptr(act, "act", (_act_dtype(p), torch.float8_e4m3fn) if fp8 else _act_dtype(p), rows * p.I),
            _ptr(act_scales, "act_scales", torch.float32, rows * p.I // 128),
            _ptr(w2, "w2", _w_dtype(p), p.E * p.H * p.I),
            _ptr(w2_scales, "w2_scales", torch.float32, p.E * (p.H // 128) * (p.I // 128)),
            _ptr(topk_weights, "topk_weights", torch.float32, p.T * p.top_k),
            _ptr(sorted_slots, "sorted_slots", torch.int32, rows),
            _ptr(offsets, "offsets", torch.int32, p.E + 1),
            _ptr(tiles, "tiles", torch.int32, 2 * moe_max_tiles(p)),
            _ptr(num_tiles, "num_tiles", torch.int32, 1),
            _ptr(slot_out, "slot_out", _TORCH_DT[p.dtype], p.T * p.top_k * p.H),
            _ptr(workspace, "workspace", torch.uint8),
            0 if workspace is None else workspace.numel() * workspace.element_size()]
    _checked(load().moe_grouped_gemm_down(ctypes.byref(p), *args, _stream(stream)),
             "moe_grouped_gemm_down")


def moe_combine(p: Problem, slot_out, slot_row, out, stream=None) -> None:
    args = [_ptr(slot_out, "slot_out", _TORCH_DT[p.dtype], p.T * p.top_k * p.H),
            _ptr(slot_row, "slot_row", torch.int32, p.T * p.top_k),
            _ptr(out, "out", _TORCH_DT[p.dtype], p.T * p.H)]
    _checked(load().moe_combine(ctypes.byref(p), *args, _stream(stream)), "moe_combine")


def moe_forward(p: Problem, x, topk_ids, topk_weights, w13, w13_scales, w2, w2_scales, out,
                workspace, stream=None) -> None:
    ws_bytes = moe_workspace_bytes(p)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        raise MoeError(MOE_ERR_WORKSPACE, "moe_forward")
    args = [_ptr(x, "x", _TORCH_DT[p.dtype], p.T * p.H),
            _ptr(topk_ids, "topk_ids", torch.int32, p.T * p.top_k),
            _ptr(topk_weights, "topk_weights", torch.float32, p.T * p.top_k),
            _ptr(w13, "w13", _w_dtype(p), p.E * 2 * p.I * p.H),
            _ptr(w13_scales, "w13_scales", torch.float32, p.E * (2 * p.I // 128) * (p.H // 128)),
            _ptr(w2, "w2", _w_dtype(p), p.E * p.H * p.I),
            _ptr(w2_scales, "w2_scales", torch.float32, p.E * (p.H // 128) * (p.I // 128)),
            _ptr(out, "out", _TORCH_DT[p.dtype], p.T * p.H),
            _ptr(workspace, "workspace")]
    _checked(load().moe_forward(ctypes.byref(p), *args, ctypes.c_size_t(ws_bytes), _stream(stream)),
             "moe_forward")


def moe_scratch_max_bytes() -> int:
    return int(load().moe_scratch_max_bytes())


def moe_forward_scratch(p: Problem, x, topk_ids, topk_weights, w13, w13_scales, w2, w2_scales,
                        out, n_invalid=None, stream=None) -> None:
    args = [_ptr(x, "x", _TORCH_DT[p.dtype], p.T * p.H),
            _ptr(topk_ids, "topk_ids", torch.int32, p.T * p.top_k),
            _ptr(topk_weights, "topk_weights", torch.float32, p.T * p.top_k),
            _ptr(w13, "w13", _w_dtype(p), p.E * 2 * p.I * p.H),
            _ptr(w13_scales, "w13_scales", torch.float32, p.E * (2 * p.I // 128) * (p.H // 128)),
            _ptr(w2, "w2", _w_dtype(p), p.E * p.H * p.I),
            _ptr(w2_scales, "w2_scales", torch.float32, p.E * (p.H // 128) * (p.I // 128)),
            _ptr(out, "out", _TORCH_DT[p.dtype], p.T * p.H),
            _ptr(n_invalid, "n_invalid", torch.int32, 1)]
    _checked(load().moe_forward_scratch(ctypes.byref(p), *args, _stream(stream)),
             "moe_forward_scratch")


# ---------------------------------------------------------------------------------------------
# rows in expert-sorted order, router, norm, products, gradients.  Every tensor of a call must be
# on the current device: the launch goes to that device's stream.  A call's host time is that of
# these checks next to 3.5 us of launch, so the common case of each is one expression (0.3 us a
# tensor) and only a tensor that fails it is looked at again, for the reason.
# ---------------------------------------------------------------------------------------------
_ROW_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float8_e4m3fn: MOE_E4M3,
           torch.uint8: MOE_E4M3}
_CODES = (torch.float8_e4m3fn, torch.uint8)
_F32, _I32, _BF16 = (torch.float32,), (torch.int32,), (torch.bfloat16,)
_OUT = (torch.bfloat16, torch.float32)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # None: torch without GPUs
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _row_dtype(t: torch.Tensor, name: str) -> int:
    dt = _ROW_DT.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if dt is None:
        raise ValueError(f"{name}: dtype {getattr(t, 'dtype', type(t))} not supported")
    return dt


def _arg(t: Optional[torch.Tensor], name: str, dtypes: tuple, numel: int, dev: int):
    """Device pointer of a contiguous tensor of `numel` elements on device `dev` (None: NULL)."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype in dtypes
            and t.numel() == numel and t.is_contiguous()):
        return t.data_ptr()
    _ptr(t, name, dtypes, numel, torch.device("cuda", dev))
    raise ValueError(f"{name}: not a dense tensor of {numel} elements on device {dev}")


def _mat(t: Optional[torch.Tensor], name: str, dtypes: tuple, shape: tuple, dev: int):
    """The same with the whole shape checked."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.get_device() == dev
            and t.dtype in dtypes and t.is_contiguous()):
        return t.data_ptr()
    if isinstance(t, torch.Tensor) and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _arg(t, name, dtypes, math.prod(shape), dev)


def _where(stream, dev: int):
    """The stream's handle; by default the current stream of `dev`."""
    if stream is None:
        return _raw_stream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"stream: of device {stream.device_index}, the current device is {dev}")
    return _stream(stream)


def _refuse_past_int32(where: str, *sizes: int) -> None:
    """Sizes read off a tensor, before ctypes would drop their upper bits."""
    if max(sizes) > 0x7FFFFFFF:
        raise MoeError(MOE_ERR_SHAPE, where)


def moe_permute(p: Problem, x, x_scales, slot_row, sorted_slots, num_tiles, rows, row_scales,
                stream=None) -> None:
    dt = _row_dtype(x, "x")
    same = _CODES if dt == MOE_E4M3 else (x.dtype,)
    rm = moe_max_padded_slots(p)
    dev = _device()
    T, H = p.T, p.H
    _checked(load().moe_permute(
        ctypes.byref(p), dt, _arg(x, "x", same, T * H, dev),
        _arg(x_scales, "x_scales", _F32, T * (H // 128), dev),
        _arg(slot_row, "slot_row", _I32, T * p.top_k, dev),
        _arg(sorted_slots, "sorted_slots", _I32, rm, dev),
        _arg(num_tiles, "num_tiles", _I32, 1, dev), _arg(rows, "rows", same, rm * H, dev),
        _arg(row_scales, "row_scales", _F32, rm * (H // 128), dev), _where(stream, dev)),
        "moe_permute")


def moe_unpermute(p: Problem, rows, slot_row, topk_weights, out, stream=None) -> None:
    dt = _row_dtype(rows, "rows")
    same = (rows.dtype,)
    dev = _device()
    T, H = p.T, p.H
    N = T * p.top_k
    _checked(load().moe_unpermute(
        ctypes.byref(p), dt, _arg(rows, "rows", same, moe_max_padded_slots(p) * H, dev),
        _arg(slot_row, "slot_row", _I32, N, dev),
        _arg(topk_weights, "topk_weights", _F32, N, dev), _arg(out, "out", same, T * H, dev),
        _where(stream, dev)), "moe_unpermute")


def moe_unpermute_bwd(p: Problem, d_out, rows, slot_row, sorted_slots, num_tiles, topk_weights,
                      d_rows, d_weights, stream=None) -> None:
    dt = _row_dtype(d_out, "d_out")
    same = (d_out.dtype,)
    rm = moe_max_padded_slots(p)
    dev = _device()
    T, H = p.T, p.H
    N = T * p.top_k
    _checked(load().moe_unpermute_bwd(
        ctypes.byref(p), dt, _arg(d_out, "d_out", same, T * H, dev),
        _arg(rows, "rows", same, rm * H, dev), _arg(slot_row, "slot_row", _I32, N, dev),
        _arg(sorted_slots, "sorted_slots", _I32, rm, dev),
        _arg(num_tiles, "num_tiles", _I32, 1, dev),
        _arg(topk_weights, "topk_weights", _F32, N, dev),
        _arg(d_rows, "d_rows", same, rm * H, dev), _arg(d_weights, "d_weights", _F32, N, dev),
        _where(stream, dev)), "moe_unpermute_bwd")


def moe_route_bwd(p: Problem, logits, renormalize: bool, topk_ids, d_weights, d_logits,
                  stream=None) -> None:
    dev = _device()
    T = p.T
    N, L = T * p.top_k, T * p.E
    _checked(load().moe_route_bwd(
        ctypes.byref(p), _arg(logits, "logits", _F32, L, dev), 1 if renormalize else 0,
        _arg(topk_ids, "topk_ids", _I32, N, dev), _arg(d_weights, "d_weights", _F32, N, dev),
        _arg(d_logits, "d_logits", _F32, L, dev), _where(stream, dev)), "moe_route_bwd")


def moe_quantize_cols_e4m3(x, xq, scales, stream=None) -> None:
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a matrix")
    m, n = x.shape
    _refuse_past_int32("moe_quantize_cols_e4m3", m, n)
    groups = -(-m // 128)
    dev = _device()
    _checked(load().moe_quantize_cols_e4m3(
        m, n, _arg(x, "x", _BF16, m * n, dev), _mat(xq, "xq", _CODES, (n, groups * 128), dev),
        _mat(scales, "scales", _F32, (n, groups), dev), _where(stream, dev)),
        "moe_quantize_cols_e4m3")


def moe_gemm_e4m3(a, a_scales, b, b_scales, b_block: int, c, stream=None) -> None:
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a: expected a matrix")
    if not isinstance(b, torch.Tensor) or b.dim() != 2:
        raise ValueError("b: expected a matrix")
    m, k = a.shape
    n = b.shape[0]
    _refuse_past_int32("moe_gemm_e4m3", m, n, k)
    if b_block != 1 and b_block != 128:           # it says how many b_scales there are
        raise MoeError(MOE_ERR_SHAPE, "moe_gemm_e4m3")
    g = k // 128
    dev = _device()
    _checked(load().moe_gemm_e4m3(
        m, n, k, _arg(a, "a", _CODES, m * k, dev), _mat(a_scales, "a_scales", _F32, (m, g), dev),
        _arg(b, "b", _CODES, n * k, dev),
        _mat(b_scales, "b_scales", _F32, (n if b_block == 1 else -(-n // 128), g), dev), b_block,
        _mat(c, "c", _OUT, (m, n), dev), _row_dtype(c, "c"), _where(stream, dev)),
        "moe_gemm_e4m3")


def moe_grouped_gemm_e4m3(p: Problem, rows, row_scales, w, w_scales, sorted_slots, offsets, tiles,
                          num_tiles, out, stream=None) -> None:
    if not isinstance(w, torch.Tensor) or w.dim() != 3 or w.shape[0] != p.E:
        raise ValueError("w: expected [E, n, k]")
    E, n, k = w.shape
    _refuse_past_int32("moe_grouped_gemm_e4m3", n, k)
    rm = moe_max_padded_slots(p)
    dev = _device()
    _checked(load().moe_grouped_gemm_e4m3(
        ctypes.byref(p), n, k, _mat(rows, "rows", _CODES, (rm, k), dev),
        _mat(row_scales, "row_scales", _F32, (rm, k // 128), dev),
        _arg(w, "w", _CODES, E * n * k, dev),
        _mat(w_scales, "w_scales", _F32, (E, -(-n // 128), k // 128), dev),
        _arg(sorted_slots, "sorted_slots", _I32, rm, dev),
        _arg(offsets, "offsets", _I32, E + 1, dev),
        _arg(tiles, "tiles", _I32, 2 * moe_max_tiles(p), dev),
        _arg(num_tiles, "num_tiles", _I32, 1, dev), _mat(out, "out", _OUT, (rm, n), dev),
        _row_dtype(out, "out"), _where(stream, dev)), "moe_grouped_gemm_e4m3")


# ---------------------------------------------------------------------------------------------
# router with scores, norm, bf16 products with an epilogue
# ---------------------------------------------------------------------------------------------
_LOGITS = (torch.float32, torch.bfloat16)


def moe_router_validate(p: Problem, r: Router) -> int:
    return load().moe_router_validate(ctypes.byref(p), ctypes.byref(r))


def moe_route_scored(p: Problem, r: Router, logits, bias, topk_ids, topk_weights,
                     stream=None) -> None:
    dt = _row_dtype(logits, "logits")
    dev = _device()
    T, N = p.T, p.T * p.top_k
    _checked(load().moe_route_scored(
        ctypes.byref(p), ctypes.byref(r), _arg(logits, "logits", _LOGITS, T * p.E, dev), dt,
        _arg(bias, "bias", _F32, p.E, dev), _arg(topk_ids, "topk_ids", _I32, N, dev),
        _arg(topk_weights, "topk_weights", _F32, N, dev), _where(stream, dev)),
        "moe_route_scored")


def moe_route_scored_bwd(p: Problem, r: Router, logits, topk_ids, d_weights, d_logits,
                         stream=None) -> None:
    dt = _row_dtype(logits, "logits")
    dev = _device()
    L, N = p.T * p.E, p.T * p.top_k
    _checked(load().moe_route_scored_bwd(
        ctypes.byref(p), ctypes.byref(r), _arg(logits, "logits", _LOGITS, L, dev), dt,
        _arg(topk_ids, "topk_ids", _I32, N, dev), _arg(d_weights, "d_weights", _F32, N, dev),
        _arg(d_logits, "d_logits", (logits.dtype,), L, dev), _where(stream, dev)),
        "moe_route_scored_bwd")


def _rows(x, name: str, where: str):
    shape = x.shape if isinstance(x, torch.Tensor) else ()
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a matrix")
    if (shape[0] | shape[1]) > 0x7FFFFFFF:
        raise MoeError(MOE_ERR_SHAPE, where)
    return shape


def moe_rms_norm(x, residual, weight, eps: float, sum, y, codes, scales, rstd,
                 stream=None) -> None:
    t, h = shape = _rows(x, "x", "moe_rms_norm")
    dt = _row_dtype(x, "x")
    same = (x.dtype,)
    dev = _device()
    _checked(load().moe_rms_norm(
        t, h, dt, _arg(x, "x", same, t * h, dev), _mat(residual, "residual", same, shape, dev),
        _arg(weight, "weight", same, h, dev), eps, _mat(sum, "sum", same, shape, dev),
        _mat(y, "y", same, shape, dev), _mat(codes, "codes", _CODES, shape, dev),
        _mat(scales, "scales", _F32, (t, h // 128), dev), _arg(rstd, "rstd", _F32, t, dev),
        _where(stream, dev)), "moe_rms_norm")


def moe_rms_norm_bwd_workspace_bytes(t: int, h: int) -> int:
    _refuse_past_int32("moe_rms_norm_bwd_workspace_bytes", t, h)
    return _checked(load().moe_rms_norm_bwd_workspace_bytes(t, h),
                    "moe_rms_norm_bwd_workspace_bytes")


def _space(workspace, dev: int):
    """Pointer and size of an optional workspace."""
    if workspace is None:
        return None, 0
    return (_arg(workspace, "workspace", (torch.uint8,), workspace.numel(), dev),
            workspace.numel())


def moe_rms_norm_bwd(d_y, d_sum, s, weight, rstd, d_x, d_weight, workspace, stream=None) -> None:
    t, h = shape = _rows(d_y, "d_y", "moe_rms_norm_bwd")
    dt = _row_dtype(d_y, "d_y")
    same = (d_y.dtype,)
    dev = _device()
    _checked(load().moe_rms_norm_bwd(
        t, h, dt, _arg(d_y, "d_y", same, t * h, dev), _mat(d_sum, "d_sum", same, shape, dev),
        _mat(s, "s", same, shape, dev), _arg(weight, "weight", same, h, dev),
        _arg(rstd, "rstd", _F32, t, dev), _mat(d_x, "d_x", same, shape, dev),
        _arg(d_weight, "d_weight", _F32, h, dev), *_space(workspace, dev), _where(stream, dev)),
        "moe_rms_norm_bwd")


def _named(value, names: dict, what: str) -> int:
    """The number of a name; a number stands for itself."""
    if isinstance(value, str):
        raise ValueError(f"{what}: {value!r}, expected one of {', '.join(names)}")
    return int(value)


def moe_gemm_bf16(layout, a, b, bias, act, residual, pre, c, stream=None) -> None:
    lay = _LAYOUT.get(layout)
    if lay is None:
        lay = _named(layout, _LAYOUT, "layout")
        if lay not in _LAYOUT.values():
            raise MoeError(MOE_ERR_SHAPE, "moe_gemm_bf16")
    ac = _ACT.get(act)
    if ac is None:
        ac = _named(act, _ACT, "act")
    a0, a1 = _rows(a, "a", "moe_gemm_bf16")
    b0, b1 = _rows(b, "b", "moe_gemm_bf16")
    m, k = (a1, a0) if lay == MOE_TN else (a0, a1)
    n, kb = (b0, b1) if lay == MOE_NT else (b1, b0)
    if k != kb:
        raise ValueError(f"b: shape {tuple(b.shape)}, its k is {kb}, that of a is {k}")
    dev = _device()
    shape = (m, n)
    dt = _row_dtype(c, "c")
    _checked(load().moe_gemm_bf16(
        m, n, k, lay, _arg(a, "a", _BF16, m * k, dev), _arg(b, "b", _BF16, n * k, dev),
        _arg(bias, "bias", _F32, n, dev), ac, _mat(residual, "residual", (c.dtype,), shape, dev),
        _mat(pre, "pre", _BF16, shape, dev), _mat(c, "c", _OUT, shape, dev), dt,
        _where(stream, dev)), "moe_gemm_bf16")


def moe_act_bwd_workspace_bytes(m: int, n: int) -> int:
    _refuse_past_int32("moe_act_bwd_workspace_bytes", m, n)
    return _checked(load().moe_act_bwd_workspace_bytes(m, n), "moe_act_bwd_workspace_bytes")


def moe_act_bwd(act, d_c, pre, d_z, d_bias, workspace, stream=None) -> None:
    m, n = shape = _rows(d_c, "d_c", "moe_act_bwd")
    dev = _device()
    ac = _ACT.get(act)
    if ac is None:
        ac = _named(act, _ACT, "act")
    _checked(load().moe_act_bwd(
        m, n, ac, _arg(d_c, "d_c", _BF16, m * n, dev),
        _mat(pre, "pre", _BF16, shape, dev), _mat(d_z, "d_z", _BF16, shape, dev),
        _arg(d_bias, "d_bias", _F32, n, dev), *_space(workspace, dev), _where(stream, dev)),
        "moe_act_bwd")
