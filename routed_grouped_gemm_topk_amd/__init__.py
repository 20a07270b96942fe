"""MI355X (gfx950) routed grouped-GEMM top-k MoE expert layer.

The computation lives in libmoe.so (hand-written HIP kernels behind the C ABI of
include/moe.h).  This package is its Python binding: ``_lib`` mirrors the C
entry points one to one; the helpers below only allocate buffers with torch
and call them.  Nothing here records for automatic differentiation: results have
no graph, also where an input requires a gradient; the gradients (unpermute_bwd,
route_bwd, route_scored_bwd, rms_norm_bwd, act_bwd, the products of moe_gemm_bf16
and moe_gemm_e4m3 in moe.h) are the caller's to run.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch

from ._lib import (  # noqa: F401
    EXPORTS,
    LIB_PATH,
    MOE_ACT_GELU,
    MOE_ACT_GELU_TANH,
    MOE_ACT_NONE,
    MOE_ACT_SILU,
    MOE_BF16,
    MOE_E4M3,
    MOE_ERR_ALIGN,
    MOE_ERR_DEVICE,
    MOE_ERR_DTYPE,
    MOE_ERR_LAUNCH,
    MOE_ERR_NULL,
    MOE_ERR_SHAPE,
    MOE_ERR_WORKSPACE,
    MOE_F32,
    MOE_MXFP4,
    MOE_NN,
    MOE_NT,
    MOE_OK,
    MOE_SCORE_SIGMOID,
    MOE_SCORE_SOFTMAX,
    MOE_TN,
    MoeError,
    Problem,
    Router,
    load,
    make_problem,
    make_router,
    moe_act_bwd,
    moe_act_bwd_workspace_bytes,
    moe_align,
    moe_block_m_for,
    moe_combine,
    moe_gemm_workspace_bytes,
    moe_forward,
    moe_forward_scratch,
    moe_gemm_bf16,
    moe_gemm_e4m3,
    moe_grouped_gemm_down,
    moe_grouped_gemm_e4m3,
    moe_grouped_gemm_up,
    moe_grouped_gemm_up_mxfp4,
    moe_max_padded_slots,
    moe_max_tiles,
    moe_permute,
    moe_pick_block_m,
    moe_quantize_cols_e4m3,
    moe_quantize_rows_e4m3,
    moe_rms_norm,
    moe_rms_norm_bwd,
    moe_rms_norm_bwd_workspace_bytes,
    moe_route,
    moe_route_align,
    moe_route_bwd,
    moe_route_scored,
    moe_route_scored_bwd,
    moe_router_validate,
    moe_scratch_max_bytes,
    moe_unpermute,
    moe_unpermute_bwd,
    moe_validate,
    moe_workspace_bytes,
    status_str,
    _where,
)


def alloc_align(p: Problem, device) -> dict:
    rows, mt = moe_max_padded_slots(p), moe_max_tiles(p)
    z = lambda n: torch.empty(n, dtype=torch.int32, device=device)  # noqa: E731
    return {"counts": z(p.E), "offsets": z(p.E + 1), "sorted_slots": z(rows),
            "slot_row": z(p.T * p.top_k), "tiles": z(2 * mt), "num_tiles": z(1),
            "n_invalid": z(1)}


def align(p: Problem, topk_ids: torch.Tensor, stream=None) -> dict:
    """Run moe_align into freshly allocated buffers; returns them by name."""
    a = alloc_align(p, topk_ids.device)
    moe_align(p, topk_ids, a["counts"], a["offsets"], a["sorted_slots"], a["slot_row"],
              a["tiles"], a["num_tiles"], a["n_invalid"], stream)
    return a


def route(p: Problem, logits: torch.Tensor, renormalize: bool, stream=None):
    """Run moe_route into fresh buffers; returns (topk_ids int32 [T,k], topk_weights fp32 [T,k])."""
    ids = torch.empty((p.T, p.top_k), dtype=torch.int32, device=logits.device)
    w = torch.empty((p.T, p.top_k), dtype=torch.float32, device=logits.device)
    moe_route(p, logits, renormalize, ids, w, stream)
    return ids, w


def route_align(p: Problem, logits: torch.Tensor, renormalize: bool, stream=None) -> dict:
    """Run moe_route_align into fresh buffers; returns align()'s buffers plus topk_ids and
    topk_weights."""
    a = alloc_align(p, logits.device)
    a["topk_ids"] = torch.empty((p.T, p.top_k), dtype=torch.int32, device=logits.device)
    a["topk_weights"] = torch.empty((p.T, p.top_k), dtype=torch.float32, device=logits.device)
    moe_route_align(p, logits, renormalize, a["topk_ids"], a["topk_weights"], a["counts"],
                    a["offsets"], a["sorted_slots"], a["slot_row"], a["tiles"], a["num_tiles"],
                    a["n_invalid"], stream)
    return a


def alloc_workspace(p: Problem, device) -> torch.Tensor:
    return torch.empty(moe_workspace_bytes(p), dtype=torch.uint8, device=device)


def alloc_gemm_workspace(p: Problem, device) -> Optional[torch.Tensor]:
    """The optional workspace of moe_grouped_gemm_up / _down (None when the problem's GEMMs
    use none)."""
    n = moe_gemm_workspace_bytes(p)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def forward(p: Problem, x, topk_ids, topk_weights, w13, w2, w13_scales=None, w2_scales=None,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """The whole layer through moe_forward.  Allocates `out` / `workspace` if not given."""
    if out is None:
        out = torch.empty((p.T, p.H), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(p, x.device)
    moe_forward(p, x, topk_ids, topk_weights, w13, w13_scales, w2, w2_scales, out, workspace,
                stream)
    return out


# ---------------------------------------------------------------------------------------------
# rows in expert-sorted order, gradients, products of e4m3 codes.  `a` is the alignment that
# align() or route_align() returns for the same problem.
# ---------------------------------------------------------------------------------------------
def _new(like: torch.Tensor, shape, dtype: torch.dtype, stream) -> torch.Tensor:
    """A matrix allocated on the stream that the call runs on, so that its memory belongs to it."""
    if stream is None:          # torch's fastest way to one: 1.3 us against 1.6
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=like.device)
    dev = torch.cuda.current_device()
    if not isinstance(stream, torch.cuda.Stream):
        # 0 names the default stream; ExternalStream(0) would be one of torch's pool streams
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream(dev)
    _where(stream, dev)                                  # of the current device, or refused
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _vec(like: torch.Tensor, n: int, dtype: torch.dtype, stream) -> torch.Tensor:
    """The same for n values in a row."""
    if stream is None:
        return torch.empty_strided((n,), (1,), dtype=dtype, device=like.device)
    return _new(like, (1, n), dtype, stream).view(n)


def permute(p: Problem, x: torch.Tensor, a: dict, x_scales: Optional[torch.Tensor] = None,
            rows: Optional[torch.Tensor] = None, row_scales: Optional[torch.Tensor] = None,
            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Token rows (fp32, bf16 or e4m3 codes with optional scales per 128 columns) in
    expert-sorted order through moe_permute; returns (rows, row_scales or None)."""
    if rows is None:
        rows = _new(x, (moe_max_padded_slots(p), p.H), x.dtype, stream)
    if row_scales is None and x_scales is not None:
        row_scales = _new(x, (moe_max_padded_slots(p), p.H // 128), torch.float32, stream)
    moe_permute(p, x, x_scales, a["slot_row"], a["sorted_slots"], a["num_tiles"], rows,
                row_scales, stream)
    return rows, row_scales


def unpermute(p: Problem, rows: torch.Tensor, a: dict,
              topk_weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Expert-sorted rows added per token with the routing weights (1 without them: the gradient
    of permute) through moe_unpermute."""
    if out is None:
        out = _new(rows, (p.T, p.H), rows.dtype, stream)
    moe_unpermute(p, rows, a["slot_row"], topk_weights, out, stream)
    return out


def unpermute_bwd(p: Problem, d_out: torch.Tensor, rows: torch.Tensor, a: dict,
                  topk_weights: Optional[torch.Tensor] = None,
                  d_rows: Optional[torch.Tensor] = None,
                  d_weights: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradient of unpermute through moe_unpermute_bwd; returns (d_rows, d_weights)."""
    if d_rows is None:
        d_rows = _new(d_out, (moe_max_padded_slots(p), p.H), d_out.dtype, stream)
    if d_weights is None:
        d_weights = _new(d_out, (p.T, p.top_k), torch.float32, stream)
    moe_unpermute_bwd(p, d_out, rows, a["slot_row"], a["sorted_slots"], a["num_tiles"],
                      topk_weights, d_rows, d_weights, stream)
    return d_rows, d_weights


def route_bwd(p: Problem, logits: torch.Tensor, renormalize: bool, topk_ids: torch.Tensor,
              d_weights: torch.Tensor, d_logits: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Gradient of route's weights with respect to the logits through moe_route_bwd."""
    if d_logits is None:
        d_logits = (torch.empty_like(logits) if stream is None
                    else _new(logits, logits.shape, torch.float32, stream))
    moe_route_bwd(p, logits, renormalize, topk_ids, d_weights, d_logits, stream)
    return d_logits


def quantize_cols_e4m3(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Transposed quantisation of a bf16 matrix [m, n] through moe_quantize_cols_e4m3; returns
    (codes [n, mp], scales [n, mp/128]), mp = m rounded up to 128."""
    m, n = x.shape
    groups = -(-m // 128)
    xq = _new(x, (n, groups * 128), torch.float8_e4m3fn, stream)
    scales = _new(x, (n, groups), torch.float32, stream)
    moe_quantize_cols_e4m3(x, xq, scales, stream)
    return xq, scales


def gemm_e4m3(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16, b_block: int = 128,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a [m, k] times b [n, k] transposed, both e4m3 codes with one scale per 128 values along k,
    through moe_gemm_e4m3."""
    if out is None:
        out = _new(a, (a.shape[0], b.shape[0]), out_dtype, stream)
    moe_gemm_e4m3(a, a_scales, b, b_scales, b_block, out, stream)
    return out


def grouped_gemm_e4m3(p: Problem, rows: torch.Tensor, row_scales: torch.Tensor, w: torch.Tensor,
                      w_scales: torch.Tensor, a: dict, out_dtype: torch.dtype = torch.bfloat16,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Expert-sorted rows (e4m3 codes) times their experts' w [E, n, k] transposed, through
    moe_grouped_gemm_e4m3."""
    if out is None:
        out = _new(rows, (moe_max_padded_slots(p), w.shape[1]), out_dtype, stream)
    moe_grouped_gemm_e4m3(p, rows, row_scales, w, w_scales, a["sorted_slots"], a["offsets"],
                          a["tiles"], a["num_tiles"], out, stream)
    return out


# ---------------------------------------------------------------------------------------------
# before the layer and beside it: router with scores, norm, bf16 products with an epilogue
# ---------------------------------------------------------------------------------------------
def route_scored(p: Problem, r: Router, logits: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Experts and weights by scores (fp32 or bf16 logits), with a bias for balance and groups,
    through moe_route_scored; returns (topk_ids int32 [T,k], topk_weights fp32 [T,k])."""
    ids = _new(logits, (p.T, p.top_k), torch.int32, stream)
    w = _new(logits, (p.T, p.top_k), torch.float32, stream)
    moe_route_scored(p, r, logits, bias, ids, w, stream)
    return ids, w


def route_scored_bwd(p: Problem, r: Router, logits: torch.Tensor, topk_ids: torch.Tensor,
                     d_weights: torch.Tensor, d_logits: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Gradient of route_scored's weights with respect to the logits through
    moe_route_scored_bwd."""
    if d_logits is None:
        d_logits = _new(logits, (p.T, p.E), logits.dtype, stream)
    moe_route_scored_bwd(p, r, logits, topk_ids, d_weights, d_logits, stream)
    return d_logits


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             want: Sequence[str] = ("y",), sum: Optional[torch.Tensor] = None,
             stream=None) -> dict:
    """Root-mean-square norm of the rows of x (plus residual) through moe_rms_norm.  `want` names
    the outputs: "y" (rows), "codes" (e4m3 codes, with "scales" per 128 columns) and "rstd" (for
    rms_norm_bwd); with a residual "sum" comes too, in `sum` if given (residual or x, say)."""
    shape = t, h = x.shape
    out = {}
    if residual is not None:
        out["sum"] = sum if sum is not None else _new(x, shape, x.dtype, stream)
    elif sum is not None:
        raise ValueError("sum: given without a residual")
    for name in want:
        if name == "y":
            out["y"] = _new(x, shape, x.dtype, stream)
        elif name == "codes":
            out["codes"] = _new(x, shape, torch.float8_e4m3fn, stream)
            out["scales"] = _new(x, (t, h // 128), torch.float32, stream)
        elif name == "rstd":
            out["rstd"] = _vec(x, t, torch.float32, stream)
        else:
            raise ValueError(f"want: {name!r}, expected 'y', 'codes' or 'rstd'")
    get = out.get
    moe_rms_norm(x, residual, weight, eps, get("sum"), get("y"), get("codes"), get("scales"),
                 get("rstd"), stream)
    return out


def rms_norm_bwd(d_y: torch.Tensor, s: torch.Tensor, weight: Optional[torch.Tensor],
                 rstd: torch.Tensor, d_sum: Optional[torch.Tensor] = None, d_weight: bool = True,
                 d_x: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of rms_norm's y through moe_rms_norm_bwd, from the rows s that it was taken of
    ("sum", or x without a residual), its rstd, and d_sum, the gradient that reaches s otherwise;
    returns (d_x, the gradient of the rows and of the residual; d_weight fp32, None if not asked
    for)."""
    t, h = d_y.shape
    if d_x is None:
        d_x = _new(d_y, (t, h), d_y.dtype, stream)
    dw = None
    if d_weight:
        dw = _vec(d_y, h, torch.float32, stream)
        if workspace is None:
            workspace = _vec(d_y, moe_rms_norm_bwd_workspace_bytes(t, h), torch.uint8, stream)
    moe_rms_norm_bwd(d_y, d_sum, s, weight, rstd, d_x, dw, workspace if d_weight else None, stream)
    return d_x, dw


def gemm_bf16(a: torch.Tensor, b: torch.Tensor, layout: str = "nt",
              bias: Optional[torch.Tensor] = None, act: str = "none",
              residual: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
              with_pre: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """act(a b + bias) + residual through moe_gemm_bf16; layout "nt": a [m,k], b [n,k]; "nn":
    a [m,k], b [k,n]; "tn": a [k,m], b [k,n].  bias fp32 [n]; residual as the output.  with_pre:
    returns (out, pre), pre the bf16 values before the activation, for act_bwd."""
    shape = (a.shape[1] if layout in ("tn", MOE_TN) else a.shape[0],
             b.shape[0] if layout in ("nt", MOE_NT) else b.shape[1])
    if out is None:
        out = _new(a, shape, out_dtype, stream)
    pre = _new(a, shape, torch.bfloat16, stream) if with_pre else None
    moe_gemm_bf16(layout, a, b, bias, act, residual, pre, out, stream)
    return (out, pre) if with_pre else out


def act_bwd(d_c: torch.Tensor, pre: Optional[torch.Tensor] = None, act: str = "none",
            d_bias: bool = False, d_z: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None,
            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of gemm_bf16's epilogue through moe_act_bwd; returns (d_z, which is d_c itself
    without an activation; the bias' gradient fp32 [n], None if not asked for)."""
    m, n = d_c.shape
    none = act in ("none", MOE_ACT_NONE)
    if none and d_z is not None:
        raise ValueError("d_z: given without an activation, where it is d_c itself")
    if none and not d_bias:
        return d_c, None
    if none:                    # nothing to multiply with: d_z is d_c
        pre = None
    elif d_z is None:
        d_z = _new(d_c, (m, n), torch.bfloat16, stream)
    db = None
    if d_bias:
        db = _vec(d_c, n, torch.float32, stream)
        if workspace is None:
            workspace = _vec(d_c, moe_act_bwd_workspace_bytes(m, n), torch.uint8, stream)
    moe_act_bwd(act, d_c, pre, d_z, db, workspace if d_bias else None, stream)
    return (d_c if none else d_z), db
