"""MI355X (gfx950) routed grouped-GEMM top-k MoE expert layer.

The computation lives in libmoe.so (hand-written HIP kernels behind the C ABI of
include/moe.h).  This package is its Python binding: ``_lib`` mirrors the C
entry points one to one; the helpers below only allocate buffers with torch
and call them.  Nothing here records for automatic differentiation: results have
no graph, also where an input requires a gradient; unpermute_bwd, route_bwd and
the products of the gradients (moe_gemm_e4m3 in moe.h) are the caller's to run.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._lib import (  # noqa: F401
    EXPORTS,
    LIB_PATH,
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
    MOE_OK,
    MoeError,
    Problem,
    load,
    make_problem,
    moe_align,
    moe_block_m_for,
    moe_combine,
    moe_gemm_workspace_bytes,
    moe_forward,
    moe_forward_scratch,
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
    moe_route,
    moe_route_align,
    moe_route_bwd,
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
