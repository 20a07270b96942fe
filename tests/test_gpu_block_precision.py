"""What the operators before the layer and beside it promise of 64 bits, where 32 would not do: groups whose
large scores cancel, weights and gradients of the router rounded once; and GELU far below 0.

Tolerances (u = 2^-24, half a step of fp32, relative; 2^-150 absolute below fp32's normal numbers):
  * the router's weights and the gradient of its logits: sums of at most 1024 terms in 64 bits, each off
    by a few 2^-53, stay within 2^-40 of the terms' magnitudes; then one rounding to fp32, and for bf16
    one more from there.
  * GELU and its slope: the part of a normal distribution below -|z| is a ratio of at most 10 u times an
    exponential, 3 u and, where z is no bf16 value, z^2 / 2 u for the rounding of its argument; two
    products more, and above 0 a difference from at least twice as much: (z^2 / 2 + 16) u.  A slope's other
    part, z phi(z): 8 u.  Exponentials below 2^-126 count as 0: at most 14 of them.
"""
import math

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_block_operators import (F64, ROUTERS, TD, U32, UBF, WAYS, close, make_logits, ref_route, scores,
                                      weights_of)
from test_gpu_operators import gen, say

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------
# groups whose values cancel
# ---------------------------------------------------------------------------------------------
def same_choice(p, r, x, bias, k, what):
    ids, w = moe.route_scored(p, r, x, bias)
    ref_ids, ref_w = ref_route(x.cpu(), bias.cpu(), r, k)
    wrong = (ids.cpu().long() != ref_ids).any(1)
    assert not wrong.any(), (what, int(wrong.sum()), ids[wrong.to(ids.device)][:3], ref_ids[wrong][:3])
    close(w.cpu(), ref_w, (50 + k) * U32 * ref_w.abs(), "weights")


def test_route_scored_a_group_whose_values_cancel(device):
    """Group 0 adds 1000 + s and s - 1000, in fp32 3e-5 too much (too little): it is not the last one kept
    nor the first one dropped, and yet its error decides."""
    p = moe.make_problem(1, 64, 64, 6, 1, "bf16")
    r = moe.make_router("sigmoid", True, 3, 2, 2)
    bias = torch.tensor([1000.0, -1000.0, 0, 0, 0, 0], device=device)
    for first, rest in [(1.28e-4, (1e-4, 8e-5)), (1.2e-4, (2e-5, 4e-5))]:
        x = torch.tensor([[first, 0.0, rest[0], rest[0], rest[1], rest[1]]], device=device)
        say("cancelling group", first)
        same_choice(p, r, x, bias, 1, first)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [3e1, 1e3, 1e5, 1e6])
def test_route_scored_forced_and_masked_experts(device, score, size):
    """A bias that forces one expert of a group and masks its others, next to groups a few 1e-6 of a
    score apart."""
    T, E, G = 4000, 64, 8
    x = 1e-4 * torch.randn((T, E), generator=gen(device, 140), device=device)
    for forced in ((0,), (5,), (2, 3, 7)):
        bias = torch.zeros(E, device=device)
        for g in forced:
            bias[g * 8:g * 8 + 8] = -size
            bias[g * 8 + 3] = size
        for k, kept, top in [(1, 4, 2), (1, 1, 2), (8, 1, 2), (8, 7, 2), (8, 4, 2), (8, 3, 1)]:
            say("forced", score, size, forced, k, kept, top)
            r = moe.make_router(score, True, G, kept, top)
            p = moe.make_problem(T, 64, 64, E, k, "bf16")
            same_choice(p, r, x, bias, k, (forced, k, kept, top))


# ---------------------------------------------------------------------------------------------
# weights and gradient of the router
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("way", WAYS, ids=str)
@pytest.mark.parametrize("c", ROUTERS, ids=str)
def test_route_scored_weights_rounded_once(device, c, way):
    T, E, k, G, kept, top = c
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    for kind in ("plain", "ties", "holes", "far"):
        for dtype in ("f32", "bf16"):
            x = make_logits(c, dtype, device, kind, 1)
            for bias in (None, 0.1 * torch.randn(E, generator=gen(device, 2), device=device)):
                say("weights", c, way, kind, dtype, bias is None)
                r = moe.make_router(*way, G, kept, top, 2.5)
                ids, w = moe.route_scored(p, r, x, bias)
                v, s = scores(x.cpu(), way[0] == "sigmoid")
                i = ids.cpu().long()
                if way == ("softmax", True):             # ratios of the chosen, however small
                    m = torch.where(i >= 0, torch.gather(v, 1, i.clamp(min=0)), -math.inf).amax(1, True)
                    s = torch.exp(v - torch.where(torch.isinf(m), 0.0, m))
                ref = weights_of(s, i, r)
                close(w.cpu(), ref, (U32 + 2.0 ** -40) * ref.abs() + 2.0 ** -149, "weights")


def formula_bwd(x, ids, dw, r):
    """Gradient of the logits in 64 bits as moe.h writes it, and the magnitudes of its terms."""
    v, s = scores(x, r.score == moe.MOE_SCORE_SIGMOID)
    T, E = v.shape
    ok = (ids >= 0) & (ids < E)
    i = torch.where(ok, ids, 0).long()
    ok = ok & (torch.gather(v, 1, i) > -math.inf)
    dw = torch.where(ok, dw.to(F64), 0.0)
    p = torch.where(ok, torch.gather(s, 1, i), 0.0)
    if r.renormalize:
        if r.score == moe.MOE_SCORE_SOFTMAX:
            m = torch.where(ok, torch.gather(v, 1, i), -math.inf).amax(1, keepdim=True)
            p = torch.where(ok, torch.exp(torch.gather(v, 1, i) - torch.where(torch.isinf(m), 0.0, m)), 0.0)
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    mean, size = (p * dw).sum(1, keepdim=True), (p * dw).abs().sum(1, keepdim=True)
    rest = torch.sigmoid(-torch.gather(v, 1, i)) if r.score == moe.MOE_SCORE_SIGMOID else 1.0
    term, mag = p * rest * dw, p * rest * dw.abs()
    if r.renormalize:
        term, mag = term - p * rest * mean, mag + p * rest * size
    zero = torch.zeros((T, E), dtype=F64)
    d, m = zero.scatter_add(1, i, torch.where(ok, term, 0.0)), zero.scatter_add(1, i, mag)
    if r.score == moe.MOE_SCORE_SOFTMAX and not r.renormalize:
        d, m = d - s * mean, m + s * size
    return r.scale * d, r.scale * m


@pytest.mark.parametrize("way", WAYS, ids=str)
@pytest.mark.parametrize("c", ROUTERS, ids=str)
def test_route_scored_bwd_rounded_once(device, c, way):
    T, E, k, G, kept, top = c
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    for kind in ("plain", "holes", "far", "twice"):
        for dtype in ("f32", "bf16"):
            say("route_scored_bwd", c, way, kind, dtype)
            x = make_logits(c, dtype, device, kind, 3)
            r = moe.make_router(*way, G, kept, top, 2.5)
            ids = moe.route_scored(p, r, x)[0]
            if kind == "twice":
                ids = ids[:, :1].expand(T, k).contiguous()
            dw = torch.randn((T, k), generator=gen(device, 4), device=device)
            d = moe.route_scored_bwd(p, r, x, ids, dw)
            ref, size = formula_bwd(x.cpu(), ids.cpu(), dw.cpu(), r)
            u = U32 if dtype == "f32" else UBF + 2 * U32
            close(d.cpu(), ref, u * ref.abs() + 2.0 ** -40 * size + 2.0 ** -133, "d_logits")


def test_route_scored_bwd_of_tiny_scores(device):
    """Shares down to exp(-100), which fp32 holds with few bits or none, times a scale of 2^60."""
    T, E, k = 40, 96, 4
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    x = -80.0 - 20.0 * torch.rand((T, E), generator=gen(device, 142), device=device)
    x[:, 5] = 0.0
    r = moe.make_router("softmax", False, scale=2.0 ** 60)
    ids = moe.route_scored(p, r, x)[0]
    dw = torch.randn((T, k), generator=gen(device, 143), device=device)
    d = moe.route_scored_bwd(p, r, x, ids, dw)
    ref, size = formula_bwd(x.cpu(), ids.cpu(), dw.cpu(), r)
    assert float(ref[:, 6:].abs().min()) > 2.0 ** -126
    close(d.cpu(), ref, U32 * ref.abs() + 2.0 ** -40 * size, "d_logits")


# ---------------------------------------------------------------------------------------------
# GELU below 0
# ---------------------------------------------------------------------------------------------
TINY = 2.0 ** -126


@pytest.mark.parametrize("m,n", [(1, 4096), (1, 4095), (70, 1000), (300, 8192)])
def test_gelu_keeps_its_digits_below_zero(device, m, n):
    z = torch.linspace(-13, 13, n, device=device)
    z[n // 2] = 0
    a, b = (torch.zeros(s, device=device).bfloat16() for s in ((m, 8), (n, 8)))
    z64 = z.to(F64)
    ref = 0.5 * z64 * torch.erfc(-z64 * math.sqrt(0.5))
    tol = (z64 * z64 / 2 + 16) * U32 * ref.abs() + TINY
    for dtype in ("f32", "bf16"):
        say("gelu", m, n, dtype)
        c = moe.gemm_bf16(a, b, bias=z, act="gelu", out_dtype=TD[dtype])
        close(c, ref.expand(m, n), (tol + (UBF * ref.abs() if dtype == "bf16" else 0)).expand(m, n), "gelu")


def test_gelu_of_far_and_special_values(device):
    z = torch.tensor([-1e38, -1e19, -1e4, -200.0, -30.0, -14.5, 0.0, 14.5, 1e4, 1e19, 1e38, math.inf, math.nan],
                     device=device)
    a, b = (torch.zeros(s, device=device).bfloat16() for s in ((2, 8), (z.numel(), 8)))
    c = moe.gemm_bf16(a, b, bias=z, act="gelu", out_dtype=torch.float32)
    ref = torch.where(z < 0, 0.0, z).to(F64)
    close(c, ref.expand(2, -1), TINY, "gelu")


def test_gelu_slope_keeps_its_digits_below_zero(device):
    """A row of d_c of ones: d_bias is the slope itself, in fp32."""
    z = torch.linspace(-13, 13, 8191, device=device).bfloat16()
    z64 = z.to(F64)
    cdf = 0.5 * torch.erfc(-z64 * math.sqrt(0.5))
    tail = z64 * torch.exp(-0.5 * z64 * z64) / math.sqrt(2 * math.pi)
    ref = cdf + tail
    tol = (16 * cdf + 8 * tail.abs() + ref.abs()) * U32 + 16 * TINY
    dz, db = moe.act_bwd(torch.ones_like(z)[None], z[None], "gelu", d_bias=True)
    close(db, ref, tol, "slope")
    close(dz[0], ref, tol + UBF * ref.abs(), "d_z")
