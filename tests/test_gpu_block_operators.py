"""The operators before the layer and beside it on the GPU, against plain computations in 64 bits.

Tolerances count roundings (u = half a step, relative: 2^-24 fp32, 2^-8 bf16):
  * route_scored: the ids are those of 64-bit scores, exactly.  Weights: a score 5 u, a sum the
    error of its terms and at most 32 + 6 additions over all experts, or k - 1 + 6 over the chosen
    ones, a quotient and the scale 2 u: (50 + k) u.
  * route_scored_bwd: a slot's term is computed in 64 bits and rounded once; softmax without
    renormalisation subtracts p_e G with p in fp32 (the rounding of l - m costs |l - m| u of a
    term, at most 8 u of the sum, expf 2 u, at most 16 + 6 additions: 40 u) and adds one rounding.
  * rms_norm: sum one fp32 addition and one rounding, as torch does it: bit for bit.  rstd from 64
    bits: 2 u.  n two more products: 4 u.  A code is as near n / scale as the nearest one, but for
    the error of n and of the quotient: 6 u of the quotient.
  * rms_norm_bwd: d_x at most 6 roundings of its parts and the mean's: 32 products of a thread
    one after another, 6 + 16 additions across threads.  d_w: the rows of a workgroup one after
    another (at least 256 workgroups, or one per set of at most 4 rows), then at most 4 + 32 + 16.
  * gemm_bf16: products of bf16 values are exact in fp32 and at most k additions of 2 u each make a
    sum: 2 k u of the sum of magnitudes.  That is far above what random operands show, so the norm
    of the error is held as well: k independent roundings of at most 2 u of the result's own size
    add up to 2 u sqrt(k).  With operands that are small integers every sum is exact.  Functions of
    the epilogue: slopes of at most 1.13 times the error of z, and 8 u of |z| of their own.
  * act_bwd: slopes are sums of at most two terms of a few roundings: 12 u (1 + |z|) of d_c.
"""
import math

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_operators import E4M3, Guarded, close, gen, say

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8
TD = {"f32": torch.float32, "bf16": torch.bfloat16}
UT = {"f32": 0.0, "bf16": UBF}
F64 = torch.float64
TINY = 2.0 ** -126                       # below it fp32 steps are no longer relative


# ---------------------------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------------------------
def scores(logits, sigmoid):
    v = logits.to(F64)
    v = torch.where(torch.isnan(v), -math.inf, v).clamp(max=torch.finfo(torch.float32).max)
    if sigmoid:
        return v, torch.sigmoid(v)
    m = v.amax(1, keepdim=True)
    e = torch.exp(v - torch.where(torch.isinf(m), 0.0, m))
    return v, e / e.sum(1, keepdim=True).clamp(min=5e-324)


def weights_of(s, ids, r):
    """Weights of the chosen ids (-1: none) from scores in 64 bits."""
    w = torch.where(ids >= 0, torch.gather(s, 1, ids.clamp(min=0).long()), 0.0)
    if r.renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return w * r.scale


def ref_route(logits, bias, r, k):
    """(ids, weights) on the CPU in 64 bits."""
    T, E = logits.shape
    G = r.n_groups
    v, s = scores(logits, r.score == moe.MOE_SCORE_SIGMOID)
    if bias is None and (r.topk_groups == G or r.group_top == 1):
        c = v.clone()
    else:
        b = torch.zeros(E, dtype=F64) if bias is None else bias.to(F64)
        b = torch.where(torch.isnan(b), -math.inf, b)
        c = torch.where(v > -math.inf, s + b, -math.inf)
    by = torch.sort(c.view(T, G, E // G), dim=2, descending=True)[0][:, :, :r.group_top]
    value = by[:, :, 0].clone()
    if by.shape[2] == 2:
        value = torch.where(by[:, :, 1] > -math.inf, value + by[:, :, 1], value)
    keep = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :r.topk_groups]
    kept = torch.zeros((T, G), dtype=torch.bool).scatter_(1, keep, True)
    c = torch.where(kept.repeat_interleave(E // G, 1), c, -math.inf)
    top, ids = torch.sort(c, dim=1, descending=True, stable=True)
    ids = torch.where(top[:, :k] > -math.inf, ids[:, :k], -1)
    return ids, weights_of(s, ids, r)


# T, E, k, groups, kept, group_top
ROUTERS = [(1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (7, 256, 8, 8, 4, 1), (65, 64, 6, 1, 1, 1),
           (5, 8, 2, 1, 1, 1), (33, 60, 5, 4, 2, 2), (9, 1024, 64, 1, 1, 1), (6, 1024, 16, 32, 3, 2),
           (4, 1023, 31, 33, 1, 2), (10, 1022, 9, 14, 5, 2), (3, 64, 4, 64, 8, 2),
           (12, 640, 10, 64, 9, 2), (300, 128, 4, 16, 16, 2), (21, 70, 20, 2, 1, 2),
           (8, 33, 33, 3, 3, 1), (2, 510, 7, 34, 12, 1)]
WAYS = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


def make_logits(c, dtype, device, kind, seed):
    T, E = c[0], c[1]
    g = gen(device, seed)
    x = 2.0 * torch.randn((T, E), generator=g, device=device)
    if kind == "ties":                         # few distinct values: the lowest ids win
        x = torch.randint(-1, 2, (T, E), generator=g, device=device).float()
    elif kind == "holes":                      # experts taken out, rows with one and with none left
        x = torch.where(torch.rand((T, E), generator=g, device=device) < 0.4, -math.inf, x)
        x[::3] = torch.where(torch.rand(x[::3].shape, generator=g, device=device) < 0.3,
                             math.nan, x[::3])
        x[0] = -math.inf
        if T > 2:
            x[1], x[2] = math.nan, -math.inf
            x[2, E // 2] = -5.0
    elif kind == "far":                        # huge spread, infinities, the lowest value
        x = x * 1e4
        x[:, 0] = math.inf
        x[:, E // 3] = torch.finfo(torch.float32).min
        x[T // 2] = -200.0
    return x.to(TD[dtype])


@pytest.mark.parametrize("way", WAYS, ids=str)
@pytest.mark.parametrize("c", ROUTERS, ids=str)
def test_route_scored(device, c, way):
    T, E, k, G, kept, top = c
    score, renorm = way
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    r = moe.make_router(score, renorm, G, kept, top, 2.5)
    for kind in ("plain", "ties", "holes", "far"):
        for dtype in ("f32", "bf16"):
            for biased in (False, True):
                say("route_scored", c, way, kind, dtype, biased)
                x = make_logits(c, dtype, device, kind, 1)
                bias = None
                if biased:
                    bias = 0.1 * torch.randn(E, generator=gen(device, 2), device=device)
                    if kind == "ties":
                        bias = (bias > 0).float()
                    elif kind == "holes" and E > 2:
                        bias[0], bias[E // 2] = -math.inf, math.nan
                ids = Guarded((T, k), torch.int32, device)
                w = Guarded((T, k), torch.float32, device)
                moe.moe_route_scored(p, r, x, bias, ids.t, w.t)
                torch.cuda.synchronize()
                assert ids.intact() and w.intact()
                ref_ids, ref_w = ref_route(x.cpu(), None if bias is None else bias.cpu(), r, k)
                assert torch.equal(ids.t.cpu().long(), ref_ids)
                close(w.t.cpu(), ref_w, (50 + k) * U32 * ref_w.abs() + TINY, "weights")


@pytest.mark.parametrize("way", WAYS, ids=str)
def test_route_scored_near_ties(device, way):
    """Scores that 32 bits do not tell apart: biases that undo the logits' differences but for a few
    parts in 2^-30, in experts and in groups."""
    T, E, k, G = 64, 64, 6, 8
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    g = gen(device, 12)
    base = torch.randn(E, generator=g, device=device)
    x = base.expand(T, E).contiguous()
    x[T // 2:] += 1e-6 * torch.randn((T // 2, E), generator=g, device=device)
    s = scores(base[None].cpu(), way[0] == "sigmoid")[1][0]
    bias = (0.5 - s).float().to(device)          # c is 0.5 but for what fp32 rounds off the bias
    for groups, kept, top in [(1, 1, 1), (G, 3, 2), (G, 2, 1)]:
        r = moe.make_router(way[0], way[1], groups, kept, top)
        for b in (bias, bias + torch.repeat_interleave(torch.arange(8, device=device) % 2, 8) * 2e-7):
            ids, w = moe.route_scored(p, r, x, b)
            ref_ids, ref_w = ref_route(x.cpu(), b.cpu(), r, k)
            assert torch.equal(ids.cpu().long(), ref_ids), (groups, kept, top)
            close(w.cpu(), ref_w, (50 + k) * U32 * ref_w.abs() + TINY, "weights")


def test_route_scored_tiny_sigmoids(device):
    """Sigmoid scores below fp32's range still have ratios to renormalise."""
    T, E, k = 9, 16, 3
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    x = -150.0 + torch.randn((T, E), generator=gen(device, 13), device=device)
    bias = torch.randn(E, generator=gen(device, 14), device=device)
    for b in (None, bias):
        r = moe.make_router("sigmoid", True, scale=2.0)
        ids, w = moe.route_scored(p, r, x, b)
        ref_ids, ref_w = ref_route(x.cpu(), None if b is None else b.cpu(), r, k)
        assert torch.equal(ids.cpu().long(), ref_ids) and float(w.sum()) > 1.9 * T
        close(w.cpu(), ref_w, (50 + k) * U32 * ref_w.abs(), "weights")


def ref_route_bwd(logits, ids, dw, r):
    """Gradient of weights_of by automatic differentiation in 64 bits."""
    v = scores(logits, True)[0]
    out = v == -math.inf
    x = torch.where(out, 0.0, v).requires_grad_(True)
    if r.score == moe.MOE_SCORE_SIGMOID:
        s = torch.where(out, 0.0, torch.sigmoid(x))
    else:
        s = torch.softmax(torch.where(out, -math.inf, x), 1)
        s = torch.where(out, 0.0, s)
    ok = (ids >= 0) & (ids < logits.shape[1])
    i = torch.where(ok, ids, 0).long()
    use = ok & ~torch.gather(out, 1, i)
    w = torch.where(use, torch.gather(s, 1, i), 0.0)
    if r.renormalize:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    loss = (torch.where(use, r.scale * w * torch.where(use, dw.to(F64), 0.0), 0.0)).sum()
    d = torch.autograd.grad(loss, x)[0]
    return torch.where(out | torch.isnan(d), 0.0, d), (s * use.any(1, keepdim=True)).detach()


@pytest.mark.parametrize("way", WAYS, ids=str)
@pytest.mark.parametrize("c", ROUTERS, ids=str)
def test_route_scored_bwd(device, c, way):
    T, E, k, G, kept, top = c
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    r = moe.make_router(way[0], way[1], G, kept, top, 2.5)
    for kind in ("plain", "holes", "excluded", "twice"):
        for dtype in ("f32", "bf16"):
            say("route_scored_bwd", c, way, kind, dtype)
            x = make_logits(c, dtype, device, kind, 3)
            ids = moe.route_scored(p, r, x)[0]
            dw = torch.randn((T, k), generator=gen(device, 4), device=device)
            if kind == "excluded":               # ids of other shards, with no gradient to speak of
                drop = torch.rand((T, k), generator=gen(device, 5), device=device) < 0.5
                ids = torch.where(drop, torch.where(ids % 2 == 0, E + ids, -1 - ids), ids).int()
                dw = torch.where(drop, math.nan, dw)
            elif kind == "twice":
                ids = ids[:, :1].expand(T, k).contiguous()
            d = Guarded((T, E), TD[dtype], device)
            moe.moe_route_scored_bwd(p, r, x, ids, dw, d.t)
            torch.cuda.synchronize()
            assert d.intact()
            ref, s = ref_route_bwd(x.cpu(), ids.cpu(), dw.cpu(), r)
            # magnitudes: every slot's term, and the share of every expert
            clean = torch.where(torch.isnan(dw), 0.0, dw).cpu().to(F64)
            size = r.scale * clean.abs().sum(1, keepdim=True) * torch.ones_like(s)
            share = s if not r.renormalize else torch.ones_like(s)
            tol = (50 + k) * U32 * size * torch.minimum(share + (ref != 0), torch.ones_like(s))
            close(d.t.cpu(), ref, tol + UT[dtype] * ref.abs() + TINY, "d_logits")


def test_route_scored_bwd_against_differences(device):
    """The gradient against difference quotients of the weights in 64 bits, the choice held."""
    T, E, k = 3, 24, 4
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    for score, renorm in WAYS:
        r = moe.make_router(score, renorm, 4, 2, 2, 1.5)
        x = torch.randn((T, E), generator=gen(device, 6), device=device)
        ids, _ = moe.route_scored(p, r, x)
        dw = torch.randn((T, k), generator=gen(device, 7), device=device)
        d = moe.route_scored_bwd(p, r, x, ids, dw).cpu().to(F64)
        i = ids.cpu().long()

        def loss(v):
            return (weights_of(scores(v, score == "sigmoid")[1], i, r) * dw.cpu().to(F64)).sum(1)
        h = 1e-5
        for e in range(E):
            step = torch.zeros((T, E), dtype=F64)
            step[:, e] = h
            v = x.cpu().to(F64)
            quotient = (loss(v + step) - loss(v - step)) / (2 * h)
            # the quotient's own error: h^2 of the third derivative (below 10), and 2^-52 / h
            close(d[:, e], quotient, torch.full((T,), 1e-6, dtype=F64), (score, renorm, e))


def test_route_scored_equals_route(device):
    """Without bias, groups and scale it is moe_route."""
    for T, E, k in [(64, 256, 8), (9, 64, 6), (5, 1000, 3)]:
        p = moe.make_problem(T, 64, 64, E, k, "bf16")
        x = torch.randn((T, E), generator=gen(device, 8), device=device)
        for renorm in (False, True):
            ids, w = moe.route(p, x, renorm)
            ids2, w2 = moe.route_scored(p, moe.make_router("softmax", renorm), x)
            assert torch.equal(ids, ids2)
            # moe_route's weights: 40 u for the sum, k additions and a quotient when renormalised
            close(w2, w.to(F64), (90 + 2 * k) * U32 * w.to(F64), "weights")


# ---------------------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------------------
NORMS = [(1, 1), (1, 8), (3, 7), (5, 64), (4, 128), (2, 513), (9, 512), (6, 640), (70, 1024),
         (3, 1030), (5, 2048), (2, 2880), (1, 4096), (300, 4099), (1, 7168), (3, 8192), (2, 9000),
         (2, 16384), (1, 20001), (2, 32768), (2001, 384)]


def norm_inputs(T, H, dtype, device, seed=1):
    g = gen(device, seed)
    x = torch.randn((T, H), generator=g, device=device).to(TD[dtype])
    res = (2 * torch.randn((T, H), generator=g, device=device)).to(TD[dtype])
    w = (1 + 0.3 * torch.randn(H, generator=g, device=device)).to(TD[dtype])
    return x, res, w


def ref_norm(s, w, eps):
    s = s.to(F64)
    r = 1 / torch.sqrt((s * s).mean(1) + eps)
    return r, s * r[:, None] * (1.0 if w is None else w.to(F64))


def check_codes(n, codes, scales, what):
    """Each code as near n / scale as the nearest e4m3 value, up to 6 u of the quotient."""
    T, H = n.shape
    v = n.view(T, H // 128, 128)
    amax = v.abs().amax(2)
    close(scales, torch.where(amax == 0, 1.0, amax / 448), 6 * U32 * amax / 448, what + " scales")
    q = (v / scales.to(F64)[:, :, None]).view(T, H)
    best = (q.float().clamp(-448, 448).to(E4M3)).to(F64)
    far = (codes.to(F64) - q).abs() - (best - q).abs() - 2 * 6 * U32 * q.abs()
    assert not torch.isnan(codes.float()).any() and float(far.max()) <= 0, what


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", NORMS, ids=str)
def test_rms_norm(device, c, dtype):
    T, H = c
    dt = TD[dtype]
    x, res, w = norm_inputs(T, H, dtype, device)
    for with_res in (False, True):
        for with_w in (True, False):
            say("rms_norm", c, dtype, with_res, with_w)
            fp8 = H % 128 == 0
            s = Guarded((T, H), dt, device) if with_res else None
            y, rstd = Guarded((T, H), dt, device), Guarded((T,), torch.float32, device)
            codes = Guarded((T, H), E4M3, device) if fp8 else None
            scales = Guarded((T, H // 128), torch.float32, device) if fp8 else None
            moe.moe_rms_norm(x, res if with_res else None, w if with_w else None, 1e-5,
                             s.t if s else None, y.t, codes.t if fp8 else None,
                             scales.t if fp8 else None, rstd.t)
            torch.cuda.synchronize()
            assert all(o.intact() for o in (s, y, rstd, codes, scales) if o)
            h = x
            if with_res:
                h = (x.float() + res.float()).to(dt)
                assert torch.equal(s.t, h)
            r, n = ref_norm(h, w if with_w else None, 1e-5)
            close(rstd.t, r, 2 * U32 * r, "rstd")
            close(y.t, n, (4 * U32 + UT[dtype]) * n.abs() + TINY, "y")
            if fp8:
                check_codes(n, codes.t, scales.t, "codes")
                only = moe.rms_norm(x, w if with_w else None, res if with_res else None, 1e-5,
                                    ["codes"])
                assert torch.equal(only["codes"].view(torch.uint8), codes.t.view(torch.uint8))
                assert torch.equal(only["scales"], scales.t)


def test_rms_norm_in_place(device):
    """The sum in the residual's and in x's own memory."""
    for T, H in [(5, 7168), (33, 640), (3, 1001)]:
        x, res, w = norm_inputs(T, H, "bf16", device)
        ref = moe.rms_norm(x, w, res)
        for own in ("x", "res"):
            a, b = x.clone(), res.clone()
            out = moe.rms_norm(a, w, b, sum=a if own == "x" else b)
            assert out["sum"] is (a if own == "x" else b)
            assert torch.equal(out["sum"], ref["sum"]) and torch.equal(out["y"], ref["y"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rms_norm_special_rows(device, dtype):
    """Rows of zeros, huge and tiny rows whose squares leave fp32, infinities, NaN: one row's never
    reaches another's."""
    T, H = 9, 1024
    x, _, w = norm_inputs(T, H, dtype, device)
    x[1] = 0
    x[2] = x[2] * 1e30
    x[3] = x[3] * 1e-30
    x[4, 5] = math.nan
    x[5, 700] = math.inf
    out = moe.rms_norm(x, w, eps=1e-6, want=("y", "codes", "rstd"))
    r, n = ref_norm(x, w, 1e-6)
    fine = [0, 1, 2, 3, 6, 7, 8]
    close(out["rstd"][fine], r[fine], 2 * U32 * r[fine] + TINY, "rstd")
    close(out["y"][fine], n[fine], (4 * U32 + UT[dtype]) * n[fine].abs() + TINY, "y")
    check_codes(n[fine], out["codes"][fine], out["scales"][fine], "codes")
    assert not out["codes"][1].float().any() and bool((out["scales"][1] == 1).all())
    assert torch.isnan(out["y"][4].float()).all() and torch.isnan(out["codes"][4].float()).all()
    row = out["y"][5].float()                     # 1 / sqrt(inf) = 0: inf * 0 is NaN, the rest 0
    assert torch.isnan(row[700]) and int(torch.isnan(row).sum()) == 1 and not row.nansum()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", NORMS + [(1, 513), (5000, 128), (1500, 2048), (700, 4096)], ids=str)
def test_rms_norm_bwd(device, c, dtype):
    T, H = c
    dt = TD[dtype]
    s, ds, w = norm_inputs(T, H, dtype, device, 2)
    dy = torch.randn((T, H), generator=gen(device, 3), device=device).to(dt)
    rstd = moe.rms_norm(s, w, want=("y", "rstd"))["rstd"]
    for with_w, with_ds, with_dw in [(True, True, True), (False, False, True), (True, False, False)]:
        say("rms_norm_bwd", c, dtype, with_w, with_ds, with_dw)
        dx = Guarded((T, H), dt, device)
        dw = Guarded((H,), torch.float32, device) if with_dw else None
        need = moe.moe_rms_norm_bwd_workspace_bytes(T, H)
        ws = Guarded((need,), torch.uint8, device) if with_dw else None
        moe.moe_rms_norm_bwd(dy, ds if with_ds else None, s, w if with_w else None, rstd, dx.t,
                             dw.t if dw else None, ws.t if ws else None)
        torch.cuda.synchronize()
        assert all(o.intact() for o in (dx, dw, ws) if o)
        r = rstd.to(F64)[:, None]
        n = s.to(F64) * r
        g = dy.to(F64) * (w.to(F64) if with_w else 1.0)
        extra = ds.to(F64) if with_ds else torch.zeros_like(g)
        ref = r * (g - n * (g * n).mean(1, keepdim=True)) + extra
        size = (r * g).abs() + (r * n * (g * n).mean(1, keepdim=True)).abs() + extra.abs()
        mean = (g * n).abs().mean(1, keepdim=True)
        tol = U32 * (6 * size + 60 * (r * n).abs() * mean) + UT[dtype] * ref.abs() + TINY
        close(dx.t, ref, tol, "d_x")
        if with_dw:
            prod = dy.to(F64) * n
            depth = math.ceil(T / 256) + 4 + 32 + 16 + 3
            close(dw.t, prod.sum(0), depth * U32 * prod.abs().sum(0) + TINY, "d_w")


def test_rms_norm_bwd_in_place_and_by_differences(device):
    T, H = 4, 96
    s, ds, w = norm_inputs(T, H, "f32", device, 5)
    dy = torch.randn((T, H), generator=gen(device, 6), device=device)
    rstd = moe.rms_norm(s, w, want=("y", "rstd"))["rstd"]
    dx, dw = moe.rms_norm_bwd(dy, s, w, rstd, ds)
    for own in (dy.clone(), ds.clone()):
        a, b = (own, ds) if torch.equal(own, dy) else (dy, own)
        assert torch.equal(moe.rms_norm_bwd(a, s, w, rstd, b, d_x=own)[0], dx)

    def loss(sv, wv):
        return (ref_norm(sv, wv, 1e-6)[1] * dy.to(F64)).sum() + (sv.to(F64) * ds.to(F64)).sum()
    h, s64, w64 = 1e-5, s.to(F64), w.to(F64)
    for t, i in [(0, 0), (1, 50), (3, 95)]:
        e = torch.zeros_like(s64)
        e[t, i] = h
        quotient = (loss(s64 + e, w64) - loss(s64 - e, w64)) / (2 * h)
        # central differences: h^2 of third derivatives (below 100), 2^-52 of the loss over h
        assert abs(float(dx[t, i]) - float(quotient)) < 2e-6 * (1 + abs(float(quotient)))
        f = torch.zeros_like(w64)
        f[i] = h
        quotient = (loss(s64, w64 + f) - loss(s64, w64 - f)) / (2 * h)
        assert abs(float(dw[i]) - float(quotient)) < 2e-6 * (1 + abs(float(quotient)))


# ---------------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------------
GEMMS = [(1, 1, 1), (1, 256, 7168), (1, 8, 8), (3, 5, 7), (2, 64, 64), (16, 16, 32), (17, 24, 40),
         (15, 40, 200), (64, 64, 64), (65, 72, 136), (8, 1000, 72), (33, 7, 130), (100, 130, 257),
         (128, 128, 128), (129, 136, 1000), (200, 328, 520), (256, 256, 256), (257, 264, 64),
         (300, 600, 1096), (513, 520, 264), (1000, 8, 512), (8, 1000, 2048), (777, 1544, 392),
         (1030, 1032, 72), (2100, 768, 128), (31, 2056, 4096), (1, 4104, 1032), (640, 3200, 200),
         (1, 5, 14001), (1501, 1503, 77), (1502, 1600, 129), (200, 331, 3001)]
LAYOUTS = ["nt", "nn", "tn"]
ACTS = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
        "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def operands(m, n, k, layout, device, seed, ints=False):
    """a and b in their layout, and as a [m, k] and b [k, n] in 64 bits."""
    g = gen(device, seed)
    sa = (k, m) if layout == "tn" else (m, k)
    sb = (n, k) if layout == "nt" else (k, n)
    if ints:
        a, b = (torch.randint(-2, 3, s, generator=g, device=device).bfloat16() for s in (sa, sb))
    else:
        a, b = (torch.randn(s, generator=g, device=device).bfloat16() for s in (sa, sb))
    a64, b64 = a.to(F64), b.to(F64)
    return a, b, (a64.t() if layout == "tn" else a64), (b64.t() if layout == "nt" else b64)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("c", GEMMS, ids=str)
def test_gemm_of_integers(device, c, layout):
    """Sums of small integers are exact, whatever the order of their additions (k times 4 stays
    below 2^24), so is bias and residual in fp32; bf16 results are rounded once."""
    m, n, k = c
    a, b, a64, b64 = operands(m, n, k, layout, device, 1, ints=True)
    g = gen(device, 2)
    bias = torch.randint(-9, 10, (n,), generator=g, device=device).float()
    z = a64 @ b64
    for dtype in ("f32", "bf16"):
        res = torch.randint(-9, 10, (m, n), generator=g, device=device).to(TD[dtype])
        for with_bias, with_res, with_pre in [(False, False, False), (True, True, True),
                                              (True, False, False), (False, True, False)]:
            say("gemm", c, layout, dtype, with_bias, with_res)
            out = Guarded((m, n), TD[dtype], device)
            pre = Guarded((m, n), torch.bfloat16, device) if with_pre else None
            moe.moe_gemm_bf16(layout, a, b, bias if with_bias else None, "none",
                              res if with_res else None, pre.t if pre else None, out.t)
            torch.cuda.synchronize()
            assert out.intact() and (not pre or pre.intact())
            want = z + (bias.to(F64) if with_bias else 0)
            if pre:
                assert torch.equal(pre.t, want.to(torch.bfloat16))
            want = want + (res.to(F64) if with_res else 0)
            assert torch.equal(out.t, want.to(TD[dtype]))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("c", [(1, 264, 520), (5, 9, 33), (70, 136, 72), (130, 200, 1000),
                               (300, 264, 4104), (515, 776, 136)], ids=str)
def test_gemm_epilogue(device, c, act, layout):
    m, n, k = c
    a, b, a64, b64 = operands(m, n, k, layout, device, 3)
    b, b64 = (b / math.sqrt(k)).bfloat16(), None
    b64 = b.to(F64).t() if layout == "nt" else b.to(F64)
    bias = torch.randn(n, generator=gen(device, 4), device=device)
    z = a64 @ b64 + bias.to(F64)
    tol_z = 2 * k * U32 * (a64.abs() @ b64.abs()) + 2 * U32 * z.abs()
    for dtype in ("f32", "bf16"):
        say("gemm epilogue", c, act, layout, dtype)
        res = torch.randn((m, n), generator=gen(device, 5), device=device).to(TD[dtype])
        out, pre = moe.gemm_bf16(a, b, layout, bias, act, res, TD[dtype], with_pre=True)
        want = ACTS[act](z) + res.to(F64)
        close(pre, z, tol_z + UBF * z.abs(), "pre")
        close(out, want, 1.13 * tol_z + 8 * U32 * (z.abs() + want.abs()) + UT[dtype] * want.abs(),
              "c")
        rms = float((out.double() - want).norm() / want.norm())
        assert rms <= 2 * U32 * math.sqrt(k) + 8 * U32 + UT[dtype], rms
        own = res.clone()                        # the result in the residual's own memory
        assert moe.gemm_bf16(a, b, layout, bias, act, own, out=own) is own
        assert torch.equal(own, out)


def test_gemm_values_past_the_ends_do_not_count(device):
    """NaN and infinities right behind the operands' last rows and columns."""
    for m, n, k in [(65, 72, 136), (130, 264, 200), (17, 40, 72), (300, 520, 1032), (1, 24, 200)]:
        for layout in LAYOUTS:
            a, b, a64, b64 = operands(m, n, k, layout, device, 6, ints=True)
            held = []
            for t in (a, b):
                buf = torch.full((t.numel() + 8192,), math.nan, dtype=torch.bfloat16, device=device)
                buf[4096:4096 + t.numel()] = t.reshape(-1)
                held.append(buf[4096:4096 + t.numel()].view(t.shape))
            out = moe.gemm_bf16(*held, layout, out_dtype=torch.float32)
            assert torch.equal(out.double(), a64 @ b64), (m, n, k, layout)


def test_gemm_nan_and_infinities_stay_in_their_rows(device):
    m, n, k = 140, 136, 200
    for layout in LAYOUTS:
        a, b, a64, b64 = operands(m, n, k, layout, device, 7)
        for bad in (math.nan, math.inf):
            x = a.clone()
            (x.t() if layout == "tn" else x)[77, 199] = bad
            out = moe.gemm_bf16(x, b, layout)
            clean = moe.gemm_bf16(a, b, layout)
            rows = torch.arange(m, device=device) != 77
            assert torch.equal(out[rows], clean[rows])
            assert not torch.isfinite(out[77].float()).any()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("c", [(1, 1), (1, 4096), (3, 7), (64, 256), (257, 1000), (2001, 2880),
                               (5000, 24), (9, 30001), (1003, 130)], ids=str)
def test_act_bwd(device, c, act):
    m, n = c
    g = gen(device, 8)
    z = (3 * torch.randn((m, n), generator=g, device=device)).bfloat16()
    dc = torch.randn((m, n), generator=g, device=device).bfloat16()
    special = torch.tensor([0.0, -0.0, 40.0, -40.0, 3e38, -3e38, math.inf, -math.inf],
                           device=device).bfloat16()
    z.view(-1)[:8] = special[:z.numel()]
    z64 = z.to(F64).clamp(-1e4, 1e4).requires_grad_(True)       # the slope is 0 or 1 from there
    slope = torch.autograd.grad(ACTS[act](z64).sum(), z64)[0]
    v = dc.to(F64) * slope
    err = 12 * U32 * (1 + z.to(F64).abs().clamp(max=30)) * dc.to(F64).abs()
    none = act == "none"
    for with_bias in (True, False):
        if none and not with_bias:
            continue
        say("act_bwd", c, act, with_bias)
        dz = None if none else Guarded((m, n), torch.bfloat16, device)
        db = Guarded((n,), torch.float32, device) if with_bias else None
        ws = Guarded((moe.moe_act_bwd_workspace_bytes(m, n),), torch.uint8, device)
        moe.moe_act_bwd(act, dc, None if none else z, dz.t if dz else None, db.t if db else None,
                        ws.t if with_bias else None)
        torch.cuda.synchronize()
        assert all(o.intact() for o in (dz, db, ws) if o)
        if dz:
            close(dz.t, v, err + UBF * v.abs() + TINY, "d_z")
        if db:
            depth = math.ceil(m / 4) + 4 + 32 + 16       # one row of workgroups, at most
            close(db.t, v.sum(0), err.sum(0) + depth * U32 * v.abs().sum(0) + TINY, "d_bias")
    if not none:
        for own in (dc.clone(), z.clone()):
            first = own if torch.equal(own.view(torch.int16), dc.view(torch.int16)) else dc
            got = moe.act_bwd(first, z if first is own else own, act, d_z=own)[0]
            assert got is own and torch.equal(own.view(torch.int16), dz.t.view(torch.int16))


def test_linear_gradients_are_those_of_the_layer(device):
    """The backward pass of act(x w^T + bias) + residual as moe.h writes it, against automatic
    differentiation in 64 bits."""
    m, n, k = 130, 72, 264
    g = gen(device, 9)
    x = torch.randn((m, k), generator=g, device=device).bfloat16()
    w = (torch.randn((n, k), generator=g, device=device) / 16).bfloat16()
    bias = torch.randn(n, generator=g, device=device)
    dy = torch.randn((m, n), generator=g, device=device).bfloat16()
    for act in ACTS:
        y, pre = moe.gemm_bf16(x, w, "nt", bias, act, with_pre=True)
        dz, db = moe.act_bwd(dy, pre, act, d_bias=True)
        dx = moe.gemm_bf16(dz, w, "nn", out_dtype=torch.float32)
        dw = moe.gemm_bf16(dz, x, "tn", out_dtype=torch.float32)
        leaves = [t.to(F64).requires_grad_(True) for t in (x, w, bias)]
        ACTS[act](leaves[0] @ leaves[1].t() + leaves[2]).backward(dy.to(F64))
        # pre and d_z are handed on in bf16, in the middle of the sums
        for got, leaf in zip((dx, dw, db), leaves):
            rel = float((got.double() - leaf.grad).norm() / leaf.grad.norm())
            assert rel <= 2 * UBF, (act, rel)
