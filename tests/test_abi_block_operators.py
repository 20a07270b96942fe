"""Refusals of the operators before the layer and beside it (router with scores, norm, bf16 products):
every bad argument is turned down on the host, before any HIP call."""
import ctypes

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe

S, D, N, A, W = (moe.MOE_ERR_SHAPE, moe.MOE_ERR_DTYPE, moe.MOE_ERR_NULL, moe.MOE_ERR_ALIGN,
                 moe.MOE_ERR_WORKSPACE)
F32, BF16, E4M3 = moe.MOE_F32, moe.MOE_BF16, moe.MOE_E4M3
ok, odd8, odd2 = (ctypes.c_void_p(4096 + d) for d in (0, 8, 2))
EPS = ctypes.c_float(1e-6)


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def problem(**kw):
    base = dict(T=16, H=192, I=256, E=24, top_k=4, dtype="bf16")
    base.update(kw)
    return moe.make_problem(**base)


BAD_ROUTERS = [dict(score=2), dict(score=-1), dict(n_groups=0), dict(n_groups=5), dict(n_groups=-1),
               dict(n_groups=4, topk_groups=0), dict(n_groups=4, topk_groups=5),
               dict(group_top=0), dict(group_top=3), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(n_groups=8, topk_groups=1)]


def test_router(lib):
    P = problem()
    good = moe.make_router("sigmoid", True, 4, 2, 2, 2.5)
    assert moe.moe_router_validate(P, good) == moe.MOE_OK
    assert moe.moe_router_validate(problem(E=130, top_k=64), moe.make_router()) == moe.MOE_OK
    assert moe.moe_router_validate(problem(E=130, top_k=65), moe.make_router()) == S
    assert moe.moe_router_validate(problem(E=130), moe.make_router(n_groups=65)) == S
    assert moe.moe_router_validate(problem(H=100), good) == S
    ref, gref = ctypes.byref(P), ctypes.byref(good)
    for f in (lib.moe_route_scored, lib.moe_route_scored_bwd):
        for kw in BAD_ROUTERS:
            assert f(ref, ctypes.byref(moe.make_router(**kw)), ok, F32, ok, ok, ok, None) == S, kw
        assert f(ref, None, ok, F32, ok, ok, ok, None) == N
        assert f(None, gref, ok, F32, ok, ok, ok, None) == N
        for bad in (E4M3, moe.MOE_MXFP4, -1):
            assert f(ref, gref, ok, bad, ok, ok, ok, None) == D
    for i in range(4):
        args = [ok] * 4                       # logits, bias | topk_ids, then the outputs
        args[i] = None
        assert lib.moe_route_scored_bwd(ref, gref, args[0], F32, *args[1:], None) == N
        if i != 1:                            # no bias is a valid call
            assert lib.moe_route_scored(ref, gref, args[0], F32, *args[1:], None) == N
        args[i] = odd2
        assert lib.moe_route_scored_bwd(ref, gref, args[0], F32, *args[1:], None) == A
        assert lib.moe_route_scored(ref, gref, args[0], F32, *args[1:], None) == A


def test_rms_norm(lib):
    def call(t=4, h=256, dt=BF16, x=ok, res=ok, w=ok, eps=EPS, s=ok, y=ok, codes=ok, scales=ok,
             rstd=ok):
        return lib.moe_rms_norm(t, h, dt, x, res, w, eps, s, y, codes, scales, rstd, None)
    for kw in [dict(t=0), dict(t=-1), dict(h=0), dict(h=32769), dict(h=192), dict(h=-128),
               dict(eps=ctypes.c_float(-1e-6)), dict(eps=ctypes.c_float(float("nan"))),
               dict(eps=ctypes.c_float(float("inf")))]:
        assert call(**kw) == S, kw
    assert call(h=192, codes=None) == S and call(h=192, scales=None) == S
    for bad in (E4M3, moe.MOE_MXFP4, 9):
        assert call(dt=bad) == D
    for kw in [dict(x=None), dict(res=None), dict(s=None), dict(codes=None), dict(scales=None),
               dict(y=None, codes=None, scales=None)]:
        assert call(**kw) == N, kw
    for kw in [dict(x=odd8), dict(res=odd8), dict(w=odd8), dict(s=odd8), dict(y=odd8),
               dict(codes=odd8), dict(scales=odd8), dict(rstd=odd2)]:
        assert call(**kw) == A, kw


def test_rms_norm_bwd(lib):
    need = moe.moe_rms_norm_bwd_workspace_bytes(4, 100)
    assert need == 1792                                   # 4 rows of 100 values, in units of 256
    big = moe.moe_rms_norm_bwd_workspace_bytes(1 << 20, 32768)
    assert big == 512 * 32768 * 4

    def call(t=4, h=100, dt=BF16, ptr=(ok,) * 5, dx=ok, dw=ok, ws=ok, n=need):
        return lib.moe_rms_norm_bwd(t, h, dt, *ptr, dx, dw, ws, n, None)
    for kw in [dict(t=0), dict(h=0), dict(h=32769)]:
        assert call(**kw) == S, kw
    assert lib.moe_rms_norm_bwd_workspace_bytes(0, 5) == S
    assert lib.moe_rms_norm_bwd_workspace_bytes(5, 32769) == S
    with pytest.raises(moe.MoeError):
        moe.moe_rms_norm_bwd_workspace_bytes(0, 5)
    assert call(dt=E4M3) == D
    assert call(n=need - 1) == W and call(ws=None) == N and call(dx=None) == N
    for i in (0, 2, 4):                                   # d_sum and the weight may be missing
        p = [ok] * 5
        p[i] = None
        assert call(ptr=p) == N
    for i in range(5):
        p = [ok] * 5
        p[i] = odd2 if i == 4 else odd8
        assert call(ptr=p) == A
    assert call(dx=odd8) == A and call(dw=odd8) == A and call(ws=odd8) == A


def test_gemm_bf16(lib):
    def call(m=16, n=32, k=64, layout=moe.MOE_NT, a=ok, b=ok, bias=ok, act=moe.MOE_ACT_SILU,
             res=ok, pre=ok, c=ok, dt=BF16):
        return lib.moe_gemm_bf16(m, n, k, layout, a, b, bias, act, res, pre, c, dt, None)
    for kw in [dict(m=0), dict(n=0), dict(k=0), dict(m=-1), dict(m=2 ** 24 + 1),
               dict(n=2 ** 24 + 1), dict(k=2 ** 24 + 1), dict(m=2 ** 24, n=2 ** 24),
               dict(m=2 ** 22, n=2 ** 15 + 16), dict(layout=3), dict(layout=-1), dict(act=4),
               dict(act=-1)]:
        assert call(**kw) == S, kw
    assert call(dt=E4M3) == D and call(dt=7) == D
    for kw in [dict(a=None), dict(b=None), dict(c=None)]:
        assert call(**kw) == N, kw
    for kw in [dict(a=odd8), dict(b=odd8), dict(c=odd8), dict(res=odd8), dict(pre=odd8),
               dict(bias=odd2)]:
        assert call(**kw) == A, kw


def test_act_bwd(lib):
    need = moe.moe_act_bwd_workspace_bytes(9, 100)
    assert need == 1280                                   # 3 rows of 100 values
    assert moe.moe_act_bwd_workspace_bytes(2 ** 24, 2 ** 24) == 2 ** 26
    assert moe.moe_act_bwd_workspace_bytes(2 ** 24, 256) == 512 * 1024

    def call(m=9, n=100, act=moe.MOE_ACT_GELU, dc=ok, pre=ok, dz=ok, db=ok, ws=ok, size=need):
        return lib.moe_act_bwd(m, n, act, dc, pre, dz, db, ws, size, None)
    for kw in [dict(m=0), dict(n=0), dict(m=2 ** 24 + 1), dict(n=2 ** 24 + 1), dict(act=4),
               dict(act=-1)]:
        assert call(**kw) == S, kw
    none = moe.MOE_ACT_NONE
    for kw in [dict(dc=None), dict(pre=None), dict(dz=None), dict(ws=None), dict(act=none),
               dict(act=none, pre=None), dict(act=none, dz=None),
               dict(act=none, pre=None, dz=None, db=None)]:
        assert call(**kw) == N, kw
    assert call(size=need - 1) == W
    for kw in [dict(dc=odd8), dict(pre=odd8), dict(dz=odd8), dict(db=odd2), dict(ws=odd8)]:
        assert call(**kw) == A, kw


def test_helpers_refuse_unknown_names():
    with pytest.raises(ValueError):
        moe.rms_norm(torch.zeros(2, 8), want=["z"])
    with pytest.raises(ValueError):
        moe.rms_norm(torch.zeros(2, 8), sum=torch.zeros(2, 8))
    with pytest.raises(KeyError):
        moe.make_router("tanh")
    a, b = torch.zeros(2, 8).bfloat16(), torch.zeros(3, 8).bfloat16()
    for kw in [dict(act="relu"), dict(layout="xx")]:
        with pytest.raises(ValueError):
            moe.moe_gemm_bf16(kw.get("layout", "nt"), a, b, None, kw.get("act", "none"), None, None,
                              a)
    with pytest.raises(moe.MoeError):
        moe.moe_gemm_bf16(3, a, b, None, "none", None, None, a)
    with pytest.raises(ValueError, match="k is"):
        moe.moe_gemm_bf16("nn", a, b, None, "none", None, None, a)
    for x in (torch.zeros(8), None, [1.0]):
        with pytest.raises(ValueError):
            moe.moe_rms_norm(x, None, None, 1e-6, None, None, None, None, None)
