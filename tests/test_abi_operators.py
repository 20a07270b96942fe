"""Refusals of the operators around the layer (rows in expert-sorted order, gradients, products of
e4m3 codes): every bad argument is turned down on the host, before any HIP call."""
import ctypes
import glob
import os
import re

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe

S, D, N, A = moe.MOE_ERR_SHAPE, moe.MOE_ERR_DTYPE, moe.MOE_ERR_NULL, moe.MOE_ERR_ALIGN
F32, BF16, E4M3 = moe.MOE_F32, moe.MOE_BF16, moe.MOE_E4M3
ok, odd8, odd2 = (ctypes.c_void_p(4096 + d) for d in (0, 8, 2))


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def problem(**kw):
    base = dict(T=16, H=192, I=256, E=8, top_k=2, dtype="bf16")
    base.update(kw)
    return ctypes.byref(moe.make_problem(**base))


def test_permute(lib):
    P = problem()
    assert lib.moe_permute(None, BF16, *[ok] * 7, None) == N
    assert lib.moe_permute(problem(H=100), BF16, *[ok] * 7, None) == S
    for bad in (moe.MOE_MXFP4, -1, 17):
        assert lib.moe_permute(P, bad, ok, None, ok, ok, ok, ok, None, None) == D
    assert lib.moe_permute(P, BF16, ok, ok, ok, ok, ok, ok, ok, None) == D        # scales of bf16 rows
    assert lib.moe_permute(P, E4M3, ok, ok, ok, ok, ok, ok, ok, None) == S        # H % 128
    P128 = problem(H=256)
    assert lib.moe_permute(P128, E4M3, ok, ok, ok, ok, ok, ok, None, None) == N   # one scale array
    assert lib.moe_permute(P128, E4M3, ok, None, ok, ok, ok, ok, ok, None) == N
    for i in (0, 2, 3, 4, 5):
        args = [ok, None, ok, ok, ok, ok, None]
        args[i] = None
        assert lib.moe_permute(P, BF16, *args, None) == N
        args[i] = odd8 if i in (0, 5) else odd2
        assert lib.moe_permute(P, BF16, *args, None) == A
    assert lib.moe_permute(P128, E4M3, ok, odd2, ok, ok, ok, ok, ok, None) == A


def test_unpermute(lib):
    P = problem()
    for bad in (E4M3, moe.MOE_MXFP4):
        assert lib.moe_unpermute(P, bad, ok, ok, ok, ok, None) == D
        assert lib.moe_unpermute_bwd(P, bad, *[ok] * 8, None) == D
    assert lib.moe_unpermute(problem(top_k=9), F32, ok, ok, ok, ok, None) == S
    for i in (0, 1, 3):
        args = [ok, ok, None, ok]                          # no weights is a valid call
        args[i] = None
        assert lib.moe_unpermute(P, F32, *args, None) == N
    assert lib.moe_unpermute(P, F32, odd8, ok, ok, ok, None) == A
    assert lib.moe_unpermute(P, F32, ok, ok, odd2, ok, None) == A
    full = [ok] * 8                    # d_out rows slot_row sorted_slots num_tiles w d_rows d_weights
    for i in (0, 1, 2, 3, 4):
        args = list(full)
        args[i] = None
        assert lib.moe_unpermute_bwd(P, BF16, *args, None) == N
    assert lib.moe_unpermute_bwd(P, BF16, *full[:6], None, None, None) == N       # nothing to write
    for i, bad in [(0, odd8), (1, odd8), (2, odd2), (5, odd2), (6, odd8), (7, odd2)]:
        args = list(full)
        args[i] = bad
        assert lib.moe_unpermute_bwd(P, BF16, *args, None) == A


def test_route_bwd(lib):
    assert lib.moe_route_bwd(problem(H=100), ok, 0, ok, ok, ok, None) == S
    assert lib.moe_route_bwd(problem(E=100, top_k=65), ok, 0, ok, ok, ok, None) == S
    for i in range(4):
        args = [ok] * 4
        args[i] = None
        assert lib.moe_route_bwd(problem(), args[0], 1, *args[1:], None) == N
        args[i] = odd2
        assert lib.moe_route_bwd(problem(), args[0], 1, *args[1:], None) == A


def test_quantize_cols(lib):
    for m, n in [(0, 8), (-1, 8), (4, 0), (4, 12), (4, -8), (2 ** 22 + 1, 8), (8, 2 ** 22 + 8),
                 (2 ** 22, 2 ** 22)]:
        assert lib.moe_quantize_cols_e4m3(m, n, ok, ok, ok, None) == S, (m, n)
    assert lib.moe_quantize_cols_e4m3(4, 8, None, ok, ok, None) == N
    assert lib.moe_quantize_cols_e4m3(4, 8, odd8, ok, ok, None) == A
    assert lib.moe_quantize_cols_e4m3(4, 8, ok, ok, odd2, None) == A


def test_gemm(lib):
    def call(m=16, n=32, k=256, ptr=(ok,) * 4, block=128, c=ok, dt=BF16):
        return lib.moe_gemm_e4m3(m, n, k, *ptr, block, c, dt, None)
    for kw in [dict(m=0), dict(n=0), dict(k=0), dict(k=64), dict(k=200), dict(m=-5),
               dict(m=2 ** 24 + 1), dict(n=2 ** 24 + 1), dict(k=2 ** 22 + 128),
               dict(m=2 ** 24, n=2 ** 24), dict(block=64), dict(block=0),
               dict(m=2 ** 22, n=2 ** 15 + 16), dict(m=2 ** 15 + 1, n=2 ** 22)]:
        assert call(**kw) == S, kw
    assert call(dt=E4M3) == D and call(dt=9) == D
    for i in range(4):
        p = [ok] * 4
        p[i] = None
        assert call(ptr=p) == N
        p[i] = odd8 if i in (0, 2) else odd2
        assert call(ptr=p) == A
    assert call(c=None) == N and call(c=odd8) == A


def test_grouped_gemm(lib):
    P8 = problem(H=256, w_dtype="e4m3")

    def call(P=P8, n=32, k=256, ptr=(ok,) * 8, out=ok, dt=BF16):
        return lib.moe_grouped_gemm_e4m3(P, n, k, *ptr, out, dt, None)
    assert call(P=problem()) == D and call(P=problem(dtype="f32")) == D
    assert call(dt=E4M3) == D
    assert call(P=problem(H=192, w_dtype="e4m3")) == S
    for kw in [dict(n=0), dict(k=0), dict(k=192), dict(n=32769), dict(k=32768 + 128), dict(n=-1)]:
        assert call(**kw) == S, kw
    # more workgroups than a launch's thread count holds: 2^19 m-blocks of 16 rows, 17 n-blocks
    many = problem(T=2 ** 20, H=256, E=8, top_k=8, w_dtype="e4m3", block_m=16)
    assert call(P=many, n=16 * 128 + 1) == S
    for i in range(8):
        p = [ok] * 8
        p[i] = None
        assert call(ptr=p) == N
        p[i] = odd8 if i in (0, 2) else odd2
        assert call(ptr=p) == A
    assert call(out=None) == N and call(out=odd8) == A


def test_binding_refuses_wrong_tensors():
    """Host tensors, wrong types and shapes are refused before the library is called."""
    p = moe.make_problem(4, 128, 128, 8, 2, "bf16")
    with pytest.raises(ValueError):
        moe._lib._mat(torch.zeros(4, 4), "x", (torch.float32,), (4, 5), 0)
    with pytest.raises(ValueError):
        moe._lib._row_dtype(torch.zeros(4, dtype=torch.float16), "x")
    with pytest.raises(ValueError):
        moe._lib._row_dtype(None, "x")
    for t in (torch.zeros(4, 4), torch.zeros(4, 4, dtype=torch.bfloat16), torch.zeros(4, 8)[:, ::2]):
        with pytest.raises(ValueError):
            moe._lib._arg(t, "x", (torch.float32,), 16, 0)
    with pytest.raises(TypeError):
        moe._lib._arg([1.0], "x", (torch.float32,), 1, 0)
    if torch.cuda.is_available():
        with pytest.raises(ValueError):
            moe.moe_unpermute(p, torch.zeros(2), torch.zeros(2), None, torch.zeros(2))


def test_copies_to_lds_wait_for_m0():
    """A load to LDS needs a wait state after the write of M0, which assembly has to hold itself."""
    found = 0
    for path in glob.glob(os.path.join(os.path.dirname(moe.__file__), "csrc", "*")):
        with open(path) as f:
            for rest in re.findall(r"s_mov_b32 m0, %\d\\n\\t(\w+)", f.read()):
                assert rest == "s_nop", path
                found += 1
    assert found >= 6
