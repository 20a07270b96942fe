"""Products of e4m3 codes on every kernel that their choice has, against 64 bits.

Dense: TILES reaches, on a device of UNITS compute units, every kernel in every form (scales of b by
block and by row, results in bf16 and fp32, rows of c that begin on 16 bytes, on an even and on an odd
number of values), with ragged last tiles and so many slices of k that every ring of stages is refilled
(test_gemm_choice.py holds it to that).  Grouped: one case at least per kernel of
launch_grouped_gemm_e4m3, with experts of one m-block and of several.

Tolerances: gemm_tol bounds every element from the sum of magnitudes.  Random operands stay far below
it, so two statements about them are held as well.  fp32 results: gemm_norm, 2^-21.  bf16 results: the
error of the product BEFORE its rounding, which `beyond_rounding` reads off the rounded one.  With
r = bf16(ref), v = ref + d the computed sum and got = bf16(v): |got - ref| <= |got - v| + |d| <=
|r - v| + |d| <= |r - ref| + 2 |d|, so the excess |got - ref| - |r - ref| of an element is between 0 and
2 |d|.  An element is rounded the other way where its distance m to a rounding border is below |d|; ref
lies anywhere in a step s, so that happens with probability |d| / s, m is uniform up to |d| and the
excess is 2 m: the excess times s has the mean d^2.  The fp8 instruction's d is 2^-16 of a result in the
root mean square (1.4e-5, measured on fp32 results of the same sums), by the row's and the column's
products a normal variable of many terms.  Held: 16 of its standard deviations, 2^-12 of
sqrt(sum of the squared products), for every element; 2^-15 in the root mean square where at least 50000
elements (some 150 of them rounded the other way, so the estimate of d^2 is good to 10%) tell it.
"""
import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_operators import (TD, Guarded, aligned, close, gemm_norm, gemm_tol, gen, operands,
                                product, row_codes, say)

pytestmark = pytest.mark.gpu

UNITS = 256                     # compute units of an MI355X
TILES = [(13, 56, 4224), (16, 60, 4224), (5, 61, 4224), (19, 56, 2176), (17, 63, 2176),
         (18, 60, 2176), (3, 7178, 4224), (12, 7216, 4224), (1, 7617, 4224), (2068, 70, 1152),
         (17, 8672, 1152), (2215, 71, 1152), (36, 8342, 1152), (37, 8255, 1152), (36, 8552, 1152),
         (92, 9543, 1152), (99, 8326, 640), (3271, 261, 640), (6572, 136, 640), (6238, 415, 1024),
         (6739, 386, 1024), (4930, 560, 1024), (6867, 679, 3200), (5186, 904, 3200),
         (5208, 930, 3200), (5506, 270, 3328), (5528, 264, 3456), (5812, 267, 3328),
         (1417, 5448, 512), (1677, 4649, 512), (1059, 7402, 512), (1415, 8363, 512),
         (5818, 2062, 512), (2576, 4728, 512)]
# 256x256 tiles whose last round runs as halves of 128 rows, the last of them with rows and without
HALVES = [(2566, 7693, 640), (3714, 5389, 640), (2309, 8624, 640), (6019, 3338, 1152)]


def squares(a, sa, b, sb, b_block):
    """sqrt(sum of the squared products) of every element."""
    sbr = sb if b_block == 1 else sb.repeat_interleave(128, 0)[: b.shape[0]]
    a64 = a.view(torch.float8_e4m3fn).double() * sa.double().repeat_interleave(128, 1)
    b64 = b.view(torch.float8_e4m3fn).double() * sbr.double().repeat_interleave(128, 1)
    return ((a64 * a64) @ (b64 * b64).t()).sqrt()


def beyond_rounding(got, ref, scale):
    """Holds the error of a bf16 result before its rounding (see above); returns its estimate."""
    near = ref.bfloat16().double()            # through fp32: off by 2^-24 of ref at most
    excess = (got.double() - ref).abs() - (near - ref).abs()
    worst = (excess - 2 * 2.0 ** -12 * scale - 2 * 2.0 ** -24 * ref.abs()).max()
    assert float(worst) <= 0.0, f"{float(worst):.3e} beyond the product's own error"
    step = torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=1e-30))) - 7)
    rms = float(((excess * step).sum().clamp(min=0.0) / (ref * ref).sum()).sqrt())
    if ref.numel() >= 50000:
        assert rms <= 2.0 ** -15, rms
    return rms


@pytest.mark.parametrize("b_block", [128, 1])
@pytest.mark.parametrize("c", TILES + HALVES, ids=str)
def test_dense(device, c, b_block):
    m, n, k = c
    say("dense", c, b_block)
    a, sa, b, sb = operands(device, m, n, k, b_block, 80)
    ref, mag = product(a, sa, b, sb, b_block)
    for dtype in ("bf16", "f32"):
        c_ = Guarded((m, n), TD[dtype], device)
        moe.moe_gemm_e4m3(a, sa, b, sb, b_block, c_.t)
        torch.cuda.synchronize()
        assert c_.intact(), dtype
        close(c_.t, ref, gemm_tol(ref, mag, k, dtype), dtype)
        if dtype == "f32":
            gemm_norm(c_.t, ref, dtype)
        else:
            say("before rounding", beyond_rounding(c_.t, ref, squares(a, sa, b, sb, b_block)))


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("m,n,k", [(1, 50000, 7168), (16, 8192, 2048), (700, 2880, 4096)])
def test_dense_before_rounding(device, m, n, k, seed):
    """The same for more operands, one row among them."""
    a, sa, b, sb = operands(device, m, n, k, 128, 81 + seed)
    ref, _ = product(a, sa, b, sb, 128)
    got = moe.gemm_e4m3(a, sa, b, sb)
    torch.cuda.synchronize()
    say("before rounding", (m, n, k), beyond_rounding(got, ref, squares(a, sa, b, sb, 128)))


# (T, E, k, block_m, n, kk)
GROUPED = [(20, 4, 2, 16, 200, 2176), (60, 3, 2, 16, 203, 2176), (200, 20, 2, 16, 1111, 896),
           (200, 40, 2, 16, 1112, 1152), (50, 3, 2, 32, 201, 1408), (20, 3, 2, 32, 200, 1408),
           (300, 12, 3, 32, 1001, 896), (100, 12, 2, 32, 1002, 1152), (60, 2, 2, 64, 129, 1408),
           (200, 2, 1, 64, 128, 1408), (400, 8, 3, 64, 1000, 896), (150, 10, 3, 64, 1279, 1152),
           (400, 8, 3, 64, 1101, 896), (150, 10, 3, 64, 1344, 1152), (700, 6, 3, 128, 1000, 896),
           (700, 6, 3, 128, 1101, 896), (90, 9, 2, 128, 1023, 1152)]


def grouped(device, T, E, k, bm, n, kk, dtype, sample):
    """One grouped product between guards; `sample` rows of every expert are compared."""
    p, a, used, ss, held = aligned(device, T, 128, E, k, bm, "all", 82, fp8=True)
    g = gen(device, 83)
    rows, rs = row_codes(torch.randn((ss.numel(), kk), generator=g, device=device))
    rows.view(torch.uint8)[~held] = 0x7F                  # no slot's: never read
    w, _ = row_codes(torch.randn((E * n, kk), generator=g, device=device))
    w = w.view(E, n, kk)
    ws = torch.rand((E, -(-n // 128), kk // 128), generator=g, device=device) + 0.1
    out = Guarded((ss.numel(), n), TD[dtype], device)
    moe.grouped_gemm_e4m3(p, rows, rs, w, ws, a, out=out.t)
    torch.cuda.synchronize()
    assert out.intact(used)
    assert not bool(out.t[:used][~held[:used]].any()), "padding rows"
    at = a["offsets"].tolist()
    for e in range(E):
        mine = torch.arange(at[e], at[e + 1], device=device)[held[at[e]:at[e + 1]]]
        if mine.numel() > sample:
            mine = mine[torch.linspace(0, mine.numel() - 1, sample, device=device).long()]
        if not mine.numel():
            continue
        args = rows.view(torch.uint8)[mine], rs[mine], w[e], ws[e], 128
        ref, mag = product(*args)
        close(out.t[mine], ref, gemm_tol(ref, mag, kk, dtype), f"expert {e}")
        if dtype == "f32":
            gemm_norm(out.t[mine], ref, dtype)
        else:
            beyond_rounding(out.t[mine], ref, squares(*args))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", GROUPED, ids=str)
def test_grouped(device, c, dtype):
    say("grouped", c, dtype)
    grouped(device, *c, dtype, 1 << 30)
