"""bf16 products on every kernel that their choice has, in every layout, against 64 bits.

TILES reaches, on a device of UNITS compute units, every kernel in every layout with rows of c that begin
on 16 bytes, on an even and on an odd number of values, with ragged last tiles and so many slices of k
that every ring of stages is refilled (test_gemm_bf16_choice.py holds it to that).  Operands, bias and
residual are small integers: the products and their sums in fp32 are exact in any order, so results
before an activation are compared bit for bit.  After one: 8 u of |z| and |c| for the function in fp32
and the residual's addition, and the rounding of the result, as in test_gpu_block_operators.py.
"""
import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_block_operators import ACTS, F64, TD, U32, UBF, operands
from test_gpu_operators import Guarded, close, gen, say

pytestmark = pytest.mark.gpu

UNITS = 256                     # compute units of an MI355X
TILES = [(3, 2, 773, "nn"), (3, 3, 773, "nn"), (3, 8, 771, "nn"), (3, 2, 796, "nt"), (3, 3, 780,
         "nt"), (3, 8, 771, "nt"), (3, 2, 777, "tn"), (3, 3, 774, "tn"), (3, 8, 772, "tn"), (139,
         8846, 203, "nn"), (130, 10481, 208, "nn"), (178, 8208, 194, "nn"), (135, 8964, 199, "nt"),
         (130, 8635, 202, "nt"), (270, 5384, 203, "nt"), (145, 8348, 218, "tn"), (156, 8077, 197,
         "tn"), (138, 8656, 206, "tn"), (1, 2, 2568, "nt"), (1, 3, 2568, "nt"), (1, 8, 2568, "nt"),
         (1, 4106, 2104, "nt"), (1, 4119, 2160, "nt"), (1, 4240, 2088, "nt"), (3, 8, 648, "nn"),
         (4287, 2, 648, "nt"), (4260, 3, 648, "nt"), (3, 8680, 800, "nt"), (33, 8584, 528, "nn"),
         (34, 8196, 552, "nt"), (34, 8295, 528, "nt"), (4414, 72, 528, "nt"), (8, 8, 513, "tn"),
         (65, 8616, 264, "nn"), (70, 8374, 280, "nt"), (66, 8989, 264, "nt"), (67, 8904, 264, "nt"),
         (72, 8440, 263, "tn"), (5444, 272, 264, "nn"), (5486, 260, 272, "nt"), (5485, 267, 264,
         "nt"), (6003, 264, 264, "nt"), (136, 10944, 269, "tn"), (6947, 520, 264, "nn"), (260,
         13340, 272, "nt"), (261, 13609, 264, "nt"), (456, 8272, 264, "nt"), (5448, 664, 257, "tn"),
         (6764, 1048, 264, "nn"), (670, 10770, 272, "nt"), (1155, 6507, 264, "nt"), (3641, 2064,
         264, "nt"), (5416, 1304, 259, "tn"), (982, 8368, 328, "nn"), (577, 13746, 328, "nt"), (652,
         12365, 344, "nt"), (782, 9912, 344, "nt"), (584, 13416, 328, "tn"), (779, 13440, 264,
         "nn"), (774, 13930, 288, "nt"), (1005, 10907, 264, "nt"), (1173, 9344, 272, "nt"), (6960,
         1560, 268, "tn"), (17, 9, 2640, "nt"), (17, 8, 2648, "nt"), (17, 10, 2640, "nt"), (17,
         2085, 2672, "nt"), (17, 2056, 2672, "nt"), (17, 2068, 2640, "nt"),
         (700, 1001, 1100, "nt"), (700, 1002, 1100, "nt"), (700, 1000, 1100, "nt"),
         (3, 3, 5301, "nt"), (19, 10, 5300, "nt"), (17, 24, 5303, "nt")]
# 256x256 tiles whose last round runs as halves of 128 rows, the last of them with rows and without
HALVES = [(1554, 11080, 272, "nn"), (1443, 12368, 264, "nn"), (1384, 12483, 264, "nt"), (1166,
          14501, 264, "nt"), (1544, 11208, 263, "tn"), (1224, 14216, 264, "tn")]


@pytest.mark.parametrize("c", TILES + HALVES, ids=str)
def test_tiles(device, c):
    m, n, k, layout = c
    say("tiles", c)
    a, b, a64, b64 = operands(m, n, k, layout, device, 60, ints=True)
    g = gen(device, 61)
    bias = torch.randint(-9, 10, (n,), generator=g, device=device).float()
    ref = a64 @ b64
    out = Guarded((m, n), torch.float32, device)
    moe.moe_gemm_bf16(layout, a, b, None, "none", None, None, out.t)
    torch.cuda.synchronize()
    assert out.intact() and torch.equal(out.t, ref.float())
    res = torch.randint(-9, 10, (m, n), generator=g, device=device).bfloat16()
    ref += bias.to(F64)
    for act in ("none", "silu"):
        out = Guarded((m, n), torch.bfloat16, device)
        pre = Guarded((m, n), torch.bfloat16, device)
        moe.moe_gemm_bf16(layout, a, b, bias, act, res, pre.t, out.t)
        torch.cuda.synchronize()
        assert out.intact() and pre.intact() and torch.equal(pre.t, ref.bfloat16()), act
        want = ACTS[act](ref) + res.to(F64)
        if act == "none":
            assert torch.equal(out.t, want.bfloat16())
        else:
            close(out.t, want, 8 * U32 * (ref.abs() + want.abs()) + UBF * want.abs(), act)
        again = torch.empty((m, n), dtype=torch.bfloat16, device=device)
        moe.moe_gemm_bf16(layout, a, b, bias, act, res, None, again)
        torch.cuda.synchronize()
        assert torch.equal(again, out.t), act
