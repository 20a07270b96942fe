"""Sizes and choices that do not fit the C entry points' 32-bit arguments are refused by the binding;
ctypes would drop their upper bits and the library would see a small, valid call."""
import pytest
import torch

import routed_grouped_gemm_topk_amd as moe

E4M3 = torch.float8_e4m3fn


def none(*shape, dtype=E4M3):
    """A tensor without memory: of the right shape, so that only the sizes are wrong."""
    return torch.empty(shape, dtype=dtype, device="meta")


def refused(call):
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.MOE_ERR_SHAPE


@pytest.mark.parametrize("m,n", [(2 ** 32 + 128, 8), (2 ** 31, 8), (8, 2 ** 32 + 8)])
def test_quantize_cols(m, n):
    groups = -(-m // 128)
    refused(lambda: moe.moe_quantize_cols_e4m3(
        none(m, n, dtype=torch.bfloat16), none(n, groups * 128),
        none(n, groups, dtype=torch.float32)))


@pytest.mark.parametrize("m,n,k", [(1, 1, 2 ** 32 + 128), (1, 1, 2 ** 31), (2 ** 32 + 1, 4, 128),
                                   (4, 2 ** 32 + 1, 128)])
def test_gemm(m, n, k):
    g = k // 128
    refused(lambda: moe.moe_gemm_e4m3(
        none(m, k), none(m, g, dtype=torch.float32), none(n, k),
        none(-(-n // 128), g, dtype=torch.float32), 128, none(m, n, dtype=torch.bfloat16)))


@pytest.mark.parametrize("b_block", [2 ** 32 + 1, 2 ** 32 + 128, 0, -1, 64])
def test_gemm_b_block(b_block):
    refused(lambda: moe.moe_gemm_e4m3(
        none(4, 256), none(4, 2, dtype=torch.float32), none(300, 256),
        none(3, 2, dtype=torch.float32), b_block, none(4, 300, dtype=torch.bfloat16)))


@pytest.mark.parametrize("n,k", [(1, 2 ** 32 + 128), (2 ** 32 + 128, 128)])
def test_grouped_gemm(n, k):
    p = moe.make_problem(4, 128, 128, 1, 1, "bf16", "e4m3", 16)
    rm = moe.moe_max_padded_slots(p)
    i32 = torch.int32
    refused(lambda: moe.moe_grouped_gemm_e4m3(
        p, none(rm, k), none(rm, k // 128, dtype=torch.float32), none(1, n, k),
        none(1, -(-n // 128), k // 128, dtype=torch.float32), none(rm, dtype=i32),
        none(2, dtype=i32), none(2 * moe.moe_max_tiles(p), dtype=i32), none(1, dtype=i32),
        none(rm, n, dtype=torch.bfloat16)))
