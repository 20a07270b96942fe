"""What the GPU tests hold about a bf16 product's error before its rounding, on made-up sums (host)."""
import pytest
import torch

from test_gpu_gemm_tiles import beyond_rounding
from test_gpu_operators import gemm_norm


def sums(error, seed=0):
    """(bf16 of sums that are off by `error` of their scale, the sums, their scale, how far off)."""
    g = torch.Generator()
    g.manual_seed(seed)
    scale = torch.exp(torch.randn(400, 500, generator=g, dtype=torch.float64))
    ref = scale * torch.randn(400, 500, generator=g, dtype=torch.float64)
    off = error * scale * torch.randn(400, 500, generator=g, dtype=torch.float64)
    v = (ref + off).float()
    return v.bfloat16(), ref, scale, v.double() - ref


@pytest.mark.parametrize("error", [0.0, 2.0 ** -24, 2.0 ** -18, 2.0 ** -16])
def test_estimate(error):
    """The estimate is the error that was planted, and passes.  An element whose sum is off by d in a
    step s is rounded the other way with probability |d| / s, its excess is then uniform up to 2 |d|,
    so what it adds to the estimate of sum(d^2) has the variance (|d| / s) (4 d^2 / 3) s^2 = 4/3
    |d|^3 s at most: held to 6 standard deviations."""
    got, ref, scale, d = sums(error)
    step = torch.exp2(torch.floor(torch.log2(ref.abs())) - 7)
    six = 6 * float((4 / 3 * d.abs() ** 3 * step).sum().sqrt())
    square = beyond_rounding(got, ref, scale) ** 2 * float((ref * ref).sum())
    assert abs(square - float((d * d).sum())) <= six


@pytest.mark.parametrize("error", [2.0 ** -14, 2.0 ** -12, 2.0 ** -9])
def test_larger_errors_are_found(error):
    """Also where the norm of the rounded result does not show them."""
    got, ref, scale, _ = sums(error)
    if error < 2.0 ** -9:
        gemm_norm(got, ref, "bf16")
    with pytest.raises(AssertionError):
        beyond_rounding(got, ref, scale)


def test_one_wrong_element_is_found():
    got, ref, scale, _ = sums(2.0 ** -16)
    at = int((ref.abs() / scale - 0.5).abs().argmin())             # an ordinary one
    got.view(-1)[at] = float(ref.view(-1)[at]) * (1 + 2.0 ** -6)
    with pytest.raises(AssertionError):
        beyond_rounding(got, ref, scale)
