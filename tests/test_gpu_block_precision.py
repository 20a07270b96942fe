"""What the operators before the layer and beside it promise of 64 bits, where 32 would not do: groups whose
large scores cancel, weights of the router rounded once.

Tolerances (u = 2^-24, half a step of fp32, relative; 2^-150 absolute below fp32's normal numbers):
  * the router's weights: sums of at most 1024 terms in 64 bits, each off by a few 2^-53, stay within
    2^-40 of the terms' magnitudes; then one rounding to fp32.
"""
import math

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_block_operators import ROUTERS, U32, WAYS, close, make_logits, ref_route, scores, weights_of
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
# weights of the router
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
