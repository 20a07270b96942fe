"""What the operators before the layer and beside it promise of 64 bits, where 32 would not do: groups whose
large scores cancel."""
import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_block_operators import U32, close, ref_route
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
