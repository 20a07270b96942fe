"""Values at the edges of their types in the operators beside the layer: signed zeros among logits that
tie, weights below fp32's normal numbers, scales below them, bf16 operands below theirs."""
import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_block_operators import F64, TD, U32, close, ref_norm, ref_route
from test_gpu_operators import E4M3, gen, say


def test_act_bwd_refuses_a_d_z_that_it_would_not_fill():
    d_c, d_z = torch.zeros((2, 8)).bfloat16(), torch.zeros((2, 8)).bfloat16()
    for d_bias in (False, True):
        with pytest.raises(ValueError, match="d_z"):
            moe.act_bwd(d_c, d_bias=d_bias, d_z=d_z)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_scored_signed_zeros(device, dtype, score):
    """-0 and 0 are the same logit: the lower id, and the lower group, come first."""
    T, E, k = 65, 64, 6
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    g = gen(device, 130)
    x = torch.where(torch.rand((T, E), generator=g, device=device) < 0.5, -0.0, 0.0)
    x[::3] -= (torch.rand((T, E), generator=g, device=device) < 0.3).float()[::3]
    x = x.to(TD[dtype])
    for r in (moe.make_router(score), moe.make_router(score, True, 8, 3, 1),
              moe.make_router(score, True, 8, 3, 2)):
        say("signed zeros", dtype, score, r)
        ids, w = moe.route_scored(p, r, x)
        ref_ids, ref_w = ref_route(x.cpu(), None, r, k)
        assert torch.equal(ids.cpu().long(), ref_ids)
        close(w.cpu(), ref_w, (50 + k) * U32 * ref_w.abs(), "weights")


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored_weights_of_tiny_scores(device, score, renorm):
    """Scores down to exp(-100), which fp32 holds with few bits or none, times a scale of 2^60: the
    weights are normal numbers and as exact as others."""
    T, E, k = 40, 32, 4
    p = moe.make_problem(T, 64, 64, E, k, "bf16")
    x = -80.0 - 20.0 * torch.rand((T, E), generator=gen(device, 131), device=device)
    x[::2, 5] = 0.0
    for r in (moe.make_router(score, renorm, scale=2.0 ** 60),
              moe.make_router(score, renorm, 4, 4, 2, 2.0 ** 60)):
        for b in (None, torch.zeros(E, device=device)):
            ids, w = moe.route_scored(p, r, x, b)
            ref_ids, ref_w = ref_route(x.cpu(), None if b is None else b.cpu(), r, k)
            assert torch.equal(ids.cpu().long(), ref_ids)
            assert float(ref_w.min()) > 2.0 ** -126
            close(w.cpu(), ref_w, (50 + k) * U32 * ref_w.abs(), "weights")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rms_norm_codes_of_tiny_groups(device, dtype):
    """A group whose values lie far below the row's: scales end at 2^-126, codes are finite and as near
    as e4m3 has them, in groups whose own scale would be 0 as well.  The quotients are n 2^126, n in
    fp32 with half a step of 2^-150 per product (of up to 4 u as elsewhere): 2^-23 of a code's unit."""
    T, H = 64, 1024
    g = gen(device, 132)
    x = torch.randn((T, H), generator=g, device=device)
    size = 2.0 ** (-100 - 50 * torch.rand((T, 7, 1), generator=g, device=device))
    x.view(T, 8, 128)[:, 1:] *= size
    x = x.to(TD[dtype])
    out = moe.rms_norm(x, eps=0.0, want=("y", "codes"))
    n = ref_norm(x, None, 0.0)[1]
    v = n.view(T, 8, 128)
    amax = v.abs().amax(2)
    assert int((amax < 2.0 ** -126).sum()) > 30 and int((amax == 0).sum()) < 200
    live = amax > 2.0 ** -148
    want = (amax / 448).clamp(min=2.0 ** -126)
    close(out["scales"][live], want[live], 6 * U32 * want[live] + 2.0 ** -149, "scales")
    q = v / out["scales"].to(F64)[:, :, None]
    codes = out["codes"].view(T, 8, 128).to(F64)
    best = q.float().clamp(-448, 448).to(E4M3).to(F64)
    far = (codes - q).abs() - (best - q).abs() - 2 * 6 * U32 * q.abs() - 2.0 ** -22
    assert not torch.isnan(codes).any()
    assert float(far[live].max()) <= 0 and not codes[amax < 2.0 ** -150].any()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
def test_gemm_of_subnormal_operands(device, layout):
    """bf16 values below 2^-126 count: times 2^100 they are ordinary products."""
    for m, n, k in [(1, 256, 520), (70, 72, 136), (300, 264, 200), (5, 7, 33)]:
        say("subnormal", m, n, k, layout)
        g = gen(device, 133)
        sa, sb = ((k, m) if layout == "tn" else (m, k)), ((n, k) if layout == "nt" else (k, n))
        a = (torch.randint(-7, 8, sa, generator=g, device=device).double() * 2.0 ** -130).bfloat16()
        b = (torch.randint(-7, 8, sb, generator=g, device=device).double() * 2.0 ** 100).bfloat16()
        a64, b64 = a.to(F64), b.to(F64)
        assert float(a64.abs().amax()) > 0
        z = (a64.t() if layout == "tn" else a64) @ (b64.t() if layout == "nt" else b64)
        out = moe.gemm_bf16(a, b, layout, out_dtype=torch.float32)
        assert torch.equal(out.double(), z)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
def test_gemm_rows_of_any_alignment_between_nan(device, layout):
    """Operands right between NaN, down to less than one load of 8 values, rows that end inside one:
    nothing beside an operand, and nothing of a row's neighbour, reaches a result."""
    for m, n, k in [(1, 1, 1), (1, 3, 5), (2, 3, 3), (7, 1, 1), (1, 7, 1), (8, 1, 1), (1, 8, 1), (1, 9, 7),
                    (3, 3, 3), (1, 20001, 3), (20001, 1, 5), (9, 9, 9), (63, 65, 66), (70, 131, 67),
                    (129, 270, 515), (1030, 1031, 65), (2049, 1027, 131), (1027, 2050, 200)]:
        say("any alignment", m, n, k, layout)
        g = gen(device, 134)
        held = []
        for shape in (((k, m) if layout == "tn" else (m, k)), ((n, k) if layout == "nt" else (k, n))):
            size = shape[0] * shape[1]
            buf = torch.full((size + 128,), float("nan"), dtype=torch.bfloat16, device=device)
            held.append(buf[64:64 + size].view(shape))
            held[-1].copy_(torch.randint(-2, 3, shape, generator=g, device=device))
        a, b = held
        out = moe.gemm_bf16(a, b, layout, out_dtype=torch.float32)
        a64, b64 = a.to(F64), b.to(F64)
        z = (a64.t() if layout == "tn" else a64) @ (b64.t() if layout == "nt" else b64)
        assert torch.equal(out.double(), z)
        # NaN in one row (column) of an operand stays in its row (column) of the result
        (a.t() if layout == "tn" else a)[m // 2] = float("nan")
        out = moe.gemm_bf16(a, b, layout, out_dtype=torch.float32)
        rows = torch.arange(m, device=device) != m // 2
        assert torch.equal(out[rows].double(), z[rows]) and torch.isnan(out[m // 2]).all()
