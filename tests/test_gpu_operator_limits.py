"""The largest sizes that the operators' calls accept in one dimension, many experts per token, one
expert's weight gradient, and dense products and the transposed quantiser in a captured graph; against
64 bits."""
import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_operators import (TD, U32, UBF, UT, Guarded, aligned, close, gemm_tol, gen, operands,
                                product, say, sorted_rows)

pytestmark = pytest.mark.gpu


def codes(device, rows, cols, g):
    """Finite e4m3 codes of every size and both signs."""
    c = torch.randint(0, 0x7F, (rows, cols), generator=g, device=device, dtype=torch.uint8)
    return c | (torch.randint(0, 2, (rows, cols), generator=g, device=device, dtype=torch.uint8) << 7)


@pytest.mark.parametrize("m,n,b_block", [(5, 40, 128), (40, 70, 1), (300, 200, 128), (2000, 1800, 128),
                                         (2100, 2300, 1), (4096, 4096, 128)])
def test_gemm_longest_k(device, m, n, b_block):
    """k = 2^22: a tile's rows span 2^30 bytes.  Rows that lie in the first and the last tiles."""
    k = 2 ** 22
    say("longest k", m, n, b_block)
    g = gen(device, 100)
    a, b = codes(device, m, k, g), codes(device, n, k, g)
    sa = torch.rand((m, k // 128), generator=g, device=device) + 0.1
    sb = torch.rand((n if b_block == 1 else -(-n // 128), k // 128), generator=g, device=device) + 0.1
    i, j = (torch.tensor(sorted({0, 1, s // 3, s - 2, s - 1}), device=device) for s in (m, n))
    ref = torch.zeros((i.numel(), j.numel()), dtype=torch.float64, device=device)
    mag = ref.clone()
    sbj = sb[j if b_block == 1 else j // 128]
    for at in range(0, k, 2 ** 18):
        s, t = slice(at, at + 2 ** 18), slice(at // 128, at // 128 + 2 ** 11)
        r, q = product(a[i][:, s], sa[i][:, t], b[j][:, s], sbj[:, t], 1)
        ref, mag = ref + r, mag + q
    for dtype in ("bf16", "f32"):
        c = moe.gemm_e4m3(a, sa, b, sb, out_dtype=TD[dtype], b_block=b_block)
        torch.cuda.synchronize()
        close(c[i][:, j], ref, gemm_tol(ref, mag, k, dtype), dtype)


@pytest.mark.parametrize("m,n", [(1, 2 ** 24), (16, 2 ** 24 - 3), (17, 2 ** 24), (2 ** 24, 3),
                                 (2 ** 24 - 5, 24), (2 ** 24, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gemm_longest_m_and_n(device, m, n, dtype):
    say("longest", m, n, dtype)
    g = gen(device, 101)
    a, b = codes(device, m, 128, g), codes(device, n, 128, g)
    sa = torch.rand((m, 1), generator=g, device=device) + 0.1
    sb = torch.rand((-(-n // 128), 1), generator=g, device=device) + 0.1
    c = Guarded((m, n), TD[dtype], device)
    moe.moe_gemm_e4m3(a, sa, b, sb, 128, c.t)
    torch.cuda.synchronize()
    assert c.intact()
    step = 2 ** 21
    for at in range(0, max(m, n), step):
        if m > n:
            s = slice(at, at + step)
            ref, mag = product(a[s], sa[s], b, sb, 128)
            got = c.t[s]
        else:
            s, t = slice(at, at + step), slice(at // 128, (at + step) // 128)
            ref, mag = product(a, sa, b[s], sb[t], 128)
            got = c.t[:, s]
        close(got, ref, gemm_tol(ref, mag, 128, dtype), (at, dtype))


@pytest.mark.parametrize("m,n", [(2 ** 22, 8), (2 ** 22 - 1, 16), (3, 2 ** 22), (130, 2 ** 21)])
def test_quantize_cols_longest(device, m, n):
    say("quantize_cols", m, n)
    x = torch.randn((m, n), generator=gen(device, 102), device=device).bfloat16()
    groups = -(-m // 128)
    xq = Guarded((n, groups * 128), torch.uint8, device)
    sc = Guarded((n, groups), torch.float32, device)
    moe.moe_quantize_cols_e4m3(x, xq.t, sc.t)
    torch.cuda.synchronize()
    assert xq.intact() and sc.intact()
    step = 2 ** 25 // (groups * 128)
    for c in range(0, n, max(step, 1)):
        part = x[:, c:c + max(step, 1)].float()
        v = torch.zeros((groups * 128, part.shape[1]), device=device)
        v[:m] = part
        v = v.t().contiguous().view(-1, groups, 128)
        amax = v.abs().amax(2)
        s = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
        q = (v / s[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, groups * 128)
        assert torch.equal(sc.t[c:c + q.shape[0]], s) and torch.equal(xq.t[c:c + q.shape[0]], q), c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,bm", [(7, 1024, 1024, 16), (90, 130, 101, 64), (1, 5, 5, 16)])
def test_many_experts_per_token(device, T, E, k, bm, dtype):
    """Rows, combine and gradient for up to 1024 slots per token."""
    H = 192
    say("experts per token", k, dtype)
    p, a, used, ss, held = aligned(device, T, H, E, k, bm, "some", 103)
    g = gen(device, 104)
    dt = TD[dtype]
    x, d_out = (torch.randn((T, H), generator=g, device=device).to(dt) for _ in range(2))
    w = torch.randn((T, k), generator=g, device=device)
    rows, _ = moe.permute(p, x, a)
    y = sorted_rows(device, ss, held, H, dt, 105)
    out = moe.unpermute(p, y, a, w)
    d_rows, d_w = moe.unpermute_bwd(p, d_out, y, a, w)
    torch.cuda.synchronize()
    tok = (ss // k).clamp(max=T - 1)
    assert torch.equal(rows[:used], torch.where(held[:, None], x[tok], 0.0)[:used])
    at = a["slot_row"].long().view(T, k)
    there = (at >= 0)[:, :, None]
    yt = torch.where(there, y.double()[at.clamp(min=0)], 0.0)
    wd = torch.where(there, w.double()[:, :, None], 0.0)
    ref, mag = (yt * wd).sum(1), (yt * wd).abs().sum(1)
    u = UT[dtype]
    close(out, ref, (k + 1) * U32 * mag + u * (ref.abs() + (k + 1) * U32 * mag) + 1e-38, "out")
    terms = yt * d_out.double()[:, None, :]
    close(d_w, terms.sum(2), (H / 64 + 8) * U32 * terms.abs().sum(2), "d_weights")
    want = (wd * d_out.double()[:, None, :])[there[:, :, 0]]
    close(d_rows[at[there[:, :, 0]]], want, (u + 2 * U32) * want.abs() + 1e-38, "d_rows")


def test_expert_weight_gradients(device):
    """d_w[e] = sum over the expert's rows of d_y x, from slices of the sorted rows, padding and all:
    the product of the codes, and within e4m3's rounding (2^-4 of each operand, and what falls below
    the smallest code) that of the tokens themselves."""
    T, H, n, E, k, bm = 500, 256, 136, 6, 2, 64
    p, a, used, ss, held = aligned(device, T, H, E, k, bm, "some", 110)
    pn = moe.make_problem(T, 192, 128, E, k, "bf16", None, bm)
    g = gen(device, 111)
    x = torch.randn((T, H), generator=g, device=device).bfloat16()
    d_out = torch.randn((T, 192), generator=g, device=device).bfloat16()
    w = torch.rand((T, k), generator=g, device=device) + 0.5
    rows, _ = moe.permute(p, x, a)
    y = sorted_rows(device, ss, held, 192, torch.bfloat16, 112)
    d_rows, _ = moe.unpermute_bwd(pn, d_out, y, a, w)
    at = a["offsets"].tolist()
    for e in range(E):
        mine = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        dy = d_rows[mine, :n].contiguous()
        q, s = moe.quantize_cols_e4m3(dy)
        qx, sx = moe.quantize_cols_e4m3(rows[mine])
        dw = moe.gemm_e4m3(q, s, qx, sx, out_dtype=torch.float32, b_block=1)
        torch.cuda.synchronize()
        ref, mag = product(q, s, qx, sx, 1)
        close(dw, ref, gemm_tol(ref, mag, q.shape[1], "f32"), f"expert {e}")
        slot = ss[mine][held[mine]]
        d64 = d_out.double()[slot // k, :n] * w.double().view(-1)[slot][:, None]
        x64 = x.double()[slot // k]
        m = slot.numel()
        sub = 2.0 ** -10 * m * (s.double().amax(1)[:, None] * x64.abs().amax() * 2
                                + sx.double().amax(1)[None, :] * d64.abs().amax() * 2)
        tol = (2 * 2.0 ** -4 + 2.0 ** -8 + UBF) * 1.01 * (d64.abs().t() @ x64.abs()) + sub
        close(dw, d64.t() @ x64, tol, f"expert {e}, its tokens")


def test_products_in_a_graph(device):
    """Dense products on kernels of every kind and the quantiser, captured once and replayed on new
    operands, with eager work between the replays."""
    shapes = [(1, 600, 1152), (40, 4100, 640), (300, 520, 2048), (1000, 2049, 256), (3718, 5402, 384)]
    sets = [[operands(device, *s, bb, 106 + i) for i, s in enumerate(shapes)] for bb in (128, 1)]
    x = torch.randn((1000, 520), generator=gen(device, 107), device=device).bfloat16()

    def work():
        out = [moe.gemm_e4m3(*ops, out_dtype=dt, b_block=bb) for bb, group in zip((128, 1), sets)
               for ops in group for dt in (torch.bfloat16, torch.float32)]
        q, s = moe.quantize_cols_e4m3(x)
        return out + [s, q.view(torch.uint8), moe.gemm_e4m3(q, s, q, s, torch.float32, 1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for rep in range(3):
        for bb, group in zip((128, 1), sets):
            for i, s in enumerate(shapes):
                for t, new in zip(group[i], operands(device, *s, bb, 200 + 10 * rep + i)):
                    t.view(torch.uint8).copy_(new.view(torch.uint8))
        x.copy_(torch.randn(x.shape, generator=gen(device, 300 + rep), device=device))
        graph.replay()
        torch.cuda.synchronize()
        eager = work()
        torch.cuda.synchronize()
        for i, (got, want) in enumerate(zip(held, eager)):
            assert torch.equal(got, want), (rep, i)
