"""The largest sizes that the operators beside the layer accept, elements past 2^31 and bytes past 2^32.

Products have operands that are small integers, so that every sum is exact in any order.  Norm, router and
their gradients treat every row for itself: rows of a large call equal, bit for bit, those of a small
call of the same rows, which other tests compare with 64 bits."""
import math

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_block_operators import F64, U32, UBF
from test_gpu_operators import Guarded, close, gen, say

pytestmark = pytest.mark.gpu


def ints(shape, g, device, low=-2, high=2):
    return torch.randint(low, high + 1, shape, generator=g, device=device, dtype=torch.int8).bfloat16()


@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
@pytest.mark.parametrize("m,n,k", [(3, 5, 2 ** 24), (16, 8, 2 ** 21), (24, 40, 2 ** 21 + 8),
                                   (72, 136, 2 ** 21), (304, 200, 2 ** 21 - 3)])
def test_gemm_longest_k(device, m, n, k, layout):
    """Up to 2^24 products of -1, 0 and 1: sums of up to 2^24, still exact."""
    say("longest k", m, n, k, layout)
    g = gen(device, 120)
    a = ints((k, m) if layout == "tn" else (m, k), g, device, -1, 1)
    b = ints((n, k) if layout == "nt" else (k, n), g, device, -1, 1)
    out = Guarded((m, n), torch.float32, device)
    moe.moe_gemm_bf16(layout, a, b, None, "none", None, None, out.t)
    torch.cuda.synchronize()
    a64, b64 = (a.t() if layout == "tn" else a), (b.t() if layout == "nt" else b)
    want = torch.zeros((m, n), dtype=F64, device=device)
    for at in range(0, k, 2 ** 20):
        want += a64[:, at:at + 2 ** 20].to(F64) @ b64[at:at + 2 ** 20].to(F64).contiguous()
    assert out.intact() and torch.equal(out.t.double(), want)


@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
@pytest.mark.parametrize("m,n,k", [(1, 2 ** 24, 8), (2 ** 24, 8, 8), (2 ** 24 - 3, 5, 16),
                                   (17, 2 ** 24 - 7, 8), (2 ** 23, 16, 72), (24, 2 ** 23, 72)])
def test_gemm_longest_m_and_n(device, m, n, k, layout):
    say("longest", m, n, k, layout)
    g = gen(device, 121)
    a = ints((k, m) if layout == "tn" else (m, k), g, device)
    b = ints((n, k) if layout == "nt" else (k, n), g, device)
    bias = torch.randint(-9, 10, (n,), generator=g, device=device).float()
    out = Guarded((m, n), torch.bfloat16, device)
    moe.moe_gemm_bf16(layout, a, b, bias, "none", None, None, out.t)
    torch.cuda.synchronize()
    assert out.intact()
    a32, b32 = (a.t() if layout == "tn" else a), (b.t() if layout == "nt" else b)
    step = 2 ** 21
    for at in range(0, max(m, n), step):
        s = slice(at, at + step)
        if m > n:
            want, got = a32[s].float() @ b32.float() + bias, out.t[s]
        else:
            want, got = a32.float() @ b32[:, s].float() + bias[s], out.t[:, s]
        assert torch.equal(got, want.bfloat16()), at


@pytest.mark.parametrize("m,n,k,layout", [(70008, 31000, 72, "nt"), (70008, 31000, 72, "nn"),
                                          (70008, 31000, 65, "tn"), (70001, 30801, 40, "nt"),
                                          (70001, 30801, 33, "nn"),
                                          (300008, 8, 8200, "nt"), (8, 300008, 8200, "nn"),
                                          (300008, 16, 8200, "tn"), (16, 300001, 8193, "nt")])
def test_gemm_past_32_bits(device, m, n, k, layout):
    """A result, or an operand, of more than 2^31 elements and 2^32 bytes, with a residual and pre
    beside the result."""
    say("past 32 bits", m, n, k, layout)
    assert max(m * n, m * k, n * k) > 2 ** 31
    g = gen(device, 122)
    a = ints((k, m) if layout == "tn" else (m, k), g, device)
    b = ints((n, k) if layout == "nt" else (k, n), g, device)
    res = ints((m, n), g, device, -9, 9)
    out, pre = Guarded((m, n), torch.bfloat16, device), Guarded((m, n), torch.bfloat16, device)
    moe.moe_gemm_bf16(layout, a, b, None, "none", res, pre.t, out.t)
    torch.cuda.synchronize()
    assert out.intact() and pre.intact()
    a32, b32 = (a.t() if layout == "tn" else a), (b.t() if layout == "nt" else b)
    step = 10000
    for i in range(0, m, step):
        rows = a32[i:i + step].float()
        for j in range(0, n, 100000):
            s = slice(i, i + step), slice(j, j + 100000)
            z = rows @ b32[:, s[1]].float().contiguous()
            assert torch.equal(pre.t[s], z.bfloat16()), s
            assert torch.equal(out.t[s], (z + res[s].float()).bfloat16()), s


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("m,n", [(70008, 31000), (70001, 30801), (1, 2 ** 24), (2 ** 24, 3)])
def test_act_bwd_past_32_bits(device, m, n, act):
    """The sums of a column are of -1, 0 and 1 where there is no activation, and so exact."""
    say("act_bwd", m, n, act)
    g = gen(device, 123)
    dc = ints((m, n), g, device, -1, 1)
    none = act == "none"
    z = None if none else (ints((m, n), g, device, -20, 20) / 8)
    dz, db = moe.act_bwd(dc, z, act, d_bias=True)
    torch.cuda.synchronize()
    want, mag = (torch.zeros(n, dtype=F64, device=device) for _ in range(2))
    err = 0
    for at in range(0, m, 10000 if n > 100 else m):
        s = slice(at, at + (10000 if n > 100 else m))
        if none:
            want += dc[s].sum(0, dtype=F64)
            continue
        x = z[s].to(F64)
        sig = torch.sigmoid(x)
        v = dc[s].to(F64) * sig * (1 + x * (1 - sig))
        e = 12 * U32 * (1 + x.abs()) * dc[s].to(F64).abs()
        close(dz[s], v, e + UBF * v.abs(), at)
        want, mag, err = want + v.sum(0), mag + v.abs().sum(0), err + e.sum(0)
    if none:
        assert dz is dc and torch.equal(db.double(), want)
    else:
        close(db, want, err + (math.ceil(m / 4) + 4 + 32 + 16) * U32 * mag, "d_bias")


# T, H: many short rows (a workgroup takes several), rows of the largest width, and more than 2^32
# bytes of them, or elements
NORMS = [(2 ** 23 + 5, 8), (2 ** 22 + 3, 520), (2 ** 17 + 3, 32768), (2 ** 18 + 1, 8193), (3, 32768)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", NORMS)
def test_norm_past_32_bits(device, T, H, dtype):
    say("norm", T, H, dtype)
    g = gen(device, 124)
    x = torch.empty((T, H), dtype=dtype, device=device).normal_(generator=g)
    dy = torch.empty((T, H), dtype=dtype, device=device).normal_(generator=g)
    w = torch.randn(H, generator=g, device=device).to(dtype)
    want = ("y", "rstd") + (("codes",) if H % 128 == 0 else ())
    out = moe.rms_norm(x, w, dy, want=want)
    dx, dw = moe.rms_norm_bwd(dy, out["sum"], w, out["rstd"], d_sum=x)
    torch.cuda.synchronize()
    total, mag = torch.zeros(H, dtype=F64, device=device), torch.zeros(H, dtype=F64, device=device)
    step = 2 ** 27 // H // 8 * 8                # slices begin on 16 bytes
    for at in range(0, T, step):
        s = slice(at, at + step)
        one = moe.rms_norm(x[s], w, dy[s], want=want)
        for name in one:
            got, ref = out[name][s], one[name]
            if name == "codes":
                got, ref = got.view(torch.uint8), ref.view(torch.uint8)
            assert torch.equal(got, ref), (at, name)
        assert torch.equal(dx[s], moe.rms_norm_bwd(dy[s], one["sum"], w, one["rstd"], x[s],
                                                   d_weight=False)[0]), at
        t = dy[s].double() * one["sum"].double() * one["rstd"].double()[:, None]
        total, mag = total + t.sum(0), mag + t.abs().sum(0)
    close(dw, total, (math.ceil(T / 4) + 4 + 4 + 32 + 16) * U32 * mag, "d_weight")


@pytest.mark.parametrize("T,E,dtype", [(2 ** 22 + 5, 1024, torch.bfloat16), (2 ** 24 + 1, 8, torch.float32),
                                       (2 ** 21 + 3, 1024, torch.float32)])
def test_router_past_32_bits(device, T, E, dtype):
    k = 2
    say("router", T, E, dtype)
    g = gen(device, 125)
    x = torch.empty((T, E), dtype=dtype, device=device).normal_(generator=g)
    bias = 0.1 * torch.randn(E, generator=g, device=device)
    dw = torch.randn((T, k), generator=g, device=device)
    p = moe.make_problem(T, 64, 64, E, k, "bf16", None, 16)
    for r in (moe.make_router("sigmoid", True, 4, 2, 2, 2.5), moe.make_router("softmax", False)):
        b = bias if r.n_groups > 1 else None
        ids, wt = moe.route_scored(p, r, x, b)
        d = moe.route_scored_bwd(p, r, x, ids, dw)
        torch.cuda.synchronize()
        step = 2 ** 27 // E
        for at in range(0, T, step):
            s = slice(at, min(at + step, T))
            q = moe.make_problem(s.stop - at, 64, 64, E, k, "bf16", None, 16)
            one = moe.route_scored(q, r, x[s], b)
            assert torch.equal(ids[s], one[0]) and torch.equal(wt[s], one[1]), at
            assert torch.equal(d[s], moe.route_scored_bwd(q, r, x[s], one[0], dw[s])), at


def test_the_same_bits_twice(device):
    """No sum depends on the order in which workgroups end."""
    g = gen(device, 126)
    T, H = 3001, 2048
    x = torch.randn((T, H), generator=g, device=device).bfloat16()
    dy = torch.randn((T, H), generator=g, device=device).bfloat16()
    w = torch.randn(H, generator=g, device=device).bfloat16()
    wo = torch.randn((1000, H), generator=g, device=device).bfloat16()
    one = torch.randn((1, H), generator=g, device=device).bfloat16()
    rstd = moe.rms_norm(x, w, want=("y", "rstd"))["rstd"]

    def results():
        dx, dw = moe.rms_norm_bwd(dy, x, w, rstd)
        dz, db = moe.act_bwd(dy, x, "gelu", d_bias=True)
        return [dx, dw, dz, db, moe.gemm_bf16(x, wo, act="silu"), moe.gemm_bf16(one, wo),
                moe.gemm_bf16(dy, x, "tn", out_dtype=torch.float32)]
    first = results()
    for _ in range(5):
        for got, want in zip(results(), first):
            assert torch.equal(got, want)
