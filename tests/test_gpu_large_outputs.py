"""The kernels that only large rows and outputs reach: loads past the caches for rows of more than
128 MB, stores past the last-level cache for outputs of more than 256 MB."""
import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_gemm_tiles import grouped
from test_gpu_operators import (TD, U32, UT, Guarded, aligned, close, gen, say, sorted_rows)

pytestmark = pytest.mark.gpu

MB = 2 ** 20
# (T, E, k, block_m, n, kk): m-blocks with several per expert and with one, bf16 outputs of 290 MB
# and more; columns that end on 16 bytes, on an even and on an odd number
PAST = [(6000, 8, 3, 128, 8190, 640), (6000, 8, 3, 64, 8189, 640), (4096, 256, 2, 64, 8184, 640),
        (2048, 128, 2, 128, 8184, 640)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", PAST, ids=str)
def test_grouped(device, c, dtype):
    T, E, k, bm, n, kk = c
    say("grouped past the cache", c, dtype)
    p = moe.make_problem(T, 128, 128, E, k, "bf16", "e4m3", bm)
    assert moe.moe_max_padded_slots(p) * n * 2 > 256 * MB
    grouped(device, *c, dtype, 40)


@pytest.mark.parametrize("c", [(2100, 2048, 16, 8, 128, "all"), (1030, 8192, 6, 6, 32, "all"),
                               (4300, 2048, 24, 8, 64, "some")], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unpermute_and_gradient(device, c, dtype):
    T, H, E, k, bm, mode = c
    if dtype == "bf16":
        T = 2 * T
    say("large rows", c, dtype)
    p, a, used, ss, held = aligned(device, T, H, E, k, bm, mode, 90)
    dt = TD[dtype]
    assert T * k * H * dt.itemsize > 128 * MB
    g = gen(device, 91)
    rows = sorted_rows(device, ss, held, H, dt, 92)
    w = torch.randn((T, k), generator=g, device=device)
    d_out = torch.randn((T, H), generator=g, device=device).to(dt)
    out = Guarded((T, H), dt, device)
    d_rows, d_w = Guarded((ss.numel(), H), dt, device), Guarded((T, k), torch.float32, device)
    moe.unpermute(p, rows, a, w, out=out.t)
    moe.unpermute_bwd(p, d_out, rows, a, w, d_rows=d_rows.t, d_weights=d_w.t)
    torch.cuda.synchronize()
    assert out.intact() and d_rows.intact(used) and d_w.intact()
    at = a["slot_row"].long().view(T, k)
    u = UT[dtype]
    for t in range(0, T, 500):                             # a slice of tokens at a time
        mine = at[t:t + 500]
        there = (mine >= 0)[:, :, None]
        y = torch.where(there, rows.double()[mine.clamp(min=0)], 0.0)
        wd = torch.where(there[:, :, 0], w[t:t + 500].double(), 0.0)[:, :, None]
        d = d_out[t:t + 500].double()[:, None, :]
        ref, mag = (y * wd).sum(1), (y * wd).abs().sum(1)
        close(out.t[t:t + 500], ref, (k + 1) * U32 * mag + u * (ref.abs() + (k + 1) * U32 * mag), "out")
        close(d_w.t[t:t + 500], (y * d).sum(2), (H / 64 + 8) * U32 * (y * d).abs().sum(2), "d_weights")
        want = (wd * d)[there[:, :, 0]]
        close(d_rows.t[mine[there[:, :, 0]]], want, (u + 2 * U32) * want.abs() + 1e-38, "d_rows")
    assert not bool(d_rows.t[:used][~held[:used]].any()), "padding rows"


def test_more_workgroups_than_a_launch_has(device):
    """So many slots that permute's and unpermute_bwd's workgroups take several parts each (a launch
    has at most 2^22 of 256 threads), and the elements lie past 2^31."""
    T, H, E, k, bm = 2 ** 23 + 5, 64, 8, 4, 16
    say("many slots", T * k)
    p, a, used, ss, held = aligned(device, T, H, E, k, bm, "all", 93)
    N = T * k
    assert -(-T * H // 8 // 256) + ss.numel() // 8 > 2 ** 22 and N // 4 > 2 ** 22
    g = gen(device, 94)
    x = torch.randn((T, H), generator=g, device=device).bfloat16()
    w = torch.rand((T, k), generator=g, device=device) + 0.5
    rows = Guarded((ss.numel(), H), torch.bfloat16, device)
    moe.permute(p, x, a, rows=rows.t)
    torch.cuda.synchronize()
    step = 2 ** 22
    for r in range(0, used, step):
        tok = (ss[r:min(r + step, used)] // k).clamp(max=T - 1)
        own = held[r:r + tok.numel(), None]
        assert torch.equal(rows.t[r:r + tok.numel()], torch.where(own, x[tok], 0.0)), r
    assert rows.intact(used)
    d_rows = Guarded((ss.numel(), H), torch.bfloat16, device)
    d_w = Guarded((T, k), torch.float32, device)
    moe.unpermute_bwd(p, x, rows.t, a, w, d_rows=d_rows.t, d_weights=d_w.t)
    torch.cuda.synchronize()
    for r in range(0, used, step):
        slot = ss[r:min(r + step, used)]
        own, slot = held[r:r + slot.numel(), None], slot.clamp(max=N - 1)
        want = (w.view(-1)[slot][:, None] * x[slot // k].float()).bfloat16()   # one product, rounded
        assert torch.equal(d_rows.t[r:r + slot.numel()], torch.where(own, want, 0.0)), r
    for t in range(0, T, step):
        sq = (x[t:t + step].double() ** 2).sum(1, keepdim=True).expand(-1, k)
        close(d_w.t[t:t + step], sq, (H / 64 + 8) * U32 * sq, "d_weights")
    assert d_rows.intact(used) and d_w.intact()
