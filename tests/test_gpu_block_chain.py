"""The operators of a block together, as a training step runs them: projection with residual, norm,
router, experts and a dense branch, the next norm, and back.  Each result against 64 bits on the values
that reached it; on other streams, on two at once, and in captured graphs."""
import contextlib
import math

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe
from test_gpu_block_operators import (F64, TINY, U32, UBF, ref_norm, ref_route, ref_route_bwd)
from test_gpu_operators import close, gen, row_codes, say
from test_operator_streams import owner

pytestmark = pytest.mark.gpu

EPS = 1e-5


def block_inputs(device, T=200, K=192, H=256, E=16, k=4, I=320, bm=32, seed=70):
    g = gen(device, seed)

    def rand(*s, scale=1.0, dtype=torch.bfloat16):
        return (scale * torch.randn(s, generator=g, device=device)).to(dtype)
    p = moe.make_problem(T, H, 128, E, k, "bf16", "e4m3", bm)
    r = moe.make_router("sigmoid", True, 4, 2, 2, 2.5)
    we, _ = row_codes(rand(E * H, H, dtype=torch.float32))
    x = dict(x=rand(T, K), s=rand(T, H), wo=rand(H, K, scale=K ** -0.5),
             bo=rand(H, dtype=torch.float32), w1=1 + rand(H, scale=0.1), w2=1 + rand(H, scale=0.1),
             gate=rand(E, H, scale=H ** -0.5), bal=rand(E, scale=0.1, dtype=torch.float32),
             we=we.view(E, H, H),
             ws=0.001 * (torch.rand((E, H // 128, H // 128), generator=g, device=device) + 0.5),
             up=rand(I, H, scale=H ** -0.5), bu=rand(I, dtype=torch.float32),
             down=rand(H, I, scale=I ** -0.5), dy=rand(T, H))
    return p, r, x


def block(p, r, x, stream=None):
    """Every value of the forward and the backward pass by name."""
    v = dict(x)
    f32, s = torch.float32, dict(stream=stream)
    v["h"] = moe.gemm_bf16(v["x"], v["wo"], "nt", v["bo"], residual=v["s"], **s)
    n1 = moe.rms_norm(v["h"], v["w1"], eps=EPS, want=("y", "codes", "rstd"), **s)
    v.update(y=n1["y"], codes=n1["codes"], scales=n1["scales"], rstd1=n1["rstd"])
    v["lg"] = moe.gemm_bf16(v["y"], v["gate"], **s)
    v["ids"], v["wt"] = moe.route_scored(p, r, v["lg"], v["bal"], **s)
    a = v["a"] = moe.align(p, v["ids"], **s)
    v["rows"], v["rs"] = moe.permute(p, v["codes"], a, v["scales"], **s)
    v["ye"] = moe.grouped_gemm_e4m3(p, v["rows"], v["rs"], v["we"], v["ws"], a, **s)
    v["mix"] = moe.unpermute(p, v["ye"], a, v["wt"], **s)
    v["z"], v["pre"] = moe.gemm_bf16(v["y"], v["up"], "nt", v["bu"], "gelu_tanh", with_pre=True, **s)
    v["d"] = moe.gemm_bf16(v["z"], v["down"], residual=v["mix"], **s)
    n2 = moe.rms_norm(v["d"], v["w2"], v["h"], EPS, ("y", "rstd"), **s)
    v.update(sum=n2["sum"], out=n2["y"], rstd2=n2["rstd"])

    v["dd"], v["dw2"] = moe.rms_norm_bwd(v["dy"], v["sum"], v["w2"], v["rstd2"], **s)
    v["dz"] = moe.gemm_bf16(v["dd"], v["down"], "nn", **s)
    v["ddown"] = moe.gemm_bf16(v["dd"], v["z"], "tn", out_dtype=f32, **s)
    v["dpre"], v["dbu"] = moe.act_bwd(v["dz"], v["pre"], "gelu_tanh", d_bias=True, **s)
    v["dup"] = moe.gemm_bf16(v["dpre"], v["y"], "tn", out_dtype=f32, **s)
    v["dy1"] = moe.gemm_bf16(v["dpre"], v["up"], "nn", **s)
    v["dye"], v["dwt"] = moe.unpermute_bwd(p, v["dd"], v["ye"], a, v["wt"], **s)
    v["dlg"] = moe.route_scored_bwd(p, r, v["lg"], v["ids"], v["dwt"], **s)
    v["dgate"] = moe.gemm_bf16(v["dlg"], v["y"], "tn", out_dtype=f32, **s)
    v["dy2"] = moe.gemm_bf16(v["dlg"], v["gate"], "nn", residual=v["dy1"], **s)
    v["dh"], v["dw1"] = moe.rms_norm_bwd(v["dy2"], v["h"], v["w1"], v["rstd1"], v["dd"], **s)
    v["dbo"] = moe.act_bwd(v["dh"], d_bias=True, **s)[1]
    v["dx"] = moe.gemm_bf16(v["dh"], v["wo"], "nn", **s)
    v["dwo"] = moe.gemm_bf16(v["dh"], v["x"], "tn", out_dtype=f32, **s)
    return v


# results that are whole tensors of every call (the sorted rows end where the used slots do)
RESULTS = ["h", "y", "codes", "scales", "rstd1", "lg", "ids", "wt", "mix", "z", "pre", "d", "sum",
           "out", "rstd2", "dd", "dw2", "dz", "ddown", "dpre", "dbu", "dup", "dy1", "dwt", "dlg",
           "dgate", "dy2", "dh", "dw1", "dbo", "dx", "dwo"]


def same(got, want, what=""):
    for name in RESULTS:
        u, w = (t[name].view(torch.uint8) if name == "codes" else t[name] for t in (got, want))
        assert torch.equal(u, w), (what, name)


def test_block(device):
    p, r, x = block_inputs(device)
    v = block(p, r, x)
    torch.cuda.synchronize()
    w = {n: t.to(F64) for n, t in v.items() if isinstance(t, torch.Tensor) and t.is_floating_point()
         and t.dtype.itemsize > 1}

    def product(name, a, b, residual=None, bias=None, u=UBF):
        k = a.shape[1]
        z = a @ b + (0 if bias is None else bias)
        want = z + (0 if residual is None else residual)
        err = 2 * k * U32 * (a.abs() @ b.abs()) + 2 * U32 * z.abs()
        close(v[name], want, err + u * (want.abs() + err) + 2 * U32 * want.abs(), name)
    product("h", w["x"], w["wo"].t(), w["s"], w["bo"])
    product("lg", w["y"], w["gate"].t())
    product("pre", w["y"], w["up"].t(), None, w["bu"])
    product("d", w["z"], w["down"].t(), w["mix"])
    product("dz", w["dd"], w["down"])
    product("ddown", w["dd"].t(), w["z"], u=U32)
    product("dup", w["dpre"].t(), w["y"], u=U32)
    product("dy1", w["dpre"], w["up"])
    product("dgate", w["dlg"].t(), w["y"], u=U32)
    product("dy2", w["dlg"], w["gate"], w["dy1"])
    product("dx", w["dh"], w["wo"])
    product("dwo", w["dh"].t(), w["x"], u=U32)

    assert torch.equal(v["sum"], (v["d"].float() + v["h"].float()).bfloat16())
    for y, s, weight in (("y", "h", "w1"), ("out", "sum", "w2")):
        want = ref_norm(w[s], w[weight], EPS)[1]
        close(v[y], want, (UBF + 4 * U32) * want.abs() + TINY, y)
    ids, wt = ref_route(v["lg"].cpu(), v["bal"].cpu(), r, p.top_k)
    assert torch.equal(v["ids"].cpu(), ids.int())
    close(v["wt"], wt.to(device), (50 + p.top_k) * U32 * wt.abs().to(device), "weights")

    def norm_bwd(dx, dw, d, s, weight, rstd, d_sum=None):
        n, t = w[s] * w[rstd][:, None], w[d] * w[weight]
        mean = (t * n).mean(1, keepdim=True)
        want = w[rstd][:, None] * (t - n * mean)
        mag = w[rstd][:, None] * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True))
        if d_sum is not None:
            want = want + w[d_sum]
        err = (32 + 6 + 16 + 6) * U32 * mag
        close(v[dx], want, err + UBF * want.abs() + 2 * U32 * want.abs() + TINY, dx)
        depth = math.ceil(p.T / 4) + 4 + 32 + 16
        close(v[dw], (w[d] * n).sum(0), (depth + 4) * U32 * (w[d] * n).abs().sum(0) + TINY, dw)
    norm_bwd("dd", "dw2", "dy", "sum", "w2", "rstd2")
    norm_bwd("dh", "dw1", "dy2", "h", "w1", "rstd1", "dd")

    z = w["pre"].clone().requires_grad_(True)
    f = torch.nn.functional.gelu(z, approximate="tanh")
    slope = torch.autograd.grad(f.sum(), z)[0]
    # z is the activation of the sum in fp32, pre that sum rounded
    close(v["z"], f.detach(), 1.13 * UBF * 1.01 * w["pre"].abs() + UBF * 1.01 * f.detach().abs()
          + 8 * U32 * w["pre"].abs() + TINY, "z")
    err = 12 * U32 * (1 + w["pre"].abs()) * w["dz"].abs()
    close(v["dpre"], w["dz"] * slope, err + UBF * (w["dz"] * slope).abs() + TINY, "dpre")
    depth = math.ceil(p.T / 4) + 4 + 32 + 16
    for name, t, e in (("dbu", w["dz"] * slope, err), ("dbo", w["dh"], torch.zeros_like(w["dh"]))):
        close(v[name], t.sum(0), e.sum(0) + depth * U32 * t.abs().sum(0) + TINY, name)

    dlg = ref_route_bwd(v["lg"].cpu(), v["ids"].cpu(), v["dwt"].cpu(), r)[0].to(device)
    size = r.scale * w["dwt"].abs().sum(1, keepdim=True) * (dlg != 0)
    close(v["dlg"], dlg, (50 + p.top_k) * U32 * size + UBF * dlg.abs() + TINY, "dlg")


def on(stream):
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def test_block_on_other_streams(device):
    """By a stream's handle, as a current stream, and two passes on two streams at once: the same
    bits, in memory of the stream of the call."""
    p, r, x = block_inputs(device, seed=71)
    other = block_inputs(device, seed=72)
    ref, ref2 = block(p, r, x), block(*other)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = block(p, r, x, stream=one)
    by_handle = block(p, r, x, stream=two.cuda_stream)
    with on(one):
        inside = block(p, r, x)
    torch.cuda.synchronize()
    for v, what in ((got, "argument"), (by_handle, "handle"), (inside, "current")):
        same(v, ref, what)
    for v, s in ((got, one), (by_handle, two), (inside, one)):
        assert {owner(v[n]) for n in RESULTS} == {s.cuda_stream}
    for rep in range(3):
        a, b = [], []
        for _ in range(3):                       # enqueued in turns, so that both are on their way
            a.append(block(p, r, x, stream=one))
            b.append(block(*other, stream=two))
        torch.cuda.synchronize()
        for v in a:
            same(v, ref, rep)
        for v in b:
            same(v, ref2, rep)


def test_blocks_in_graphs(device):
    """Two passes captured once each, replayed on new inputs one after the other and at once, with
    eager passes between the replays."""
    sets = [block_inputs(device, seed=73), block_inputs(device, T=77, I=328, seed=74)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, held = [], []
    for args in sets:
        streams[0].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[0]):
            block(*args)
        torch.cuda.current_stream().wait_stream(streams[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(block(*args))
        graphs.append(graph)
    for rep in range(4):
        say("replay", rep)
        for (p, _, x), shape in zip(sets, ({}, dict(T=77, I=328))):
            new = block_inputs(device, seed=80 + rep, **shape)[2]
            for n, t in x.items():
                if n not in ("we", "ws"):
                    t.copy_(new[n])
        torch.cuda.synchronize()
        if rep % 2:
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        else:
            for graph in graphs:
                graph.replay()
                block(*sets[0])
        torch.cuda.synchronize()
        for args, v in zip(sets, held):
            same(v, block(*args), rep)


def test_one_token(device):
    """The same for a single token, the form that serving runs, against the token in a batch: norm,
    router and the gradients of both treat every row for itself."""
    p, r, x = block_inputs(device, seed=75)
    v = block(p, r, x)
    p1 = moe.make_problem(1, p.H, 128, p.E, p.top_k, "bf16", "e4m3", 16)
    for t in (0, 63, p.T - 1):
        one = slice(t, t + 1)
        n = moe.rms_norm(v["h"][one], v["w1"], eps=EPS, want=("y", "codes", "rstd"))
        ids, wt = moe.route_scored(p1, r, v["lg"][one], v["bal"])
        dlg = moe.route_scored_bwd(p1, r, v["lg"][one], ids, v["dwt"][one])
        dh, _ = moe.rms_norm_bwd(v["dy2"][one], v["h"][one], v["w1"], n["rstd"], v["dd"][one])
        for got, name in ((n["y"], "y"), (n["codes"].view(torch.uint8), "codes"),
                          (n["scales"], "scales"), (ids, "ids"), (wt, "wt"), (dlg, "dlg"),
                          (dh, "dh")):
            want = v[name].view(torch.uint8) if name == "codes" else v[name]
            assert torch.equal(got, want[one]), (t, name)
