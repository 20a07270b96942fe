"""Measured cases of the operators around the routed expert products.

  permute      token rows gathered into the padded expert-sorted order of the alignment
  unpermute    expert-sorted rows brought back to token order and added with the routing
               weights, and the gradient of that (of the rows and of the weights)
  route_bwd    the gradient of the router's top-k softmax weights with respect to its logits
  gemm         products of 8-bit (e4m3) codes with one scale per 128 values: dense (weights
               scaled per 128x128 block), over expert-sorted rows, and the weight gradient
               (both operands quantised along the tokens, then multiplied)

With `own` false every operator is computed from elementary torch operations; with `own` true
by the package's entry points.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _scale(amax):
    """amax / 448 as the IEEE quotient (a division by a Python number may multiply by its
    reciprocal instead, which moves values that lie midway between two codes); 1 for zeros."""
    return torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))


# ---------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # a prefill batch of 256 experts, rows already quantised for the fp8 expert products
        dict(name="permute_e4m3_256_experts", op="permute", T=2048, H=7168, E=256, R=256, k=8,
             bm=128, dtype="e4m3", bias=0.0),
        # a skewed prefill batch, top-6 of 64 experts with a router bias, bf16 rows
        dict(name="permute_bf16_skewed", op="permute", T=8192, H=2048, E=64, R=64, k=6, bm=256,
             dtype="bf16", bias=2.0),
        # one decoded token: eight expert rows back into one output row, latency only
        dict(name="unpermute_bf16_one_token", op="unpermute", T=1, H=7168, E=256, R=256, k=8,
             bm=16, dtype="bf16", bias=0.0, weighted=True),
        # a training step of the skewed batch: the combine and its gradient
        dict(name="unpermute_train_bf16_skewed", op="unpermute_train", T=8192, H=2048, E=64,
             R=64, k=6, bm=256, dtype="bf16", bias=2.0),
        # one expert-parallel shard (16 of 128 experts, most slots belong to others), fp32, an
        # odd number of tokens
        dict(name="unpermute_train_f32_shard", op="unpermute_train", T=2001, H=2880, E=16, R=128,
             k=4, bm=128, dtype="f32", bias=0.0),
        # router gradient, 256 experts, weights not renormalised
        dict(name="route_bwd_256_experts", op="route_bwd", T=2048, E=256, k=8, renorm=False),
        # router gradient, 8 experts, top-2 renormalised
        dict(name="route_bwd_8_experts_renorm", op="route_bwd", T=4096, E=8, k=2, renorm=True),
        # one decoded token through a dense 8-bit projection (a shared expert's gate and up)
        dict(name="gemm_one_token", op="gemm", M=1, n=4096, kk=7168, out="bf16"),
        # a prefill batch through a dense 8-bit projection
        dict(name="gemm_prefill", op="gemm", M=4096, n=14336, kk=4096, out="bf16"),
        # weight gradient of a dense 8-bit projection over an odd number of tokens
        dict(name="gemm_weight_gradient", op="wgrad", M=4001, n=2048, kk=7168),
        # decode batch over 8 large experts: weight streaming
        dict(name="grouped_decode_8_experts", op="grouped", T=64, E=8, R=8, k=2, bm=32, n=4096,
             kk=14336, out="bf16"),
        # prefill batch over 256 experts, the down product
        dict(name="grouped_prefill_256_experts", op="grouped", T=2048, E=256, R=256, k=8, bm=128,
             n=7168, kk=2048, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "unpermute_train", "route_bwd", "gemm", "gemm",
                     "wgrad", "grouped"])
    E = _log(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 8192)
    if op == "route_bwd":
        return dict(op=op, T=T, E=rng.choice([E, _log(rng, 2, 1024)]) if k <= 2 else E, k=k,
                    renorm=rng.random() < 0.5)
    R = E * rng.choice([1, 1, 1, 4])
    if op in ("permute", "unpermute", "unpermute_train"):
        dtype = rng.choice(["bf16", "bf16", "f32"] + (["e4m3"] if op == "permute" else []))
        H = 64 * _log(rng, 1, 128)
        H = max(128, H // 128 * 128) if dtype == "e4m3" else H
        bm = rng.choice([16, 32, 64, 128] + ([256] if dtype == "bf16" else []))
        while T > 1 and (T * k + E * bm) * H > 2048 * 8 * 7168:
            T = (T + 1) // 2
        c = dict(op=op, T=T, H=H, E=E, R=R, k=k, bm=bm, dtype=dtype,
                 bias=rng.choice([0.0, 0.0, 2.0]))
        if op == "unpermute":
            c["weighted"] = rng.random() < 0.8
        return c
    if op == "gemm":
        M, n, kk = _log(rng, 1, 8192), _log(rng, 16, 16384), 128 * _log(rng, 1, 112)
        while M * n * kk > 4096 * 14336 * 4096:
            M = (M + 1) // 2
        return dict(op=op, M=M, n=n, kk=kk, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "wgrad":
        return dict(op=op, M=_log(rng, 1, 4096), n=8 * _log(rng, 8, 384), kk=8 * _log(rng, 8, 896))
    E = min(E, 64)
    k = min(k, E)
    return dict(op=op, T=min(T, 4096), E=E, R=E * rng.choice([1, 1, 2]), k=k,
                bm=rng.choice([16, 32, 64, 128]), n=16 * _log(rng, 8, 256),
                kk=128 * _log(rng, 1, 32), out=rng.choice(["bf16", "bf16", "f32"]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _row_codes(x):
    """Per-(row, 128-column group) e4m3 codes and fp32 scales."""
    m, c = x.shape
    v = x.float().view(m, c // 128, 128)
    a = v.abs().amax(2)
    s = _scale(a)
    return (v / s[:, :, None]).clamp(-448, 448).to(E4M3).view(m, c), s


def _block_codes(w):
    """Per-128x128-block e4m3 codes and fp32 scales; the last row block may be ragged."""
    n, c = w.shape
    nb = -(-n // 128)
    v = torch.zeros((nb * 128, c), device=w.device)
    v[:n] = w
    v = v.view(nb, 128, c // 128, 128)
    a = v.abs().amax((1, 3))
    s = _scale(a)
    q = (v / s[:, None, :, None]).clamp(-448, 448).to(E4M3).view(nb * 128, c)
    return q[:n].contiguous(), s


def _routing(case, g):
    """Top-k ids and renormalised weights from logits N(0,1) (plus a per-expert bias) over R
    experts; ids from E on belong to other shards."""
    T, R, k = case["T"], case["R"], case["k"]
    lg = _randn(g, T, R) + case.get("bias", 0.0) * _randn(g, R)[None, :]
    p, ids = torch.softmax(lg, 1).topk(k, 1)
    return ids.to(torch.int32), (p / p.sum(1, keepdim=True)).contiguous()


def _alignment(case, ids):
    """The padded expert-sorted slot list of the routing, as the alignment gives it."""
    T, E, k, bm = case["T"], case["E"], case["k"], case["bm"]
    N, dev = T * k, ids.device
    rows_max = N + min(E, N) * (bm - 1)
    tiles_max = rows_max // bm
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + bm - 1) // bm * bm
    offsets = torch.zeros(E + 1, dtype=torch.long, device=dev)
    offsets[1:] = padded.cumsum(0)
    first = torch.zeros(E + 1, dtype=torch.long, device=dev)
    first[1:] = counts.cumsum(0)
    e = key[order]
    keep = e < E
    e, slots = e[keep], order[keep]
    row = offsets[e] + torch.nonzero(keep)[:, 0] - first[e]
    sorted_slots = torch.full((rows_max,), N, dtype=torch.int32, device=dev)
    sorted_slots[row] = slots.to(torch.int32)
    slot_row = torch.full((N,), -1, dtype=torch.int32, device=dev)
    slot_row[slots] = row.to(torch.int32)
    starts = torch.arange(tiles_max, device=dev) * bm
    tile_e = torch.searchsorted(offsets[1:].contiguous(), starts, right=True)
    live = starts < offsets[E]
    tiles = torch.where(live[:, None], torch.stack([tile_e, starts], 1),
                        torch.full((tiles_max, 2), -1, device=dev))
    i32 = torch.int32
    return {"sorted_slots": sorted_slots, "slot_row": slot_row, "offsets": offsets.to(i32),
            "tiles": tiles.to(i32).contiguous().view(-1),
            "num_tiles": live.sum().to(i32).view(1)}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "route_bwd":
        s["logits"] = 2 * _randn(g, case["T"], case["E"])
        s["ids"] = s["logits"].topk(case["k"], 1)[1].to(torch.int32).contiguous()
        s["dw"] = _randn(g, case["T"], case["k"])
        return s
    if op == "gemm":
        s["a"], s["a_scales"] = _row_codes(_randn(g, case["M"], case["kk"]).bfloat16())
        s["b"], s["b_scales"] = _block_codes(0.02 * _randn(g, case["n"], case["kk"]))
        return s
    if op == "wgrad":
        s["dy"] = (0.1 * _randn(g, case["M"], case["n"])).bfloat16()
        s["x"] = _randn(g, case["M"], case["kk"]).bfloat16()
        return s
    ids, s["w"] = _routing(case, g)
    s.update(_alignment(case, ids))
    rows_max = s["sorted_slots"].numel()
    live = (s["sorted_slots"] < case["T"] * case["k"])[:, None]
    if op == "grouped":
        n, kk = case["n"], case["kk"]
        a, sc = _row_codes(_randn(g, rows_max, kk).bfloat16() * live)
        s["rows"], s["row_scales"] = a, sc
        s["b"] = torch.empty((case["E"], n, kk), dtype=E4M3, device="cuda")
        s["b_scales"] = torch.empty((case["E"], -(-n // 128), kk // 128), device="cuda")
        for e in range(case["E"]):
            s["b"][e], s["b_scales"][e] = _block_codes(0.02 * _randn(g, n, kk))
        s["out_buf"] = torch.zeros((rows_max, n), dtype=TYPES[case["out"]], device="cuda")
        return s
    T, H = case["T"], case["H"]
    if op == "permute":
        x = _randn(g, T, H).bfloat16()
        if case["dtype"] == "e4m3":
            s["x"], s["x_scales"] = _row_codes(x)
            s["rows_buf"] = torch.zeros((rows_max, H), dtype=torch.uint8, device="cuda").view(E4M3)
            s["scales_buf"] = torch.zeros((rows_max, H // 128), device="cuda")
        else:
            s["x"], s["x_scales"] = x.to(TYPES[case["dtype"]]), None
            s["rows_buf"] = torch.zeros((rows_max, H), dtype=s["x"].dtype, device="cuda")
            s["scales_buf"] = None
        return s
    dt = TYPES[case["dtype"]]
    s["rows"] = (_randn(g, rows_max, H) * live).to(dt)
    if op == "unpermute_train":
        s["d_out"] = _randn(g, T, H).to(dt)
        s["d_rows_buf"] = torch.zeros((rows_max, H), dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _problem(s):
    """The problem description that a user's program makes once and keeps."""
    import routed_grouped_gemm_topk_amd as moe
    if "problem" not in s:
        fp8 = s["op"] == "grouped" or s.get("dtype") == "e4m3"
        s["problem"] = moe.make_problem(s["T"], s.get("H", 128), 128, s["E"], s["k"],
                                        "bf16" if fp8 else s.get("dtype", "bf16"),
                                        "e4m3" if fp8 else None, s.get("bm", 0))
    return moe, s["problem"]


def _run_own(s):
    import routed_grouped_gemm_topk_amd as moe
    op = s["op"]
    if op == "gemm":
        return moe.gemm_e4m3(s["a"], s["a_scales"], s["b"], s["b_scales"],
                             out_dtype=TYPES[s["out"]])
    if op == "wgrad":
        dyt, dys = moe.quantize_cols_e4m3(s["dy"])
        xt, xs = moe.quantize_cols_e4m3(s["x"])
        dw = moe.gemm_e4m3(dyt, dys, xt, xs, out_dtype=torch.float32, b_block=1)
        return {"dw": dw, "dyt": dyt, "dys": dys, "xt": xt, "xs": xs}
    moe, p = _problem(s)
    if op == "route_bwd":
        return moe.route_bwd(p, s["logits"], s["renorm"], s["ids"], s["dw"])
    if op == "permute":
        rows, scales = moe.permute(p, s["x"], s, s["x_scales"], rows=s["rows_buf"],
                                   row_scales=s["scales_buf"])
        return [rows] if scales is None else [rows, scales]
    if op == "unpermute":
        return moe.unpermute(p, s["rows"], s, s["w"] if s["weighted"] else None)
    if op == "unpermute_train":
        out = moe.unpermute(p, s["rows"], s, s["w"])
        d_rows, d_w = moe.unpermute_bwd(p, s["d_out"], s["rows"], s, s["w"],
                                        d_rows=s["d_rows_buf"])
        return {"out": out, "d_rows": d_rows, "d_w": d_w}
    return moe.grouped_gemm_e4m3(p, s["rows"], s["row_scales"], s["b"], s["b_scales"], s,
                                 out=s["out_buf"])


def _groups(codes, scales):
    """codes [..., c] times scales [..., c/128], in fp32."""
    v = codes.to(torch.float32).unflatten(-1, (-1, 128))
    return (v * scales[..., None]).flatten(-2)


def _blocks(codes, scales):
    """codes [..., n, c] times scales [..., ceil(n/128), c/128], in fp32."""
    return _groups(codes, scales.repeat_interleave(128, -2)[..., : codes.shape[-2], :])


def _quantize_cols(x):
    m, c = x.shape
    v = torch.zeros((-(-m // 128) * 128, c), device=x.device)
    v[:m] = x
    v = v.t().contiguous().view(c, -1, 128)
    a = v.abs().amax(2)
    s = _scale(a)
    return (v / s[:, :, None]).clamp(-448, 448).to(E4M3).view(c, -1), s


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "gemm":
        out = _groups(s["a"], s["a_scales"]) @ _blocks(s["b"], s["b_scales"]).t()
        return out.to(TYPES[s["out"]])
    if op == "wgrad":
        dyt, dys = _quantize_cols(s["dy"])
        xt, xs = _quantize_cols(s["x"])
        return {"dw": _groups(dyt, dys) @ _groups(xt, xs).t(), "dyt": dyt, "dys": dys, "xt": xt,
                "xs": xs}
    k = s["k"]
    if op == "route_bwd":
        ids, dw = s["ids"].long(), s["dw"]
        if s["renorm"]:
            lg = torch.gather(s["logits"], 1, ids)
            w = torch.exp(lg - lg.amax(1, keepdim=True))
            w = w / w.sum(1, keepdim=True)
            d = w * (dw - (w * dw).sum(1, keepdim=True))
            return torch.zeros_like(s["logits"]).scatter(1, ids, d)
        p = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        g = torch.zeros_like(p).scatter(1, ids, dw)
        return p * (g - (p * g).sum(1, keepdim=True))
    N = s["T"] * k
    slots = s["sorted_slots"].long()
    held = (slots < N)[:, None]
    token = (slots // k).clamp(max=s["T"] - 1)
    if op == "permute":
        if s["x_scales"] is None:
            return [torch.where(held, s["x"][token], torch.zeros((), dtype=s["x"].dtype,
                                                                 device="cuda"))]
        rows = s["x"].view(torch.uint8)[token] * held
        in_tile = torch.arange(slots.numel(), device="cuda") < s["num_tiles"] * s["bm"]
        scales = torch.where(held, s["x_scales"][token], in_tile[:, None].float())
        return [rows.view(E4M3), scales]
    if op == "grouped":
        bm = s["bm"]
        tiles = s["tiles"].view(-1, 2)[:, 0].long()
        nt = tiles.numel()
        w = _blocks(s["b"], s["b_scales"])[tiles.clamp(min=0)]
        a = _groups(s["rows"][: nt * bm], s["row_scales"][: nt * bm]).view(nt, bm, -1)
        c = torch.bmm(a, w.transpose(1, 2)) * (tiles >= 0)[:, None, None]
        out = torch.zeros((slots.numel(), s["n"]), dtype=TYPES[s["out"]], device="cuda")
        out[: nt * bm] = c.view(nt * bm, -1)
        return out
    at = s["slot_row"].long()
    there = (at >= 0)[:, None]
    rows = torch.where(there, s["rows"][at.clamp(min=0)].float(), 0.0).view(s["T"], k, -1)
    w = s["w"] if op == "unpermute_train" or s["weighted"] else torch.ones_like(s["w"])
    out = (rows * w[:, :, None]).sum(1).to(s["rows"].dtype)
    if op == "unpermute":
        return out
    d = s["d_out"].float()
    d_w = (rows * d[:, None, :]).sum(2)
    d_rows = torch.where(held, d[token] * s["w"].view(-1)[slots.clamp(max=N - 1)][:, None], 0.0)
    return {"out": out, "d_rows": d_rows.to(s["rows"].dtype), "d_w": d_w}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "route_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        read = k if case["renorm"] else E           # renormalised: the chosen logits alone
        return {"bytes": 4.0 * T * (read + E + 2 * k), "flops": 4.0 * T * E}
    if op == "gemm":
        M, n, c = case["M"], case["n"], case["kk"]
        elt = 2 if case["out"] == "bf16" else 4
        return {"bytes": M * c * (1 + 4 / 128) + n * c * (1 + 4 / 128 / 128) + elt * M * n,
                "flops": 2.0 * M * n * c}
    if op == "wgrad":
        M, n, c = case["M"], case["n"], case["kk"]
        return {"bytes": M * (n + c) * (2 + 1 + 4 / 128) + 4.0 * n * c,
                "flops": 2.0 * M * n * c}
    T, E, k = case["T"], case["E"], case["k"]
    held = T * k * E / case["R"]                    # slots of local experts, expected
    if op == "grouped":
        n, c = case["n"], case["kk"]
        elt = 2 if case["out"] == "bf16" else 4
        active = E * (1 - (1 - 1 / case["R"]) ** (T * k))
        return {"bytes": held * (c * (1 + 4 / 128) + elt * n) + active * n * c,
                "flops": 2.0 * held * n * c}
    H = case["H"]
    elt = {"bf16": 2, "f32": 4, "e4m3": 1 + 4 / 128}[case["dtype"]]
    tokens = T * (1 - (1 - E / case["R"]) ** k)     # tokens with a local expert, expected
    if op == "permute":
        return {"bytes": (tokens + held) * H * elt + 4.0 * held, "flops": 0}
    if op == "unpermute":
        return {"bytes": (T + held) * H * elt + 8.0 * T * k, "flops": 2.0 * held * H}
    # combine: rows in, out; gradient: d_out, rows in, d_rows
    return {"bytes": (2 * T + 3 * held) * H * elt + 16.0 * T * k, "flops": 5.0 * held * H}


# ---------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------
def _e4m3_nearest(v):
    """The e4m3 value nearest to v, ties to even: 3 mantissa bits from 2^-6 up, steps of 2^-9
    below, at most 448 (fp64 throughout; v is an fp32 quotient)."""
    a = v.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _exact_cols(x):
    """Transposed quantisation: (codes' values [c, mp], scales [c, mp/128])."""
    m, c = x.shape
    groups = -(-m // 128)
    v = torch.zeros((c, groups * 128), dtype=torch.float32, device=x.device)
    v[:, :m] = x.float().t()
    v = v.view(c, groups, 128)
    amax = v.double().abs().max(2)[0]
    # fp32 quotients: a 64-bit one rounded to fp32 is the same value
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax)).float()
    q = _e4m3_nearest((v.double() / s.double().unsqueeze(2)).float().double())
    return q.view(c, -1), s.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "gemm":
        M, n, c = case["M"], case["n"], case["kk"]
        total = torch.zeros((M, n), dtype=f64, device="cuda")
        for g in range(c // 128):
            at = slice(128 * g, 128 * g + 128)
            part = s["a"][:, at].to(f64) @ s["b"][:, at].to(f64).t()
            col = s["b_scales"][:, g].to(f64).repeat_interleave(128)[:n]
            total += part * s["a_scales"][:, g].to(f64)[:, None] * col[None, :]
        return total
    if op == "wgrad":
        dyt, dys = _exact_cols(s["dy"])
        xt, xs = _exact_cols(s["x"])
        total = torch.zeros((case["n"], case["kk"]), dtype=f64, device="cuda")
        for g in range(dys.shape[1]):
            at = slice(128 * g, 128 * g + 128)
            total += (dyt[:, at] * dys[:, g, None]) @ (xt[:, at] * xs[:, g, None]).t()
        return {"dw": total, "dyt": dyt, "dys": dys, "xt": xt, "xs": xs}
    k = case["k"]
    if op == "route_bwd":
        lg = s["logits"].double()
        ids, dw = s["ids"].long(), s["dw"].double()
        p = torch.softmax(lg, 1)
        d = torch.zeros_like(lg)
        picked = torch.gather(p, 1, ids)
        w = picked / picked.sum(1, keepdim=True) if case["renorm"] else picked
        mean = (w * dw).sum(1)
        if not case["renorm"]:
            d -= p * mean[:, None]
            return d.scatter_add(1, ids, w * dw)
        return d.scatter_add(1, ids, w * (dw - mean[:, None]))
    N = case["T"] * k
    slots = s["sorted_slots"].long()
    rows_at = torch.nonzero(slots < N)[:, 0]        # rows that hold a slot
    slot = slots[rows_at]
    if op == "permute":
        v = torch.zeros((slots.numel(), case["H"]), dtype=f64, device="cuda")
        v[rows_at] = s["x"].to(f64)[slot // k]
        if s["x_scales"] is None:
            return [v]
        sc = torch.zeros((slots.numel(), case["H"] // 128), dtype=f64, device="cuda")
        sc[: int(s["num_tiles"]) * case["bm"]] = 1.0
        sc[rows_at] = s["x_scales"].double()[slot // k]
        return [v, sc]
    if op == "grouped":
        out = torch.zeros((slots.numel(), case["n"]), dtype=f64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if lo == hi:
                continue
            sb = s["b_scales"][e].double().repeat_interleave(128, 0)[: case["n"]]
            w = s["b"][e].to(f64) * sb.repeat_interleave(128, 1)
            a = s["rows"][lo:hi].to(f64) * s["row_scales"][lo:hi].double().repeat_interleave(128, 1)
            out[lo:hi] = a @ w.t()
        return out
    T, H = case["T"], case["H"]
    w = s["w"].double().view(-1)
    if op == "unpermute" and not case["weighted"]:
        w = torch.ones_like(w)
    y = s["rows"].double()[rows_at]
    out = torch.zeros((T, H), dtype=f64, device="cuda")
    for j in range(k):                              # one slot of a token at a time
        mine = slot % k == j
        out[slot[mine] // k] += y[mine] * w[slot[mine], None]
    if op == "unpermute":
        return out
    d = s["d_out"].double()[slot // k]
    d_rows = torch.zeros((slots.numel(), H), dtype=f64, device="cuda")
    d_rows[rows_at] = d * w[slot, None]
    d_w = torch.zeros(N, dtype=f64, device="cuda")
    d_w[slot] = (d * y).sum(1)
    return {"out": out, "d_rows": d_rows, "d_w": d_w.view(T, k)}
