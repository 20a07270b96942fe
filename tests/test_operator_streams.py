"""Which stream the memory of an operator's outputs belongs to: the one that the call runs on, whatever
names it."""
import contextlib

import pytest
import torch

import routed_grouped_gemm_topk_amd as moe


def test_handle_0_allocates_on_the_default_stream(monkeypatch):
    """On the host, with torch.cuda's stream calls recorded."""
    entered = []

    def enter(stream):
        entered.append(stream)
        return contextlib.nullcontext()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 70 + (device or 0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: 90 + handle)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    for handle, stream in ((0, 70), (5, 95)):
        t = moe._new(torch.empty(2), (2, 3), torch.float32, handle)
        assert t.shape == (2, 3) and t.is_contiguous()
        assert entered.pop() == stream and not entered


def owner(t):
    """The handle of the stream that a device tensor's memory was allocated on."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no segment holds the tensor")


@pytest.mark.gpu
def test_memory_belongs_to_the_stream_of_the_call(device):
    """Every helper that allocates, with the current stream, the default stream by its handle and as
    a Stream, and another stream by its handle and as a Stream."""
    T, H, E, k = 40, 256, 8, 2
    g = torch.Generator(device=device)
    g.manual_seed(1)
    p = moe.make_problem(T, H, 128, E, k, "bf16", "e4m3", 16)
    lg = torch.randn((T, E), generator=g, device=device)
    x = torch.randn((T, H), generator=g, device=device).bfloat16()
    codes = torch.randint(0, 0x70, (256, H), generator=g, device=device, dtype=torch.uint8)
    rm = moe.moe_max_padded_slots(p)
    rows8 = torch.zeros((rm, H), device=device, dtype=torch.uint8)
    w8 = torch.zeros((E, 128, H), device=device, dtype=torch.uint8)
    one = lambda *s: torch.ones(s, device=device)  # noqa: E731
    a = moe.route_align(p, lg, True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0 and side.cuda_stream != 0
    for s, want in ((None, 0), (0, 0), (default.cuda_stream, 0), (default, 0),
                    (side.cuda_stream, side.cuda_stream), (side, side.cuda_stream)):
        rows, _ = moe.permute(p, x, a, stream=s)
        outs = [rows, *moe.permute(p, rows8[:T], a, one(T, H // 128), stream=s),
                moe.unpermute(p, rows, a, a["topk_weights"], stream=s),
                *moe.unpermute_bwd(p, x, rows, a, a["topk_weights"], stream=s),
                moe.route_bwd(p, lg, True, a["topk_ids"], a["topk_weights"], stream=s),
                *moe.quantize_cols_e4m3(x, stream=s),
                moe.gemm_e4m3(codes, one(256, H // 128), codes, one(2, H // 128), stream=s),
                moe.grouped_gemm_e4m3(p, rows8, one(rm, H // 128), w8, one(E, 1, H // 128), a,
                                      stream=s)]
        torch.cuda.synchronize()
        assert [owner(t) for t in outs] == [want] * len(outs), s
