"""Calls that take MXFP4 weights launch on the current device and refuse tensors and weights of another one before
anything is enqueued. The other device is played by the answer of torch.cuda.current_device(), so one GPU is enough."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu

H, I, E, T = 256, 128, 2, 3


@pytest.fixture
def calls():
    import mixture_experts_layer_select_amd as L
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    shapes = ((E, 2 * I, H // 2), (E, H, I // 2), (E, 2 * I, H // 32), (E, H, I // 32))
    w = L.make_weights(L.MXFP4, E, H, I, *[u8(*s) for s in shapes])
    x, xs, off = u8(T, H // 2), u8(T, H // 32), torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    y, slots = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    n = L.moe_expert_ffn_workspace_size(w, T)
    ws = u8(n)
    few = u8(L.moe_layer_few_workspace_size(w, T, E, 1))
    ids, tw = torch.zeros((T, 1), dtype=torch.int32, device=DEV), torch.zeros((T, 1), device=DEV)
    return dict(
        ffn=lambda w=w, x=x: L.moe_expert_ffn(w, x, xs, off, E, T, y, ws, n),
        gate_up=lambda w=w, x=x: L.moe_expert_ffn_gate_up(w, x, xs, off, E, T, ws, n),
        tokens=lambda w=w, x=x: L.moe_expert_ffn_gate_up_tokens(w, x, xs, T, 1, slots, off, E, T, ws, n),
        down=lambda w=w, x=y: L.moe_expert_ffn_down(w, off, E, T, x, ws, n),
        noalloc=lambda w=w, x=x: L.moe_expert_ffn_noalloc(w, x, xs, off, E, T, y),
        few=lambda w=w, x=y: L.moe_layer_few(x, None, None, T, E, 1, L.SIGMOID, True, w, 0, ids, tw, y, few, few.numel()))


@pytest.mark.parametrize("name", ["ffn", "gate_up", "tokens", "down", "noalloc", "few"])
def test_another_device_is_refused(calls, name, monkeypatch):
    call = calls[name]
    call()  # on its own device the same call goes through
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="tensor on cuda:0, the current device is cuda:1"):
        call()


def test_weights_of_another_device_are_refused(monkeypatch):
    import mixture_experts_layer_select_amd as L
    w = L.make_weights(L.MXFP4, 1, H, I, *[torch.zeros(1, 1, dtype=torch.uint8, device=DEV)] * 4)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="weights on cuda:0, the current device is cuda:1"):
        L.moe_expert_ffn(w, None, None, None, 1, 0, None, None, 0, 0)


def test_current_stream_by_either_way(monkeypatch):
    """Calls without a stream go to torch's current one, with torch's raw handle and without it."""
    from mixture_experts_layer_select_amd import _lib
    side = torch.cuda.Stream()
    for raw in (_lib._raw_stream, None):
        monkeypatch.setattr(_lib, "_raw_stream", raw)
        assert _lib._stream() == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(side):
            assert _lib._stream() == side.cuda_stream != torch.cuda.default_stream().cuda_stream
        assert _lib._stream(side) == side.cuda_stream


@pytest.mark.parametrize("handle", [False, True])
def test_quantize_mxfp4_allocates_on_its_stream(handle):
    """Freed codes go back to the stream that wrote them: the next tensor there takes their memory, one of the current
    stream does not, so nothing is written over while the other stream works."""
    import mixture_experts_layer_select_amd as L
    side = torch.cuda.Stream()
    x = torch.randn((4096, 16384), device=DEV)
    torch.cuda.synchronize()
    want = L.quantize_mxfp4(x)
    codes, scales = L.quantize_mxfp4(x, side.cuda_stream if handle else side)
    side.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    at, n = codes.data_ptr(), codes.numel()
    del codes
    here = torch.empty(n, dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(side):
        there = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert here.data_ptr() != at and there.data_ptr() == at


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("name", ["forward", "forward_few", "forward_block", "forward_fused"])
def test_layer_of_another_device_is_refused(fmt, name, monkeypatch):
    """Before its first step: not even buffers are made."""
    import mixture_experts_layer_select_amd as L
    w13, w2 = torch.zeros((E, 2 * I, H), device=DEV), torch.zeros((E, H, I), device=DEV)
    if fmt == "mxfp4":
        (w13, s13), (w2, s2) = L.quantize_mxfp4(w13), L.quantize_mxfp4(w2)
    else:
        w13, w2, s13, s2 = w13.to(torch.bfloat16), w2.to(torch.bfloat16), None, None
    router = dict(w=torch.zeros((E, H), dtype=torch.bfloat16, device=DEV), bias=None, scoring=L.SIGMOID)
    layer = L.MoELayer(fmt, H, I, 1, w13, w2, s13, s2, router=router)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="x: on cuda:0, the current device is cuda:1"):
        getattr(layer, name)(x)
    assert not layer._bufs
