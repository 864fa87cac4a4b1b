"""The training calls launch on the current device and refuse tensors of another one, or of the host, before anything is
enqueued (the other device is played by the answer of torch.cuda.current_device()); gradients made under a stream."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu

E, H, I, T, k = 8, 64, 32, 6, 2


@pytest.fixture
def calls():
    import mixture_experts_layer_select_amd as L
    f = lambda *s: torch.zeros(s, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    off, rng = i32(E + 1), torch.zeros(2, dtype=torch.int64, device=DEV)
    x, w, y = f(T, H), f(E, I, H), f(T, I)
    return dict(
        forward=lambda t=x: L.moe_grouped_gemm(t, w, None, L.F32, off, E, T, I, H, y, L.F32, False),
        dx=lambda t=y: L.moe_grouped_gemm_dx(t, w, None, L.F32, off, E, T, I, H, x, L.F32, False),
        dw=lambda t=y: L.moe_grouped_gemm_dw(t, x, L.F32, off, E, T, I, H, w, None, L.F32, False),
        swiglu=lambda t=x: L.moe_swiglu(t, L.F32, None, T, I, 0.5, rng, y),
        swiglu_grad=lambda t=x: L.moe_swiglu_grad(t, y, L.F32, None, T, I, 0.5, rng, t, None),
        dropout=lambda t=x: L.moe_dropout(t, None, L.F32, t.numel(), 0.5, rng, t),
        combine=lambda t=x: L.moe_combine_grad(t, f(T, H), L.F32, i32(T, 1), f(T, 1), T, 1, H, None, -1, f(T, H), f(T, 1)),
        route=lambda t=x: L.moe_route_grad(t, i32(T, k), f(T, k), T, H, k, L.SIGMOID, True, f(T, H), L.F32))


@pytest.mark.parametrize("name", ["forward", "dx", "dw", "swiglu", "swiglu_grad", "dropout", "combine", "route"])
def test_another_device_is_refused(calls, name, monkeypatch):
    call = calls[name]
    call()
    torch.cuda.synchronize()
    shape = (T, I) if name in ("dx", "dw") else (T, H)
    with pytest.raises(ValueError, match="tensor on cpu"):
        call(torch.zeros(shape))
    with pytest.raises(ValueError, match="not contiguous"):
        call(torch.zeros(shape[::-1], device=DEV).t())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="tensor on cuda:0, the current device is cuda:1"):
        call()


def layer(L):
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: (torch.randn(s, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    return L.MoELayer("bf16", H, I, k, r(E, 2 * I, H), r(E, H, I),
                      router=dict(w=r(E, H), bias=torch.zeros(E, device=DEV), scoring=L.SIGMOID))


def test_layer_of_another_device_is_refused(monkeypatch):
    import mixture_experts_layer_select_amd as L
    m = layer(L)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="x: on cuda:0, the current device is cuda:1"):
        m.forward_train(torch.zeros((T, H), dtype=torch.bfloat16, device=DEV))
    assert not m._bufs


def test_gradients_are_made_on_the_stream():
    """A backward without gradients on a stream, while the current stream is busy: their zeros do not come late."""
    import mixture_experts_layer_select_amd as L
    m = layer(L)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    want = m.backward(m.forward_train(x), x)
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    got = m.backward(m.forward_train(x, stream=side), x, stream=side)
    torch.cuda.synchronize()
    for n in ("w13", "w2", "router_w", "router_bias"):
        assert torch.equal(getattr(got, n), getattr(want, n)), n
