"""Training steps of odd layers: experts that are no multiple of the types' 16 bytes with the routing handed in."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    import mixture_experts_layer_select_amd as pkg
    return pkg


def rand(seed, *shape, dt=BF, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


@pytest.mark.parametrize("fmt,E", [("bf16", 60), ("f32", 9)])
def test_given_routing_beside_a_router_of_any_size(L, fmt, E):
    """The same bits as a layer without a router."""
    T, H, I, k, dt = 21, 64, 40, 4, BF if fmt == "bf16" else F32
    w13, w2 = rand(1, E, 2 * I, H, dt=dt, std=H ** -0.5), rand(2, E, H, I, dt=dt, std=I ** -0.5)
    x, dout = rand(3, T, H, dt=dt), rand(4, T, H, dt=dt)
    ids = rand(5, T, E, dt=F32).topk(k, 1).indices.to(torch.int32)
    tw = torch.rand((T, k), device=DEV)
    got = []
    for router in (None, dict(w=rand(6, E, H, dt=dt), bias=torch.zeros(E, device=DEV), scoring=L.SIGMOID)):
        m = L.MoELayer(fmt, H, I, k, w13, w2, router=router)
        step = m.forward_train(x, ids, tw)
        out = step.out.clone()
        g = m.backward(step, dout)
        got.append((out, g.dx, g.w13, g.w2, g.topk_w))
    for a, b in zip(*got):
        assert torch.equal(a, b) and (a != 0).any()


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_inputs_of_any_alignment(L, fmt):
    """x, dout and the residual one element behind an allocation: the bits of aligned ones."""
    T, E, H, I, k, dt = 19, 8, 72, 24, 2, BF if fmt == "bf16" else F32
    w13, w2 = rand(1, E, 2 * I, H, dt=dt, std=H ** -0.5), rand(2, E, H, I, dt=dt, std=I ** -0.5)
    m = L.MoELayer(fmt, H, I, k, w13, w2, router=dict(w=rand(3, E, H, dt=dt, std=0.2), bias=rand(4, E, dt=F32),
                                                      scoring=L.SIGMOID))
    tensors, got = [rand(s, T, H, dt=dt) for s in (5, 6, 7)], []
    for off in (0, 1):
        x, dout, res = (torch.empty(T * H + 1, device=DEV, dtype=dt)[off:off + T * H].view(T, H).copy_(t) for t in tensors)
        step = m.forward_train(x, residual=res)
        out = step.out.clone()
        g = m.backward(step, dout)
        got.append((out, step.topk_ids.clone(), g.dx.clone(), g.w13, g.w2, g.router_w, g.router_bias))
    for a, b in zip(*got):
        assert torch.equal(a, b) and (a != 0).any()


def test_residual_and_output_dropout_on_shares(L):
    """The residual in one share's call and one mask for the output: the shares' outputs add up to the whole layer's, and so
    do their gradients of x. fp32; the sums of the parts are taken in another order, of at most k + 2 terms, each of which went
    through products of at most 64 terms."""
    T, E, H, I, k = 24, 16, 64, 32, 4
    w13, w2 = rand(1, E, 2 * I, H, dt=F32, std=H ** -0.5), rand(2, E, H, I, dt=F32, std=I ** -0.5)
    router = dict(w=rand(3, E, H, dt=F32, std=0.2), bias=None, scoring=L.SIGMOID)
    x, dout, res = (rand(s, T, H, dt=F32) for s in (4, 5, 6))
    rng = torch.tensor([[1, 2], [3, 4]], device=DEV)
    whole = L.MoELayer("f32", H, I, k, w13, w2, router=router)
    step = whole.forward_train(x, residual=res, out_dropout=0.25, rng=rng)
    out, grads = step.out.clone(), whole.backward(step, dout)
    outs, dxs, parts = [], [], []
    for base in (0, 8):
        m = L.MoELayer("f32", H, I, k, w13[base:base + 8].contiguous(), w2[base:base + 8].contiguous(), router=router,
                       expert_base=base)
        step = m.forward_train(x, residual=None if base else res, out_dropout=0.25, rng=rng)
        outs.append(step.out.clone())
        parts.append((m, step, m.backward(step, dout)))
        dxs.append(parts[-1][2].dx)
    total = parts[0][2].topk_w + parts[1][2].topk_w
    parts[0][0].gate_backward(parts[0][1], total, parts[0][2])
    for got, want in ((sum(outs), out), (sum(dxs), grads.dx), (parts[0][2].router_w, grads.router_w)):
        err = (got.double() - want.double()).norm() / want.double().norm()
        assert err <= (k + 2 + 3 * 64) * 2.0 ** -24, float(err)
