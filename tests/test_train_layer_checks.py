"""MoELayer's training calls without a GPU: which steps, tensors and sizes they refuse, before anything is enqueued. The
library's calls are recorded instead of launched; calls without tensors (checks of sizes alone) reach the library."""
import types

import pytest
import torch

E, H, I, K, T = 8, 64, 32, 2, 6
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    import os

    import mixture_experts_layer_select_amd as pkg
    if not os.path.exists(pkg._lib.LIB_PATH):
        pkg.build()
    return pkg


@pytest.fixture
def calls(L, monkeypatch):
    made = []

    def recorded(name, real):
        def call(*args, **kw):
            if not any(isinstance(a, torch.Tensor) for a in args):
                return real(*args, **kw)
            made.append(name)
        return call
    for name in ("moe_route", "moe_route_select", "moe_permute", "moe_grouped_gemm", "moe_grouped_gemm_dx",
                 "moe_grouped_gemm_dw", "moe_swiglu", "moe_swiglu_grad", "moe_dropout", "moe_combine",
                 "moe_combine_grad", "moe_route_grad"):
        monkeypatch.setattr(L._lib, name, recorded(name, getattr(L._lib, name)))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(synchronize=lambda: None))
    return made


def layer(L, router=E, bias=True, dt=BF, base=0, E_local=E):
    r = None
    if router:
        r = dict(w=torch.zeros(router, H, dtype=dt), bias=torch.zeros(router) if bias else None, scoring=L.SIGMOID)
    return L.MoELayer("bf16" if dt == BF else "f32", H, I, K, torch.zeros(E_local, 2 * I, H, dtype=dt),
                      torch.zeros(E_local, H, I, dtype=dt), router=r, expert_base=base)


def tokens(n=T, dt=BF):
    return torch.zeros(n, H, dtype=dt)


# ---------------------------------------------------------------- the gate's part of which step
def share(L):
    """Half of a router's experts: backward leaves the gate's part to gate_backward."""
    return layer(L, router=2 * E)


def test_gate_of_a_share(L, calls):
    m = share(L)
    step = m.forward_train(tokens())
    grads = m.backward(step, tokens())
    assert "moe_route_grad" not in calls
    grads.dx = grads.dx.clone()  # as a sum over GPUs would be
    m.gate_backward(step, grads.topk_w, grads)
    assert calls.count("moe_route_grad") == 1


def test_gate_refuses_a_stale_step(L, calls):
    """A later forward_train of as many tokens took the logits and picks."""
    m = share(L)
    step = m.forward_train(tokens())
    grads = m.backward(step, tokens())
    m.forward_train(tokens(T + 1))  # another size: other buffers
    later = m.forward_train(tokens())
    del calls[:]
    with pytest.raises(RuntimeError, match="no longer"):
        m.gate_backward(step, grads.topk_w, grads)
    assert not calls
    m.backward(later, tokens(), grads)
    with pytest.raises(RuntimeError, match="no longer"):
        m.gate_backward(step, grads.topk_w, grads)
    m.gate_backward(later, grads.topk_w, grads)


@pytest.mark.parametrize("done", [0, 1, 2])
@pytest.mark.parametrize("between", [1, 2, 3])
def test_gate_refuses_every_older_step(L, calls, done, between):
    """Whatever was done with the step and with the later ones: forward_train, its backward, its gate's part."""
    m = share(L)
    step = m.forward_train(tokens())
    grads = m.backward(step, tokens()) if done else m.new_grads()
    if done == 2:
        m.gate_backward(step, grads.topk_w, grads)
    for _ in range(between):
        later = m.forward_train(tokens())
        for then in (lambda: None, lambda: m.backward(later, tokens(), grads),
                     lambda: m.gate_backward(later, torch.zeros(T, K), grads)):
            then()
            for call in (lambda: m.gate_backward(step, torch.zeros(T, K), grads), lambda: m.backward(step, tokens())):
                with pytest.raises(RuntimeError):
                    call()


def test_gate_refuses_another_layers_step(L, calls):
    one, two = share(L), share(L)
    steps = [m.forward_train(tokens()) for m in (one, two)]
    grads = [m.backward(s, tokens()) for m, s in zip((one, two), steps)]
    del calls[:]
    with pytest.raises(RuntimeError, match="no longer"):
        one.gate_backward(steps[1], grads[1].topk_w, grads[0])
    assert not calls
    three = share(L)
    with pytest.raises(RuntimeError, match="no longer"):
        three.gate_backward(steps[1], grads[1].topk_w, grads[1])


def test_gate_refuses_a_step_ahead_of_its_backward(L, calls):
    m = share(L)
    grads = m.backward(m.forward_train(tokens()), tokens())
    step = m.forward_train(tokens())
    del calls[:]
    with pytest.raises(RuntimeError, match="not yet"):
        m.gate_backward(step, grads.topk_w, grads)
    assert not calls
    m.backward(step, tokens(), grads)
    m.gate_backward(step, grads.topk_w, grads)


def test_gate_refuses_a_second_part(L, calls):
    """Its part is added to dx: once for each step, and backward has added it where all experts are here."""
    m = share(L)
    step = m.forward_train(tokens())
    grads = m.backward(step, tokens())
    m.gate_backward(step, grads.topk_w, grads)
    whole = layer(L)
    all_here = whole.forward_train(tokens())
    got = whole.backward(all_here, tokens())
    assert calls.count("moe_route_grad") == 2
    for a, s, g in ((m, step, grads), (whole, all_here, got)):
        with pytest.raises(RuntimeError, match="already"):
            a.gate_backward(s, g.topk_w, g)
    assert calls.count("moe_route_grad") == 2


def test_gate_refuses_given_routing_in_the_layers_own_buffers(L, calls):
    """Picks of an earlier step handed in again are handed in: the logits need not be theirs."""
    m = share(L)
    first = m.forward_train(tokens())
    step = m.forward_train(tokens(), first.topk_ids, first.topk_w)
    grads = m.backward(step, tokens())
    with pytest.raises(ValueError, match="not routed"):
        m.gate_backward(step, grads.topk_w, grads)


def test_gate_refuses_dx_of_another_type(L, calls):
    m = share(L)
    step = m.forward_train(tokens())
    grads = m.backward(step, tokens())
    dx, grads.dx = grads.dx, grads.dx.float()
    with pytest.raises(TypeError, match="grads.dx"):
        m.gate_backward(step, grads.topk_w, grads)
    grads.dx = dx
    m.gate_backward(step, grads.topk_w, grads)


def test_a_step_refused_by_the_gate_keeps_its_backward(L, calls):
    m = share(L)
    step = m.forward_train(tokens())
    with pytest.raises(RuntimeError):
        m.gate_backward(step, torch.zeros(T, K), m.new_grads())
    m.backward(step, tokens())
    with pytest.raises(RuntimeError, match="later step"):
        m.backward(step, tokens())


# ---------------------------------------------------------------- inputs in the layer's own buffers
def test_inputs_in_the_steps_buffers_are_refused(L, calls):
    """The next step of as many tokens writes its output before it reads the residual, and before backward reads x."""
    m = layer(L)
    step = m.forward_train(tokens())
    del calls[:]
    for kw, name in ((dict(x=tokens(), residual=step.out), "residual"), (dict(x=step.out), "x"),
                     (dict(x=step.dx), "x"), (dict(x=step.b.x_perm[3:3 + T]), "x"),
                     (dict(x=tokens(), residual=step.b.y_perm[1:1 + T]), "residual")):
        with pytest.raises(ValueError, match=f"^{name}: lies in the layer's buffers for {T} tokens"):
            m.forward_train(**kw)
    assert not calls
    m.backward(step, tokens())  # and the step is still the layer's


def test_inputs_beside_the_steps_buffers_are_taken(L, calls):
    m, other = layer(L), layer(L)
    step = m.forward_train(tokens())
    other.forward_train(step.out, residual=step.out)
    m.forward_train(step.out[:T - 1], residual=step.out[1:])  # of another size: other buffers
    m.forward_train(tokens(), residual=step.dx)  # which backward alone writes
    m.forward_train(tokens(0), residual=tokens(0))


# ---------------------------------------------------------------- ahead of the first launch
@pytest.mark.parametrize("name", ["dropout", "out_dropout"])
@pytest.mark.parametrize("p", [1.0, -0.1, 0.999999, float("nan")])
def test_dropout_is_refused_ahead_of_the_launches(L, calls, name, p):
    m, rng = layer(L), torch.zeros((2, 2), dtype=torch.int64)
    step = m.forward_train(tokens(), dropout=0.5, out_dropout=0.25, rng=rng)
    del calls[:]
    with pytest.raises(L.MoEError) as e:
        m.forward_train(tokens(), rng=rng, **{name: p})
    assert e.value.status == "MOE_ERR_INVALID_ARG" and not calls
    m.backward(step, tokens())  # its buffers are not taken
    with pytest.raises(L.MoEError):
        m.forward_train(tokens(T + 3), rng=rng, **{name: p})
    assert ("train", T + 3) not in m._bufs


# ---------------------------------------------------------------- sizes
@pytest.mark.parametrize("dt,experts", [(BF, 60), (BF, 9), (torch.float32, 6), (torch.float32, 9)])
def test_any_number_of_experts_where_the_routing_is_given(L, calls, dt, experts):
    """The gate's products run along the experts in whole 16 bytes; a step with its routing handed in makes none."""
    m = layer(L, router=experts, dt=dt, E_local=experts)
    with pytest.raises(ValueError, match=f"the router's experts = {experts} is not a multiple of"):
        m.forward_train(tokens(dt=dt))
    assert not calls
    step = m.forward_train(tokens(dt=dt), torch.zeros((T, K), dtype=torch.int32), torch.ones(T, K))
    grads = m.backward(step, tokens(dt=dt))
    assert "moe_route" not in calls and "moe_route_grad" not in calls
    with pytest.raises(ValueError, match="not routed"):
        m.gate_backward(step, grads.topk_w, grads)


# ---------------------------------------------------------------- buffers
@pytest.mark.parametrize("name,at", [("empty", 3), ("empty", 12), ("empty_like", 1), ("empty_like", 2), ("ones", 1),
                                     ("ones", 2), ("tensor", 1), ("empty", 15)])
def test_memory_that_runs_out_on_the_first_step(L, calls, monkeypatch, name, at):
    """The step fails with the allocation's own error, leaves nothing behind, and runs once there is memory."""
    m, x, real, made = layer(L), tokens(), getattr(torch, name), []

    def allocate(*args, **kw):
        made.append(0)
        if len(made) == at:
            raise torch.OutOfMemoryError("out of memory")
        return real(*args, **kw)
    monkeypatch.setattr(torch, name, allocate)
    with pytest.raises(torch.OutOfMemoryError):
        m.forward_train(x)
    assert not m._bufs and not calls
    monkeypatch.setattr(torch, name, real)
    m.backward(m.forward_train(x), tokens())


def test_training_holds_no_workspace_of_inference(L, calls):
    """From 4096 tokens on inference routes through a workspace, and its experts keep their intermediate in another."""
    m = L.MoELayer("bf16", 128, 128, 2, torch.zeros(E, 256, 128, dtype=BF), torch.zeros(E, 128, 128, dtype=BF),
                   router=dict(w=torch.zeros(E, 128, dtype=BF), bias=None, scoring=L.SIGMOID))
    x = torch.zeros(4096, 128, dtype=BF)
    b = m.forward_train(x).b
    assert b.ws_ffn.numel() <= 1 and b.ws_route is None and "moe_route" in calls
    inference = m.buffers(4096)
    assert inference is not b and inference.ws_route is not None
    assert inference.ws_ffn.numel() == L.moe_expert_ffn_workspace_size(m.weights, 3 * 4096)


def off_by_one(*shape):
    """A tensor that begins one element behind an allocation."""
    n = 1
    for s in shape:
        n *= s
    return torch.zeros(n + 1, dtype=BF)[1:].view(shape)


def test_sizes_are_refused_ahead_of_the_launches(L, calls):
    """What the library's calls of a step refuse is refused with nothing launched and no buffers made."""
    def step(m, n=3):
        m.forward_train(torch.zeros(n, m.H, dtype=BF), torch.zeros((n, m.k), dtype=torch.int32), torch.zeros(n, m.k))

    def plain(experts, h, i, k):
        return L.MoELayer("bf16", h, i, k, torch.zeros(experts, 2 * i, h, dtype=BF), torch.zeros(experts, h, i, dtype=BF))
    for m, match in ((plain(257, 8, 8, 2), "E_local=257"), (plain(1, 8, 8, 257), "k=257"),
                     (plain(1, 65544, 8, 1), "K=65544"), (plain(1, 8, 32776, 1), "N=65552")):
        with pytest.raises(L.MoEError, match=match) as e:
            step(m)
        assert e.value.status == "MOE_ERR_UNSUPPORTED" and not m._bufs, match
    wide = layer(L, router=264)
    with pytest.raises(L.MoEError, match="E=264"):
        wide.forward_train(tokens())
    step(wide)  # handed in
    del calls[:]
    with pytest.raises(L.MoEError, match="unknown scoring"):
        m = layer(L)
        m.router["scoring"] = 7
        m.forward_train(tokens())
    with pytest.raises(ValueError, match="expected .T, 64."):
        layer(L).forward_train(torch.zeros((), dtype=BF))
    m = plain(1, 8, 8, 255)
    n = 2 ** 30 // 256 + 1
    with pytest.raises(ValueError, match="more than 2.30 rows"):
        m.forward_train(torch.empty(n, 8, dtype=BF), torch.empty((n, 255), dtype=torch.int32), torch.empty(n, 255))
    assert not m._bufs and not calls


@pytest.mark.parametrize("name", ["w13", "w2", "shared w13", "shared w2"])
def test_weights_off_their_alignment_are_refused(L, calls, name):
    def make(what, *shape):
        return off_by_one(*shape) if what == name else torch.zeros(shape, dtype=BF)
    m = L.MoELayer("bf16", H, I, K, make("w13", E, 2 * I, H), make("w2", E, H, I),
                   shared=dict(w13=make("shared w13", 2 * I, H), w2=make("shared w2", H, I)),
                   router=dict(w=torch.zeros(E, H, dtype=BF), bias=None, scoring=L.SIGMOID))
    with pytest.raises(ValueError, match=f"^{name}: not 16-byte aligned"):
        m.forward_train(tokens())
    assert not calls and not m._bufs


@pytest.mark.parametrize("name", ["w13", "w2", "shared_w13", "shared_w2", "router_w"])
def test_gradients_off_their_alignment_are_refused(L, calls, name):
    """Ahead of the launches: the step keeps its buffers and takes a backward with others."""
    m = L.MoELayer("bf16", H, I, K, torch.zeros(E, 2 * I, H, dtype=BF), torch.zeros(E, H, I, dtype=BF),
                   shared=dict(w13=torch.zeros(2 * I, H, dtype=BF), w2=torch.zeros(H, I, dtype=BF)),
                   router=dict(w=torch.zeros(E, H, dtype=BF), bias=torch.zeros(E), scoring=L.SIGMOID))
    step, grads = m.forward_train(tokens()), m.new_grads()
    good = getattr(grads, name)
    setattr(grads, name, torch.zeros(good.numel() + 1)[1:].view(good.shape))
    del calls[:]
    with pytest.raises(ValueError, match=f"^grads.{name}: not 16-byte aligned"):
        m.backward(step, tokens(), grads)
    assert not calls
    setattr(grads, name, good)
    grads.router_bias = torch.zeros(E + 1)[1:]  # any
    m.backward(step, tokens(), grads)


def test_a_router_off_its_alignment_is_refused_ahead_of_the_gradients(L, calls):
    for m in (layer(L), share(L)):
        m.router["w"] = off_by_one(*m.router["w"].shape)
        step = m.forward_train(tokens())
        del calls[:]
        with pytest.raises(ValueError, match="^the router's w: not 16-byte aligned"):
            grads = m.backward(step, tokens())
            assert not step.routed_here
            del calls[:]
            m.gate_backward(step, grads.topk_w, grads)
        assert not calls


def test_dx_off_its_alignment_is_refused(L, calls):
    m = share(L)
    step = m.forward_train(tokens())
    grads = m.backward(step, tokens())
    dx, grads.dx = grads.dx, off_by_one(T, H)
    with pytest.raises(ValueError, match="^grads.dx: not 16-byte aligned"):
        m.gate_backward(step, grads.topk_w, grads)
    grads.dx = dx
    m.gate_backward(step, grads.topk_w, grads)


@pytest.mark.parametrize("rng", [torch.zeros(1, dtype=torch.int64), torch.zeros(2, 2), torch.zeros(2, 4)[:, ::2]])
def test_rng_is_not_looked_at_without_dropout(L, calls, monkeypatch, rng):
    """No call is handed a tensor that nothing has checked."""
    m = layer(L)
    seen = []
    for name in ("moe_swiglu", "moe_swiglu_grad", "moe_dropout"):
        monkeypatch.setattr(L._lib, name, lambda *args: seen.append(any(a is rng for a in args)))
    step = m.forward_train(tokens(), residual=tokens(), rng=rng)
    m.backward(step, tokens())
    assert len(seen) == 3 and not any(seen)
