"""A training step of the layer: forward_train and backward against a float64 layer differentiated by autograd, the calls
one by one, graphs, differences, the dropouts, accumulation, refusals."""
import pytest
import torch

import train_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    import mixture_experts_layer_select_amd as pkg
    return pkg


def weights(E, H, I, dt, seed=0, E_all=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, std: (torch.randn(s, generator=g, device=DEV) * std).to(dt)
    return dict(w13=r(E, 2 * I, H, std=H ** -0.5), w2=r(E, H, I, std=I ** -0.5), s13=r(2 * I, H, std=H ** -0.5),
                s2=r(1, H, I, std=I ** -0.5), rw=r(E_all or E, H, std=2 * H ** -0.5),
                rb=torch.randn(E_all or E, generator=g, device=DEV) * 0.1)


def make(L, fmt, E, H, I, k, shared=True, router=True, bias=True, scoring=None, renorm=True, base=0, E_all=None, seed=0):
    w = weights(E, H, I, BF if fmt == "bf16" else F32, seed, E_all)
    layer = L.MoELayer(fmt, H, I, k, w["w13"], w["w2"], shared=dict(w13=w["s13"], w2=w["s2"]) if shared else None,
                       router=dict(w=w["rw"], bias=w["rb"] if bias else None,
                                   scoring=L.SIGMOID if scoring is None else scoring, renormalize=renorm)
                       if router else None, expert_base=base)
    return layer, w


def reference(L, layer, w, x, ids, given_w=None, residual=None, p=0.0, p_out=0.0, rng=None, row_to_slot=None):
    """The layer in float64 on the CPU with the picks held fixed; leaves for the gradients."""
    k, E, base = layer.k, layer.E_local, layer.expert_base
    T, H = x.shape
    leaf = lambda t: None if t is None else t.double().cpu().clone().requires_grad_()
    v = dict(x=leaf(x), w13=leaf(w["w13"]), w2=leaf(w["w2"]), s13=leaf(w["s13"].reshape(2 * layer.I, H)),
             s2=leaf(w["s2"].reshape(H, layer.I)), rw=leaf(w["rw"]), rb=leaf(w["rb"]), topk_w=leaf(given_w))
    ids = ids.long().cpu()
    if given_w is None:
        r = layer.router
        logits = v["x"] @ v["rw"].t() + (v["rb"] if r["bias"] is not None else 0)
        picked = logits.gather(1, ids)
        if r["scoring"] == L.SIGMOID:
            tw = torch.sigmoid(picked)
            tw = tw / tw.sum(1, keepdim=True) if r["renormalize"] else tw
        else:
            tw = torch.softmax(picked, 1) if r["renormalize"] else torch.softmax(logits, 1).gather(1, ids)
    else:
        tw = v["topk_w"]
    out = torch.zeros((T, H), dtype=torch.float64)
    rows = row_to_slot.cpu().tolist()
    factor = None if p == 0 else train_ref.factor(rng[0].cpu(), len(rows) * layer.I, p).view(-1, layer.I)
    for row, slot in enumerate(rows):
        if slot < 0:
            break
        t, j = (slot // k, slot % k) if slot < T * k else (slot - T * k, -1)
        e = -1 if j < 0 else int(ids[t, j]) - base
        gu = (v["s13"] if j < 0 else v["w13"][e]) @ v["x"][t]
        a = torch.nn.functional.silu(gu[:layer.I]) * gu[layer.I:]
        if factor is not None:
            a = a * factor[row]
        y = (v["s2"] if j < 0 else v["w2"][e]) @ a
        out = out.index_add(0, torch.tensor([t]), (y if j < 0 else tw[t, j] * y)[None])
    if p_out:
        out = out * train_ref.factor(rng[1].cpu(), T * H, p_out).view(T, H)
    return out + (0 if residual is None else residual.double().cpu()), v


def near(got, ref, fmt, name, roundings=9):
    """In the norm. bf16: every tensor between two calls is rounded by half a step (x's gradient has gone through gu, a, y or
    dy, da, dgu, the rows' dx, their sum, dlogits and the gate's part: nine), each rounding's effect carried on by
    operators of norm about one; twice that for those that are above one. fp32: sums of up to 2^10 terms, worth
    2^-24 of the terms' norm each, through the same chain."""
    unit = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -24 * 2 ** 5  # sqrt of the 2^10 terms, whose roundings do not line up
    ref = ref.to(got.device) if isinstance(ref, torch.Tensor) else ref
    err = (got.double() - ref).norm() / ref.norm().clamp(min=1e-30)
    assert err <= 2 * roundings * unit, (name, float(err))


def compare(layer, grads, v, fmt, routed=True):
    near(grads.dx, v["x"].grad, fmt, "dx")
    near(grads.w13, v["w13"].grad, fmt, "w13")
    near(grads.w2, v["w2"].grad, fmt, "w2")
    if layer.shared is not None:
        near(grads.shared_w13.view_as(v["s13"]), v["s13"].grad, fmt, "s13")
        near(grads.shared_w2.view_as(v["s2"]), v["s2"].grad, fmt, "s2")
    if routed and layer.k == 1 and layer.router.get("renormalize"):
        # the one pick's weight is s / s = 1 whatever its logit
        assert (grads.router_w == 0).all() and (grads.router_bias == 0).all()
    elif routed:
        near(grads.router_w, v["rw"].grad, fmt, "router")
        if layer.router["bias"] is not None:
            near(grads.router_bias, v["rb"].grad, fmt, "bias")


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,H,I,k,shared,scoring,renorm", [
    (1, 8, 64, 40, 2, True, 1, True), (7, 8, 72, 24, 3, False, 1, False), (33, 16, 136, 72, 4, True, 0, True),
    (20, 24, 64, 8, 8, True, 0, False), (65, 8, 256, 264, 1, True, 1, True)])
def test_step(L, T, E, H, I, k, shared, scoring, renorm, fmt):
    layer, w = make(L, fmt, E, H, I, k, shared=shared, scoring=scoring, renorm=renorm, bias=T != 7)
    g = torch.Generator(device=DEV).manual_seed(T)
    dt = BF if fmt == "bf16" else F32
    x, dout = (torch.randn((T, H), generator=g, device=DEV).to(dt) for _ in range(2))
    step = layer.forward_train(x)
    out = step.out.clone()
    ref, v = reference(L, layer, w, x, step.topk_ids, row_to_slot=step.b.row_to_slot)
    near(out, ref.detach(), fmt, "out")
    grads = layer.backward(step, dout)
    (ref * dout.double().cpu()).sum().backward()
    compare(layer, grads, v, fmt)
    # inference gives the same output where its kernels are the same products
    if fmt == "f32":
        near(layer.forward(x).out, ref.detach(), fmt, "inference")


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
def test_dropout_and_residual(L, fmt):
    T, E, H, I, k = 19, 8, 64, 48, 2
    layer, w = make(L, fmt, E, H, I, k)
    g = torch.Generator(device=DEV).manual_seed(3)
    dt = BF if fmt == "bf16" else F32
    x, dout, res = (torch.randn((T, H), generator=g, device=DEV).to(dt) for _ in range(3))
    rng = torch.tensor([[5, 6], [7, 8]], device=DEV)
    step = layer.forward_train(x, dropout=0.25, out_dropout=0.5, residual=res, rng=rng)
    ref, v = reference(L, layer, w, x, step.topk_ids, residual=res, p=0.25, p_out=0.5, rng=rng,
                       row_to_slot=step.b.row_to_slot)
    near(step.out, ref.detach(), fmt, "out")
    grads = layer.backward(step, dout)
    (ref * dout.double().cpu()).sum().backward()
    compare(layer, grads, v, fmt)


def test_given_routing_on_a_share(L):
    """An expert share with the routing handed in: picks elsewhere add nothing, the weights' gradients come back."""
    T, E, H, I, k, base = 30, 8, 64, 32, 3, 4
    layer, w = make(L, "f32", E, H, I, k, router=False, base=base)
    g = torch.Generator(device=DEV).manual_seed(4)
    x, dout = (torch.randn((T, H), generator=g, device=DEV) for _ in range(2))
    ids = torch.rand((T, 20), generator=g, device=DEV).topk(k, 1).indices.to(torch.int32)
    tw = torch.rand((T, k), generator=g, device=DEV)
    step = layer.forward_train(x, ids, tw)
    ref, v = reference(L, layer, w, x, ids, given_w=tw, row_to_slot=step.b.row_to_slot)
    near(step.out, ref.detach(), "f32", "out")
    grads = layer.backward(step, dout)
    (ref * dout.double().cpu()).sum().backward()
    compare(layer, grads, v, "f32", routed=False)
    near(grads.topk_w, v["topk_w"].grad, "f32", "topk_w")
    with pytest.raises(ValueError, match="not routed"):
        layer.gate_backward(step, grads.topk_w, grads)


def test_shares_add_up(L):
    """Two shares of the experts with the router on both: dx, the picks' weights' gradients and, from their sum, the gate's
    equal the whole layer's."""
    T, E, H, I, k = 24, 16, 64, 32, 4
    whole, w = make(L, "f32", E, H, I, k, shared=False)
    g = torch.Generator(device=DEV).manual_seed(6)
    x, dout = (torch.randn((T, H), generator=g, device=DEV) for _ in range(2))
    want = whole.backward(whole.forward_train(x), dout)
    parts = []
    for base in (0, 8):
        layer = L.MoELayer("f32", H, I, k, w["w13"][base:base + 8].contiguous(), w["w2"][base:base + 8].contiguous(),
                           router=whole.router, expert_base=base)
        step = layer.forward_train(x)
        parts.append((layer, step, layer.backward(step, dout)))
    total = parts[0][2].topk_w + parts[1][2].topk_w
    near(total, want.topk_w.double(), "f32", "topk_w")
    layer, step, grads = parts[0]
    layer.gate_backward(step, total, grads)
    near(grads.router_w, want.router_w.double(), "f32", "router")
    near(grads.router_bias, want.router_bias.double(), "f32", "bias")
    near(grads.dx + parts[1][2].dx, want.dx.double(), "f32", "dx")
    near(torch.cat([p[2].w13 for p in parts]), want.w13.double(), "f32", "w13")


def test_accumulate(L):
    layer, _ = make(L, "bf16", 8, 64, 32, 2)
    g = torch.Generator(device=DEV).manual_seed(7)
    xs = [torch.randn((9 + i, 64), generator=g, device=DEV).to(BF) for i in range(2)]
    ds = [torch.randn((9 + i, 64), generator=g, device=DEV).to(BF) for i in range(2)]
    steps = [layer.forward_train(x) for x in xs]  # of different sizes: both alive
    one = [layer.backward(s, d) for s, d in zip(steps, ds)]
    both = layer.new_grads()
    for x, d in zip(xs, ds):
        layer.backward(layer.forward_train(x), d, both, accumulate=True)
    for name in ("w13", "w2", "shared_w13", "shared_w2", "router_w", "router_bias"):
        a, b = getattr(one[0], name), getattr(one[1], name)
        err = (getattr(both, name).double() - (a.double() + b.double())).abs()
        assert (err <= 2.0 ** -23 * (a.abs() + b.abs())).all(), name
    with pytest.raises(ValueError, match="accumulate"):
        layer.backward(layer.forward_train(xs[0]), ds[0], accumulate=True)


def test_graph(L):
    """Forward and backward captured, replayed with a moving offset between eager steps of another size: the eager bits."""
    layer, _ = make(L, "bf16", 16, 128, 64, 4)
    g = torch.Generator(device=DEV).manual_seed(8)
    x, dout = (torch.randn((21, 128), generator=g, device=DEV).to(BF) for _ in range(2))
    other = torch.randn((5, 128), generator=g, device=DEV).to(BF)
    rng = torch.tensor([[1, 0], [2, 0]], device=DEV)
    move = torch.tensor([[0, 1], [0, 1]], device=DEV)
    names = ("w13", "w2", "shared_w13", "shared_w2", "router_w", "router_bias", "dx")

    def run(grads, r):
        step = layer.forward_train(x, dropout=0.1, out_dropout=0.2, rng=r)
        return step, layer.backward(step, dout, grads)
    want = []
    for i in range(3):
        step, grads = run(layer.new_grads(), rng + i * move)
        want.append([step.out.clone()] + [getattr(grads, n).clone() for n in names])
    grads = layer.new_grads()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step, _ = run(grads, rng)
        rng.add_(move)
    for i in range(3):
        graph.replay()
        layer.backward(layer.forward_train(other), other)
        torch.cuda.synchronize()
        for got, ref in zip([step.out] + [getattr(grads, n) for n in names], want[i]):
            assert torch.equal(got, ref)
    assert not torch.equal(want[0][0], want[1][0])


def test_stream(L):
    layer, _ = make(L, "bf16", 8, 64, 32, 2)
    x = torch.randn((12, 64), device=DEV).to(BF)
    want = layer.backward(layer.forward_train(x), x)
    want = [want.dx.clone(), want.w13, want.router_bias]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step = layer.forward_train(x, stream=s)
    with torch.cuda.stream(s):
        grads = layer.new_grads()
    got = layer.backward(step, x, grads, stream=s)
    s.synchronize()
    for a, b in zip((got.dx, got.w13, got.router_bias), want):
        assert torch.equal(a, b)


def test_other_stream_first(L):
    """A layer whose first step runs on a stream of its own, and a capture without a step before it."""
    layer, _ = make(L, "bf16", 8, 64, 32, 2)
    again, _ = make(L, "bf16", 8, 64, 32, 2)
    x = torch.randn((12, 64), device=DEV).to(BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        grads = layer.new_grads()
    got = layer.backward(layer.forward_train(x, stream=s), x, grads, stream=s)
    s.synchronize()
    want = again.backward(again.forward_train(x), x)
    for n in ("dx", "w13", "router_w", "router_bias"):
        assert torch.equal(getattr(got, n), getattr(want, n)), n
    third, _ = make(L, "bf16", 8, 64, 32, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(graph):
            third.forward_train(x)
    torch.cuda.synchronize()


def test_no_tokens(L):
    layer, _ = make(L, "bf16", 8, 64, 32, 2)
    x = torch.empty((0, 64), device=DEV, dtype=BF)
    grads = layer.backward(layer.forward_train(x), x)
    assert grads.dx.shape == (0, 64)
    for g in (grads.w13, grads.w2, grads.shared_w13, grads.shared_w2, grads.router_w, grads.router_bias):
        assert (g == 0).all()


def test_inference_keeps_its_buffers(L):
    """A forward between forward_train and backward changes nothing; a later forward_train of the same size does."""
    layer, _ = make(L, "bf16", 8, 128, 128, 2)
    g = torch.Generator(device=DEV).manual_seed(9)
    x, z = (torch.randn((10, 128), generator=g, device=DEV).to(BF) for _ in range(2))
    want = layer.backward(layer.forward_train(x), x).w13
    step = layer.forward_train(x)
    layer.forward(z)
    got = layer.backward(step, x)
    assert torch.equal(got.w13, want)
    with pytest.raises(RuntimeError, match="later step"):
        layer.backward(step, x)  # its buffers hold gradients
    step = layer.forward_train(x)
    layer.forward_train(z)
    with pytest.raises(RuntimeError, match="later step"):
        layer.backward(step, x)


def test_against_differences(L):
    """Central differences of sum(c out) in fp32 along random directions of x and of the weights, picks held fixed by their
    margins: h^2 / 6 of the third derivative (taken as 4 times the gradient's scale) and the values' rounding over h."""
    layer, w = make(L, "f32", 8, 32, 16, 2, seed=3)
    g = torch.Generator(device=DEV).manual_seed(10)
    x = torch.randn((6, 32), generator=g, device=DEV)
    c = torch.randn((6, 32), generator=g, device=DEV)
    rng = torch.tensor([[3, 1], [4, 1]], device=DEV)
    kw = dict(dropout=0.25, out_dropout=0.25, rng=rng)
    step = layer.forward_train(x, **kw)
    ids = step.topk_ids.clone()
    grads = layer.backward(step, c)
    grads.dx = grads.dx.clone()
    h = 2.0 ** -8
    params = [(x, grads.dx), (w["w13"], grads.w13), (w["w2"], grads.w2), (w["s13"], grads.shared_w13),
              (w["s2"], grads.shared_w2), (w["rw"], grads.router_w), (w["rb"], grads.router_bias)]
    for p, grad in params:
        v = torch.randn(p.shape, generator=g, device=DEV)
        v /= v.norm()
        keep, value = p.clone(), []
        for sign in (1, -1):
            p.copy_(keep + sign * h * v)
            step = layer.forward_train(x, **kw)
            assert torch.equal(step.topk_ids, ids)
            value.append((step.out.double() * c.double()).sum())
            size = float((step.out * c).abs().sum())
        moved = float((grad.double() * keep.double()).abs().sum()) * 2.0 ** -24 / h  # the points' own rounding
        p.copy_(keep)
        slope, want = float(value[0] - value[1]) / (2 * h), float((grad.double() * v.double()).sum())
        tol = h * h / 6 * 4 * float(grad.norm()) + size * 2.0 ** -18 / h + moved
        assert abs(slope - want) <= tol, (p.shape, slope, want, tol)


def test_refusals(L):
    layer, w = make(L, "bf16", 8, 64, 32, 2)
    x = torch.randn((4, 64), device=DEV).to(BF)
    rng = torch.zeros((2, 2), dtype=torch.int64, device=DEV)
    for kw, err in ((dict(dropout=0.1), "needs rng"), (dict(dropout=0.1, rng=rng[0]), "shape"),
                    (dict(out_dropout=0.1, rng=rng.int()), "dtype"), (dict(residual=x[:2]), "shape"),
                    (dict(residual=x.float()), "dtype")):
        with pytest.raises((ValueError, TypeError), match=err):
            layer.forward_train(x, **kw)
    for p in (1.0, -0.1, float("nan")):
        with pytest.raises(L.MoEError):
            layer.forward_train(x, dropout=p, rng=rng)
    step = layer.forward_train(x)
    for bad in (x.float(), x[:2], x.t().contiguous()):
        with pytest.raises((ValueError, TypeError)):
            layer.backward(step, bad)
    grads = layer.new_grads()
    for name, bad in (("w13", None), ("w2", grads.w2[:4]), ("router_w", grads.router_w.to(BF)),
                      ("shared_w13", grads.shared_w13.t().contiguous().t())):
        keep = getattr(grads, name)
        setattr(grads, name, bad)
        with pytest.raises((ValueError, TypeError), match=f"grads.{name}"):
            layer.backward(step, x, grads)
        setattr(grads, name, keep)
    other, _ = make(L, "bf16", 8, 64, 32, 2)
    with pytest.raises(RuntimeError):
        other.backward(step, x)
    layer.backward(step, x, grads)  # none of these touched the step
    fp8 = L.MoELayer("fp8", 256, 128, 2, torch.zeros((4, 256, 256), dtype=torch.uint8, device=DEV),
                     torch.zeros((4, 256, 128), dtype=torch.uint8, device=DEV), torch.ones((4, 2, 2), device=DEV),
                     torch.ones((4, 2, 1), device=DEV))
    with pytest.raises(ValueError, match="f32 or bf16"):
        fp8.forward_train(torch.zeros((4, 256), device=DEV, dtype=BF))
    odd, _ = make(L, "bf16", 9, 64, 32, 2)
    with pytest.raises(ValueError, match="multiple of 8"):
        odd.forward_train(x)


def test_batch_of_the_layer(L):
    """A batch at the layer's widths: finite, and every weight gradient equal to the calls one by one."""
    T, E, H, I, k = 300, 16, 7168, 2048, 8
    layer, w = make(L, "bf16", E, H, I, k)
    g = torch.Generator(device=DEV).manual_seed(12)
    x, dout = (torch.randn((T, H), generator=g, device=DEV).to(BF) for _ in range(2))
    step = layer.forward_train(x)
    off, r2s, s2r = step.b.offsets.clone(), step.b.row_to_slot.clone(), step.b.slot_to_row.clone()
    y, gu, xp, tw = step.b.y_perm.clone(), step.gu.clone(), step.b.x_perm.clone(), step.topk_w.clone()
    grads = layer.backward(step, dout)
    R = T * k + T
    counts = off.tolist()
    rows = r2s.long()[:R]
    token = torch.where(rows < T * k, rows // k, rows - T * k)
    weight = torch.where(rows < T * k, tw.flatten()[rows.clamp(max=T * k - 1)], torch.ones_like(tw.flatten()[:1]))
    assert torch.equal(xp[:R], x[token])
    dy = (dout[token].float() * weight[:, None]).to(BF)
    for name, a, b, got in (("w2", dy, None, grads.w2),):
        g_, u_ = gu[:R].float().chunk(2, 1)
        act = (torch.nn.functional.silu(g_) * u_).to(BF)
        ref, mag = train_ref.grouped("weights", dy, act, counts)
        # act may round to the neighbour of the kernel's: half a step of it more
        err = (got.double() - ref[:E]).abs()
        assert (err <= (2.0 ** -8 + R * 2.0 ** -23) * mag[:E]).all(), name
    assert all(torch.isfinite(t).all() for t in (grads.dx, grads.w13, grads.router_w, grads.router_bias))
