"""The MXFP4 layer and the block around it as a program runs them: weights quantised on the GPU, prompt and
few-token forms, graphs, and every step against 64 bits on the previous step's own outputs."""
import pytest
import torch

import mx_ref
from gpu_util import DEV, say
from mx_ref import F64, U
from test_gpu_10_mxfp4 import check
from test_gpu_11_norm import close, rms

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 256, 8, 3


def _lib():
    import mixture_experts_layer_select_amd as L
    return L


def rand(shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


class Case:
    def __init__(self, shared=True):
        L = _lib()
        self.w13, self.w2 = rand((E + 1, 2 * I, H), 1, 0.05), rand((E + 1, H, I), 2, 0.05)
        c13, s13 = L.quantize_mxfp4(self.w13.to(DEV))
        c2, s2 = L.quantize_mxfp4(self.w2.to(DEV))
        self.v13, self.v2 = mx_ref.quantize(self.w13)[2], mx_ref.quantize(self.w2)[2]
        sh = dict(w13=c13[E], w13_scale=s13[E], w2=c2[E], w2_scale=s2[E]) if shared else None
        self.router = rand((E, H), 3, 0.05).to(DEV)
        self.layer = L.MoELayer("mxfp4", H, I, K, c13[:E], c2[:E], s13[:E], s2[:E], shared=sh,
                                router=dict(w=self.router, bias=None, scoring=L.SIGMOID, renormalize=True))
        self.shared = shared

    def combined(self, n, ids, w, y_rounded):
        """The layer's sum for tokens n with its own routing, and the bound of fp32 and (y_rounded) bf16 rows."""
        xv = mx_ref.quantize(n)[2]
        out, bound = torch.zeros(n.shape, dtype=F64), torch.zeros(n.shape, dtype=F64)
        half = 2.0 ** -8 if y_rounded else 0.0
        for e in range(E + 1):
            hit = (ids == e)
            rows = torch.nonzero(hit.any(1)).flatten() if e < E else torch.arange(len(n)) if self.shared else []
            if not len(rows):
                continue
            wt = (w * hit).sum(1)[rows].to(F64)[:, None] if e < E else torch.ones((len(rows), 1), dtype=F64)
            y, dy = mx_ref.expert(xv[rows], self.v13[e], self.v2[e])
            out[rows] += wt * y
            bound[rows] += wt * (dy + half * (y.abs() + dy) + 2 * (K + 1) * U * y.abs())
        return out, bound


@pytest.mark.parametrize("T,shared", [(1, True), (16, False), (65, True), (300, True)])
def test_layer_forward_and_few(T, shared):
    L = _lib()
    say(f"[mx layer] T={T} shared={shared}")
    c = Case(shared)
    x = rand((T, H), 10 + T)
    b = c.layer.forward(x.to(DEV))
    ids, w = b.topk_ids.cpu(), b.topk_w.cpu()
    want, bound = c.combined(x, ids, w, True)
    check("forward", b.out, want, bound)
    if c.layer.uses_few(T):
        b2 = c.layer.forward_few(x.to(DEV))
        assert torch.equal(b2.topk_ids.cpu(), ids) and torch.equal(b2.topk_w.cpu(), w)
        want, bound = c.combined(x, ids, w, False)
        check("few", b2.out, want, bound)
        given = c.layer.forward_few(x.to(DEV), ids.to(DEV), w.to(DEV)).out
        check("few with the routing handed in", given, want, bound)


@pytest.mark.parametrize("T", [1, 33])
def test_block(T):
    """pre_norm -> route -> experts -> combine_norm, each step against 64 bits."""
    c = Case()
    x, d = rand((T, H), 20), rand((T, H), 21)
    gain, post = 1 + rand((H,), 22, 0.1, torch.float32), 1 + rand((H,), 23, 0.1, torch.float32)
    gate = rand((T, H), 24, 0.5)
    b = c.layer.forward_block(x.to(DEV), d.to(DEV), delta_scale=0.5, gain=gain.to(DEV), post_gain=post.to(DEV),
                              gate=gate.to(DEV), alpha=0.75)
    h = x.to(F64) + 0.5 * d.to(F64)
    eps = float(torch.tensor(1e-6))
    close("h", b.h, h, U * h.abs(), torch.bfloat16)
    n = h * rms(h, eps) * gain.to(F64)
    close("n", b.n, n, 56 * U * n.abs(), torch.bfloat16)
    s, ds = c.combined(b.n.cpu(), b.topk_ids.cpu(), b.topk_w.cpu(), True)
    r = rms(s, eps)
    # first order, and its square for the rest: |d(s r)| <= r ds + |s| r^3 mean(|s| ds)
    lean = r ** 2 * (s.abs() * ds + ds ** 2).mean(1, keepdim=True)
    v = s * r * post.to(F64)
    dv = (r * ds + s.abs() * r * lean) * post.to(F64).abs() * (1 + 2 * lean) + 56 * U * v.abs()
    f = 0.75 * gate.to(F64)
    want = b.h.cpu().to(F64) + f * v
    check("block out", b.out, want, f.abs() * dv + 4 * U * (f * v).abs() + U * want.abs())


def test_block_refusals():
    c = Case()
    x = rand((4, H), 30).to(DEV)
    with pytest.raises(TypeError):
        c.layer.forward_block(x, gain=torch.ones(H, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        c.layer.forward_block(x, gate=torch.ones((3, H), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        c.layer.forward_block(x, delta=x[:2])
    with pytest.raises(ValueError):
        c.layer.forward_block(x[:, :256].t().contiguous().t())
    L = _lib()
    with pytest.raises(ValueError):
        L.quantize_mxfp4(torch.zeros((4, 48), device=DEV))
    with pytest.raises(ValueError):
        L.quantize_mxfp4(torch.zeros((64, 4), device=DEV).t())
    with pytest.raises(ValueError):  # a tensor that is on no GPU
        L.moe_pre_norm(torch.zeros((1, 64)), None, 0.0, None, 0.0, L.F32, 1, 64, None, torch.zeros((1, 64)))


def test_graph_replays_follow_new_inputs():
    """The block and the few-token layer captured in one graph; replays between eager work equal eager calls."""
    c = Case()
    x = rand((5, H), 40).to(DEV)
    gain = torch.ones(H, device=DEV)

    def step():
        return c.layer.forward_block(x, gain=gain, post_gain=gain)
    few = lambda: c.layer.forward_few(x)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        few()
    torch.cuda.synchronize()
    kept = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept.copy_(step().out)
        out = few().out
    for seed in (41, 42, 41):
        x.copy_(rand((5, H), seed))
        g.replay()
        torch.cuda.synchronize()
        got = kept.clone(), out.clone()
        want = step().out.clone(), few().out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
