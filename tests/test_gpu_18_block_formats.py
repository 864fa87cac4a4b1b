"""forward_block in every format, with the router of large batches, without tokens and on its own buffers: the norms
against 64 bits, the layer between them against forward on the same rows, bit for bit."""
import pytest
import torch

from gpu_util import DEV, say
from mx_ref import F64, U
from test_gpu_11_norm import close, rms

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 128, 8, 2


def _lib():
    import mixture_experts_layer_select_amd as L
    return L


def rand(shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def make(fmt, shared):
    L = _lib()
    act = torch.float32 if fmt == "f32" else torch.bfloat16
    w13, w2 = rand((E + 1, 2 * I, H), 1, 0.05, torch.float32), rand((E + 1, H, I), 2, 0.05, torch.float32)
    if fmt == "mxfp4":
        (c13, s13), (c2, s2) = L.quantize_mxfp4(w13.to(DEV)), L.quantize_mxfp4(w2.to(DEV))
    elif fmt == "fp8":
        c13, c2 = ((w * 64).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV) for w in (w13, w2))
        s13 = torch.full((E + 1, 2 * I // 128, H // 128), 1 / 64, device=DEV)
        s2 = torch.full((E + 1, H // 128, I // 128), 1 / 64, device=DEV)
    else:
        c13, c2, s13, s2 = w13.to(act).to(DEV), w2.to(act).to(DEV), None, None
    part = lambda t, sl: None if t is None else t[sl].contiguous()
    sh = dict(w13=c13[E], w2=c2[E], w13_scale=part(s13, E), w2_scale=part(s2, E)) if shared else None
    head = slice(0, E)
    router = dict(w=rand((E, H), 3, 0.05, act).to(DEV), bias=None, scoring=L.SIGMOID, renormalize=True)
    return L.MoELayer(fmt, H, I, K, part(c13, head), part(c2, head), part(s13, head), part(s2, head), shared=sh,
                      router=router), act


@pytest.mark.parametrize("fmt,T,shared", [("f32", 5, True), ("bf16", 1, False), ("bf16", 70, True), ("fp8", 33, True),
                                          ("fp8", 9, False), ("mxfp4", 40, False), ("bf16", 4097, True),
                                          ("fp8", 4096, True), ("mxfp4", 4100, True)])
def test_block(fmt, T, shared):
    say(f"[block] {fmt} T={T} shared={shared}")
    layer, act = make(fmt, shared)
    x, d, gate = rand((T, H), 4, 1.0, act), rand((T, H), 5, 1.0, act), rand((1, H), 6, 0.5, act)
    gain, post = 1 + rand((H,), 7, 0.1, torch.float32), 1 + rand((H,), 8, 0.1, torch.float32)
    b = layer.forward_block(x.to(DEV), d.to(DEV), delta_scale=0.5, gain=gain.to(DEV), post_gain=post.to(DEV),
                            gate=gate.to(DEV), alpha=0.75)
    eps = float(torch.tensor(1e-6))
    h = x.to(F64) + 0.5 * d.to(F64)
    n = h * rms(h, eps) * gain.to(F64)
    close("h", b.h, h, U * h.abs(), act)
    close("n", b.n, n, 56 * U * n.abs(), act)
    f = make(fmt, shared)[0].forward(b.n)
    same = lambda p, q: torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    rows = int(f.offsets[E + (1 if shared else 0)])
    assert same(f.topk_ids, b.topk_ids) and same(f.topk_w, b.topk_w) and same(f.slot_to_row, b.slot_to_row)
    assert same(f.y_perm[:rows], b.y_perm[:rows])
    # the combine and its norm in 64 bits on the layer's own rows, bounds as in test_gpu_11_norm
    y, w, at = f.y_perm.cpu().to(F64), f.topk_w.cpu().to(F64), f.slot_to_row.cpu().view(T, K).long()
    assert bool((at >= 0).all())
    parts = y[at] * w[..., None]
    own = y[int(f.offsets[E]):][:T] if shared else torch.zeros((T, H), dtype=F64)
    c = parts.sum(1) + own
    dc = (K + 1) * U * (parts.abs().sum(1) + own.abs())
    r = rms(c, eps)
    ddc = dc.square().mean(1, keepdim=True).sqrt()
    rel = (2 * c.square().mean(1, keepdim=True).sqrt() * ddc + ddc ** 2) * r ** 2
    v = c * r * post.to(F64)
    dv = dc * r * post.to(F64).abs() + v.abs() * (52 * U + rel)
    g = 0.75 * gate.to(F64)
    want = b.h.cpu().to(F64) + g * v
    close("out", b.out, want, g.abs() * dv + 4 * U * (g * v).abs() + U * want.abs(), act)


@pytest.mark.parametrize("fmt", ["f32", "bf16", "fp8", "mxfp4"])
def test_no_tokens(fmt):
    layer, act = make(fmt, True)
    x = torch.empty((0, H), dtype=act, device=DEV)
    assert layer.forward_block(x, x, gain=torch.ones(H, device=DEV)).out.shape == (0, H)
    if fmt == "mxfp4":
        assert layer.forward_few(x).out.shape == (0, H)
        c, s = _lib().quantize_mxfp4(x)
        assert c.shape == (0, H // 2) and s.shape == (0, H // 32)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 65])
def test_blocks_one_after_another(T):
    """A block whose input is the block before's own buffers: its residual stream as x, its output as delta."""
    x, gain = rand((T, H), 9).to(DEV), (1 + rand((H,), 10, 0.1, torch.float32)).to(DEV)
    layer, other = make("mxfp4", True)[0], make("mxfp4", True)[0]
    b = layer.forward_block(x, gain=gain, post_gain=gain)
    for _ in range(3):
        h, out = b.h.clone(), b.out.clone()
        want = other.forward_block(h, out, delta_scale=0.5, gain=gain, post_gain=gain)
        b = layer.forward_block(b.h, b.out, delta_scale=0.5, gain=gain, post_gain=gain)
        assert torch.equal(b.h, want.h) and torch.equal(b.n, want.n) and torch.equal(b.out, want.out)
