"""Plain 64-bit forms of the training operators, for their tests (not a test module)."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a rounding step, relative


def philox(seed: int, offset: int, blocks) -> np.ndarray:
    """Words [n, 4] of Philox4x32-10 for the block numbers."""
    m32 = np.uint64(0xFFFFFFFF)
    b = np.asarray(blocks, np.uint64)
    c = [b & m32, b >> np.uint64(32), np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & m32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).astype(np.uint32)


def threshold(p: float) -> int:
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def factor(rng, n: int, p: float, first: int = 0) -> torch.Tensor:
    """What dropout multiplies elements first ... first + n - 1 by (0 or the scale), float64 on the CPU."""
    t = threshold(p)
    if t == 0:
        return torch.ones(n, dtype=torch.float64)
    seed, offset = [int(v) & (2 ** 64 - 1) for v in rng.tolist()]
    b0 = first // 8
    w = philox(seed, offset, np.arange(b0, (first + n + 7) // 8, dtype=np.uint64))
    bits = np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[first - 8 * b0:][:n]
    return torch.from_numpy((bits >= t) * (65536 / (65536 - t)))


def drop(v, f):
    return torch.where(f != 0, v * f, torch.zeros_like(v))


def rng_tensor(seed, offset, device):
    return torch.tensor([seed, offset], dtype=torch.int64, device=device)


def grouped(form, a, b, offsets):
    """Result and the sum of the products' magnitudes, float64, on the inputs' device. forward: x, w;
    input: dy, w; weights: dy, x. Rows are those of the groups."""
    out, mag = [], []
    for j, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        p = a[lo:hi].double()
        if form == "forward":
            q = b[j].double().t().contiguous()
        elif form == "input":
            q = b[j].double()
        else:
            p, q = p.t().contiguous(), b[lo:hi].double()
        out.append(p @ q)
        mag.append(p.abs() @ q.abs())
    if form == "weights":
        return torch.stack(out), torch.stack(mag)
    return torch.cat(out), torch.cat(mag)


def silu_parts(g):
    s = torch.sigmoid(g)
    return g * s, s * (1 + g * torch.sigmoid(-g))  # silu and its derivative


def route_grad(logits, ids, dw, sigmoid, renorm):
    """d sum(w * dw) / d logits in float64 by autograd; ids may repeat and lie outside the experts."""
    lg = logits.double().requires_grad_()
    E = lg.shape[1]
    ok = (ids >= 0) & (ids < E)
    picked = lg.gather(1, ids.clamp(0, E - 1).long())
    if sigmoid:
        w = torch.sigmoid(picked) * ok
    elif renorm:
        w = torch.exp(picked - picked.detach().amax(1, keepdim=True)) * ok
    else:
        w = torch.softmax(lg, 1).gather(1, ids.clamp(0, E - 1).long()) * ok
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad((w * dw.double()).sum(), lg)[0], w.detach()
