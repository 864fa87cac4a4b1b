"""64-bit references of the MXFP4 path with derived error bounds (not a test module).

Quantisation is exact, so it is compared bit for bit. Where a quantised value
depends on fp32 arithmetic (the intermediate A), an element is undecided if
its 64-bit value lies so near a rounding threshold, or its block's largest so
near a power of two, that fp32's error may move it; the bound of what follows
counts one step (a block: the coarser grid's) for each undecided element."""
from __future__ import annotations

import torch

F64 = torch.float64
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64)
EDGES = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=F64)
U = 2.0 ** -24  # half a step of fp32


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def exponents(b):
    """e of each block's scale 2^e; b [..., 32] float64."""
    amax = b.abs().amax(-1)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -300)))
    e = torch.where(torch.pow(2.0, e) > amax, e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= amax, e + 1, e)
    return torch.where(amax > 0, (e - 2).clamp(-127, 127), torch.zeros_like(e))


def quantize(x):
    """(codes uint8 [.., K/2], scale bytes uint8 [.., K/32], values float64) of x (CPU)."""
    b = x.to(F64).unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    e = exponents(b)
    m = b.abs() * torch.pow(torch.tensor(2.0, dtype=F64), -e)[..., None]
    lo = torch.bucketize(m, EDGES)
    hi = torch.bucketize(m, EDGES, right=True)
    idx = torch.where(lo % 2 == 0, lo, hi)  # on a threshold: the even code
    sign = torch.signbit(b)
    values = torch.where(sign, -GRID[idx], GRID[idx]) * torch.pow(2.0, e)[..., None]
    code = torch.where(bad[..., None], torch.zeros_like(idx), idx + 8 * sign).flatten(-2).to(torch.uint8)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    values = torch.where(bad[..., None], torch.full_like(values, torch.nan), values)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte, values.flatten(-2)


def values(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.where(c >= 8, -GRID[c % 8], GRID[c % 8])
    s = torch.pow(torch.tensor(2.0, dtype=F64), scales.to(F64) - 127)
    s = torch.where(scales == 255, torch.full_like(s, torch.nan), s)
    return v * s.repeat_interleave(32, -1)


def expert(x, w13, w2):
    """One expert on quantised rows x: (y, bound of fp32's error in y without its last rounding), all float64.

    A matrix instruction adds at most 128 exact products and the sum so far, in any order, and at least 64; so a
    product passes through at most 128 + K/64 fp32 additions, and the sum is within that many U of sum|p|.
    __expf(-g) is within (4 + |g|) * 2U relative, and the remaining operations of SiLU and its product within 4U."""
    I = w13.shape[0] // 2
    h = x @ w13.t()
    dh = (128 + x.shape[1] // 64) * U * (x.abs() @ w13.abs().t())
    g, u = h[:, :I], h[:, I:]
    dg, du = dh[:, :I], dh[:, I:]
    s = torch.sigmoid(g)
    a = g * s * u
    da = 1.1 * dg * u.abs() + (g * s).abs() * du + dg * du + a.abs() * (12 + 2 * g.abs()) * U
    b, db = a.unflatten(-1, (-1, 32)), da.unflatten(-1, (-1, 32))
    e = exponents(b)
    step = torch.pow(2.0, e)[..., None]
    q = quantize(a)[2]
    m, dm = b.abs() / step, db / step
    near = ((m[..., None] - EDGES).abs() <= dm[..., None]).any(-1)
    moved = torch.where(near, 2 * step, torch.zeros_like(m))  # at most the grid's widest step
    amax, top = b.abs().amax(-1), db.amax(-1)
    loose = (exponents(b.abs() + top[..., None]) != e) | (exponents((b.abs() - top[..., None]).clamp(min=0)) != e)
    moved = torch.where(loose[..., None] & (amax > 0)[..., None], 4 * step, moved).flatten(-2)
    y = q @ w2.t()
    return y, moved @ w2.abs().t() + (128 + I // 64) * U * (q.abs() @ w2.abs().t())
