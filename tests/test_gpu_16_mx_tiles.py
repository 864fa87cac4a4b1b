"""MXFP4 grouped products on every tile height: 64, 128 and 256 rows, one to four 64-row blocks in a tile, two and three
load stages, several items per workgroup, K of one step, of odd steps and of an odd last half, contiguous and gathered
rows. The height that a case is meant to reach is computed by the kernel's rule from this card's CUs and asserted.

Every row's bits are compared with a call of at most 64 rows (64-row tiles: the path that test_gpu_10_mxfp4 checks), and
rows at the edges of blocks and tiles with 64 bits."""
import functools

import numpy as np
import pytest
import torch

import mx_ref
from gpu_util import DEV, say
from test_gpu_10_mxfp4 import check, quantized, run_ffn

pytestmark = pytest.mark.gpu


def tile_height(rows, n_blocks, max_rows):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    most = (max_rows + 63) // 64 + min(len(rows), max_rows)
    grid = min((most * n_blocks + 7) // 8 * 8, cus // 8 * 8)
    for h in (64, 128):
        if sum(-(-r // h) for r in rows) <= grid // n_blocks:
            return h
    return 256


class RandomCodes:
    """Experts of random codes and scales of 2^-9 to 2^-6."""

    def __init__(self, H, I, E, shared, seed):
        import mixture_experts_layer_select_amd as L
        g = torch.Generator().manual_seed(seed)
        n = E + (1 if shared else 0)
        draw = lambda r, c: (torch.randint(0, 256, (n, r, c // 2), generator=g, dtype=torch.uint8),
                             torch.randint(118, 122, (n, r, c // 32), generator=g, dtype=torch.uint8))
        self.H, self.I, self.E = H, I, E
        self.c13, self.s13 = draw(2 * I, H)
        self.c2, self.s2 = draw(H, I)
        d = [t.to(DEV) for t in (self.c13, self.c2, self.s13, self.s2)]
        sh = [t[E] for t in d] if shared else [None] * 4
        self.w = L.make_weights(L.MXFP4, E, H, I, *[t[:E].contiguous() for t in d], *sh)

    def reference(self, x, e):
        return mx_ref.expert(x, mx_ref.values(self.c13[e], self.s13[e]), mx_ref.values(self.c2[e], self.s2[e]))


@functools.lru_cache(maxsize=1)
def experts(H, I, E, shared):
    return RandomCodes(H, I, E, shared, H + I)


def edges(n):
    return sorted({r for r in (0, 31, 32, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, n // 2, n - 1) if r < n})


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


MIXED = [600, 3, 250, 64, 0, 1, 513, 66]
PAST = [257, 193, 129, 65, 1]
EIGHT = [128, 65, 64, 100, 128, 127, 128, 70]
CASES = [  # H, I, rows, shared, height of gate/up and of down
    (256, 8192, PAST, False, 256, 64),             # gate/up: one K step
    (256, 8192, MIXED, True, 256, 64),             # ... three items a workgroup
    (512, 8192, [128, 65, 64, 100], False, 128, 64),
    (768, 8192, [256, 255, 192, 2], True, 256, 64),   # three K steps
    (1280, 4096, [700, 191, 129, 0, 33], False, 256, 64),  # five
    (8192, 128, PAST, False, 64, 256),             # down: half a K step
    (8192, 256, MIXED, True, 64, 256),             # one, more than one item a workgroup
    (8192, 512, EIGHT, False, 64, 128),            # two
    (8192, 384, [200, 192, 129, 128, 65, 64, 256], True, 64, 256),  # one and a half
    (8192, 640, [257, 300, 191, 1], False, 64, 256)]  # two and a half


@pytest.mark.parametrize("H,I,rows,shared,gate_up,down", CASES)
def test_every_height(H, I, rows, shared, gate_up, down):
    say(f"[mx tiles] H={H} I={I} rows={rows}")
    G, R = len(rows), sum(rows)
    offsets = [0] + np.cumsum(rows).tolist()
    assert tile_height(rows, I // 128, R + 5) == gate_up and tile_height(rows, H // 256, R + 5) == down
    assert tile_height([64], I // 128, 64) == tile_height([64], H // 256, 64) == 64
    ex = experts(H, I, G - shared, shared)
    x, xs, xv = quantized((R + 5, H), 1.0, 50)
    y = run_ffn(x, xs, ex, offsets, R + 5)
    assert bool((y[R:] == 3.0).all()), "rows behind the last group were written"
    for _ in range(4):
        assert same(run_ffn(x, xs, ex, offsets, R + 5), y)
    for e in range(G):
        a, b = offsets[e], offsets[e + 1]
        for i in range(a, b, 64):
            n = min(64, b - i)
            part = run_ffn(x[i:i + n].contiguous(), xs[i:i + n].contiguous(), ex, [0] * (e + 1) + [n] * (G - e), n)
            assert same(part, y[i:i + n]), (e, i - a)
        if b > a:
            at = [a + r for r in edges(b - a)]
            want, bound = ex.reference(xv[at], e)
            check(f"group {e} of {b - a}", y[at], want, bound)


@pytest.mark.parametrize("H,I,rows", [(256, 8192, [257, 129, 0, 65, 2]), (768, 4096, [450, 193, 1, 64]),
                                      (512, 8192, [64, 30, 1])])
def test_gathered_rows_on_tall_tiles(H, I, rows):
    """Token rows through row_to_slot, the shared group behind, against the same rows laid out, bit for bit."""
    T, E = sum(rows), len(rows)
    rows = rows + [T]
    offsets = [0] + np.cumsum(rows).tolist()
    assert tile_height(rows, I // 128, 2 * T) > 64
    ex = experts(H, I, E, True)
    x, xs, _ = quantized((T, H), 1.0, 51)
    token = torch.cat([torch.randperm(T, generator=torch.Generator().manual_seed(52)), torch.arange(T)])
    slots = torch.cat([token[:T], T + token[T:]]).to(torch.int32).to(DEV)
    got = run_ffn(x, xs, ex, offsets, 2 * T, (T, 1, slots))
    tk = token.to(DEV)
    assert same(got, run_ffn(x[tk].contiguous(), xs[tk].contiguous(), ex, offsets, 2 * T))


def test_nan_of_the_next_row_on_tall_tiles():
    """An odd last half of K in tiles of 256 rows: every other row of the intermediate and some rows of w2 are NaN."""
    H, I, rows = 8192, 640, [300, 700]
    assert tile_height(rows, H // 256, 1000) == 256
    ex = RandomCodes(H, I, 2, False, 53)
    x, xs, _ = quantized((1000, H), 1.0, 54)
    clean = run_ffn(x, xs, ex, [0, 300, 1000], 1000)
    bad = xs.clone()
    bad[1::2] = 255
    ex.w._tensors[3][:, 8::16] = 255
    y = run_ffn(x, bad, ex, [0, 300, 1000], 1000).float()
    keep = torch.ones(H, dtype=torch.bool, device=DEV)
    keep[8::16] = False
    assert torch.equal(y[0::2][:, keep], clean[0::2][:, keep].float())
    assert bool(torch.isnan(y[1::2]).all()) and bool(torch.isnan(y[:, 8::16]).all())
