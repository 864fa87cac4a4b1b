"""SiLU of the MXFP4 experts at its far negative end, in the grouped product and in the layer for a few tokens.

The gate is summed from numbers that MXFP4 holds exactly, so it is exact in fp32; exp(-g) is still finite there, so
g / (1 + exp(-g)) is a normal fp32 number, and an up product of 2^120 brings it back to ordinary size."""
import pytest
import torch

import mx_ref
from gpu_util import DEV
from test_gpu_10_mxfp4 import check, run_ffn

pytestmark = pytest.mark.gpu

H, I = 256, 128
PARTS = {-88.0: (-64.0, -24.0), -87.5: (-64.0, -24.0, 0.5), -80.0: (-64.0, -16.0), -4.5: (-4.0, -0.5)}


class OneExpert:
    """Gate sums of g in every column, up sums of `up`, a random down matrix."""

    def __init__(self, g, up):
        import mixture_experts_layer_select_amd as L
        w13 = torch.zeros((2 * I, H), dtype=torch.float64)
        for i, v in enumerate(PARTS[g]):
            w13[:I, 32 * i] = v
        w13[I:, 32 * 7] = up
        w2 = torch.randn((H, I), generator=torch.Generator().manual_seed(3))
        c13, s13, self.v13 = mx_ref.quantize(w13)
        c2, s2, self.v2 = mx_ref.quantize(w2)
        assert torch.equal(self.v13, w13)
        on = lambda t: t[None].contiguous().to(DEV)
        self.H, self.I = H, I
        self.w = L.make_weights(L.MXFP4, 1, H, I, on(c13), on(c2), on(s13), on(s2))


def ones(T):
    x = torch.zeros((T, H))
    x[:, ::32] = 1.0
    return x


def reference(xv, ex, g):
    """(y, bound). The gate and up sums have at most four terms on one binary grid, so fp32 holds them exactly and the
    intermediate is off by its own operations alone: (12 + 2|g|) U, as mx_ref.expert counts them. No element lies that
    near a threshold, so its code is decided."""
    h = xv @ ex.v13.t()
    assert bool((h[:, :I] == g).all())
    a = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
    m = a.abs() / torch.pow(2.0, mx_ref.exponents(a.unflatten(-1, (-1, 32)))).repeat_interleave(32, -1)
    edges = torch.cat([mx_ref.EDGES, torch.tensor([4.0, 8.0], dtype=torch.float64)])
    assert float(((m[..., None] - edges).abs() / m[..., None]).min()) > (12 + 2 * abs(g)) * mx_ref.U
    q = mx_ref.quantize(a)[2]
    y = q @ ex.v2.t()
    assert bool((y != 0).any(1).all())
    return y, (128 + I // 64) * mx_ref.U * (q.abs() @ ex.v2.abs().t())


@pytest.mark.parametrize("g", sorted(PARTS))
@pytest.mark.parametrize("form", ["grouped", "few"])
def test_far_negative_gate(form, g):
    import mixture_experts_layer_select_amd as L
    T = 3
    ex = OneExpert(g, 2.0 ** 120 if g < -50 else 1.0)
    x = ones(T)
    codes, scales, xv = mx_ref.quantize(x)
    want, bound = reference(xv, ex, g)
    if form == "grouped":
        out = run_ffn(codes.to(DEV), scales.to(DEV), ex, [0, T], T)
    else:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(L.moe_layer_few_workspace_size(ex.w, T, 1, 1), dtype=torch.uint8, device=DEV)
        L.moe_layer_few(x.to(torch.bfloat16).to(DEV), None, None, T, 1, 1, L.SIGMOID, True, ex.w, 0,
                        torch.zeros((T, 1), dtype=torch.int32, device=DEV), torch.ones((T, 1), device=DEV), out, ws,
                        ws.numel())
        bound = bound + 4 * mx_ref.U * want.abs()  # the weighted sum: one product, one sum
    check(f"{form} g={g}", out, want, bound)
