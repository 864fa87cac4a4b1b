"""The gate's gradient at confident picks: the error is held against the gradient's own size, s (1 - s), which is a
millionth of the weight at a logit of 14, in both kernels (up to eight picks, and more)."""
import pytest
import torch

import train_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def L():
    import mixture_experts_layer_select_amd as pkg
    return pkg


def size_and_reference(logits, ids, dw, renorm):
    """s (1 - s) |dw|, or w (1 - s) (|dw| + sum w |dw|), and the gradient, of the picks in float64; 1 - s as 1 / (1 + e^l)."""
    l, dw = logits.double().gather(1, ids.long()), dw.double()
    s, rest = 1 / (1 + torch.exp(-l)), 1 / (1 + torch.exp(l))
    if not renorm:
        return s * rest * dw.abs(), s * rest * dw
    w = s / s.sum(1, keepdim=True)
    return w * rest * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True)), w * rest * (dw - (w * dw).sum(1, keepdim=True))


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("lo,hi", [(8, 20), (-20, -8), (-3, 3), (20, 80), (-80, -20)])
@pytest.mark.parametrize("T,E,k", [(203, 24, 2), (64, 256, 8), (33, 64, 20)])
def test_confident_picks(L, T, E, k, lo, hi, renorm, dt):
    """Units of 2^-24, to first order. exp of a number that is held exactly: 2. s and 1 - s: the sum in the denominator 1,
    of exp at most half of its 2 (what is in it is at most 1 of 1 + e), a division of at most 5: 7, and 9 with exp in the
    numerator. s (1 - s) dw: 7 + 9 + 2 = 18.
    Renormalised, in terms of w (1 - s) (|dw| + D), D = sum w |dw|: w has its s 9, the sum of k terms k + 9, a division 5; times
    1 - s 9 + 1, times the difference 1; the difference dw - D, D's error k + 23 + 1 + k and its own rounding 1.
    In all (k + 34) + (2 k + 25) = 3 k + 59. What is rounded to the output's type is off by half a step more; numbers
    below fp32's normal ones by 2^-149 a step."""
    g = torch.Generator(device=DEV).manual_seed(T)
    logits = torch.rand((T, E), generator=g, device=DEV) * (hi - lo) + lo
    ids = logits.topk(k, 1).indices.to(torch.int32)
    dw = torch.randn((T, k), generator=g, device=DEV)
    out = torch.full((T, E), 5.0, device=DEV, dtype=dt)
    L.moe_route_grad(logits, ids, dw, T, E, k, L.SIGMOID, renorm, out, L.F32 if dt == F32 else L.BF16)
    size, ref = size_and_reference(logits, ids, dw, renorm)
    got = out.double().gather(1, ids.long())
    units = 3 * k + 59 if renorm else 18
    tol = units * U * 1.01 * size + train_ref.HALF[dt] * 1.01 * ref.abs() * (dt == BF) + 1e-40
    err = (got - ref).abs()
    assert (err <= tol).all(), float((err / size).max() / U)
    rest = out.clone()
    rest.scatter_(1, ids.long(), 0)
    assert (rest == 0).all()


def test_a_gate_that_is_sure_still_learns(L):
    """At logits of 18 and more the gradient is small, not zero."""
    logits = torch.tensor([[18.0, 24.0, 30.0, 60.0]], device=DEV)
    ids = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    out = torch.empty_like(logits)
    L.moe_route_grad(logits, ids, torch.ones_like(logits), 1, 4, 4, L.SIGMOID, False, out, L.F32)
    want = torch.exp(-logits.double()) / (1 + torch.exp(-logits.double())) ** 2
    assert ((out.double() / want - 1).abs() <= 18 * U * 1.01).all()
