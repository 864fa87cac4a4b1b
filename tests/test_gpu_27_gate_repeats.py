"""The gate's gradient where most tokens pick an expert several times: every pick's part arrives, on repeated runs too."""
import pytest
import torch

from test_gpu_22_route_grads import run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def L():
    import mixture_experts_layer_select_amd as pkg
    return pkg


@pytest.mark.parametrize("sigmoid,renorm", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T,E,k,experts", [(1, 8, 8, 1), (37, 256, 8, 2), (1000, 64, 7, 3), (64, 12, 2, 1), (129, 40, 20, 4)])
def test_repeated_picks(L, T, E, k, experts, sigmoid, renorm):
    g = torch.Generator(device=DEV).manual_seed(T + k)
    logits = torch.randn((T, E), generator=g, device=DEV)
    ids = torch.randint(E - experts, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    dw = torch.randn((T, k), generator=g, device=DEV)
    first = run(L, logits, ids, dw, sigmoid, renorm, torch.float32)
    for _ in range(3):
        assert torch.equal(run(L, logits, ids, dw, sigmoid, renorm, torch.float32), first)
    if sigmoid and not renorm:  # each pick's part by itself is known: their sum, with equal parts in any order
        ones = torch.ones_like(dw)
        same = torch.full_like(ids, E - 1)
        one = run(L, logits, same[:, :1].contiguous(), ones[:, :1].contiguous(), True, False, torch.float32)
        many = run(L, logits, same, ones, True, False, torch.float32)
        assert ((many.double() - k * one.double()).abs() <= k * k * 2.0 ** -24 * one.double().abs()).all()
        assert (many[:, E - 1] > 0).all()
