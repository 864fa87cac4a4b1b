"""moe_layer_few on the paths that its sizes choose: the K split and the columns of its kernels by H, segments by I, the
number of groups, and calls without any group. Against 64 bits, as in test_gpu_12_few."""
import pytest
import torch

from gpu_util import DEV, say
from test_gpu_10_mxfp4 import Experts, check
from test_gpu_12_few import few, reference, tokens

pytestmark = pytest.mark.gpu


def _lib():
    import mixture_experts_layer_select_amd as L
    return L


@pytest.mark.parametrize("T,k,I", [(1, 1, 128), (1, 1, 2176), (16, 8, 2304), (3, 2, 16384)])
def test_no_local_pick_and_no_shared_expert(T, k, I):
    """No group at all, with one segment of K and with several: zeros, and nothing is looked up."""
    say(f"[few none] T={T} k={k} I={I}")
    ex = Experts(256, I, 2, False, 41)
    ids = torch.arange(T * k).reshape(T, k) % 30 + 2
    _, _, out = few(ex, tokens(T, 256, 1), ids, torch.ones((T, k)), base=0, E=64)
    assert bool((out == 0).all())
