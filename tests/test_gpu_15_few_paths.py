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


@pytest.mark.parametrize("H", [2048, 2304, 2816, 3840, 4096, 4352, 5888, 6144, 6400])
@pytest.mark.parametrize("T,k,E,I,shared", [(5, 2, 4, 128, True), (16, 3, 6, 384, False)])
def test_widths(H, T, k, E, I, shared):
    """2, 4 and 8 waves to an item's K, with K steps that they share unevenly; 8, 16, 24 and 32 output columns a
    workgroup, with a shorter last one."""
    say(f"[few widths] H={H} T={T} I={I}")
    ex = Experts(H, I, E, shared, 42)
    x = tokens(T, H, H)
    g = torch.Generator().manual_seed(H + T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    w = torch.rand((T, k), generator=g)
    _, _, out = few(ex, x, ids, w)
    want, bound = reference(x, ids, w, ex)
    check(f"few {H} x {I}", out, want, bound)


@pytest.mark.parametrize("I,shared", [(128, True), (128, False), (384, True), (640, False), (1152, True), (2176, True)])
def test_every_pick_another_expert(I, shared):
    """16 tokens of 8 picks, no two alike: 128 groups, or 129 with the shared expert, with 1, 2, 4 and 8 waves to K."""
    T, k, H = 16, 8, 256
    ex = Experts(H, I, T * k, shared, 43)
    x = tokens(T, H, I)
    ids = torch.randperm(T * k, generator=torch.Generator().manual_seed(I)).reshape(T, k)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(44))
    _, _, out = few(ex, x, ids, w)
    want, bound = reference(x, ids, w, ex)
    check(f"few of {T * k} experts, I={I}", out, want, bound)
    for t in (0, 7, 15):  # and the same bits as alone
        assert torch.equal(few(ex, x[t:t + 1], ids[t:t + 1], w[t:t + 1])[2][0], out[t])


def test_r1_layer_with_16_tokens():
    """The largest call of the R1 layer, 256 experts and the shared one, about 102 of them hit: every token as alone."""
    L = _lib()
    H, I, E, T, k = 7168, 2048, 256, 16, 8
    g = torch.Generator(device=DEV).manual_seed(45)
    codes = lambda n, r, c: torch.randint(0, 256, (n, r, c // 2), generator=g, dtype=torch.uint8, device=DEV)
    scales = lambda n, r, c: torch.randint(117, 121, (n, r, c // 32), generator=g, dtype=torch.uint8, device=DEV)
    w = L.make_weights(L.MXFP4, E, H, I, codes(E, 2 * I, H), codes(E, H, I), scales(E, 2 * I, H), scales(E, H, I),
                       codes(1, 2 * I, H), codes(1, H, I), scales(1, 2 * I, H), scales(1, H, I))
    router = tokens(E, H, 46, 0.02).to(DEV)
    x = tokens(T, H, 47).to(DEV)

    def call(a, b):
        n = b - a
        ids = torch.empty((n, k), dtype=torch.int32, device=DEV)
        tw = torch.empty((n, k), device=DEV)
        out = torch.empty((n, H), dtype=torch.bfloat16, device=DEV)
        ws = torch.full((L.moe_layer_few_workspace_size(w, n, E, k),), 0xFF, dtype=torch.uint8, device=DEV)
        L.moe_layer_few(x[a:b], router, None, n, E, k, L.SIGMOID, True, w, 0, ids, tw, out, ws, ws.numel())
        torch.cuda.synchronize()
        return ids, tw, out
    ids, tw, out = call(0, T)
    assert len(ids.unique()) > 64 and bool(torch.isfinite(out).all()) and bool((out != 0).any(1).all())
    for t in range(T):
        one = call(t, t + 1)
        assert torch.equal(one[0][0], ids[t]) and torch.equal(one[1][0], tw[t]) and torch.equal(one[2][0], out[t])


def test_output_over_the_tokens():
    """out may be x, routed by the call."""
    L = _lib()
    T, k, E, H, I = 9, 2, 6, 512, 256
    ex = Experts(H, I, E, True, 48)
    x, router = tokens(T, H, 49).to(DEV), tokens(E, H, 50, 0.05).to(DEV)
    ids, tw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    ws = torch.empty(L.moe_layer_few_workspace_size(ex.w, T, E, k), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x)
    for o in (out, x):
        L.moe_layer_few(x, router, None, T, E, k, L.SIGMOID, True, ex.w, 0, ids, tw, o, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(x, out)
