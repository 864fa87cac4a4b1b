"""moe_layer_few against 64 bits: routing equal to moe_route's, the output within the experts' bounds (mx_ref.expert),
the routing weights' fp32 error and one bf16 rounding."""
import pytest
import torch

import mx_ref
from gpu_util import DEV, say
from mx_ref import F64, U
from test_gpu_10_mxfp4 import Experts, check

pytestmark = pytest.mark.gpu


def _lib():
    import mixture_experts_layer_select_amd as L
    return L


def tokens(T, H, seed, std=1.0):
    return (torch.randn((T, H), generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def reference(x, ids, w, ex, base=0):
    """(out, bound) in float64 for given ids (any values) and fp32 weights."""
    T, H = x.shape
    xv = mx_ref.quantize(x)[2]
    out, bound, mass = (torch.zeros((T, H), dtype=F64) for _ in range(3))
    n = ids.shape[1] + 1
    for t in range(T):
        picks = [(int(e) - base, float(w[t, j])) for j, e in enumerate(ids[t].tolist()) if 0 <= int(e) - base < ex.E]
        if ex.shared:
            picks.append((ex.E, 1.0))
        for e, wt in picks:
            y, dy = ex.reference(xv[t:t + 1], e)
            out[t] += wt * y[0]
            bound[t] += abs(wt) * dy[0]
            mass[t] += abs(wt) * y[0].abs()
    return out, bound + 2 * n * U * mass


def few(ex, x, ids=None, w=None, router=None, bias=None, k=None, E=None, base=0, scoring=None, renorm=True, ws=None):
    L = _lib()
    T, H = x.shape
    E = E or ex.E
    k = ids.shape[1] if ids is not None else k
    if ws is None:
        ws = torch.full((L.moe_layer_few_workspace_size(ex.w, T, E, k),), 0xFF, dtype=torch.uint8, device=DEV)
    i = torch.full((T, k), -7, dtype=torch.int32, device=DEV) if ids is None else ids.to(torch.int32).to(DEV)
    v = torch.zeros((T, k), device=DEV) if w is None else w.to(DEV)
    out = torch.full((T, H), 9.0, dtype=torch.bfloat16, device=DEV)
    L.moe_layer_few(x.to(DEV), router, bias, T, E, k, L.SIGMOID if scoring is None else scoring, renorm, ex.w, base, i, v,
                    out, ws, ws.numel())
    torch.cuda.synchronize()
    return i.cpu(), v.cpu(), out


@pytest.mark.parametrize("T,k,E,H,I,shared", [
    (1, 1, 1, 256, 128, False), (1, 2, 8, 512, 256, True), (3, 3, 5, 768, 384, False), (16, 8, 16, 256, 128, True),
    (7, 4, 40, 1280, 640, True), (16, 1, 3, 512, 1152, False), (2, 8, 8, 1024, 2176, True)])
def test_routed_against_64_bits(T, k, E, H, I, shared):
    L = _lib()
    say(f"[few] T={T} k={k} E={E} H={H} I={I} shared={shared}")
    ex = Experts(H, I, E, shared, H + E)
    x = tokens(T, H, T)
    router = tokens(E, H, 91, 0.05).to(DEV)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(4)).to(DEV)
    for scoring, renorm in ((L.SIGMOID, True), (L.SOFTMAX, True), (L.SOFTMAX, False), (L.SIGMOID, False)):
        ids, w, out = few(ex, x, router=router, bias=bias, k=k, scoring=scoring, renorm=renorm)
        want_ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
        want_w, logits = torch.empty((T, k), device=DEV), torch.empty((T, E), device=DEV)
        L.moe_route(x.to(DEV), router, bias, L.BF16, T, H, E, k, scoring, renorm, logits, want_ids, want_w)
        assert torch.equal(ids, want_ids.cpu()) and torch.equal(w, want_w.cpu())
    want, bound = reference(x, ids, w, ex)
    check("few out", out, want, bound)


def test_r1_width():
    ex = Experts(7168, 2048, 3, True, 17, 0.02)
    x = tokens(4, 7168, 2)
    ids = torch.tensor([[0, 2], [1, 0], [2, 1], [2, 0]])
    w = torch.tensor([[.7, .3], [.5, .5], [.9, .1], [.2, .8]])
    _, _, out = few(ex, x, ids, w)
    want, bound = reference(x, ids, w, ex)
    check("few r1", out, want, bound)


def test_widest():
    """H = 8192, the widest layer the call takes."""
    ex = Experts(8192, 128, 2, False, 18, 0.02)
    x = tokens(16, 8192, 3)
    ids = (torch.arange(16) % 2)[:, None]
    w = torch.full((16, 1), 0.5)
    _, _, out = few(ex, x, ids, w)
    want, bound = reference(x, ids, w, ex)
    check("few 8192", out, want, bound)


def test_given_routing_edges():
    """Ids of other GPUs, negative and huge ids, an id twice in a row of picks, a token with no local pick, an expert
    base; without a shared expert such a token's output is zero."""
    ex = Experts(512, 256, 4, False, 19)
    x = tokens(5, 512, 5)
    big = 2 ** 31 - 1
    ids = torch.tensor([[10, 11, 9], [12, 12, 13], [0, -1, big], [13, 14, -(2 ** 31)], [11, 10, 12]])
    w = torch.tensor([[.5, .25, .25], [.5, .2, .3], [1., 1., 1.], [.6, .4, 5.], [.1, .2, .7]])
    _, _, out = few(ex, x, ids, w, base=10, E=64)
    want, bound = reference(x, ids, w, ex, base=10)
    check("few edges", out, want, bound)
    assert bool((out[2] == 0).all())
    # no pick is local at all
    _, _, out = few(ex, x, torch.full((5, 3), 3), w, base=10, E=64)
    assert bool((out == 0).all())


def test_nan_reaches_its_own_tokens_alone():
    ex = Experts(512, 256, 3, True, 20)
    x = tokens(4, 512, 6)
    ids, w = torch.tensor([[0], [1], [0], [2]]), torch.ones((4, 1))
    _, _, clean = few(ex, x, ids, w)
    y = x.clone()
    y[1, 17] = float("nan")
    _, _, out = few(ex, y, ids, w)
    assert bool(torch.isnan(out[1].float()).all())
    assert torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])
    ex.w._tensors[2][2, 9, 1] = 255  # a w13 scale of expert 2, picked by token 3 alone
    _, _, out = few(ex, x, ids, w)
    assert bool(torch.isnan(out[3].float()).any())
    assert torch.equal(out[:3], clean[:3])
    y = x.clone()
    y[0, 5] = float("inf")
    _, _, out = few(ex, y, ids, w)
    assert torch.equal(out[1:3], clean[1:3])


def test_more_tokens_do_not_change_a_token():
    """A token's output has the same bits alone and among 16, and from call to call."""
    ex = Experts(1024, 384, 12, True, 21)
    x = tokens(16, 1024, 7)
    ids = torch.stack([torch.randperm(12, generator=torch.Generator().manual_seed(t))[:3] for t in range(16)])
    w = torch.rand((16, 3), generator=torch.Generator().manual_seed(99))
    _, _, all16 = few(ex, x, ids, w)
    assert torch.equal(all16, few(ex, x, ids, w)[2])
    for t in (0, 5, 15):
        # the experts of other tokens add exact zeros nowhere: a token sums its own picks in ascending order
        _, _, one = few(ex, x[t:t + 1], ids[t:t + 1], w[t:t + 1])
        assert torch.equal(one[0], all16[t])


def test_captured_and_replayed():
    L = _lib()
    T, k, E, H, I = 3, 2, 6, 512, 256
    ex = Experts(H, I, E, True, 22)
    router = tokens(E, H, 92, 0.05).to(DEV)
    x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(L.moe_layer_few_workspace_size(ex.w, T, E, k), dtype=torch.uint8, device=DEV)

    def call():
        L.moe_layer_few(x, router, None, T, E, k, L.SIGMOID, True, ex.w, 0, ids, w, out, ws, ws.numel())
    x.copy_(tokens(T, H, 1))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (1, 2, 3, 2):
        x.copy_(tokens(T, H, seed))
        g.replay()
        torch.cuda.synchronize()
        got = (ids.clone(), w.clone(), out.clone())
        out.fill_(5)
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (ids, w, out)))


def test_two_streams_with_a_workspace_each():
    """Calls that overlap on two streams, each with its own workspace, give what they give alone."""
    L = _lib()
    ex = Experts(2048, 1024, 16, True, 23)
    router = tokens(16, 2048, 93, 0.05).to(DEV)
    sides = []
    for n in range(2):
        x = tokens(8 + n, 2048, 40 + n)
        sides.append((x, few(ex, x, router=router, k=4)[2]))
    streams = [torch.cuda.Stream() for _ in sides]
    state = []
    for (x, _), st in zip(sides, streams):
        T = x.shape[0]
        state.append((x.to(DEV), torch.empty((T, 4), dtype=torch.int32, device=DEV), torch.empty((T, 4), device=DEV),
                      torch.empty((T, 2048), dtype=torch.bfloat16, device=DEV),
                      torch.zeros(L.moe_layer_few_workspace_size(ex.w, T, 16, 4), dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, i, w, o, ws), st in zip(state, streams):
            L.moe_layer_few(x, router, None, x.shape[0], 16, 4, L.SIGMOID, True, ex.w, 0, i, w, o, ws, ws.numel(), st)
    torch.cuda.synchronize()
    for (_, want), (_, _, _, o, _) in zip(sides, state):
        assert torch.equal(o, want)


@pytest.mark.parametrize("T,k,E,H,I,shared", [
    (16, 8, 16, 512, 2176, True),    # more (expert, token) rows than are held at a time, two segments of K each
    (16, 8, 9, 256, 4224, False),    # three segments, the last of one step and a half-filled one
    (9, 2, 3, 256, 16384, True),     # the widest intermediate
    (16, 4, 64, 768, 128, True)])
def test_many_rows_and_segments(T, k, E, H, I, shared):
    ex = Experts(H, I, E, shared, 31)
    x = tokens(T, H, 33)
    g = torch.Generator().manual_seed(T + E)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    w = torch.rand((T, k), generator=g)
    _, _, out = few(ex, x, ids, w)
    want, bound = reference(x, ids, w, ex)
    check(f"few {T}x{k} of {E}, {H}x{I}", out, want, bound)
    assert torch.equal(out, few(ex, x, ids, w)[2])


def test_most_local_experts():
    """512 local experts behind a base, picks at both ends of the range and next to it."""
    ex = Experts(256, 128, 512, True, 32)
    x = tokens(4, 256, 34)
    ids = torch.tensor([[100, 611], [99, 612], [611, 610], [131, 132]])
    w = torch.tensor([[.5, .5], [.4, .6], [.3, .7], [1., 2.]])
    _, _, out = few(ex, x, ids, w, base=100, E=700)
    want, bound = reference(x, ids, w, ex, base=100)
    check("few 512", out, want, bound)
