"""Gradients of the combine and of the gate against float64: types, widths, picks that are not local, repeated and
foreign ids, large k, in-place rows, extremes."""
import pytest
import torch

import train_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    import mixture_experts_layer_select_amd as pkg
    return pkg


def maps(T, k, shared, seed, local=0.8):
    g = torch.Generator().manual_seed(seed)
    on = torch.rand(T * k, generator=g) < local
    R = int(on.sum())
    row = torch.full((T * k,), -1, dtype=torch.int32)
    row[on] = torch.randperm(R, generator=g).to(torch.int32)
    off = torch.tensor([0, R, R + (T if shared else 0)], dtype=torch.int32)
    return row.to(DEV), off.to(DEV), R


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("T,k,H,shared", [(1, 1, 1, False), (1, 8, 64, True), (17, 3, 129, True), (3, 256, 40, False),
                                          (130, 8, 512, True), (5, 8, 7168, True), (900, 2, 2056, False),
                                          (2100, 5, 24, True), (9, 4, 20000, True)])
def test_combine_grad(L, T, k, H, shared, dt):
    code = L.F32 if dt == F32 else L.BF16
    g = torch.Generator(device=DEV).manual_seed(T + H)
    row, off, R = maps(T, k, shared, T)
    n = R + (T if shared else 0)
    y = torch.randn((n + 3, H), generator=g, device=DEV).to(dt)
    dout = torch.randn((T, H), generator=g, device=DEV).to(dt)
    w = torch.rand((T, k), generator=g, device=DEV)
    dy, dw = torch.full_like(y, 5.0), torch.full((T, k), 5.0, device=DEV)
    sg = 1 if shared else -1
    L.moe_combine_grad(dout, y, code, row, w, T, k, H, off, sg, dy, dw)
    d, r = dout.double(), row.long().view(T, k)
    ref = torch.full((n + 3, H), 5.0, dtype=torch.float64, device=DEV)
    local = r >= 0
    ref[r[local]] = (w.double()[..., None] * d[:, None])[local]
    if shared:
        ref[R:n] = d
    err = (dy.double() - ref).abs()
    assert (err <= (train_ref.HALF[dt] * 1.01 + 2.0 ** -23) * ref.abs()).all()
    prod = y[r.clamp(min=0)].double() * d[:, None]
    dref, mag = prod.sum(2) * local, prod.abs().sum(2)
    assert ((dw.double() - dref).abs() <= (H + 2) * 2.0 ** -24 * mag).all()
    assert (dw[~local] == 0).all()
    # without the weights' gradient, and over y
    d2 = torch.full_like(y, 5.0)
    L.moe_combine_grad(dout, None, code, row, w, T, k, H, off, sg, d2, None)
    assert torch.equal(d2, dy)
    yi, dwi = y.clone(), torch.empty_like(dw)
    L.moe_combine_grad(dout, yi, code, row, w, T, k, H, off, sg, yi, dwi)
    assert torch.equal(yi[:n], dy[:n]) and torch.equal(yi[n:], y[n:]) and torch.equal(dwi, dw)


def test_combine_and_its_gradient_agree(L):
    """<dout, combine(y)> = <combine_grad(dout), y> for moe_permute's own maps, fp32."""
    T, k, E, H = 57, 4, 12, 96
    g = torch.Generator(device=DEV).manual_seed(3)
    ids = torch.rand((T, 2 * E), generator=g, device=DEV).topk(k, 1).indices.to(torch.int32)
    x = torch.randn((T, H), generator=g, device=DEV)
    cap = T * k + T
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, off, r2s, s2r = (torch.empty(n, **i32) for n in (E + 1, E + 2, cap, T * k))
    xp = torch.empty((cap, H), device=DEV)
    ws = torch.empty(L.moe_permute_workspace_size(T, k, E), dtype=torch.uint8, device=DEV)
    L.moe_permute(ids, T, k, 3, E, True, x, L.F32, H, L.F32, counts, off, r2s, s2r, xp, None, ws, ws.numel())
    y, dout = torch.randn((cap, H), generator=g, device=DEV), torch.randn((T, H), generator=g, device=DEV)
    w = torch.rand((T, k), generator=g, device=DEV)
    out, dy, dw = torch.empty_like(x), torch.zeros_like(y), torch.empty_like(w)
    L.moe_combine(y, L.F32, s2r, w, T, k, H, off, E, out, L.F32)
    L.moe_combine_grad(dout, y, L.F32, s2r, w, T, k, H, off, E, dy, dw)
    a, b = (out.double() * dout.double()).sum(), (dy.double() * y.double()).sum()
    size = (dy.double() * y.double()).abs().sum()
    assert abs(float(a - b)) <= 16 * 2.0 ** -24 * float(size)
    # and linear in the weights: sum(w dw) is the routed part of the same sum
    R = int(off[E])
    assert abs(float((w.double() * dw.double()).sum() - (dy[:R].double() * y[:R].double()).sum())) <= (
        (H + 4) * 2.0 ** -24 * float(size))


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 2), (203, 24, 2), (64, 256, 8), (33, 255, 255), (1000, 130, 70)])
def test_route_grad(L, T, E, k, sigmoid, renorm, dt):
    g = torch.Generator(device=DEV).manual_seed(T)
    logits = torch.randn((T, E), generator=g, device=DEV) * 2
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1).indices.to(torch.int32)
    dw = torch.randn((T, k), generator=g, device=DEV)
    run(L, logits, ids, dw, sigmoid, renorm, dt)


def run(L, logits, ids, dw, sigmoid, renorm, dt):
    T, E = logits.shape
    k = ids.shape[1]
    out = torch.full((T, E), 5.0, device=DEV, dtype=dt)
    L.moe_route_grad(logits, ids, dw, T, E, k, L.SIGMOID if sigmoid else L.SOFTMAX, renorm, out,
                     L.F32 if dt == F32 else L.BF16)
    ref, w = train_ref.route_grad(logits, ids, dw, sigmoid, renorm)
    # fp32: weights and sums of k (E) terms to (k + E + 16) units of 2^-24; the terms' magnitudes are |dw| and, for the
    # mean that is taken off, sum |w dw|, each times the weight
    mean = (w * dw.double().abs()).sum(1, keepdim=True)
    ok = (ids >= 0) & (ids < E)
    mag = torch.zeros_like(ref).scatter_add_(1, ids.clamp(0, E - 1).long(), w * ok * (dw.double().abs() + mean))
    if not sigmoid and not renorm:
        mag = mag + torch.softmax(logits.double(), 1) * mean
    tol = train_ref.HALF[dt] * 1.01 * ref.abs() + (k + E + 16) * 2.0 ** -24 * mag + 1e-37
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())
    return out


@pytest.mark.parametrize("sigmoid,renorm", [(True, True), (True, False), (False, True), (False, False)])
def test_route_grad_odd_ids(L, sigmoid, renorm):
    """The same expert twice in a token's picks, and ids that name no expert."""
    logits = torch.randn((6, 20), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    ids = torch.tensor([[3, 3, 7], [0, 19, 0], [-1, 4, 5], [20, 1, 2], [7, 7, 7], [2 ** 31 - 1, -2 ** 31, 9]],
                       dtype=torch.int32, device=DEV)
    dw = torch.randn((6, 3), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    run(L, logits, ids, dw, sigmoid, renorm, F32)


def test_route_grad_extremes(L):
    """Far logits: saturated scores have no gradient and no NaN; a shift of every logit changes nothing for softmax."""
    logits = torch.full((4, 64), -1e4, device=DEV)
    logits[:, :4] = torch.tensor([1e4, 50.0, -50.0, 0.0], device=DEV)
    ids = torch.arange(4, device=DEV, dtype=torch.int32).repeat(4, 1)
    dw = torch.ones((4, 4), device=DEV) * torch.tensor([1.0, -2.0, 3.0, 0.5], device=DEV)
    for scoring in (L.SIGMOID, L.SOFTMAX):
        for renorm in (True, False):
            out = torch.empty_like(logits)
            L.moe_route_grad(logits, ids, dw, 4, 64, 4, scoring, renorm, out, L.F32)
            assert torch.isfinite(out).all() and (out[:, 4:] == 0).all()
    half = torch.randint(-8, 8, (9, 40), device=DEV).float() / 2
    ids = torch.rand((9, 40), device=DEV).topk(5, 1).indices.to(torch.int32)
    dw = torch.randn((9, 5), device=DEV)
    for renorm in (True, False):
        a, b = torch.empty_like(half), torch.empty_like(half)
        L.moe_route_grad(half, ids, dw, 9, 40, 5, L.SOFTMAX, renorm, a, L.F32)
        L.moe_route_grad(half + 1024, ids, dw, 9, 40, 5, L.SOFTMAX, renorm, b, L.F32)
        assert torch.equal(a, b)


def test_route_grad_against_differences(L):
    """moe_route's own weights differentiated: x = one-hot rows make the logits anything, fp32. Error: h^2 / 6 of the
    third derivative (below 1 here for each score) times |dw|, and the weights' rounding over h."""
    T, E, k, h = 12, 16, 4, 2.0 ** -5
    g = torch.Generator(device=DEV).manual_seed(5)
    logits = torch.randperm(T * E, generator=g, device=DEV).view(T, E).float() / 32  # picks do not change within h
    dw = torch.randn((T, k), generator=g, device=DEV)
    eye = torch.eye(T, 16, device=DEV)

    def route(lg, scoring, renorm):
        w_router = torch.zeros((E, 16), device=DEV)
        w_router[:, :T] = lg.t()
        out = torch.empty((T, E), device=DEV)
        ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
        w = torch.empty((T, k), device=DEV)
        L.moe_route(eye, w_router, None, L.F32, T, 16, E, k, scoring, renorm, out, ids, w)
        return out, ids, w
    for scoring in (L.SIGMOID, L.SOFTMAX):
        for renorm in (True, False):
            lg, ids, _ = route(logits, scoring, renorm)
            d = torch.empty_like(lg)
            L.moe_route_grad(lg, ids, dw, T, E, k, scoring, renorm, d, L.F32)
            for s in range(3):
                v = torch.randn((T, E), generator=g, device=DEV)
                v /= v.abs().max() * 4  # |h v| <= 1/128, the logits lie 1/32 apart
                _, iu, wu = route(logits + h * v, scoring, renorm)
                _, il, wl = route(logits - h * v, scoring, renorm)
                assert torch.equal(iu, ids) and torch.equal(il, ids)
                slope = ((wu.double() - wl.double()) * dw.double()).sum() / (2 * h)
                want = (d.double() * v.double()).sum()
                size = float(dw.abs().sum())
                assert abs(float(slope - want)) <= size * (h * h / 6 * 8 * float(v.abs().max()) ** 3 + 2.0 ** -21 / h)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_grad_many_tokens(L, sigmoid):
    """More tokens than one grid of work items holds (2^26 of one wave each): the last ones, and some before."""
    T, E, k = 2 ** 26 + 5, 4, 1
    logits = torch.randn((T, E), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    ids = torch.randint(0, E, (T, k), device=DEV, dtype=torch.int32, generator=torch.Generator(device=DEV).manual_seed(2))
    dw = torch.randn((T, k), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    out = torch.full((T, E), 5.0, device=DEV)
    L.moe_route_grad(logits, ids, dw, T, E, k, L.SIGMOID if sigmoid else L.SOFTMAX, False, out, L.F32)
    for at in (slice(0, 9), slice(2 ** 21 - 4, 2 ** 21 + 4), slice(T // 2, T // 2 + 9), slice(T - 9, T)):
        part = torch.empty_like(out[at])
        L.moe_route_grad(logits[at].contiguous(), ids[at].contiguous(), dw[at].contiguous(), len(part), E, k,
                         L.SIGMOID if sigmoid else L.SOFTMAX, False, part, L.F32)
        assert torch.equal(out[at], part)
    assert not (out == 5).any()


@pytest.mark.parametrize("k", [1, 17])
def test_combine_grad_many_tokens(L, k):
    """More tokens than one launch takes."""
    T, H = 2 ** 21 // ((k + 7) // 8) + 3, 8
    row = torch.arange(T * k, dtype=torch.int32, device=DEV).flip(0)
    y = torch.randn((T * k + T, H), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    dout = torch.randint(-3, 4, (T, H), device=DEV).float()
    w = torch.full((T, k), 0.5, device=DEV)
    off = torch.tensor([0, T * k, T * k + T], dtype=torch.int32, device=DEV)
    dy, dw = torch.full_like(y, 9.0), torch.empty_like(w)
    L.moe_combine_grad(dout, y, L.F32, row, w, T, k, H, off, 1, dy, dw)
    assert torch.equal(dy[T * k:], dout)
    assert torch.equal(dy[:T * k], (dout * 0.5).repeat_interleave(k, 0).flip(0))
    prod = y[row.long()].view(T, k, H).double() * dout[:, None].double()
    assert ((dw.double() - prod.sum(2)).abs() <= 10 * 2.0 ** -24 * prod.abs().sum(2)).all()
