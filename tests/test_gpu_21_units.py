"""Gated units, their gradient and dropout against float64: types, odd widths and alignments, rows left out, infinities
in dropped places, in-place calls, the counter past 32 bits, graphs with a moving offset, differences."""
import pytest
import torch

import train_ref
from train_ref import drop, factor, rng_tensor

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    import mixture_experts_layer_select_amd as pkg
    return pkg


def code(L, dt):
    return L.F32 if dt == F32 else L.BF16


def units_ref(gu, da, f):
    """float64 on the CPU: a, dgu and their error bounds before the output's rounding. The fp32 steps (exp, the
    divide, up to six products and sums) are worth 2^-20 of each term's magnitude for |g| <= 16: exp(-g) is exact to
    a few units of 2^-24 with expf, and to |g| / ln 2 units of 2^-24 with the hardware's exp2 of a rounded product."""
    I = gu.shape[1] // 2
    g, u = gu.double().cpu().split(I, 1)
    silu, slope = train_ref.silu_parts(g)
    f = f.view(-1, I)
    a = drop(silu * u, f)
    if da is None:
        return a, None, None
    w = drop(da.double().cpu(), f)
    s = torch.sigmoid(g)
    mag = torch.cat([(w * u).abs() * s * (1 + g.abs()), (w * silu).abs()], 1)
    on = f != 0  # w holds dropout's factor
    return a, torch.cat([torch.where(on, w * u * slope, 0.0), torch.where(on, w * silu, 0.0)], 1), mag


def check(got, ref, mag, dt):
    err = (got.double().cpu() - ref).abs()
    tol = train_ref.HALF[dt] * 1.01 * ref.abs() + 2.0 ** -20 * mag + 1e-37
    assert (err <= tol).all(), (float(err.max()), (err - tol).argmax())


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("rows,I", [(1, 1), (1, 8), (3, 7), (5, 13), (33, 64), (129, 200), (64, 2048), (17, 1031)])
def test_units(L, rows, I, dt, p):
    g = torch.Generator(device=DEV).manual_seed(rows + I)
    gu = (torch.randn((rows + 2, 2 * I), generator=g, device=DEV) * 3).to(dt)
    da = torch.randn((rows + 2, I), generator=g, device=DEV).to(dt)
    rng = rng_tensor(123456789012345, 3 << 40, DEV)
    f = factor(rng.cpu(), rows * I, p)
    n_rows = torch.tensor([rows], dtype=torch.int32, device=DEV)
    a = torch.full((rows + 2, I), 5.0, device=DEV, dtype=dt)
    L.moe_swiglu(gu, code(L, dt), n_rows, rows + 2, I, p, rng, a)
    ref, dref, dmag = units_ref(gu[:rows], da[:rows], f)
    check(a[:rows], ref, ref.abs(), dt)
    assert (a[rows:] == 5).all()
    a2, dgu = torch.full_like(a, 5.0), torch.full_like(gu, 5.0)
    L.moe_swiglu_grad(gu, da, code(L, dt), n_rows, rows + 2, I, p, rng, dgu, a2)
    assert torch.equal(a2, a)
    check(dgu[:rows], dref, dmag, dt)
    assert (dgu[rows:] == 5).all()
    # without a; in place; every row where no count is given
    d2 = torch.full_like(gu, 5.0)
    L.moe_swiglu_grad(gu, da, code(L, dt), n_rows, rows + 2, I, p, rng, d2, None)
    assert torch.equal(d2, dgu)
    gi, di = gu.clone(), da.clone()
    L.moe_swiglu_grad(gi, di, code(L, dt), n_rows, rows + 2, I, p, rng, gi, di)
    assert torch.equal(gi[:rows], dgu[:rows]) and torch.equal(di[:rows], a[:rows])
    assert torch.equal(gi[rows:], gu[rows:]) and torch.equal(di[rows:], da[rows:])
    full = torch.full_like(a, 5.0)
    L.moe_swiglu(gu, code(L, dt), None, rows + 2, I, p, rng, full)
    check(full, units_ref(gu, None, factor(rng.cpu(), (rows + 2) * I, p))[0],
          units_ref(gu, None, factor(rng.cpu(), (rows + 2) * I, p))[0].abs(), dt)


@pytest.mark.parametrize("count", [0, -3, 100])
def test_row_count_is_clamped(L, count):
    gu = torch.randn((4, 16), device=DEV)
    a = torch.full((4, 8), 5.0, device=DEV)
    L.moe_swiglu(gu, L.F32, torch.tensor([count], dtype=torch.int32, device=DEV), 4, 8, 0.0, None, a)
    assert bool((a == 5).all()) == (count <= 0)


def test_units_extremes(L):
    """Large gates saturate without NaN; a dropped place is zero whatever stood there, in the value and the gradient."""
    rows, I = 64, 64
    rng = rng_tensor(9, 1, DEV)
    f = factor(rng.cpu(), rows * I, 0.5).view(rows, I)
    for dt in (BF, F32):
        gu = torch.full((rows, 2 * I), 2.0, device=DEV, dtype=dt)
        gu[:, 0::4] = 3e4
        gu[:, 1::4] = -3e4
        da = torch.ones((rows, I), device=DEV, dtype=dt)
        a, dgu = torch.empty_like(da), torch.empty_like(gu)
        L.moe_swiglu_grad(gu, da, code(L, dt), None, rows, I, 0.0, None, dgu, a)
        assert torch.isfinite(a).all() and torch.isfinite(dgu).all()
        assert (a[:, 1::4] == 0).all() and (dgu[:, 1:I:4] == 0).all()  # silu of a large negative, and its slope
        for bad in (float("nan"), float("inf"), float("-inf")):
            gu[:] = bad
            da[:] = bad
            L.moe_swiglu_grad(gu, da, code(L, dt), None, rows, I, 0.5, rng, dgu, a)
            gone = (f == 0).to(DEV)
            assert (a[gone] == 0).all() and (dgu[:, :I][gone] == 0).all() and (dgu[:, I:][gone] == 0).all()
            assert not torch.isfinite(dgu[:, I:][~gone]).any()


@pytest.mark.parametrize("p", [0.0, 0.1, 0.9])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 4096, 65537, 3_000_001])
def test_dropout(L, n, dt, p):
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randn(n, generator=g, device=DEV).to(dt)
    res = torch.randn(n, generator=g, device=DEV).to(dt)
    rng = rng_tensor(-7, 12, DEV)  # as 64 unsigned bits
    f = factor(rng.cpu(), n, p)
    out = torch.empty_like(x)
    L.moe_dropout(x, None, code(L, dt), n, p, rng, out)
    ref = drop(x.double().cpu(), f)
    assert ((out.double().cpu() - ref).abs() <= (train_ref.HALF[dt] * 1.01 + 2.0 ** -23) * ref.abs()).all()
    L.moe_dropout(x, res, code(L, dt), n, p, rng, out)
    both = ref + res.double().cpu()
    assert ((out.double().cpu() - both).abs() <= train_ref.HALF[dt] * 1.01 * both.abs() + 2.0 ** -22 * ref.abs()
            + 2.0 ** -23 * both.abs()).all()
    for t, args in ((x.clone(), "x"), (res.clone(), "residual")):  # written over an input
        L.moe_dropout(t if args == "x" else x, t if args == "residual" else res, code(L, dt), n, p, rng, t)
        assert torch.equal(t, out)


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_dropout_alignment(L, dt):
    """Tensors that start between 16-byte lines: the same bits as aligned ones."""
    n = 1001
    x, res = torch.randn(n + 3, device=DEV).to(dt), torch.randn(n + 5, device=DEV).to(dt)
    rng = rng_tensor(1, 2, DEV)
    a, b = x[3:].clone(), res[5:].clone()
    whole, out = torch.empty_like(a), torch.zeros(n + 1, device=DEV, dtype=dt)
    L.moe_dropout(a, b, code(L, dt), n, 0.3, rng, whole)
    L.moe_dropout(x[3:], res[5:], code(L, dt), n, 0.3, rng, out[1:])
    assert torch.equal(out[1:], whole) and out[0] == 0


def test_dropout_special_values(L):
    x = torch.full((4096,), float("nan"), device=DEV)
    rng = rng_tensor(4, 4, DEV)
    gone = (factor(rng.cpu(), 4096, 0.5) == 0).to(DEV)
    out = torch.empty_like(x)
    L.moe_dropout(x, torch.ones_like(x), L.F32, 4096, 0.5, rng, out)
    assert (out[gone] == 1).all() and torch.isnan(out[~gone]).all()


def test_dropout_past_32_bits(L):
    """More than 2^32 elements: the last ones use their own blocks."""
    n = 2 ** 32 + 1000
    x = torch.ones(n, device=DEV, dtype=BF)
    rng = rng_tensor(11, 0, DEV)
    L.moe_dropout(x, None, L.BF16, n, 0.5, rng, x)
    f = factor(rng.cpu(), 5000, 0.5, first=n - 5000)
    assert torch.equal(x[-5000:].double().cpu(), f)
    assert not torch.equal(x[:5000].double().cpu(), f)


def test_dropout_share_and_independence(L):
    """The dropped share of 2^22 elements, and of pairs under two offsets, within six standard deviations."""
    n, p = 2 ** 22, 0.3
    q = train_ref.threshold(p) / 65536
    x = torch.ones(n, device=DEV)
    masks = []
    for rng in (rng_tensor(5, 0, DEV), rng_tensor(5, 1, DEV), rng_tensor(6, 0, DEV)):
        out = torch.empty_like(x)
        L.moe_dropout(x, None, L.F32, n, p, rng, out)
        masks.append((out == 0).double())
    for m in masks:
        assert abs(float(m.mean()) - q) <= 6 * (q * (1 - q) / n) ** 0.5
    for a, b in ((0, 1), (0, 2), (1, 2)):
        assert abs(float((masks[a] * masks[b]).mean()) - q * q) <= 6 * (q * q * (1 - q * q) / n) ** 0.5
    assert abs(float((masks[0][1:] * masks[0][:-1]).mean()) - q * q) <= 6 * (2 * q * q / n) ** 0.5  # neighbours


def test_graph_draws_anew(L):
    """A captured forward and backward with a moving offset in device memory."""
    rows, I = 40, 72
    gu, da = torch.randn((rows, 2 * I), device=DEV).to(BF), torch.randn((rows, I), device=DEV).to(BF)
    rng, one = rng_tensor(21, 0, DEV), torch.tensor([0, 1], device=DEV)
    a, dgu = torch.empty_like(da), torch.empty_like(gu)
    L.moe_swiglu(gu, L.BF16, None, rows, I, 0.5, rng, a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_swiglu(gu, L.BF16, None, rows, I, 0.5, rng, a)
        L.moe_swiglu_grad(gu, da, L.BF16, None, rows, I, 0.5, rng, dgu, None)
        rng.add_(one)
    seen = []
    for i in range(3):
        want, dwant = torch.empty_like(a), torch.empty_like(dgu)
        now = rng_tensor(21, i, DEV)
        L.moe_swiglu(gu, L.BF16, None, rows, I, 0.5, now, want)
        L.moe_swiglu_grad(gu, da, L.BF16, None, rows, I, 0.5, now, dwant, None)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(dgu, dwant)
        seen.append(a.clone())
    assert not torch.equal(seen[0], seen[1])


def test_units_gradient_against_differences(L):
    """Central differences of sum(c * a) with fp32 calls: h^2 / 6 of the third derivative (below 1 for the sum of unit
    directions here) and the rounding of the two values, 2^-22 of the summed magnitudes over h."""
    rows, I, h = 8, 24, 2.0 ** -6
    g = torch.Generator(device=DEV).manual_seed(8)
    gu = torch.randn((rows, 2 * I), generator=g, device=DEV)
    c = torch.randn((rows, I), generator=g, device=DEV)
    rng = rng_tensor(2, 2, DEV)
    dgu = torch.empty_like(gu)
    L.moe_swiglu_grad(gu, c, L.F32, None, rows, I, 0.25, rng, dgu, None)

    def value(v):
        a = torch.empty_like(c)
        L.moe_swiglu(v, L.F32, None, rows, I, 0.25, rng, a)
        return (a.double() * c.double()).sum(), float((a * c).abs().sum())
    for s in range(5):
        v = torch.randn(gu.shape, generator=g, device=DEV)
        v /= v.norm()
        (up, mag), (down, _) = value(gu + h * v), value(gu - h * v)
        slope = float(up - down) / (2 * h)
        third = 4 * float((c.abs() * (1 + gu[:, I:].abs())).max())  # |silu'''| < 1, dropout's scale 4/3, mixed terms
        # the points themselves are rounded to fp32: |gu| 2^-24 each, times the gradient
        moved = float((dgu.abs() * gu.abs()).sum()) * 2.0 ** -24 / h
        assert abs(slope - float((dgu * v).double().sum())) <= h * h / 6 * third + mag * 2.0 ** -22 / h + moved
