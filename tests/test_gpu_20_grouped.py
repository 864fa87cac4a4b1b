"""Grouped products against float64: forms, types, ragged and empty groups, sizes around the tiles, what lies behind
the rows, other groups' infinities, accumulation, the last group's weights apart, streams and graphs."""
import pytest
import torch

import train_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMS = ("forward", "input", "weights")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    import mixture_experts_layer_select_amd as pkg
    return pkg


def make(counts, N, K, dt, seed=1, behind=7):
    g = torch.Generator(device=DEV).manual_seed(seed)
    R = sum(counts)
    x = torch.full((R + behind, K), float("nan"), device=DEV, dtype=dt)
    dy = torch.full((R + behind, N), float("nan"), device=DEV, dtype=dt)
    x[:R] = torch.randn((R, K), generator=g, device=DEV).to(dt)
    dy[:R] = torch.randn((R, N), generator=g, device=DEV).to(dt)
    w = torch.randn((len(counts), N, K), generator=g, device=DEV).to(dt)
    offsets = torch.tensor([0] + counts, device=DEV).cumsum(0).to(torch.int32)
    return x, dy, w, offsets


def empty_out(form, counts, N, K, out_dt, rows):
    shape = (len(counts), N, K) if form == "weights" else (rows, N if form == "forward" else K)
    return torch.full(shape, 37.0, device=DEV, dtype=out_dt)


def call(L, form, x, dy, w, offsets, N, K, out, accumulate=False, last=None, stream=None, n_groups=None):
    code = lambda t: L.F32 if t == F32 else L.BF16
    n, rows, dt, odt = n_groups or len(offsets) - 1, x.shape[0], code(x.dtype), code(out.dtype)
    if form == "forward":
        L.moe_grouped_gemm(x, w, last, dt, offsets, n, rows, N, K, out, odt, accumulate, stream)
    elif form == "input":
        L.moe_grouped_gemm_dx(dy, w, last, dt, offsets, n, rows, N, K, out, odt, accumulate, stream)
    else:
        L.moe_grouped_gemm_dw(dy, x, dt, offsets, n, rows, N, K, out, last, odt, accumulate, stream)


def reference(form, x, dy, w, offsets):
    a, b = {"forward": (x, w), "input": (dy, w), "weights": (dy, x)}[form]
    return train_ref.grouped(form, a, b, offsets.tolist())


def contraction(form, N, K, offsets):
    o = offsets.tolist()
    return {"forward": K, "input": N, "weights": max(b - a for a, b in zip(o, o[1:]))}[form]


def check(got, ref, mag, length, extra=0.0):
    """One rounding of the output (half a step), and fp32 sums of `length` exact products in any order: each addition
    rounds or truncates a partial that the magnitudes bound (2^-23 of it)."""
    err = (got.double() - ref).abs()
    tol = train_ref.HALF[got.dtype] * 1.01 * ref.abs() + (length + 2) * 2.0 ** -23 * mag + extra + 1e-37
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float(err.max()), bad.nonzero()[0].tolist())


COUNTS = {
    "one row": [1],
    "single rows": [1, 1, 0, 1],
    "ragged": [5, 0, 64, 65, 0, 127, 1],
    "tall": [300, 257, 256, 0, 31],
    "empty": [0, 0, 0],
    "one group": [611],
}
SIZES = [(8, 8), (24, 40), (136, 264), (512, 256), (264, 1032)]


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: c.replace(" ", "-"))
@pytest.mark.parametrize("form", FORMS)
def test_product(L, form, counts, N, K):
    counts = COUNTS[counts]
    for dt, out_dt in ((BF, BF), (BF, F32), (F32, F32)):
        x, dy, w, off = make(counts, N, K, dt)
        out = empty_out(form, counts, N, K, out_dt, x.shape[0])
        call(L, form, x, dy, w, off, N, K, out)
        ref, mag = reference(form, x, dy, w, off)
        R = sum(counts)
        got = out if form == "weights" else out[:R]
        check(got, ref, mag, contraction(form, N, K, off))
        if form != "weights":
            assert (out[R:] == 37).all()  # rows behind the last group


@pytest.mark.parametrize("form", FORMS)
def test_fp32_sizes_of_four(L, form):
    counts, N, K = [3, 70, 129], 12, 148
    x, dy, w, off = make(counts, N, K, F32)
    out = empty_out(form, counts, N, K, F32, x.shape[0])
    call(L, form, x, dy, w, off, N, K, out)
    ref, mag = reference(form, x, dy, w, off)
    check(out if form == "weights" else out[:202], ref, mag, contraction(form, N, K, off))


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("form", FORMS)
def test_accumulate(L, form, dt):
    counts, N, K = [70, 0, 200, 9], 136, 72
    x, dy, w, off = make(counts, N, K, dt)
    for out_dt in {dt, F32}:
        out = empty_out(form, counts, N, K, out_dt, x.shape[0])
        out.copy_(torch.randn(out.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)))
        before = out.clone()
        call(L, form, x, dy, w, off, N, K, out, accumulate=True)
        ref, mag = reference(form, x, dy, w, off)
        R = sum(counts)
        n = out.shape[0] if form == "weights" else R
        check(out[:n], ref + before[:n].double(), mag + before[:n].double().abs(), contraction(form, N, K, off))
        assert torch.equal(out[n:], before[n:])
        if form == "weights":
            assert torch.equal(out[1], before[1])  # the group without rows


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("form", FORMS)
def test_last_group_apart(L, form, dt):
    """The shared expert's weights in a tensor of their own: the same bits."""
    counts, N, K = [40, 13, 150], 72, 136
    x, dy, w, off = make(counts, N, K, dt)
    whole = empty_out(form, counts, N, K, dt, x.shape[0])
    call(L, form, x, dy, w, off, N, K, whole)
    if form == "weights":
        routed, last = torch.zeros((2, N, K), device=DEV, dtype=dt), torch.zeros((N, K), device=DEV, dtype=dt)
        call(L, form, x, dy, w, off, N, K, routed, last=last)
        assert torch.equal(torch.cat([routed, last[None]]), whole)
        only = torch.zeros((N, K), device=DEV, dtype=dt)
        call(L, form, x, dy, w, off[:2].contiguous(), N, K, only, n_groups=1)
        assert torch.equal(only, whole[0])
    else:
        out = empty_out(form, counts, N, K, dt, x.shape[0])
        call(L, form, x, dy, w[:2].contiguous(), off, N, K, out, last=w[2].contiguous())
        assert torch.equal(out, whole)
        one = empty_out(form, counts, N, K, dt, x.shape[0])
        call(L, form, x, dy, None, off[:2].contiguous(), N, K, one, last=w[0].contiguous(), n_groups=1)
        assert torch.equal(one[:40], whole[:40])


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("form", FORMS)
def test_other_groups_do_not_leak(L, form, dt):
    """Infinities and NaN in one group's rows and weights stay in its outputs; lengths that end inside a step."""
    N, K = 200, 328
    for counts in ([37, 5, 90], [130, 61, 259]):
        x, dy, w, off = make(counts, N, K, dt)
        lo, hi = off[1], off[2]
        x[lo:hi], dy[lo:hi], w[1] = float("nan"), float("inf"), float("nan")
        out = empty_out(form, counts, N, K, F32, x.shape[0])
        call(L, form, x, dy, w, off, N, K, out)
        ref, mag = reference(form, x, dy, w, off)
        keep = [0, 2] if form == "weights" else [i for i in range(sum(counts)) if not lo <= i < hi]
        check(out[keep], ref[keep], mag[keep], contraction(form, N, K, off))
        bad = out[1] if form == "weights" else out[lo:hi]
        assert not torch.isfinite(bad).any()


def test_rows_above_the_bound_are_left_out(L):
    """Offsets past max_rows (inconsistent maps) are cut there."""
    counts, N, K = [20, 30], 64, 64
    x, dy, w, off = make(counts, N, K, BF, behind=0)
    short = x[:35].contiguous()
    out = torch.full((50, N), 37.0, device=DEV, dtype=BF)
    L.moe_grouped_gemm(short, w, None, L.BF16, off, 2, 35, N, K, out, L.BF16, False)
    ref, mag = train_ref.grouped("forward", short, w, [0, 20, 35])
    check(out[:35], ref, mag, K)
    assert (out[35:] == 37).all()
    dw = torch.empty((2, N, K), device=DEV)
    L.moe_grouped_gemm_dw(dy[:35].contiguous(), short, L.BF16, off, 2, 35, N, K, dw, None, L.F32, False)
    ref, mag = train_ref.grouped("weights", dy[:35], short, [0, 20, 35])
    check(dw, ref, mag, 20)


@pytest.mark.parametrize("form", FORMS)
def test_many_groups(L, form):
    g = torch.Generator().manual_seed(2)
    counts = torch.randint(0, 5, (1025,), generator=g).tolist()
    N, K = 40, 24
    x, dy, w, off = make(counts, N, K, BF)
    out = empty_out(form, counts, N, K, F32, x.shape[0])
    call(L, form, x, dy, w, off, N, K, out)
    ref, mag = reference(form, x, dy, w, off)
    check(out if form == "weights" else out[:sum(counts)], ref, mag, contraction(form, N, K, off))


@pytest.mark.parametrize("form", FORMS)
def test_offsets_past_32_bits(L, form):
    """Row operands of more than 2^32 bytes: the last group's rows."""
    N, K = (40, 32768) if form != "input" else (32768, 40)
    counts = [66000, 500]
    x = torch.zeros((66500, K), device=DEV, dtype=BF)
    dy = torch.zeros((66500, N), device=DEV, dtype=BF)
    g = torch.Generator(device=DEV).manual_seed(4)
    x[66000:] = torch.randn((500, K), generator=g, device=DEV)
    dy[66000:] = torch.randn((500, N), generator=g, device=DEV)
    w = torch.randn((2, N, K), generator=g, device=DEV).to(BF)
    off = torch.tensor([0, 66000, 66500], device=DEV, dtype=torch.int32)
    out = empty_out(form, counts, N, K, F32, 66500)
    call(L, form, x, dy, w, off, N, K, out)
    a, b = {"forward": (x[66000:], w[1:]), "input": (dy[66000:], w[1:]), "weights": (dy[66000:], x[66000:])}[form]
    ref, mag = train_ref.grouped(form, a, b, [0, 500])
    check(out[1:] if form == "weights" else out[66000:], ref, mag, 32768)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("form", FORMS)
def test_shares_of_the_layer(L, form):
    """An expert share at the layer's widths, rows from one to several tiles an expert."""
    counts, N, K = [1, 300, 17, 0, 129, 64, 513], 2048, 7168
    x, dy, w, off = make(counts, N, K, BF)
    out = empty_out(form, counts, N, K, BF, x.shape[0])
    call(L, form, x, dy, w, off, N, K, out)
    ref, mag = reference(form, x, dy, w, off)
    check(out if form == "weights" else out[:sum(counts)], ref, mag, contraction(form, N, K, off))


def test_streams_graph_and_repeats(L):
    """The three forms on two streams at once and in a graph that replays between eager work: the same bits."""
    counts, N, K = [100, 0, 333, 41], 264, 520
    x, dy, w, off = make(counts, N, K, BF)
    eager = {}
    for f in FORMS:
        eager[f] = empty_out(f, counts, N, K, BF, x.shape[0])
        call(L, f, x, dy, w, off, N, K, eager[f])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [{f: empty_out(f, counts, N, K, BF, x.shape[0]) for f in FORMS} for _ in streams]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        for f in FORMS:
            call(L, f, x, dy, w, off, N, K, o[f], stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for f in FORMS:
            assert torch.equal(o[f], eager[f])
    gout = {f: empty_out(f, counts, N, K, BF, x.shape[0]) for f in FORMS}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f in FORMS:
            call(L, f, x, dy, w, off, N, K, gout[f])
    for i in range(3):
        x.mul_(2)  # exact: every product of x doubles
        dy.mul_(2)
        graph.replay()
        torch.cuda.synchronize()
        for f in FORMS:
            factor = 2.0 ** (i + 1) if f != "weights" else 4.0 ** (i + 1)
            n = len(counts) if f == "weights" else sum(counts)
            assert torch.equal(gout[f][:n].float(), eager[f][:n].float() * factor)


@pytest.mark.parametrize("out_dt", [BF, F32], ids=str)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("form", ["forward", "input"])
def test_few_tiles_long_contraction(L, form, accumulate, out_dt):
    """Calls of few tiles split their contraction over waves: lengths around the long steps, several items a workgroup."""
    for counts, out_cols, length in (([3, 0, 9], 64, 4096), ([64, 1], 200, 264), ([17], 72, 256), ([30, 40], 136, 1032),
                                     ([2] * 40, 128, 2056), ([5, 60, 33], 64, 8)):
        N, K = (out_cols, length) if form == "forward" else (length, out_cols)
        x, dy, w, off = make(counts, N, K, BF)
        out = empty_out(form, counts, N, K, out_dt, x.shape[0])
        before = out.clone()
        call(L, form, x, dy, w, off, N, K, out, accumulate=accumulate)
        ref, mag = reference(form, x, dy, w, off)
        R = sum(counts)
        if accumulate:
            ref, mag = ref + 37, mag + 37
        check(out[:R], ref, mag, length)
        assert torch.equal(out[R:], before[R:])


@pytest.mark.parametrize("seed", range(24))
def test_drawn_sizes(L, seed):
    """Sizes over the whole range of tile heights and widths, rows from one to several tiles a group, each form in turn."""
    import random
    rng = random.Random(seed)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    form, f32 = FORMS[seed % 3], seed % 8 == 7
    unit = 4 if f32 else 8
    N, K = unit * log(2, 500), unit * log(2, 500)
    n = rng.randint(1, 40)
    mean = log(1, 600)
    counts = [rng.choice((0, 1, rng.randint(0, mean), rng.randint(0, 2 * mean))) for _ in range(n)]
    while sum(counts) * N * K > 2e11:
        counts = [c // 2 for c in counts]
    dt = F32 if f32 else BF
    out_dt = F32 if f32 else rng.choice((BF, F32))
    x, dy, w, off = make(counts, N, K, dt, seed=seed)
    out = empty_out(form, counts, N, K, out_dt, x.shape[0])
    call(L, form, x, dy, w, off, N, K, out)
    ref, mag = reference(form, x, dy, w, off)
    R = sum(counts)
    check(out if form == "weights" else out[:R], ref, mag, contraction(form, N, K, off))
    if form != "weights":
        assert (out[R:] == 37).all()


@pytest.mark.parametrize("form,counts,N,K", [
    ("forward", [300] * 20, 1024, 192), ("forward", [120] * 40, 4096, 72), ("forward", [180] * 24, 2048, 136),
    ("forward", [40] * 33, 4096, 320), ("input", [300] * 20, 192, 1024), ("input", [120] * 40, 72, 4096),
    ("input", [180] * 24, 136, 2048), ("input", [40] * 33, 320, 4096), ("weights", [40] * 9, 1000, 904),
    ("weights", [100, 0, 31, 33, 64, 1, 129, 2, 511], 520, 776)])
def test_several_items_a_workgroup(L, form, counts, N, K):
    """More items than CUs: each height and width, loads of the next item under the stores of the last."""
    for out_dt in (BF, F32):
        x, dy, w, off = make(counts, N, K, BF)
        out = empty_out(form, counts, N, K, out_dt, x.shape[0])
        call(L, form, x, dy, w, off, N, K, out)
        ref, mag = reference(form, x, dy, w, off)
        R = sum(counts)
        check(out if form == "weights" else out[:R], ref, mag, contraction(form, N, K, off))
