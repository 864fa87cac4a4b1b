"""MXFP4 on the GPU: quantisation bit for bit against the 64-bit rule, reading back, and the expert FFN against
64 bits within bounds derived from its fp32 sums (mx_ref.expert) plus one bf16 rounding."""
import numpy as np
import pytest
import torch

import mx_ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def _lib():
    import mixture_experts_layer_select_amd as L
    return L


def gpu_quantize(x):
    L = _lib()
    rows, cols = x.shape
    codes = torch.full((rows, cols // 2), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, cols // 32), 0xA5, dtype=torch.uint8, device=DEV)
    L.moe_quantize_mxfp4(x, L.dtype_code(x), rows, cols, codes, scales)
    return codes, scales


def special(cols):
    """Rows of thresholds, ties, zeros, denormals, the type's extremes, infinities and NaN."""
    x = torch.zeros(12, cols)
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    for r, s in enumerate((2.0 ** -120, 2.0 ** -3, 1.0, 2.0 ** 100)):
        x[r, :18] = torch.cat([t, -t]) * s
        x[r, 20] = 4.0 * s
    x[4, 0], x[4, 1] = 3.38e38, -1e30
    x[5, :4] = torch.tensor([2.0 ** -126, -(2.0 ** -130), 2.0 ** -133, 2.0 ** -127])
    x[6, 5] = float("inf")
    x[7, 7] = float("nan")
    x[8, 9] = -float("inf")
    x[9, :3] = torch.tensor([2.0 ** -133, 0.0, -0.0])
    x[10, 31] = -1.0
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (13, 7168), (257, 160), (1000, 2048)])
def test_quantize_and_read_back(dtype, rows, cols):
    L = _lib()
    say(f"[mx quantize] {dtype} {rows}x{cols}")
    g = torch.Generator().manual_seed(rows * 31 + cols)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g).float())
    x = torch.cat([x, special(cols)]).to(dtype)
    codes, scales = gpu_quantize(x.to(DEV))
    want_codes, want_scales, want = mx_ref.quantize(x)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(codes.cpu(), want_codes)
    for out_dt in (torch.bfloat16, torch.float32):
        out = torch.full(x.shape, 7.0, dtype=out_dt, device=DEV)
        L.moe_dequantize_mxfp4(codes, scales, x.shape[0], cols, out, L.dtype_code(out))
        assert torch.equal(out.cpu().to(torch.float64).nan_to_num(12345.0), want.nan_to_num(12345.0))


def test_read_back_every_code_and_scale():
    L = _lib()
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).contiguous()
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16).contiguous()
    want = mx_ref.values(codes, scales)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.empty((256, 512), dtype=dt, device=DEV)
        L.moe_dequantize_mxfp4(codes.to(DEV), scales.to(DEV), 256, 512, out, L.dtype_code(out))
        # 6 * 2^127 and 4 * 2^127 are above either type's range; the rest is exact
        w = want.to(dt).to(torch.float64)
        assert torch.equal(out.cpu().to(torch.float64).nan_to_num(12345.0, 1e300, -1e300),
                           w.nan_to_num(12345.0, 1e300, -1e300))


def test_quantize_more_than_32_bit_offsets():
    """A tensor of more than 2^32 elements: its last rows are quantised like a small tensor's."""
    L = _lib()
    cols, rows = 1 << 16, (1 << 16) + 3
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    tail = torch.randn((5, cols), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[-5:] = tail.to(DEV)
    codes, scales = gpu_quantize(x)
    want_codes, want_scales, _ = mx_ref.quantize(tail)
    assert torch.equal(codes[-5:].cpu(), want_codes) and torch.equal(scales[-5:].cpu(), want_scales)
    assert int(codes[:-5].view(torch.int64).abs().max()) == 0 and bool((scales[:-5] == 127).all())
    out = torch.empty_like(x)
    L.moe_dequantize_mxfp4(codes, scales, rows, cols, out, L.BF16)
    assert torch.equal(out[-5:].cpu().to(torch.float64), mx_ref.values(want_codes, want_scales))


# ---------------------------------------------------------------- expert FFN
def quantized(shape, std, seed):
    """(codes, scales on the GPU, values float64 on the CPU)"""
    x = torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std
    codes, scales, v = mx_ref.quantize(x)
    return codes.contiguous().to(DEV), scales.contiguous().to(DEV), v


class Experts:
    def __init__(self, H, I, E, shared, seed, std=0.05):
        L = _lib()
        self.H, self.I, self.E, self.shared = H, I, E, shared
        n = E + (1 if shared else 0)
        w13 = [quantized((2 * I, H), std, seed * 1000 + 2 * e) for e in range(n)]
        w2 = [quantized((H, I), std, seed * 1000 + 2 * e + 1) for e in range(n)]
        self.v13, self.v2 = [w[2] for w in w13], [w[2] for w in w2]
        st = lambda ws, i: torch.stack([w[i] for w in ws[:E]])
        sh = [w13[E][0], w2[E][0], w13[E][1], w2[E][1]] if shared else [None] * 4
        self.w = L.make_weights(L.MXFP4, E, H, I, st(w13, 0), st(w2, 0), st(w13, 1), st(w2, 1), *sh)

    def reference(self, x, e):
        return mx_ref.expert(x, self.v13[e], self.v2[e])


def check(name, got, want, bound, dtype=torch.bfloat16):
    """got within half a step of its type of a value within `bound` of want."""
    got, half = got.cpu().to(torch.float64), mx_ref.half_step(dtype)
    err = (got - want).abs()
    tol = bound + half * (want.abs() + bound)
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    say(f"[{name}] worst error / tolerance {worst:.3f}")
    assert worst <= 1.0, f"{name}: {worst}"


SIZES = [  # H, I, rows of each group (the last one shared where `shared`), shared
    (256, 128, [1], False),
    (256, 128, [0, 0, 3], False),
    (512, 384, [5, 0, 33, 64, 65, 1], True),
    (768, 640, [129, 256, 257, 0, 31, 32], False),
    (1280, 128, [300, 2, 511], True),
    (256, 1152, [64, 96, 128, 160], True),
]


def run_ffn(x, xs, ex, offsets, max_rows, slots=None):
    L = _lib()
    n = L.moe_expert_ffn_workspace_size(ex.w, max_rows)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    y = torch.full((max_rows, ex.H), 3.0, dtype=torch.bfloat16, device=DEV)
    groups = len(offsets) - 1
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    if slots is None:
        L.moe_expert_ffn(ex.w, x, xs, off, groups, max_rows, y, ws, n)
    else:
        T, k, row_to_slot = slots
        L.moe_expert_ffn_gate_up_tokens(ex.w, x, xs, T, k, row_to_slot, off, groups, max_rows, ws, n)
        L.moe_expert_ffn_down(ex.w, off, groups, max_rows, y, ws, n)
    return y


@pytest.mark.parametrize("H,I,rows,shared", SIZES)
def test_expert_ffn_against_64_bits(H, I, rows, shared):
    say(f"[mx ffn] H={H} I={I} rows={rows} shared={shared}")
    ex = Experts(H, I, len(rows) - shared, shared, H + I + sum(rows))
    offsets = [0] + np.cumsum(rows).tolist()
    R = offsets[-1]
    x, xs, xv = quantized((R + 5, H), 1.0, 7)
    y = run_ffn(x, xs, ex, offsets, R + 5)
    assert bool((y[R:] == 3.0).all()), "rows behind the last group were written"
    for e in range(len(rows)):
        a, b = offsets[e], offsets[e + 1]
        want, bound = ex.reference(xv[a:b], e)
        check(f"group {e} of {b - a}", y[a:b], want, bound)


def test_expert_ffn_r1_width():
    ex = Experts(7168, 2048, 2, False, 11, 0.02)
    rows = [17, 70]
    x, xs, xv = quantized((87, 7168), 1.0, 8)
    y = run_ffn(x, xs, ex, [0, 17, 87], 87)
    for e, (a, b) in enumerate(((0, 17), (17, 87))):
        want, bound = ex.reference(xv[a:b], e)
        check(f"r1 group of {b - a}", y[a:b], want, bound)


def routed(T, k, E, seed, shared):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    flat = ids.flatten()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E).tolist()
    if shared:
        order = torch.cat([order, T * k + torch.arange(T)])
        counts.append(T)
    return ids, order.to(torch.int32), [0] + np.cumsum(counts).tolist()


@pytest.mark.parametrize("T,k,E,shared,H,I", [(1, 1, 3, False, 256, 128), (37, 3, 5, True, 512, 256),
                                              (400, 2, 3, True, 256, 256)])
def test_token_rows_equal_permuted_rows(T, k, E, shared, H, I):
    """Gate/up through row_to_slot against the same rows laid out contiguously, bit for bit."""
    ex = Experts(H, I, E, shared, 5)
    _, order, offsets = routed(T, k, E, 9, shared)
    x, xs, _ = quantized((T, H), 1.0, 21)
    token = torch.where(order < T * k, order // k, order - T * k).long()
    R = offsets[-1]
    cap = T * k + T
    slots = torch.full((cap,), -1, dtype=torch.int32)
    slots[:R] = order
    got = run_ffn(x, xs, ex, offsets, cap, (T, k, slots.to(DEV)))
    tk = token.to(DEV)
    want = run_ffn(x[tk].contiguous(), xs[tk].contiguous(), ex, offsets, R)
    assert torch.equal(got[:R].view(torch.int16), want.view(torch.int16))
    assert bool((got[R:] == 3.0).all())


def test_slots_out_of_range_stay_inside_the_token_buffers():
    """A slot outside [0, T*k+T) reads some token's row or zeros, as documented, and its own row alone is affected."""
    T, k, H, I = 9, 2, 256, 128
    ex = Experts(H, I, 2, False, 6)
    x, xs, xv = quantized((T, H), 1.0, 22)
    slots = torch.tensor([0, 5, 1 << 30, 7, 12], dtype=torch.int32)
    y = run_ffn(x, xs, ex, [0, 3, 5], 5, (T, k, slots.to(DEV)))
    for r in (0, 1, 3, 4):
        want, bound = ex.reference(xv[int(slots[r]) // k][None], 0 if r < 3 else 1)
        check(f"row {r}", y[r:r + 1], want, bound)


def test_nan_stays_in_its_row_and_its_columns():
    """A NaN scale of one activation row reaches that row alone; one of a weight row reaches its expert alone."""
    H, I = 512, 256
    ex = Experts(H, I, 2, False, 12)
    x, xs, xv = quantized((40, H), 1.0, 23)
    clean = run_ffn(x, xs, ex, [0, 20, 40], 40)
    bad = xs.clone()
    bad[7, 3] = 255
    y = run_ffn(x, bad, ex, [0, 20, 40], 40)
    assert bool(torch.isnan(y[7].float()).all())
    keep = [r for r in range(40) if r != 7]
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))
    saved = ex.w._tensors[3][1, 5, 2].clone()   # w2 scales of expert 1, output column 5
    ex.w._tensors[3][1, 5, 2] = 255
    y = run_ffn(x, xs, ex, [0, 20, 40], 40)
    ex.w._tensors[3][1, 5, 2] = saved
    assert bool(torch.isnan(y[20:, 5].float()).all())
    y[20:, 5] = clean[20:, 5]
    assert torch.equal(y.view(torch.int16), clean.view(torch.int16))


def test_offsets_past_the_buffer_are_clamped():
    """Offsets beyond max_rows write nothing behind the buffer's rows (as for the other formats)."""
    H, I = 256, 128
    ex = Experts(H, I, 2, False, 13)
    x, xs, xv = quantized((10, H), 1.0, 24)
    y = run_ffn(x, xs, ex, [0, 4, 1000], 10)
    want, bound = ex.reference(xv[4:], 1)
    check("clamped group", y[4:], want, bound)


def test_noalloc_equals_workspace():
    L = _lib()
    ex = Experts(512, 256, 3, True, 14)
    x, xs, _ = quantized((120, 512), 1.0, 25)
    offsets = [0, 50, 50, 90, 120]
    want = run_ffn(x, xs, ex, offsets, 120)
    y = torch.zeros_like(want)
    L.moe_expert_ffn_noalloc(ex.w, x, xs, torch.tensor(offsets, dtype=torch.int32, device=DEV), 4, 120, y)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("shared", [False, True])
def test_expert_ffn_with_the_most_experts(shared):
    """512 local experts, nearly all of them empty, with and without the shared group behind them."""
    H, I, E = 256, 128, 512
    ex = Experts(H, I, E, shared, 15)
    rows = [0] * (E + shared)
    for e, r in ((0, 3), (63, 1), (64, 70), (255, 2), (510, 257), (511, 5)):
        rows[e] = r
    if shared:
        rows[E] = 9
    offsets = [0] + np.cumsum(rows).tolist()
    R = offsets[-1]
    x, xs, xv = quantized((R, H), 1.0, 26)
    y = run_ffn(x, xs, ex, offsets, R)
    for e in range(len(rows)):
        if rows[e]:
            a, b = offsets[e], offsets[e + 1]
            want, bound = ex.reference(xv[a:b], e)
            check(f"group {e} of {b - a}", y[a:b], want, bound)


@pytest.mark.parametrize("R", [20, 100, 200])
def test_nan_of_the_next_row_stays_out_of_an_odd_last_half(R):
    """I % 256 = 128: the last K step of the down product holds only 128 of I; the row behind is all NaN."""
    H, I = 256, 384
    ex = Experts(H, I, 1, False, 16)
    x, xs, _ = quantized((R, H), 1.0, 27)
    clean = run_ffn(x, xs, ex, [0, R], R)
    bad = xs.clone()
    bad[1::2] = 255                                 # every other intermediate row is NaN
    ex.w._tensors[3][0, 8::16] = 255                # ... and output columns 8, 24, ...
    y = run_ffn(x, bad, ex, [0, R], R).float()
    keep = torch.ones(H, dtype=torch.bool, device=DEV)
    keep[8::16] = False
    assert torch.equal(y[0::2][:, keep], clean[0::2][:, keep].float())
    assert bool(torch.isnan(y[1::2]).all()) and bool(torch.isnan(y[:, 8::16]).all())


def test_two_graphs_share_a_workspace():
    """Quantisation and both products captured twice over one workspace; replays alternate with eager calls."""
    L = _lib()
    H, I, T = 768, 384, 150
    ex = Experts(H, I, 3, True, 17)
    off = torch.tensor([0, 40, 40, 150, 300], dtype=torch.int32, device=DEV)
    n = L.moe_expert_ffn_workspace_size(ex.w, 300)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    slots = torch.cat([torch.randperm(T, generator=torch.Generator().manual_seed(1)), T + torch.arange(T)])
    slots = slots.to(torch.int32).to(DEV)

    class Side:
        def __init__(self):
            self.x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            self.codes = torch.empty((T, H // 2), dtype=torch.uint8, device=DEV)
            self.scales = torch.empty((T, H // 32), dtype=torch.uint8, device=DEV)
            self.y = torch.empty((300, H), dtype=torch.bfloat16, device=DEV)

        def call(self):
            L.moe_quantize_mxfp4(self.x, L.BF16, T, H, self.codes, self.scales)
            L.moe_expert_ffn_gate_up_tokens(ex.w, self.codes, self.scales, T, 1, slots, off, 4, 300, ws, n)
            L.moe_expert_ffn_down(ex.w, off, 4, 300, self.y, ws, n)

    sides = [Side(), Side()]
    graphs = []
    for s in sides:
        s.x.copy_(torch.randn((T, H), generator=torch.Generator().manual_seed(2)))
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            s.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.call()
        graphs.append(g)
    for seed in (5, 6, 7):
        for i, s in enumerate(sides):
            s.x.copy_(torch.randn((T, H), generator=torch.Generator().manual_seed(10 * seed + i)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [s.y.clone() for s in sides]
        for s, y in zip(sides, got):
            s.y.fill_(4)
            s.call()
            torch.cuda.synchronize()
            assert torch.equal(s.y.view(torch.int16), y.view(torch.int16))


def test_two_streams_with_a_workspace_each():
    """Calls that overlap on two streams give what they give alone."""
    L = _lib()
    ex = Experts(2048, 1024, 4, False, 18)
    want, state = [], []
    for i in range(2):
        R = 300 + 41 * i
        x, xs, _ = quantized((R, 2048), 1.0, 40 + i)
        offsets = [0, 20, 160, 160 + i, R]
        want.append(run_ffn(x, xs, ex, offsets, R))
        n = L.moe_expert_ffn_workspace_size(ex.w, R)
        state.append((x, xs, torch.tensor(offsets, dtype=torch.int32, device=DEV), R,
                      torch.zeros((R, 2048), dtype=torch.bfloat16, device=DEV),
                      torch.empty(n, dtype=torch.uint8, device=DEV), n, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, xs, off, R, y, ws, n, st in state:
            L.moe_expert_ffn(ex.w, x, xs, off, 4, R, y, ws, n, st)
    torch.cuda.synchronize()
    for w, s in zip(want, state):
        assert torch.equal(s[4].view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("rows", [[203, 17, 17, 0, 40], [256, 1, 129], [700, 64, 65, 500], [2000]])
def test_rows_do_not_depend_on_the_tiles(rows):
    """A row's bits are the same whatever the other groups are, and so whatever height its tile gets."""
    H, I = 512, 384
    ex = Experts(H, I, len(rows), False, 19)
    offsets = [0] + np.cumsum(rows).tolist()
    R = offsets[-1]
    x, xs, xv = quantized((R, H), 1.0, 28)
    y = run_ffn(x, xs, ex, offsets, R)
    for e in range(len(rows)):
        a, b = offsets[e], offsets[e + 1]
        for n in {1, 60, rows[e] // 2, rows[e]} & set(range(1, rows[e] + 1)):
            alone = run_ffn(x[a:a + n].contiguous(), xs[a:a + n].contiguous(), ex, [0] * (e + 1) + [n] * (len(rows) - e), n)
            assert torch.equal(alone.view(torch.int16), y[a:a + n].view(torch.int16)), (e, n)
