"""The norms where the launch shape or the addresses differ from test_gpu_11_norm's: more rows than one grid of
work items holds, and rows at addresses that no vector access may take."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu

MANY = (1 << 26) + 5  # times 64 threads: more than 2^32 work items
H = 8


def _lib():
    import mixture_experts_layer_select_amd as L
    return L


def bits(a):
    return a.view(torch.int16)


def test_pre_norm_of_more_rows_than_one_grid():
    """The whole equals its two halves, each of which is one grid."""
    L = _lib()
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((MANY, H), generator=g, device=DEV, dtype=torch.bfloat16)
    n, want = torch.zeros_like(x), torch.zeros_like(x)
    L.moe_pre_norm(x, None, 0.0, None, 1e-6, L.BF16, MANY, H, None, n)
    half = 1 << 25
    for a, b in ((0, half), (half, MANY)):
        L.moe_pre_norm(x[a:b], None, 0.0, None, 1e-6, L.BF16, b - a, H, None, want[a:b])
    assert bool((want[-1] != 0).all()) and torch.equal(bits(n), bits(want))


def test_combine_norm_of_more_tokens_than_one_grid():
    """One pick a token and a shared row, a gate and a residual for each; the halves take their part of every input."""
    L = _lib()
    g = torch.Generator(device=DEV).manual_seed(2)
    draw = lambda: torch.randn((MANY, H), generator=g, device=DEV, dtype=torch.bfloat16)
    y, res = torch.cat([draw(), draw()]), draw()
    gate = res.flip(0).contiguous()
    rows = torch.arange(MANY - 1, -1, -1, dtype=torch.int32, device=DEV)
    w = torch.rand((MANY, 1), generator=g, device=DEV)
    gain = torch.rand(H, generator=g, device=DEV) + 0.5

    def call(a, b, out):
        off = torch.tensor([0, MANY + a, 2 * MANY], dtype=torch.int32, device=DEV)  # the shared rows of tokens a on
        L.moe_combine_norm(y, L.BF16, rows[a:b], w[a:b], b - a, 1, H, off, 1, gain, 1e-6, gate[a:b], b - a, 0.5,
                           res[a:b], out[a:b], L.BF16)
    out, want = torch.zeros_like(res), torch.zeros_like(res)
    call(0, MANY, out)
    half = 1 << 25
    call(0, half, want)
    call(half, MANY, want)
    assert bool((want[-1] != 0).any()) and torch.equal(bits(out), bits(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,width", [(5, 64), (3, 7168), (2, 8200), (4, 1001)])
def test_pre_norm_in_place_of_either_input(T, width, dtype):
    """h_out over x and over delta, at one and two chunks a thread, with and without vector accesses."""
    L = _lib()
    g = torch.Generator().manual_seed(T + width)
    x, d = (torch.randn((T, width), generator=g).to(dtype).to(DEV) for _ in range(2))
    gain = (torch.rand(width, generator=g) + 0.5).to(DEV)
    dt = L.BF16 if dtype == torch.bfloat16 else L.F32
    h, n = torch.empty_like(x), torch.empty_like(x)
    L.moe_pre_norm(x, d, 0.75, gain, 1e-6, dt, T, width, h, n)
    for which in (0, 1):
        pair, n2 = (x.clone(), d.clone()), torch.empty_like(x)
        L.moe_pre_norm(*pair, 0.75, gain, 1e-6, dt, T, width, pair[which], n2)
        assert torch.equal(pair[which], h) and torch.equal(n2, n) and torch.equal(pair[1 - which], (x, d)[1 - which])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,width,which", [(3, 512, "y"), (3, 512, "gain"), (4, 1024, "gate"), (2, 7168, "residual"),
                                           (5, 2056, "out"), (2, 8200, "all"), (7, 64, "all")])
def test_combine_norm_at_any_alignment(T, width, which, dtype):
    """Each buffer, and all of them, one element past a vector boundary: the threads' columns and the order of every
    sum stay what they are, so the bits are those of the aligned call."""
    L = _lib()
    k, dt = 3, L.BF16 if dtype == torch.bfloat16 else L.F32
    g = torch.Generator().manual_seed(T + width)
    draw = lambda *s, t=dtype: torch.randn(s, generator=g).to(t).to(DEV)

    def odd(t, name):
        if which not in (name, "all"):
            return t
        room = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)
        room[1:1 + t.numel()] = t.flatten()
        return room[1:1 + t.numel()].view(t.shape)
    y, gate, res, gain = draw(T * k + T, width), draw(T, width), draw(T, width), draw(width, t=torch.float32)
    rows = torch.randperm(T * k, generator=g).to(torch.int32)
    rows[1] = -1
    rows, w = rows.to(DEV), draw(T, k, t=torch.float32)
    off = torch.tensor([0, T * k, T * k + T], dtype=torch.int32, device=DEV)

    def call(y, gain, gate, res, out):
        L.moe_combine_norm(y, dt, rows, w, T, k, width, off, 1, gain, 1e-6, gate, T, 0.5, res, out, dt)
        return out
    want = call(y, gain, gate, res, torch.zeros_like(res))
    got = call(odd(y, "y"), odd(gain, "gain"), odd(gate, "gate"), odd(res, "residual"), odd(torch.zeros_like(res), "out"))
    assert torch.equal(got, want) and bool((want != 0).any(1).all())
