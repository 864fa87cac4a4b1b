"""moe_pre_norm and moe_combine_norm against 64 bits.

Tolerances count fp32 roundings (U = 2^-24 each, relative): the sum of squares adds at most 16 terms in a thread, 6
levels in a wave and 16 waves (all terms positive), so with the mean, eps, square root and division 1/rms is within
48 U; the elementwise products add 4 U; then one rounding to the output's type."""
import pytest
import torch

from gpu_util import DEV, say
from mx_ref import F64, U, half_step

pytestmark = pytest.mark.gpu


def _lib():
    import mixture_experts_layer_select_amd as L
    return L


def rand(shape, seed, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def close(name, got, want, bound, dtype):
    half = half_step(dtype)
    tiny = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133  # the smallest step of the type
    err = (got.cpu().to(F64) - want).abs()
    tol = bound + half * (want.abs() + bound) + tiny
    worst = float((err / tol).max())
    say(f"[{name}] worst error / tolerance {worst:.3f}")
    assert worst <= 1.0, f"{name}: {worst}"


def rms(v, eps):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


SHAPES = [(1, 1), (3, 7), (2, 64), (5, 100), (4, 512), (9, 513), (3, 3001), (2, 4096), (2, 4104), (1, 2048), (2, 2049),
          (17, 2056), (3, 7168), (2, 8192), (2, 8200), (1, 16384), (2, 16383), (300, 1280)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_pre_norm(T, H, dtype):
    L = _lib()
    dt = L.BF16 if dtype == torch.bfloat16 else L.F32
    for delta_on, gain_on, h_on in ((True, True, True), (False, True, False), (True, False, True)):
        x, d = rand((T, H), T + H, 2.0, dtype), rand((T, H), T + H + 1, 0.5, dtype)
        gain = 1 + rand((H,), 3, 0.2)
        scale, eps = -0.7, 1e-5
        h_out = torch.full((T, H), 9.0, dtype=dtype, device=DEV)
        n_out = torch.full((T, H), 9.0, dtype=dtype, device=DEV)
        L.moe_pre_norm(x.to(DEV), d.to(DEV) if delta_on else None, scale, gain.to(DEV) if gain_on else None, eps, dt, T,
                       H, h_out if h_on else None, n_out)
        s32 = float(torch.tensor(scale, dtype=torch.float32))
        e32 = float(torch.tensor(eps, dtype=torch.float32))
        h = x.to(F64) + (s32 * d.to(F64) if delta_on else 0)
        dh = U * h.abs()
        g = gain.to(F64) if gain_on else torch.ones(H, dtype=F64)
        r = rms(h, e32)
        n = h * r * g
        if h_on:
            close(f"h {T}x{H}", h_out, h, dh, dtype)
        # U of h's own rounding moves the mean square by at most 2 U
        close(f"n {T}x{H}", n_out, n, 56 * U * n.abs(), dtype)


def test_pre_norm_in_place_and_unaligned():
    """h_out over x, over delta, and rows at addresses that no vector load may take, equal the plain call."""
    L = _lib()
    T, H = 7, 1024
    x, d, gain = rand((T, H), 1, 1.0, torch.bfloat16).to(DEV), rand((T, H), 2, 1.0, torch.bfloat16).to(DEV), rand((H,), 3).to(DEV)
    h, n = torch.empty_like(x), torch.empty_like(x)
    L.moe_pre_norm(x, d, 0.5, gain, 1e-6, L.BF16, T, H, h, n)
    for which in (0, 1):
        a, b, n2 = x.clone(), d.clone(), torch.empty_like(x)
        L.moe_pre_norm(a, b, 0.5, gain, 1e-6, L.BF16, T, H, (a, b)[which], n2)
        assert torch.equal((a, b)[which], h) and torch.equal(n2, n)
    buf = torch.empty(T * H + 8, dtype=torch.bfloat16, device=DEV)
    odd = buf[1:1 + T * H].view(T, H)
    odd.copy_(x)
    n2 = torch.empty_like(x)
    L.moe_pre_norm(odd, d, 0.5, gain, 1e-6, L.BF16, T, H, None, n2)
    # another order of the sum of squares: 1/rms within 2 * 48 U of the other's, so at most one bf16 step apart
    assert float(((n2.float() - n.float()).abs() / n.float().abs().clamp(min=1e-20)).max()) <= 2 * half_step(torch.bfloat16) * 1.01


def test_pre_norm_extremes():
    """A zero row with eps > 0 gives zeros; a NaN or infinity stays in its row."""
    L = _lib()
    x = rand((4, 256), 5)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 9] = float("inf")
    n = torch.empty((4, 256), device=DEV)
    L.moe_pre_norm(x.to(DEV), None, 0.0, None, 1e-6, L.F32, 4, 256, None, n)
    n = n.cpu()
    assert bool((n[0] == 0).all()) and bool(torch.isnan(n[1]).all())
    assert bool(torch.isnan(n[2, 9])) and bool((n[2, :9] == 0).all())
    close("row 3", n[3:], x[3:].to(F64) * rms(x[3:].to(F64), 1e-6), 56 * U * 4.0, torch.float32)


@pytest.mark.parametrize("y_dt,out_dt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                         (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,k,H,shared,parts", [
    (1, 1, 1, False, "ngr"), (3, 2, 7, True, "ngr"), (5, 8, 64, True, "n"), (2, 8, 7168, True, "ngr"),
    (4, 3, 2050, False, "gr"), (2, 256, 128, True, "nr"), (3, 4, 8200, True, "ng"), (1, 2, 16384, False, "ngr"),
    (130, 8, 1024, True, "ngr"), (6, 9, 520, False, ""), (4, 2, 512, True, "ngr"), (3, 2, 3001, True, "ngr"),
    (2, 3, 4096, False, "nr")])
def test_combine_norm(T, k, H, shared, parts, y_dt, out_dt):
    """parts: n = post norm, g = gate, r = residual. Every third token has no local pick."""
    L = _lib()
    S = T * k
    g = torch.Generator().manual_seed(T * 7 + k)
    row = torch.randperm(S, generator=g).to(torch.int32)
    row[torch.rand(S, generator=g) < 0.2] = -1
    row.view(T, k)[2::3] = -1
    y = rand((S + T, H), 31, 1.0, y_dt)
    tw = torch.rand((T, k), generator=g)
    off = torch.tensor([0, S, S + T], dtype=torch.int32)
    gain, res = 1 + rand((H,), 4, 0.2), rand((T, H), 6, 2.0, out_dt)
    eps, alpha = float(torch.tensor(1e-6)), -0.8
    a32 = float(torch.tensor(alpha))
    for gate_rows in (1, T):
        gate = rand((gate_rows, H), 5, 0.7, out_dt)
        out = torch.full((T, H), 9.0, dtype=out_dt, device=DEV)
        L.moe_combine_norm(y.to(DEV), L.dtype_code(y), row.to(DEV), tw.to(DEV), T, k, H, off.to(DEV), 1 if shared else -1,
                           gain.to(DEV) if "n" in parts else None, eps, gate.to(DEV) if "g" in parts else None, gate_rows,
                           alpha, res.to(DEV) if "r" in parts else None, out, L.dtype_code(out))
        w = torch.where(row.view(T, k) >= 0, tw, torch.zeros_like(tw)).to(F64)
        picked = y[row.view(T, k).clamp(min=0).long()].to(F64)
        c = (picked * w[..., None]).sum(1) + (y[S:].to(F64) if shared else 0)
        dc = (k + 1) * U * ((picked.abs() * w[..., None]).sum(1) + (y[S:].to(F64).abs() if shared else 0))
        n, dn = c, dc
        if "n" in parts:
            r = rms(c, eps)
            gg = gain.to(F64)
            n = c * r * gg
            # the mean square moves by at most 2 rms dc + dc^2 (dc rms below): relative change of r half of that
            ddc = dc.square().mean(1, keepdim=True).sqrt()
            rel = (2 * c.square().mean(1, keepdim=True).sqrt() * ddc + ddc ** 2) * r ** 2
            dn = dc * r * gg.abs() + n.abs() * (52 * U + rel)
        f = a32 * (gate.to(F64) if "g" in parts else 1)
        want = f * n + (res.to(F64) if "r" in parts else 0)
        bound = torch.as_tensor(f).abs() * dn + 4 * U * (f * n).abs() + U * want.abs()
        close(f"combine {T}x{k}x{H} {parts or '-'}", out, want, bound, out_dt)


def test_combine_norm_in_place_and_bits():
    """out over residual equals a separate buffer; two calls give the same bits."""
    L = _lib()
    T, k, H = 33, 8, 7168
    y = rand((T * k + T, H), 1, 1.0, torch.bfloat16).to(DEV)
    row = torch.randperm(T * k, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)
    tw, off = torch.rand((T, k), device=DEV), torch.tensor([0, T * k, T * k + T], dtype=torch.int32, device=DEV)
    res, gain = rand((T, H), 3, 1.0, torch.bfloat16).to(DEV), rand((H,), 4).to(DEV)
    call = lambda r, o: L.moe_combine_norm(y, L.BF16, row, tw, T, k, H, off, 1, gain, 1e-6, None, 1, 0.5, r, o, L.BF16)
    a, b, c = torch.empty_like(res), torch.empty_like(res), res.clone()
    call(res, a)
    call(res, b)
    call(c, c)
    assert torch.equal(a, b) and torch.equal(a, c)


def test_combine_norm_leaves_out_what_is_not_picked():
    """NaN in rows that no token picked, and weights of non-local picks, do not reach the output."""
    L = _lib()
    T, k, H = 4, 2, 256
    y = torch.full((T * k + T, H), float("nan"))
    y[:3] = rand((3, H), 8)
    row = torch.tensor([0, -1, -1, 1, 2, -1, -1, -1], dtype=torch.int32)
    tw = torch.where(row.view(T, k) >= 0, torch.full((T, k), 0.5), torch.full((T, k), float("nan")))
    out = torch.empty((T, H), device=DEV)
    L.moe_combine_norm(y.to(DEV), L.F32, row.to(DEV), tw.to(DEV), T, k, H, None, -1, None, 0.0, None, 1, 1.0, None, out, L.F32)
    out = out.cpu()
    for t, r in ((0, 0), (1, 1), (2, 2)):
        assert torch.equal(out[t], 0.5 * y[r])
    assert bool((out[3] == 0).all())


def test_many_tokens():
    """More tokens than any other test (the grid's whole range): the last ones equal a small call's."""
    L = _lib()
    T, H = 70000, 256
    x = rand((T, H), 12, 1.0, torch.bfloat16).to(DEV)
    n, small = torch.empty_like(x), torch.empty_like(x[-3:])
    L.moe_pre_norm(x, None, 0.0, None, 1e-6, L.BF16, T, H, None, n)
    L.moe_pre_norm(x[-3:], None, 0.0, None, 1e-6, L.BF16, 3, H, None, small)
    assert torch.equal(n[-3:], small)
