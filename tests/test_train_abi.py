"""The training entry points without a GPU: refusals before anything is enqueued, calls with nothing to do, and the
reference's random numbers against published ones."""
import numpy as np
import pytest
import torch

import train_ref


@pytest.fixture(scope="module")
def L():
    import os

    import mixture_experts_layer_select_amd as pkg
    if not os.path.exists(pkg._lib.LIB_PATH):
        pkg.build()
    return pkg


P = 4096  # an aligned address that no accepted call is given


def refused(L, status, call, **kw):
    with pytest.raises(L.MoEError) as e:
        call(**kw)
    assert e.value.status == "MOE_ERR_" + status, (kw, str(e.value))


def test_philox_known_answers():
    """The generator's published answers: counter and key of zeros, of ones, and of pi's digits."""
    assert train_ref.philox(0, 0, [0])[0].tolist() == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 2 ** 64 - 1
    assert train_ref.philox(ones, ones, [ones])[0].tolist() == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    w = train_ref.philox(0x299F31D0A4093822, 0x0370734413198A2E, [0x85A308D3243F6A88])[0]
    assert w.tolist() == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_factor_slices():
    rng = torch.tensor([77, 5])
    whole = train_ref.factor(rng, 400, 0.3)
    for first, n in ((0, 1), (3, 100), (8, 8), (131, 269)):
        assert torch.equal(train_ref.factor(rng, n, 0.3, first), whole[first:first + n])
    assert set(whole.tolist()) == {0.0, 65536 / (65536 - 19661)}


@pytest.mark.parametrize("name", ["moe_grouped_gemm", "moe_grouped_gemm_dx", "moe_grouped_gemm_dw"])
def test_grouped_refusals(L, name):
    f = getattr(L, name)
    dw = name.endswith("dw")

    def call(a=P, b=P, last=None, dt=L.BF16, off=P, n=4, rows=100, N=64, K=64, out=P, out_dt=L.BF16):
        if dw:
            f(a, b, dt, off, n, rows, N, K, out, last, out_dt, 0, 0)
        else:
            f(a, b, last, dt, off, n, rows, N, K, out, out_dt, 0, 0)
    for kw, status in [(dict(n=0), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"),
                       (dict(K=-8), "INVALID_ARG"), (dict(dt=L.FP8_E4M3), "UNSUPPORTED"),
                       (dict(dt=L.MXFP4), "UNSUPPORTED"), (dict(out_dt=L.FP8_E4M3), "UNSUPPORTED"),
                       (dict(dt=L.F32), "UNSUPPORTED"),  # bf16 out of fp32
                       (dict(n=1026), "UNSUPPORTED"), (dict(N=60), "UNSUPPORTED"), (dict(K=68), "UNSUPPORTED"),
                       (dict(K=62, dt=L.F32, out_dt=L.F32), "UNSUPPORTED"), (dict(N=65544), "UNSUPPORTED"),
                       (dict(a=None), "INVALID_ARG"), (dict(b=None), "INVALID_ARG"), (dict(off=None), "INVALID_ARG"),
                       (dict(out=None), "INVALID_ARG"), (dict(a=P + 8), "INVALID_ARG"), (dict(b=P + 2), "INVALID_ARG"),
                       (dict(out=P + 4), "INVALID_ARG"), (dict(last=P + 8), "INVALID_ARG")]:
        refused(L, status, call, **kw)
    if dw:
        refused(L, "INVALID_ARG", call, out=None, last=P, n=2)
    else:
        refused(L, "UNSUPPORTED", call, rows=2 ** 31 - 1, N=65536, K=65536)
        refused(L, "INVALID_ARG", call, b=None, last=P, n=2)
        call(rows=0, a=None, b=None, off=None, out=None)


@pytest.mark.parametrize("name", ["moe_grouped_gemm", "moe_grouped_gemm_dx", "moe_grouped_gemm_dw"])
@pytest.mark.parametrize("rows", [2 ** 30 + 1, 2 ** 31 - 256, 2 ** 31 - 1])
def test_grouped_refuses_rows_past_32_bits(L, name, rows):
    """A group's rows are rounded up to whole tiles in 32 bits. Narrow matrices keep the number of tiles small, so only
    the rows' own limit refuses these; without pointers, a call that gets past it enqueues nothing either."""
    f = getattr(L, name)
    for n, status in ((rows, "UNSUPPORTED"), (2 ** 30, "INVALID_ARG")):
        with pytest.raises(L.MoEError) as e:
            if name.endswith("dw"):
                f(None, None, L.BF16, None, 1, n, 8, 8, None, None, L.BF16, 0, 0)
            else:
                f(None, None, None, L.BF16, None, 1, n, 8, 8, None, L.BF16, 0, 0)
        assert e.value.status == "MOE_ERR_" + status, (n, str(e.value))


def test_dropout_refusals(L):
    def call(x=P, dt=L.BF16, n=100, p=0.5, rng=P, out=P):
        L.moe_dropout(x, None, dt, n, p, rng, out, 0)
    for kw, status in [(dict(n=-1), "INVALID_ARG"), (dict(dt=L.FP8_E4M3), "UNSUPPORTED"), (dict(p=-0.1), "INVALID_ARG"),
                       (dict(p=1.0), "INVALID_ARG"), (dict(p=float("nan")), "INVALID_ARG"),
                       (dict(p=0.999999), "INVALID_ARG"), (dict(rng=None), "INVALID_ARG"),
                       (dict(rng=P + 4), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG")]:
        refused(L, status, call, **kw)
    call(n=0, x=None, out=None)
    call(n=0, p=0.0, rng=None)


@pytest.mark.parametrize("grad", [False, True])
def test_units_refusals(L, grad):
    def call(gu=P, da=P, dt=L.BF16, rows=10, I=64, p=0.5, rng=P, out=P):
        if grad:
            L.moe_swiglu_grad(gu, da, dt, None, rows, I, p, rng, out, None, 0)
        else:
            L.moe_swiglu(gu, dt, None, rows, I, p, rng, out, 0)
    for kw, status in [(dict(rows=-1), "INVALID_ARG"), (dict(I=0), "INVALID_ARG"), (dict(dt=L.MXFP4), "UNSUPPORTED"),
                       (dict(I=2 ** 24 + 1), "UNSUPPORTED"), (dict(p=1.5), "INVALID_ARG"),
                       (dict(rng=None), "INVALID_ARG"), (dict(gu=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG")]:
        refused(L, status, call, **kw)
    if grad:
        refused(L, "INVALID_ARG", call, da=None)
    call(rows=0, gu=None, da=None, out=None)


def test_combine_grad_refusals(L):
    def call(dout=P, y=P, dt=L.BF16, slots=P, w=P, T=4, k=2, H=64, off=None, shared=-1, dy=P, dw=P):
        L.moe_combine_grad(dout, y, dt, slots, w, T, k, H, off, shared, dy, dw, 0)
    for kw, status in [(dict(T=-1), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"),
                       (dict(k=257), "UNSUPPORTED"), (dict(H=2 ** 24 + 8), "UNSUPPORTED"),
                       (dict(dt=L.FP8_E4M3), "UNSUPPORTED"), (dict(dout=None), "INVALID_ARG"),
                       (dict(y=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"), (dict(w=None), "INVALID_ARG"),
                       (dict(dy=None), "INVALID_ARG"), (dict(shared=1), "INVALID_ARG")]:
        refused(L, status, call, **kw)
    call(T=0, dout=None, y=None, slots=None, w=None, dy=None, dw=None)


def test_route_grad_refusals(L):
    def call(logits=P, ids=P, dw=P, T=4, E=16, k=2, scoring=L.SIGMOID, out=P, dt=L.F32):
        L.moe_route_grad(logits, ids, dw, T, E, k, scoring, True, out, dt, 0)
    for kw, status in [(dict(T=-1), "INVALID_ARG"), (dict(k=17), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"),
                       (dict(E=257), "UNSUPPORTED"), (dict(scoring=7), "INVALID_ARG"), (dict(dt=L.MXFP4), "UNSUPPORTED"),
                       (dict(logits=None), "INVALID_ARG"), (dict(ids=None), "INVALID_ARG"),
                       (dict(dw=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG")]:
        refused(L, status, call, **kw)
    call(T=0, logits=None, ids=None, dw=None, out=None)


def test_host_tensors_and_views_are_refused(L):
    """The binding hands over dense tensors of the current device only."""
    t = torch.zeros(8, 8)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        L.moe_dropout(t, None, L.F32, 64, 0.0, None, t, 0)


def test_layer_refusals(L):
    """Formats and sizes that forward_train does not take, found before the device is touched."""
    def layer(fmt, E=8, H=64, I=32, router=8):
        dt = dict(bf16=torch.bfloat16, f32=torch.float32, fp8=torch.uint8)[fmt]
        kw = dict(w13_scale=torch.ones(E, 1, 1), w2_scale=torch.ones(E, 1, 1)) if fmt == "fp8" else {}
        return L.MoELayer(fmt, H, I, 2, torch.zeros(E, 2 * I, H, dtype=dt), torch.zeros(E, H, I, dtype=dt),
                          router=dict(w=torch.zeros(router, H, dtype=dt), bias=None, scoring=L.SIGMOID), **kw)
    for args, err in (((dict(fmt="fp8", H=256, I=128)), "f32 or bf16"), (dict(fmt="bf16", E=9, router=9), "multiple of 8"),
                      (dict(fmt="bf16", I=36), "multiple of 8"), (dict(fmt="f32", H=66), "multiple of 4")):
        with pytest.raises(ValueError, match=err):
            layer(**args).forward_train(torch.zeros(3, args.get("H", 64), dtype=torch.bfloat16))
    ok = layer("bf16")
    with pytest.raises(TypeError):
        ok.forward_train(torch.zeros(3, 64))
    with pytest.raises(ValueError, match="needs rng"):
        ok.forward_train(torch.zeros(3, 64, dtype=torch.bfloat16), dropout=0.5)
    g = ok.new_grads()
    assert g.w13.shape == ok.w13.shape and g.w13.dtype == torch.float32 and g.router_bias is None and g.shared_w13 is None
