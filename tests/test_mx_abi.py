"""The MXFP4, norm and few-token entry points without a GPU: refusals before anything is enqueued, no-ops,
workspace sizes."""
import pytest
import torch

import mx_ref


@pytest.fixture(scope="module")
def L():
    import os

    import mixture_experts_layer_select_amd as pkg
    if not os.path.exists(pkg._lib.LIB_PATH):
        pkg.build()
    return pkg


P = 4096  # an aligned address that no accepted call is given


def refused(L, status, fn, *args):
    with pytest.raises(L.MoEError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("name", ["moe_quantize_mxfp4", "moe_dequantize_mxfp4"])
def test_quantize_refusals(L, name):
    if name == "moe_quantize_mxfp4":
        def call(x=P, dt=L.BF16, rows=4, cols=64, codes=P, scales=P):
            L.moe_quantize_mxfp4(x, dt, rows, cols, codes, scales, 0)
    else:
        def call(x=P, dt=L.BF16, rows=4, cols=64, codes=P, scales=P):
            L.moe_dequantize_mxfp4(codes, scales, rows, cols, x, dt, 0)
    for kw, status in [(dict(rows=-1), "INVALID_ARG"), (dict(cols=0), "INVALID_ARG"), (dict(cols=48), "UNSUPPORTED"),
                       (dict(dt=L.FP8_E4M3), "UNSUPPORTED"), (dict(dt=L.MXFP4), "UNSUPPORTED"),
                       (dict(x=None), "INVALID_ARG"), (dict(codes=None), "INVALID_ARG"),
                       (dict(scales=None), "INVALID_ARG"), (dict(x=P + 8), "INVALID_ARG"),
                       (dict(codes=P + 2), "INVALID_ARG")]:
        refused(L, "MOE_ERR_" + status, lambda kw=kw: call(**kw))
    call(rows=0, x=None, codes=None, scales=None)


def test_ffn_refusals(L):
    w = lambda H=512, I=256, E=4, **kw: L.make_weights(L.MXFP4, E, H, I, kw.get("w13", P), P, kw.get("s13", P), P,
                                                       kw.get("ws13"), kw.get("ws13"), kw.get("ss13"), kw.get("ss13"))
    n = L.moe_expert_ffn_workspace_size(w(), 100)
    assert n >= 100 * (128 + 8)
    f = L.moe_expert_ffn
    refused(L, "MOE_ERR_WORKSPACE", f, w(), P, P, P, 4, 100, P, P, n - 1, 0)
    refused(L, "MOE_ERR_INVALID_ARG", f, w(), P, None, P, 4, 100, P, P, n, 0)       # activations without scales
    refused(L, "MOE_ERR_INVALID_ARG", f, w(), P + 4, P, P, 4, 100, P, P, n, 0)      # misaligned activations
    refused(L, "MOE_ERR_INVALID_ARG", f, w(s13=None), P, P, P, 4, 100, P, P, n, 0)  # weights without scales
    refused(L, "MOE_ERR_INVALID_ARG", f, w(w13=P + 8), P, P, P, 4, 100, P, P, n, 0)
    refused(L, "MOE_ERR_INVALID_ARG", f, w(s13=P + 2), P, P, P, 4, 100, P, P, n, 0)
    refused(L, "MOE_ERR_INVALID_ARG", f, w(), P, P, P, 5, 100, P, P, n, 0)          # shared group without weights
    refused(L, "MOE_ERR_INVALID_ARG", f, w(ws13=P), P, P, P, 5, 100, P, P, n, 0)    # ... without scales
    for H, I in ((384, 256), (512, 192), (16640, 256), (512, 16512)):
        refused(L, "MOE_ERR_UNSUPPORTED", f, w(H, I), P, P, P, 4, 100, P, P, 1 << 40, 0)
        assert L.moe_expert_ffn_workspace_size(w(H, I), 100) == 0
    refused(L, "MOE_ERR_UNSUPPORTED", f, w(E=513), P, P, P, 513, 100, P, P, 1 << 40, 0)
    assert L.moe_expert_ffn_workspace_size(w(E=512), 100) == n
    g = L.moe_expert_ffn_gate_up_tokens
    refused(L, "MOE_ERR_INVALID_ARG", g, w(), P, P, 10, 2, None, P, 4, 100, P, n, 0)
    refused(L, "MOE_ERR_UNSUPPORTED", g, w(), P, P, 1 << 23, 2, P, P, 4, 100, P, n, 0)  # T*H = 2^32
    f(w(), None, None, None, 4, 0, None, None, 0, 0)  # no rows
    refused(L, "MOE_ERR_UNSUPPORTED", L.moe_permute, P, 4, 2, 0, 4, 0, P, L.BF16, 512, L.MXFP4, P, P, P, P, P, P, P,
            1 << 20, 0)
    refused(L, "MOE_ERR_UNSUPPORTED", L.moe_layer_fused, P, P, None, 4, 4, 2, L.SIGMOID, 1, w(), P, P, P, P, 1 << 30, 0)


def test_few_refusals(L):
    w = L.make_weights(L.MXFP4, 16, 512, 256, P, P, P, P)
    n = L.moe_layer_few_workspace_size(w, 16, 16, 8)
    assert n >= 256 + (16 * 8 + 16) * 256 * 4

    def call(w=w, x=P, router=P, T=4, E=16, k=2, scoring=L.SIGMOID, base=0, ids=P, out=P, ws=P, ws_bytes=n):
        L.moe_layer_few(x, router, None, T, E, k, scoring, True, w, base, ids, P, out, ws, ws_bytes, 0)
    bf = L.make_weights(L.BF16, 16, 512, 256, P, P)
    tall = L.make_weights(L.MXFP4, 16, 8448, 256, P, P, P, P)
    half = L.make_weights(L.MXFP4, 16, 512, 256, P, P, P, P, P, None)
    bare = L.make_weights(L.MXFP4, 16, 512, 256, P, P, P, P, P, P)
    for kw, status in [(dict(w=bf), "UNSUPPORTED"), (dict(w=tall), "UNSUPPORTED"), (dict(w=half), "INVALID_ARG"),
                       (dict(w=bare), "INVALID_ARG"), (dict(T=17), "UNSUPPORTED"), (dict(T=-1), "INVALID_ARG"),
                       (dict(k=9), "UNSUPPORTED"), (dict(k=17), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"),
                       (dict(E=257), "UNSUPPORTED"), (dict(E=8), "INVALID_ARG"), (dict(base=1), "INVALID_ARG"),
                       (dict(base=-1), "INVALID_ARG"), (dict(scoring=7), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"),
                       (dict(ids=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
                       (dict(x=P + 2), "INVALID_ARG"), (dict(ws=P + 16), "INVALID_ARG"),
                       (dict(ws_bytes=256), "WORKSPACE"), (dict(ws=None), "WORKSPACE")]:
        refused(L, "MOE_ERR_" + status, lambda kw=kw: call(**kw))
    call(T=0, x=None, router=None, ids=None, out=None, ws=None)


def test_norm_refusals(L):
    def pre(x=P, dt=L.BF16, T=4, H=64, eps=1e-6, h=P, n=2 * P):
        L.moe_pre_norm(x, None, 0.0, None, eps, dt, T, H, h, n, 0)

    def post(y=P, y_dt=L.BF16, T=4, k=2, H=64, off=P, sg=-1, eps=1e-6, gate=None, rows=1, out=P, dt=L.BF16):
        L.moe_combine_norm(y, y_dt, P, P, T, k, H, off, sg, None, eps, gate, rows, 1.0, None, out, dt, 0)
    for f, kw, status in [(pre, dict(T=-1), "INVALID_ARG"), (pre, dict(H=0), "INVALID_ARG"),
                          (pre, dict(H=16385), "UNSUPPORTED"), (pre, dict(dt=L.MXFP4), "UNSUPPORTED"),
                          (pre, dict(eps=-1.0), "INVALID_ARG"), (pre, dict(eps=float("nan")), "INVALID_ARG"),
                          (pre, dict(x=None), "INVALID_ARG"), (pre, dict(n=None), "INVALID_ARG"),
                          (pre, dict(n=P), "INVALID_ARG"),
                          (post, dict(T=-1), "INVALID_ARG"), (post, dict(k=0), "INVALID_ARG"),
                          (post, dict(k=257), "UNSUPPORTED"), (post, dict(H=16385), "UNSUPPORTED"),
                          (post, dict(y_dt=L.FP8_E4M3), "UNSUPPORTED"), (post, dict(dt=L.FP8_E4M3), "UNSUPPORTED"),
                          (post, dict(eps=-1.0), "INVALID_ARG"), (post, dict(gate=P, rows=2), "INVALID_ARG"),
                          (post, dict(y=None), "INVALID_ARG"), (post, dict(out=None), "INVALID_ARG"),
                          (post, dict(sg=3, off=None), "INVALID_ARG")]:
        refused(L, "MOE_ERR_" + status, lambda f=f, kw=kw: f(**kw))
    pre(T=0, x=None, n=None)
    post(T=0, y=None, out=None)


def test_reference_quantisation():
    """The tests' own quantisation: thresholds, ties to the even code, saturation, the scale of a block."""
    row = torch.zeros(1, 32)
    row[0, :20] = torch.tensor([4, .25, .2500001, .75, .7499999, 1.25, 1.2500001, 1.75, 1.7499999, 2.5, 2.5000002, 3.5,
                                3.4999998, 5, 5.0000005, 6, 7, 7.9999995, -0.25, -7])
    codes, byte, v = mx_ref.quantize(row)
    assert byte.item() == 127
    want = [4, 0, .5, 1, .5, 1, 1.5, 2, 1.5, 2, 3, 4, 3, 4, 6, 6, 6, 6, 0, -6]
    assert v[0, :20].tolist() == want
    assert torch.equal(mx_ref.values(codes, byte), v)
    for amax, b in ((8.0, 128), (7.99, 127), (0.0, 127), (2.0 ** -126, 0), (2.0 ** -140, 0), (3e38, 252),
                    (float("inf"), 255), (float("nan"), 255)):
        row = torch.zeros(1, 32)
        row[0, 3] = amax
        assert mx_ref.quantize(row)[1].item() == b, amax
