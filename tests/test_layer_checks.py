"""MoELayer's own checks of arguments, without a GPU: each refuses before anything is enqueued."""
import pytest
import torch

H, I, E, K = 256, 128, 4, 2


@pytest.fixture(scope="module")
def L():
    import os

    import mixture_experts_layer_select_amd as pkg
    if not os.path.exists(pkg._lib.LIB_PATH):
        pkg.build()
    return pkg


def layer(L, E_local=E, n_router=E, base=0, k=K):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    router = None
    if n_router:
        router = dict(w=torch.zeros((n_router, H), dtype=torch.bfloat16), bias=None, scoring=L.SIGMOID)
    return L.MoELayer("mxfp4", H, I, k, u8(E_local, 2 * I, H // 2), u8(E_local, H, I // 2),
                      u8(E_local, 2 * I, H // 32), u8(E_local, H, I // 32), router=router, expert_base=base)


@pytest.mark.parametrize("base", [0, 4])
def test_post_norm_of_an_expert_share_is_refused(L, base):
    """A share's combine is a partial sum: its norm is no part of the block's."""
    x = torch.zeros((3, H), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="post_gain: the layer holds 4 of 8 experts"):
        layer(L, n_router=8, base=base).forward_block(x, post_gain=torch.ones(H))


def test_uses_few_holds_the_limits_of_the_call(L):
    """Each limit of moe_layer_few from both sides; the router's size counts only where the layer routes."""
    assert all(layer(L).uses_few(T) for T in (0, 1, 16)) and not layer(L).uses_few(17)
    assert layer(L, n_router=256).uses_few(1) and not layer(L, n_router=257).uses_few(1)
    assert layer(L, n_router=257).uses_few(1, routed=True)
    bare = layer(L, n_router=0)
    assert bare.uses_few(16, routed=True) and not bare.uses_few(16)
    assert layer(L, k=8, n_router=8).uses_few(1) and not layer(L, k=9, n_router=9).uses_few(1)
    for key, good, bad in (("E_local", 512, 513), ("H", 8192, 8448), ("H", 512, 384), ("I", 16384, 16512), ("I", 384, 192)):
        m = layer(L)
        setattr(m, key, good)
        assert m.uses_few(1, routed=True), (key, good)
        setattr(m, key, bad)
        assert not m.uses_few(1, routed=True), (key, bad)


class On(torch.Tensor):
    """A host tensor that says it lies on GPU `at`."""

    def get_device(self):
        return self.at


def test_weights_on_two_devices_are_refused(L):
    def on(at):
        t = torch.zeros(1, dtype=torch.uint8).as_subclass(On)
        t.at = at
        return t
    with pytest.raises(ValueError, match=r"several devices: \[0, 1\]"):
        L.make_weights(L.MXFP4, 1, H, I, on(0), on(0), on(0), on(1))
    L.make_weights(L.MXFP4, 1, H, I, on(1), on(1), on(1), on(1))


@pytest.mark.parametrize("shape", [(), (4, 0), (0,), (4, 48), (31,)])
def test_quantize_mxfp4_refuses_rows_that_are_no_blocks(L, shape):
    with pytest.raises(ValueError, match="not a multiple of 32"):
        L.quantize_mxfp4(torch.zeros(shape))


def test_mxfp4_weights_of_other_sizes_are_refused(L):
    """The kernels read what H and I say: a tensor that is smaller, wider or missing is refused when the layer is made."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    good = dict(w13=u8(E, 2 * I, H // 2), w2=u8(E, H, I // 2), w13_scale=u8(E, 2 * I, H // 32), w2_scale=u8(E, H, I // 32))
    shared = {n: t[0] for n, t in good.items()}

    def make(shared=None, **kw):
        w = {**good, **kw}
        return L.MoELayer("mxfp4", H, I, K, w["w13"], w["w2"], w["w13_scale"], w["w2_scale"], shared=shared)
    make()
    make(shared)
    make({n: t[None] for n, t in shared.items()})
    for name, t in good.items():
        bad = [t[:, :-1], t[..., :-1], t.to(torch.int16), torch.cat([t, t], -1), None]
        for b in bad[:-1] if name == "w13" else bad:
            with pytest.raises(ValueError, match=f"^{name}: "):
                make(**{name: b})
        for b in (t, t[0, 1:], t[0].to(torch.float32), None):
            with pytest.raises(ValueError, match=f"^shared {name}: "):
                make({**shared, name: b})
    with pytest.raises(ValueError, match="^w2: "):
        make(w2=good["w2"][:3])  # fewer experts than w13
