"""One MoE layer on one GPU: buffers plus the four C-ABI calls in order.

route -> permute -> expert FFN -> combine ([Moreh-EP] Overview and
Parallelization: gating picks k experts per token, the expert FFNs run on the
tokens routed to them, an always-on shared expert runs on every token, and
the results are combined with the routing weights). This module only
allocates device buffers (torch) and passes pointers to libmoe.so; all
arithmetic happens in the library's kernels.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib as L


@dataclass
class LayerBuffers:
    T: int
    logits: Optional[torch.Tensor]
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    row_to_slot: torch.Tensor
    slot_to_row: torch.Tensor
    x_perm: Optional[torch.Tensor]  # None when fp8 gate/up reads the token rows
    x_perm_scale: Optional[torch.Tensor]
    y_perm: torch.Tensor
    out: torch.Tensor
    ws_perm: torch.Tensor
    ws_ffn: torch.Tensor
    ws_route: Optional[torch.Tensor] = None  # moe_route_select's workspace (large batches)
    # fp8 token codes [T, H] and scales [H/128, T] (moe_quantize_tokens), or MXFP4
    # codes [T, H/2] and scale bytes [T, H/32] (moe_quantize_mxfp4)
    x_tok: Optional[torch.Tensor] = None
    x_tok_scale: Optional[torch.Tensor] = None
    h: Optional[torch.Tensor] = None  # forward_block: the residual stream before the layer
    n: Optional[torch.Tensor] = None  # forward_block: the layer's normed input


@dataclass
class TrainStep:
    """What backward needs of a forward_train: its inputs by reference, and the
    layer's buffers for T training tokens, which the next forward_train of as
    many tokens fills again."""
    x: torch.Tensor
    b: LayerBuffers
    gu: torch.Tensor      # [T*k+T, 2I] gate and up rows; their gradient after backward
    a: torch.Tensor       # [T*k+T, I] gated units
    dx: torch.Tensor      # [T, H]
    dtopk_w: torch.Tensor  # [T, k]
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    routed: bool          # by this layer's router
    routed_here: bool     # and all of its experts are this layer's
    dropout: float
    out_dropout: float
    rng: Optional[torch.Tensor]
    serial: int

    @property
    def out(self) -> torch.Tensor:
        return self.b.out


@dataclass
class LayerGrads:
    """Gradients as backward returns them: of the inputs (dx in the activation
    dtype; topk_w fp32), and of the weights in fp32, shaped as the weights."""
    w13: torch.Tensor
    w2: torch.Tensor
    shared_w13: Optional[torch.Tensor] = None
    shared_w2: Optional[torch.Tensor] = None
    router_w: Optional[torch.Tensor] = None
    router_bias: Optional[torch.Tensor] = None
    dx: Optional[torch.Tensor] = None
    topk_w: Optional[torch.Tensor] = None


class MoELayer:
    """Weights of one GPU's expert share (+ optional shared expert and router).

    fmt: "f32", "bf16", "fp8" or "mxfp4". Expert weights are device tensors
    w13 [E_local, 2I, H], w2 [E_local, H, I] (uint8 e4m3 codes for fp8, with
    w13_scale [E_local, 2I/128, H/128], w2_scale [E_local, H/128, I/128];
    uint8 codes [E_local, 2I, H/2], [E_local, H, I/2] for mxfp4, with scale
    bytes w13_scale [E_local, 2I, H/32], w2_scale [E_local, H, I/32], as
    quantize_mxfp4 makes them).
    router: dict(w=[E, H], bias=[E] or None, scoring, renormalize) or None
    when the routing is handed in (expert-parallel share).

    Calls for the same number of tokens share their buffers and workspaces, the
    outputs among them: calls of one layer must not overlap on two streams, and
    a result is read or copied before the next call.
    """

    def __init__(self, fmt: str, H: int, I: int, k: int, w13, w2, w13_scale=None, w2_scale=None,
                 shared: Optional[dict] = None, router: Optional[dict] = None, expert_base: int = 0):
        self.fmt = fmt
        self.H, self.I, self.k = H, I, k
        self.E_local = w13.shape[0]
        self.expert_base = expert_base
        self.dt = {"f32": L.F32, "bf16": L.BF16, "fp8": L.FP8_E4M3, "mxfp4": L.MXFP4}[fmt]
        self.act_dt = L.F32 if fmt == "f32" else L.BF16
        self.w13, self.w2, self.w13_scale, self.w2_scale = w13, w2, w13_scale, w2_scale
        self.shared = shared
        self.router = router
        sh = shared or {}
        if fmt == "mxfp4":
            self._check_mxfp4(sh)
        self.weights = L.make_weights(self.dt, self.E_local, H, I, w13, w2, w13_scale, w2_scale,
                                      sh.get("w13"), sh.get("w2"), sh.get("w13_scale"),
                                      sh.get("w2_scale"))
        self.n_groups = self.E_local + (1 if shared is not None else 0)
        self._bufs = {}
        self._trains = set()  # (tokens, routed by the layer) whose sizes the training calls take

    def _check_mxfp4(self, sh: dict):
        """Codes and scale bytes of the sizes that the kernels read; the
        shared expert's with or without a leading dimension of 1."""
        E, H, I = self.E_local, self.H, self.I
        sizes = dict(w13=(2 * I, H // 2), w2=(H, I // 2), w13_scale=(2 * I, H // 32), w2_scale=(H, I // 32))
        for name, size in sizes.items():
            given = [(name, getattr(self, name), ((E, *size),))]
            if self.shared is not None:
                given.append((f"shared {name}", sh.get(name), (size, (1, *size))))
            for label, t, shapes in given:
                if t is None or t.element_size() != 1 or tuple(t.shape) not in shapes:
                    have = "missing" if t is None else f"{t.dtype} of shape {tuple(t.shape)}"
                    raise ValueError(f"{label}: {have}, expected bytes of shape {shapes[0]}")

    # fp8 layers with a shared expert quantise each token once and let gate/up
    # read its token's row (moe_quantize_tokens + moe_expert_ffn_gate_up_tokens)
    # instead of copying every routed row into x_perm; the result is the same
    # bit for bit. Without a shared group moe_permute quantises each routed row
    # straight from x in one pass, and gate/up on the contiguous rows is faster
    # than the gathered reads. mxfp4 layers always read token rows (a row is a
    # quarter of its bf16 copy).
    FP8_FROM_TOKENS = True

    def uses_tokens(self) -> bool:
        return self.fmt == "mxfp4" or (self.fmt == "fp8" and self.FP8_FROM_TOKENS and self.shared is not None)

    # Batches of at least this many tokens route through moe_route_select
    # (same ids and weights as moe_route; faster once the MFMA pass has a few
    # thousand tokens, slower for a decode batch). The logits buffer is then
    # left unfilled.
    ROUTE_SELECT_MIN_T = 4096

    def uses_route_select(self, T: int) -> bool:
        r = self.router
        if r is None or self.act_dt != L.BF16 or T < self.ROUTE_SELECT_MIN_T:
            return False
        E = r["w"].shape[0]
        return (self.H % 32 == 0 and self.H <= 8192 and E <= 256
                and (r["scoring"] == L.SIGMOID or r.get("renormalize", True)))

    # ------------------------------------------------------------------ buffers
    def buffers(self, T: int, device=None, key=None) -> LayerBuffers:
        key = T if key is None else key
        if key not in self._bufs:
            self._bufs[key] = self._new_buffers(T, device or self.w13.device)
        return self._bufs[key]

    def _new_buffers(self, T: int, device, training: bool = False) -> LayerBuffers:
        """For training without the workspaces of the steps that it does not call: the
        fused experts' intermediate alone is as large as that many rows of I."""
        k, H = self.k, self.H
        cap = T * k + T
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        act = torch.float32 if self.fmt == "f32" else torch.bfloat16
        E = self.router["w"].shape[0] if self.router is not None else 0
        xdt = torch.uint8 if self.fmt == "fp8" else act
        ws_p = L.moe_permute_workspace_size(T, k, self.E_local)
        ws_f = 0 if training else L.moe_expert_ffn_workspace_size(self.weights, cap)
        b = LayerBuffers(
            T=T,
            logits=torch.empty((T, E), **f32) if E else None,
            topk_ids=torch.empty((T, k), **i32),
            topk_w=torch.empty((T, k), **f32),
            counts=torch.empty(self.E_local + 1, **i32),
            offsets=torch.empty(self.E_local + 2, **i32),
            row_to_slot=torch.empty(cap, **i32),
            slot_to_row=torch.empty(T * k, **i32),
            x_perm=None if self.uses_tokens() else torch.empty((cap, H), dtype=xdt, device=device),
            x_perm_scale=(torch.empty((H // 128, cap), **f32)
                          if self.fmt == "fp8" and not self.uses_tokens() else None),
            y_perm=torch.empty((cap, H), dtype=act, device=device),
            out=torch.empty((T, H), dtype=act, device=device),
            ws_perm=torch.empty(max(ws_p, 1), dtype=torch.uint8, device=device),
            ws_ffn=torch.empty(max(ws_f, 1), dtype=torch.uint8, device=device),
        )
        if self.uses_tokens():
            if self.fmt == "mxfp4":
                b.x_tok = torch.empty((T, H // 2), dtype=torch.uint8, device=device)
                b.x_tok_scale = torch.empty((T, H // 32), dtype=torch.uint8, device=device)
            else:
                b.x_tok = torch.empty((T, H), dtype=torch.uint8, device=device)
                b.x_tok_scale = torch.empty((H // 128, T), **f32)
        if self.uses_route_select(T) and not training:
            b.ws_route = torch.empty(L.moe_route_select_workspace_size(T, E), dtype=torch.uint8,
                                     device=device)
        return b

    # ------------------------------------------------------------------ steps
    def route(self, x: torch.Tensor, b: LayerBuffers, stream=None):
        r = self.router
        T, H = x.shape
        E = r["w"].shape[0]
        if b.ws_route is not None:
            L.moe_route_select(x, r["w"], r.get("bias"), self.act_dt, T, H, E, self.k, r["scoring"],
                               r.get("renormalize", True), b.topk_ids, b.topk_w, b.ws_route,
                               b.ws_route.numel(), stream)
        else:
            L.moe_route(x, r["w"], r.get("bias"), self.act_dt, T, H, E, self.k, r["scoring"],
                        r.get("renormalize", True), b.logits, b.topk_ids, b.topk_w, stream)

    def permute(self, x: torch.Tensor, b: LayerBuffers, topk_ids=None, stream=None):
        T = x.shape[0]
        ids = b.topk_ids if topk_ids is None else topk_ids
        L.moe_permute(ids, T, self.k, self.expert_base, self.E_local, self.shared is not None, x,
                      self.act_dt, self.H, self.dt if self.fmt == "fp8" else self.act_dt, b.counts,
                      b.offsets, b.row_to_slot, b.slot_to_row, b.x_perm, b.x_perm_scale, b.ws_perm,
                      b.ws_perm.numel(), stream)
        if self.fmt == "mxfp4":
            L.moe_quantize_mxfp4(x, self.act_dt, T, self.H, b.x_tok, b.x_tok_scale, stream)
        elif self.uses_tokens():
            L.moe_quantize_tokens(x, self.act_dt, T, self.H, b.x_tok, b.x_tok_scale, stream)

    def gate_up(self, b: LayerBuffers, stream=None):
        cap = b.T * self.k + b.T
        if self.uses_tokens():
            L.moe_expert_ffn_gate_up_tokens(self.weights, b.x_tok, b.x_tok_scale, b.T, self.k,
                                            b.row_to_slot, b.offsets, self.n_groups, cap, b.ws_ffn,
                                            b.ws_ffn.numel(), stream)
        else:
            L.moe_expert_ffn_gate_up(self.weights, b.x_perm, b.x_perm_scale, b.offsets,
                                     self.n_groups, cap, b.ws_ffn, b.ws_ffn.numel(), stream)

    def down(self, b: LayerBuffers, stream=None):
        cap = b.T * self.k + b.T
        L.moe_expert_ffn_down(self.weights, b.offsets, self.n_groups, cap, b.y_perm, b.ws_ffn,
                              b.ws_ffn.numel(), stream)

    def ffn(self, b: LayerBuffers, stream=None):
        self.gate_up(b, stream)
        self.down(b, stream)

    def combine(self, b: LayerBuffers, topk_w=None, stream=None):
        w = b.topk_w if topk_w is None else topk_w
        L.moe_combine(b.y_perm, self.act_dt, b.slot_to_row, w, b.T, self.k, self.H, b.offsets,
                      self.E_local if self.shared is not None else -1, b.out, self.act_dt, stream)

    def check_inputs(self, x: torch.Tensor, topk_ids=None, topk_w=None):
        """x must be [T, H] in the layer's activation dtype on the weights'
        device, which is the current one; given routing must be int32 ids and
        fp32 weights [T, k]."""
        act = torch.float32 if self.fmt == "f32" else torch.bfloat16
        dev = self.w13.device
        L.expect(x, "x", (act,), dev)
        if x.is_cuda and x.get_device() != torch.cuda.current_device():
            raise ValueError(f"x: on {x.device}, the current device is cuda:{torch.cuda.current_device()}")
        if x.dim() != 2 or x.shape[1] != self.H:
            raise ValueError(f"x: shape {tuple(x.shape)}, expected [T, {self.H}]")
        if (topk_ids is None) != (topk_w is None):
            raise ValueError("routing must be given as both topk_ids and topk_w, or neither")
        if topk_ids is None and self.router is None:
            raise ValueError("the layer has no router: pass topk_ids and topk_w")
        for t, name, dt in ((topk_ids, "topk_ids", torch.int32), (topk_w, "topk_w", torch.float32)):
            if t is not None:
                L.expect(t, name, (dt,), dev)
                if tuple(t.shape) != (x.shape[0], self.k):
                    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{x.shape[0]}, {self.k}]")

    # the one-launch layer (moe_layer_fused) takes batches up to this size
    FUSED_MAX_T = 256

    def fused_workspace(self, T: int) -> torch.Tensor:
        """The fused layer's workspace for T tokens, zeroed once at allocation
        (its barrier words must start at zero; every call leaves them so)."""
        key = ("fused", T)
        if key not in self._bufs:
            E = self.router["w"].shape[0]
            n = L.moe_layer_fused_workspace_size(self.weights, T, E, self.k)
            self._bufs[key] = torch.zeros(max(n, 256), dtype=torch.uint8, device=self.w13.device)
        return self._bufs[key]

    def forward_fused(self, x: torch.Tensor, stream=None) -> LayerBuffers:
        """The whole layer in one launch (routing by this layer's router, all
        experts local): the same ids, weights and output as forward()."""
        self.check_inputs(x)
        T = x.shape[0]
        b = self.buffers(T, x.device)
        ws = self.fused_workspace(T)
        r = self.router
        L.moe_layer_fused(x, r["w"], r.get("bias"), T, r["w"].shape[0], self.k, r["scoring"],
                          r.get("renormalize", True), self.weights, b.topk_ids, b.topk_w, b.out, ws,
                          ws.numel(), stream)
        return b

    # forward_few takes batches of mxfp4 experts up to this size; forward and
    # forward_block run the separate steps at every size
    FEW_MAX_T = 16

    def uses_few(self, T: int, routed: bool = False) -> bool:
        """Whether forward_few takes T tokens (moe_layer_few's limits), routed
        by this layer or, with routed=True, by the caller."""
        return (self.fmt == "mxfp4" and T <= self.FEW_MAX_T and self.k <= 8 and self.E_local <= 512
                and self.H % 256 == 0 and self.H <= 8192 and self.I % 128 == 0 and self.I <= 16384
                and (routed or (self.router is not None and self.router["w"].shape[0] <= 256)))

    def few_workspace(self, T: int) -> torch.Tensor:
        """forward_few's workspace for T tokens."""
        key = ("few", T)
        if key not in self._bufs:
            n = L.moe_layer_few_workspace_size(self.weights, T, self._n_experts(), self.k)
            self._bufs[key] = torch.empty(max(n, 256), dtype=torch.uint8, device=self.w13.device)
        return self._bufs[key]

    def _n_experts(self) -> int:
        return self.router["w"].shape[0] if self.router is not None else max(self.expert_base + self.E_local, self.k)

    def forward_few(self, x: torch.Tensor, topk_ids=None, topk_w=None, stream=None) -> LayerBuffers:
        """The layer for at most 16 tokens with mxfp4 experts (moe_layer_few):
        forward's ids and weights, and its output without the expert outputs'
        rounding to bf16. The fp32 sums are taken in another order, so an
        element of the intermediate that lies next to a rounding threshold may
        get the neighbouring 4-bit code or block scale."""
        self.check_inputs(x, topk_ids, topk_w)
        T = x.shape[0]
        b = self.buffers(T, x.device)
        ws = self.few_workspace(T)
        r = self.router if topk_ids is None else None
        L.moe_layer_few(x, r["w"] if r else None, r.get("bias") if r else None, T, self._n_experts(), self.k,
                        r["scoring"] if r else L.SIGMOID, r.get("renormalize", True) if r else True, self.weights,
                        self.expert_base, b.topk_ids if r else topk_ids, b.topk_w if r else topk_w, b.out, ws,
                        ws.numel(), stream)
        return b

    def forward(self, x: torch.Tensor, topk_ids=None, topk_w=None, stream=None) -> LayerBuffers:
        """The whole layer. Routing comes from the router unless given."""
        self.check_inputs(x, topk_ids, topk_w)
        b = self.buffers(x.shape[0], x.device)
        if topk_ids is None:
            self.route(x, b, stream)
        self.permute(x, b, topk_ids, stream)
        self.ffn(b, stream)
        self.combine(b, topk_w, stream)
        return b

    def forward_block(self, x: torch.Tensor, delta=None, *, delta_scale: float = 1.0, gain=None, post_gain=None,
                      eps: float = 1e-6, gate=None, alpha: float = 1.0, stream=None) -> LayerBuffers:
        """The block around the layer: h = x + delta_scale * delta and its RMS
        norm with `gain` (moe_pre_norm), the layer on the normed rows, then
        h + alpha * gate * norm(combine) (moe_combine_norm; no post norm when
        post_gain is None). gain, post_gain [H] fp32; gate [1, H] or [T, H] in
        the layer's activation dtype. b.h holds h, b.n the normed rows, b.out
        the block's output.

        Where this GPU holds a part of the router's experts, the combine is this
        part's sum: b.out is then h + alpha * gate * that sum, and h (and the
        shared expert, if the layer has it) is in every GPU's output. The norm
        of the whole sum cannot be had from norms of its parts, so post_gain is
        refused there."""
        self.check_inputs(x)
        if post_gain is not None and self.router["w"].shape[0] != self.E_local:
            raise ValueError(f"post_gain: the layer holds {self.E_local} of {self.router['w'].shape[0]} experts, and "
                             "the norm of a partial sum is not a part of the sum's norm")
        act, dev = x.dtype, self.w13.device
        for t, name, dt in ((delta, "delta", act), (gain, "gain", torch.float32),
                            (post_gain, "post_gain", torch.float32), (gate, "gate", act)):
            L.expect(t, name, (dt,), dev)
        T, H = x.shape
        for t, name, shapes in ((delta, "delta", ((T, H),)), (gain, "gain", ((H,),)), (post_gain, "post_gain", ((H,),)),
                                (gate, "gate", ((1, H), (T, H)))):
            if t is not None and tuple(t.shape) not in shapes:
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected one of {shapes}")
        b = self.buffers(T, x.device)
        if b.h is None:
            b.h, b.n = torch.empty_like(x), torch.empty_like(x)
        L.moe_pre_norm(x, delta, delta_scale, gain, eps, self.act_dt, T, H, b.h, b.n, stream)
        self.route(b.n, b, stream)
        self.permute(b.n, b, None, stream)
        self.ffn(b, stream)
        L.moe_combine_norm(b.y_perm, self.act_dt, b.slot_to_row, b.topk_w, T, self.k, H, b.offsets,
                           self.E_local if self.shared is not None else -1, post_gain, eps, gate,
                           1 if gate is None else gate.shape[0], alpha, b.h, b.out, self.act_dt, stream)
        return b

    # ------------------------------------------------------------------ training
    def _check_train(self, T: int, routed: bool):
        """Everything about the layer and T that a step's calls refuse, ahead of the first of them."""
        if self.fmt not in ("f32", "bf16"):
            raise ValueError(f"training needs f32 or bf16 weights, not {self.fmt}")
        if (T, routed) in self._trains:
            return
        unit = 8 if self.fmt == "bf16" else 4
        sizes = dict(H=self.H, I=self.I)
        if routed and self.router is not None:  # the gate's products run along the experts
            sizes["the router's experts"] = self.router["w"].shape[0]
        for name, n in sizes.items():
            if n % unit:
                raise ValueError(f"training in {self.fmt}: {name} = {n} is not a multiple of {unit}")
        if T * self.k + T > 1 << 30:
            raise ValueError(f"training: {T} tokens of {self.k} picks are more than 2^30 rows")
        sh, dt = self.shared or {}, self.act_dt
        for name, t in (("w13", self.w13), ("w2", self.w2), ("shared w13", sh.get("w13")), ("shared w2", sh.get("w2"))):
            self._check_aligned(t, name)
        # the calls without tokens: they check their sizes, and launch nothing
        if routed and self.router is not None:
            r = self.router
            L.moe_route(None, None, None, dt, 0, self.H, r["w"].shape[0], self.k, r["scoring"],
                        r.get("renormalize", True), None, None, None, 0)
        L.moe_permute(None, 0, self.k, self.expert_base, self.E_local, self.shared is not None, None, dt, self.H, dt, None,
                      None, None, None, None, None, None, 0, 0)
        for N, K in ((2 * self.I, self.H), (self.H, self.I)):
            L.moe_grouped_gemm(None, None, None, dt, None, self.n_groups, 0, N, K, None, dt, False, 0)
        L.moe_combine(None, dt, None, None, 0, self.k, self.H, None, -1, None, dt, 0)
        self._trains.add((T, routed))

    @staticmethod
    def _check_aligned(t, name: str):
        if t is not None and t.data_ptr() % 16:
            raise ValueError(f"{name}: not 16-byte aligned, as the grouped products need it")

    def _check_rng(self, rng, *p):
        if any(p):
            if rng is None:
                raise ValueError("dropout needs rng")
            L.expect(rng, "rng", (torch.int64,), self.w13.device)
            if tuple(rng.shape) != (2, 2):
                raise ValueError(f"rng: shape {tuple(rng.shape)}, expected (2, 2)")
            for each in p:
                if not 0.0 <= each <= 0.99:  # the library's check of p alone: no elements, nothing to launch
                    L.moe_dropout(None, None, self.act_dt, 0, each, rng.data_ptr(), None, 0)

    def _check_apart(self, x, residual):
        """The step writes its buffers before it reads the residual (which may lie in
        what backward alone writes) and before backward reads x."""
        forward, backward = self._bufs.get(("written", x.shape[0]), ((), ()))
        for t, name, own in ((x, "x", forward + backward), (residual, "residual", forward)):
            if t is None:
                continue
            first = t.data_ptr()
            past = first + t.numel() * t.element_size()
            if any(first < end and at < past for at, end in own):
                raise ValueError(f"{name}: lies in the layer's buffers for {x.shape[0]} tokens, which the step writes (pass "
                                 "a copy)")

    def forward_train(self, x: torch.Tensor, topk_ids=None, topk_w=None, *, dropout: float = 0.0, residual=None,
                      out_dropout: float = 0.0, rng=None, stream=None) -> TrainStep:
        """The layer with what its gradients need kept (f32 and bf16 weights):
        out = residual + drop(combine(...)), with `dropout` inside the experts (on
        the gated units) and `out_dropout` on the layer's output. rng: int64
        [2, 2] on the device, seed and offset of the experts' dropout and of the
        output's, read when the calls run and again by backward, so it changes
        only after backward. x is read again by backward. One step per number of
        tokens: the next forward_train of as many tokens takes its buffers, out
        among them, so neither x nor residual may be in them. The first of a size
        makes them and waits for the device; it is not captured.

        Where this GPU holds a part of the router's experts, out is residual +
        drop(this part's sum): hand the residual (and the shared expert) to one
        GPU. out_dropout goes over the sum if all of them draw from the same
        rng[1]. rng[0] counts this GPU's rows, so equal ones repeat each other's
        masks inside the experts: give each GPU its own."""
        self._check_train(x.shape[0] if x.dim() else 0, topk_ids is None)
        self.check_inputs(x, topk_ids, topk_w)
        self._check_rng(rng, dropout, out_dropout)
        T = x.shape[0]
        L.expect(residual, "residual", (x.dtype,), x.device)
        if residual is not None and residual.shape != x.shape:
            raise ValueError(f"residual: shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
        self._check_apart(x, residual)
        step = self._train_step(x, topk_ids, topk_w, dropout, out_dropout, rng)
        b, r, cap, dt = step.b, self.router, T * self.k + T, self.act_dt
        if topk_ids is None:  # at every size by moe_route, which leaves the logits that the gate's gradient reads
            L.moe_route(x, r["w"], r.get("bias"), dt, T, self.H, r["w"].shape[0], self.k, r["scoring"],
                        r.get("renormalize", True), b.logits, b.topk_ids, b.topk_w, stream)
        self.permute(x, b, step.topk_ids, stream)
        sh = self.shared or {}
        L.moe_grouped_gemm(b.x_perm, self.w13, sh.get("w13"), dt, b.offsets, self.n_groups, cap, 2 * self.I, self.H,
                           step.gu, dt, False, stream)
        L.moe_swiglu(step.gu, dt, self._n_rows(b), cap, self.I, dropout, rng if dropout else None, step.a, stream)
        L.moe_grouped_gemm(step.a, self.w2, sh.get("w2"), dt, b.offsets, self.n_groups, cap, self.H, self.I, b.y_perm,
                           dt, False, stream)
        self.combine(b, step.topk_w, stream)
        if residual is not None or out_dropout:
            L.moe_dropout(b.out, residual, dt, b.out.numel(), out_dropout, rng[1] if out_dropout else None,
                          b.out, stream)
        return step

    def _n_rows(self, b: LayerBuffers):
        return b.offsets[self.n_groups:]  # rows in use

    def _train_step(self, x, topk_ids, topk_w, dropout, out_dropout, rng) -> TrainStep:
        T, dev = x.shape[0], x.device
        key = ("train buffers", T)
        if key not in self._bufs:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError(f"the first forward_train of {T} tokens makes the layer's buffers: run it once before "
                                   "the capture")
            b, cap = self._new_buffers(T, dev, training=True), T * self.k + T
            rest = dict(gu=torch.empty((cap, 2 * self.I), dtype=x.dtype, device=dev),
                        a=torch.empty((cap, self.I), dtype=x.dtype, device=dev),
                        dx=torch.empty_like(x), dtopk_w=torch.empty_like(b.topk_w))
            # constants: one for each pick and, for column sums, eight for each token; the gate's one group and its buffers
            E = self.router["w"].shape[0] if self.router is not None else 0
            constants = (
                torch.ones((T, self.k), dtype=torch.float32, device=dev), torch.ones((T, 8), dtype=x.dtype, device=dev),
                torch.tensor([0, T], dtype=torch.int32, device=dev), torch.empty((T, E), dtype=x.dtype, device=dev),
                torch.empty((E, 8), dtype=torch.float32, device=dev))
            # from where to where the buffers lie, those that backward alone writes apart
            own = {n: (t.data_ptr(), t.data_ptr() + t.nbytes) for n, t in {**vars(b), **rest}.items()
                   if isinstance(t, torch.Tensor)}
            last = tuple(own.pop(n) for n in ("dx", "dtopk_w"))
            torch.cuda.current_stream().synchronize()  # the constants are there for every stream
            # all of them or, where memory ran out on the way, none
            self._bufs.update({("train", T): b, key: rest, ("constants", T): constants, ("serial", T): 0,
                               ("written", T): (tuple(own.values()), last)})
        b = self._bufs[("train", T)]
        self._bufs[("serial", T)] += 3  # its backward and gate_backward move it on by one each
        here = topk_ids is None
        return TrainStep(x=x, b=b, **self._bufs[key], topk_ids=b.topk_ids if here else topk_ids,
                         topk_w=b.topk_w if here else topk_w, routed=here,
                         routed_here=here and self.router["w"].shape[0] == self.E_local, dropout=dropout,
                         out_dropout=out_dropout, rng=rng, serial=self._bufs[("serial", T)])

    def _holds(self, step: TrainStep, calls: int) -> bool:
        """Whether this layer's buffers hold the step after `calls` of its backward and gate_backward."""
        T = step.x.shape[0]
        return step.b is self._bufs.get(("train", T)) and self._bufs[("serial", T)] == step.serial + calls

    def new_grads(self) -> LayerGrads:
        """Zeroed weight gradients, to pass to backward."""
        def zeros(t):
            return None if t is None else torch.zeros(t.shape, dtype=torch.float32, device=t.device)
        sh, r = self.shared or {}, self.router or {}
        return LayerGrads(zeros(self.w13), zeros(self.w2), zeros(sh.get("w13")), zeros(sh.get("w2")), zeros(r.get("w")),
                          zeros(r.get("bias")))

    def _check_grads(self, grads: LayerGrads):
        sh, r = self.shared or {}, self.router or {}
        for name, like in (("w13", self.w13), ("w2", self.w2), ("shared_w13", sh.get("w13")),
                           ("shared_w2", sh.get("w2")), ("router_w", r.get("w")), ("router_bias", r.get("bias"))):
            t = getattr(grads, name)
            if like is None:
                continue
            if t is None or t.shape != like.shape:
                raise ValueError(f"grads.{name}: {'missing' if t is None else tuple(t.shape)}, expected {tuple(like.shape)}")
            L.expect(t, f"grads.{name}", (torch.float32,), like.device)
            if name != "router_bias":
                self._check_aligned(t, f"grads.{name}")

    def backward(self, step: TrainStep, dout: torch.Tensor, grads: Optional[LayerGrads] = None,
                 accumulate: bool = False, stream=None) -> LayerGrads:
        """Gradients of a step from its output's gradient dout [T, H] (the
        residual's is dout itself). The weights' go to `grads` (new_grads()
        unless given), added to what is there with accumulate; dx and topk_w are
        the layer's buffers. Where the step was routed by this layer's router
        over experts that are all here, the gate's part is in dx and in router_w
        and router_bias. Otherwise grads.topk_w is what its weights got here:
        with routing handed in, the caller's to carry on; on an expert share,
        summed over the GPUs that share the experts and given to gate_backward
        (dx is then this share's part of a sum as well). A step's buffers hold its
        gradients afterwards: one backward per step."""
        T, b, dt, H, I = step.x.shape[0], step.b, self.act_dt, self.H, self.I
        if not self._holds(step, 0):
            raise RuntimeError("the step's buffers hold a later step or its gradients")
        L.expect(dout, "dout", (step.x.dtype,), step.x.device)
        if dout.shape != step.x.shape:
            raise ValueError(f"dout: shape {tuple(dout.shape)}, expected {tuple(step.x.shape)}")
        if grads is None:
            if accumulate:
                raise ValueError("accumulate needs the gradients to add to")
            with self._on(stream):  # zeroed there, ahead of what is written
                grads = self.new_grads()
        self._check_grads(grads)
        if step.routed_here:
            self._check_aligned(self.router["w"], "the router's w")
        self._bufs[("serial", T)] += 1
        sh, cap, n = self.shared or {}, T * self.k + T, self.n_groups
        if step.out_dropout:
            L.moe_dropout(dout, None, dt, dout.numel(), step.out_dropout, step.rng[1], step.dx, stream)
            dout = step.dx
        dy = b.y_perm
        L.moe_combine_grad(dout, b.y_perm, dt, b.slot_to_row, step.topk_w, T, self.k, H, b.offsets,
                           self.E_local if self.shared is not None else -1, dy, step.dtopk_w, stream)
        # a's buffer takes its gradient, and a again from gu, whose buffer takes its own
        L.moe_grouped_gemm_dx(dy, self.w2, sh.get("w2"), dt, b.offsets, n, cap, H, I, step.a, dt, False, stream)
        L.moe_swiglu_grad(step.gu, step.a, dt, self._n_rows(b), cap, I, step.dropout,
                          step.rng if step.dropout else None, step.gu, step.a, stream)
        L.moe_grouped_gemm_dw(dy, step.a, dt, b.offsets, n, cap, H, I, grads.w2, grads.shared_w2, L.F32, accumulate,
                              stream)
        L.moe_grouped_gemm_dw(step.gu, b.x_perm, dt, b.offsets, n, cap, 2 * I, H, grads.w13, grads.shared_w13, L.F32,
                              accumulate, stream)
        L.moe_grouped_gemm_dx(step.gu, self.w13, sh.get("w13"), dt, b.offsets, n, cap, 2 * I, H, dy, dt, False, stream)
        # the rows are copies of their tokens' x: the copies' gradients summed
        L.moe_combine(dy, dt, b.slot_to_row, self._bufs[("constants", T)][0], T, self.k, H, b.offsets,
                      self.E_local if self.shared is not None else -1, step.dx, dt, stream)
        grads.dx, grads.topk_w = step.dx, step.dtopk_w
        if step.routed_here:
            self._gate_backward(step, step.dtopk_w, grads, accumulate, stream)
        return grads

    def gate_backward(self, step: TrainStep, dtopk_w: torch.Tensor, grads: LayerGrads, accumulate: bool = False,
                      stream=None):
        """The gate's part of a step's gradients from those of its picks'
        weights [T, k]: added to grads.dx, and router_w and router_bias. backward
        calls it unless the experts are shared with other GPUs; there it belongs
        into the sum of their dx once. It reads the step's logits and picks, so it
        comes after the step's backward and before the next forward_train of as
        many tokens, once. grads.dx may be another tensor than backward's (a sum
        over GPUs)."""
        r, T = self.router, step.x.shape[0]
        if r is None or not step.routed:
            raise ValueError("the step was not routed by this layer's router")
        if not self._holds(step, 1):
            raise RuntimeError("the layer's buffers hold this step's backward no longer, or not yet, or its gate's part "
                               "is made already")
        L.expect(dtopk_w, "dtopk_w", (torch.float32,), step.x.device)
        if tuple(dtopk_w.shape) != (T, self.k):
            raise ValueError(f"dtopk_w: shape {tuple(dtopk_w.shape)}, expected [{T}, {self.k}]")
        self._check_grads(grads)
        if grads.dx is None or grads.dx.shape != step.x.shape:
            raise ValueError("grads.dx: backward's, of this step, is needed")
        L.expect(grads.dx, "grads.dx", (step.x.dtype,), step.x.device)
        self._check_aligned(grads.dx, "grads.dx")
        self._check_aligned(r["w"], "the router's w")
        self._gate_backward(step, dtopk_w, grads, accumulate, stream)

    def _gate_backward(self, step: TrainStep, dtopk_w: torch.Tensor, grads: LayerGrads, accumulate: bool, stream):
        r, T, dt, H = self.router, step.x.shape[0], self.act_dt, self.H
        self._bufs[("serial", T)] += 1
        E = r["w"].shape[0]
        _, ones, offsets, dlogits, dbias = self._bufs[("constants", T)]
        L.moe_route_grad(step.b.logits, step.topk_ids, dtopk_w, T, E, self.k, r["scoring"], r.get("renormalize", True),
                         dlogits, dt, stream)
        L.moe_grouped_gemm_dx(dlogits, r["w"], None, dt, offsets, 1, T, E, H, grads.dx, dt, True, stream)
        x = step.x
        if x.data_ptr() % 16:  # the other calls take any x
            with self._on(stream):
                x = x.clone()
        L.moe_grouped_gemm_dw(dlogits, x, dt, offsets, 1, T, E, H, grads.router_w, None, L.F32, accumulate, stream)
        if grads.router_bias is not None:  # column sums: a product with columns of ones
            L.moe_grouped_gemm_dw(dlogits, ones, dt, offsets, 1, T, E, 8, dbias, None, L.F32,
                                  False, stream)
            with self._on(stream):
                (grads.router_bias.add_ if accumulate else grads.router_bias.copy_)(dbias[:, 0])

    @staticmethod
    def _on(stream):
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(L.stream_of(stream))


def quantize_mxfp4(x: torch.Tensor, stream=None):
    """(codes [..., K/2], scale bytes [..., K/32]) of a bf16 or fp32 tensor
    [..., K] (moe_quantize_mxfp4), as MoELayer takes expert weights. With a
    stream they are allocated on it, so that memory freed behind the call is
    not handed to other streams' work while that stream may still use it."""
    L.expect(x, "x", (torch.float32, torch.bfloat16))
    K = x.shape[-1] if x.dim() else 0
    if K == 0 or K % 32:
        raise ValueError(f"x: last dimension of shape {tuple(x.shape)} is not a multiple of 32 (32 or more)")
    with MoELayer._on(stream):
        codes = torch.empty(x.shape[:-1] + (K // 2,), dtype=torch.uint8, device=x.device)
        scales = torch.empty(x.shape[:-1] + (K // 32,), dtype=torch.uint8, device=x.device)
    L.moe_quantize_mxfp4(x, L.dtype_code(x), x.numel() // K, K, codes, scales, stream)
    return codes, scales
