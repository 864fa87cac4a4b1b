"""Measured cases of the 4-bit expert path: microscaled (MXFP4) quantisation, the expert FFN on MXFP4
weights, the norms around the block, and the whole layer for a few tokens.

`run` computes a case in elementary torch operations, or, where `own` is true, by the library's calls.
Sizes are those of the R1 layer (H = 7168, I = 2048, top-8 of 256 experts, 32 experts a GPU) and odd
ones beside them.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32            # elements that share one E8M0 scale
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    ffn = dict(op="ffn", H=7168, I=2048, E=256, local=32, k=8)
    norm = dict(H=7168, dtype="bf16")
    few = dict(op="few", H=7168, I=2048, E=256, local=256, k=8, shared=True)
    return [
        # the tokens of a decode step on their way into the experts, an odd number of them
        dict(name="quantize decode", op="quantize", rows=13, cols=7168, dtype="bf16"),
        # one expert's gate and up matrix from a float32 checkpoint
        dict(name="quantize weights", op="quantize", rows=4096, cols=7168, dtype="f32"),
        # 128 tokens of the whole expert-parallel group: about four rows for each local expert
        dict(name="experts decode", **ffn, tokens=128, shared=True),
        # a 4096-token batch of the group: about 127 rows for each local expert
        dict(name="experts share", **ffn, tokens=4096, shared=False),
        # a prompt batch: about 512 rows an expert, matrix-bound
        dict(name="experts prompt", **ffn, tokens=16384, shared=False),
        # a small model's layer: odd row counts, experts that nobody picks
        dict(name="experts small", op="ffn", H=1280, I=384, E=24, local=9, k=2, tokens=203, shared=True),
        # one token before its block
        dict(name="pre norm one", op="pre_norm", T=1, delta=True, **norm),
        # a prompt before its block, an odd number of tokens
        dict(name="pre norm prompt", op="pre_norm", T=16383, delta=True, **norm),
        # a decode step behind its experts, the gate one vector for all tokens
        dict(name="combine norm decode", op="combine_norm", T=16, k=8, shared=True, gate_rows=1, **norm),
        # a prompt behind its experts, a gate for every token
        dict(name="combine norm prompt", op="combine_norm", T=4097, k=8, shared=True, gate_rows=4097, **norm),
        # single-stream decoding
        dict(name="few one", T=1, **few),
        # a handful of streams
        dict(name="few eight", T=8, **few),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "ffn", "pre_norm", "combine_norm", "few"))
    if op == "quantize":
        cols = BLOCK * _log(rng, 1, 256)
        return dict(op=op, rows=_log(rng, 1, max(1, (4096 * 7168) // cols)), cols=cols,
                    dtype=rng.choice(("bf16", "f32")))
    if op == "pre_norm":
        H = _log(rng, 64, 8192)
        return dict(op=op, T=_log(rng, 1, 16000), H=H, dtype=rng.choice(("bf16", "f32")),
                    delta=rng.random() < 0.7)
    if op == "combine_norm":
        T = _log(rng, 1, 4000)
        return dict(op=op, T=T, H=8 * _log(rng, 8, 900), k=rng.randint(1, 8), dtype=rng.choice(("bf16", "f32")),
                    shared=rng.random() < 0.5, gate_rows=rng.choice((1, T)))
    H, I = 256 * rng.randint(2, 28), 128 * rng.randint(1, 16)
    if op == "ffn":
        local = rng.randint(2, 32)
        E = local * rng.randint(1, 8)
        k = rng.randint(1, min(8, E))
        return dict(op=op, H=H, I=I, E=E, local=local, k=k, shared=rng.random() < 0.5,
                    tokens=_log(rng, 1, max(2, 14000 * E // (local * k + E))))
    E = rng.choice((8, 24, 56))
    return dict(op=op, H=H, I=I, E=E, local=E, k=rng.randint(1, 8), shared=rng.random() < 0.5, T=rng.randint(1, 16))


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _pack(v, e):
    """E2M1 codes of v (multiples of the block's 2^e) and the E8M0 bytes, as a checkpoint holds them."""
    m = v.abs() * torch.exp2(-e)
    code = torch.bucketize(m, torch.tensor(E2M1, device=DEV)[1:], right=True) + 8 * (v < 0)
    code = code.to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _weights(g, n, rows, cols):
    codes = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n, rows, cols // BLOCK), dtype=torch.uint8, device=DEV)
    for j in range(n):
        v, e = _mx(torch.randn((rows, cols), generator=g, device=DEV) * 0.02)
        codes[j], scales[j] = _pack(v, e)
    return codes, scales


def _experts(g, case):
    H, I = case["H"], case["I"]
    s = {}
    s["w13"], s["w13_scale"] = _weights(g, case["local"], 2 * I, H)
    s["w2"], s["w2_scale"] = _weights(g, case["local"], H, I)
    if case["shared"]:
        s["ws13"], s["ws13_scale"] = _weights(g, 1, 2 * I, H)
        s["ws2"], s["ws2_scale"] = _weights(g, 1, H, I)
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "quantize":
        x = torch.randn((case["rows"], case["cols"]), generator=g, device=DEV)
        s["x"] = (x * torch.exp2(torch.randn((case["rows"], 1), generator=g, device=DEV))).to(_dtype(case))
    elif op == "pre_norm":
        T, H, dt = case["T"], case["H"], _dtype(case)
        s["x"] = _randn(g, (T, H), 1.5, dt)
        s["delta"] = _randn(g, (T, H), 0.7, dt) if case["delta"] else None
        s["gain"] = 1.0 + _randn(g, (H,), 0.1, torch.float32)
    elif op == "combine_norm":
        T, H, k, dt = case["T"], case["H"], case["k"], _dtype(case)
        # every pick local but one in sixteen, rows in a shuffled order, shared rows behind them
        local = torch.rand(T * k, generator=g, device=DEV) < 15 / 16
        order = torch.randperm(T * k, generator=g, device=DEV)
        rank = torch.empty_like(order)
        rank[order[local[order]]] = torch.arange(int(local.sum()), device=DEV)
        s["slot_to_row"] = torch.where(local, rank, torch.full_like(rank, -1)).to(torch.int32)
        R = int(local.sum())
        s["offsets"] = torch.tensor([0, R, R + T], dtype=torch.int32, device=DEV)
        s["y"] = _randn(g, (T * k + T, H), 0.4, dt)
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        s["topk_w"] = w / w.sum(1, keepdim=True)
        s["gain"] = 1.0 + _randn(g, (H,), 0.1, torch.float32)
        s["gate"] = _randn(g, (case["gate_rows"], H), 0.5, dt)
        s["residual"] = _randn(g, (T, H), 1.5, dt)
    elif op == "ffn":
        # a batch of the expert-parallel group, uniform picks; this GPU keeps the tokens that pick one
        # of its experts. How many rows each expert gets belongs to the case, which tokens they are to the seed.
        ids = torch.rand((case["tokens"], case["E"]), generator=_gen(5), device=DEV).topk(case["k"], dim=1).indices
        ids = ids[(ids < case["local"]).any(1)]
        ids = ids if len(ids) else torch.arange(case["k"], device=DEV)[None]
        ids = ids[torch.randperm(len(ids), generator=g, device=DEV)]
        T, k = ids.shape
        slots = torch.nonzero((ids < case["local"]).flatten()).flatten()
        slots = slots[torch.sort(ids.flatten()[slots], stable=True).indices]
        counts = torch.bincount(ids.flatten()[slots], minlength=case["local"])
        if case["shared"]:
            slots = torch.cat([slots, T * k + torch.arange(T, device=DEV)])
            counts = torch.cat([counts, torch.tensor([T], device=DEV)])
        s["T"], s["rows"], s["most"] = T, int(counts.sum()), int(counts.max())
        s["row_to_slot"] = slots.to(torch.int32)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["x"] = _randn(g, (T, case["H"]), 1.0, torch.bfloat16)
        s.update(_experts(g, case))
    else:
        s["x"] = _randn(g, (case["T"], case["H"]), 1.0, torch.bfloat16)
        s["router"] = _randn(g, (case["E"], case["H"]), 0.006, torch.bfloat16)
        s["bias"] = _randn(g, (case["E"],), 0.1, torch.float32)
        s.update(_experts(g, case))
    return s


# ---------------------------------------------------------------- plain forms
def _mx(x):
    """The values that MXFP4 holds for x (in blocks of 32, as [..., n, 32]) and each block's exponent."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127).float()
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    m = b.abs() * torch.exp2(-e)
    q = 0.5 * ((m > 0.25).float() + (m >= 0.75) + (m > 1.25) + (m >= 1.75))
    q = q + (m > 2.5) + (m >= 3.5) + 2 * (m > 5).float()
    return torch.copysign(q, b) * torch.exp2(e), e


def _quantized(x):
    return _mx(x)[0].flatten(-2)


def _values(codes, scales):
    """float32 values of packed codes and scale bytes."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(-2).unflatten(-1, (-1, BLOCK))
    return (v * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _both(s, name):
    """Routed weights and, behind them, the shared expert's, as float32 [groups, rows, cols]."""
    w = _values(s[name], s[name + "_scale"])
    shared = "ws" + name[1:]
    return torch.cat([w, _values(s[shared], s[shared + "_scale"])]) if shared in s else w


def _swiglu(h):
    g, u = h.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _plain_ffn(s):
    T, k = s["T"], s["case"]["k"]
    slot = s["row_to_slot"].long()
    token = torch.where(slot < T * k, slot // k, slot - T * k)
    off = s["offsets"].long()
    row = torch.arange(s["rows"], device=DEV)
    group = torch.searchsorted(off[1:], row, right=True)
    at = (group, row - off[group])
    x = torch.zeros((len(off) - 1, s["most"], s["case"]["H"]), device=DEV)
    x[at] = _quantized(s["x"])[token]
    a = _quantized(_swiglu(torch.bmm(x, _both(s, "w13").transpose(1, 2))))
    return torch.bmm(a, _both(s, "w2").transpose(1, 2))[at].to(torch.bfloat16)


def _route(x, s):
    """Gating in 64 bits: picks by logit (ties to the lower index) and their sigmoid weights."""
    logits = x @ s["router"].double().t() + s["bias"].double()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    l, ids = order.values[:, : s["case"]["k"]], order.indices[:, : s["case"]["k"]]
    w = 1 / (1 + torch.exp(-l))
    return ids, w / w.sum(1, keepdim=True)


def _plain_few(s):
    T = s["case"]["T"]
    ids, w = _route(s["x"].double(), s)
    w = w.float()
    hit, where = torch.unique(ids, return_inverse=True)
    p = torch.zeros((T, len(hit)), device=DEV).scatter_add_(1, where, w)
    if s["case"]["shared"]:
        p = torch.cat([p, torch.ones((T, 1), device=DEV)], 1)
    pick = {n: v if n.startswith("ws") else v[hit] for n, v in s.items() if n.startswith(("w13", "w2", "ws"))}
    x = _quantized(s["x"]).expand(p.shape[1], -1, -1)
    a = _quantized(_swiglu(torch.bmm(x, _both(pick, "w13").transpose(1, 2))))
    y = torch.bmm(a, _both(pick, "w2").transpose(1, 2))
    out = (y * p.t()[:, :, None]).sum(0)
    return dict(ids=ids.to(torch.int32), weights=w, out=out.to(torch.bfloat16))


def _combined(s, dt):
    """sum_j w_j y[row_j], non-local picks left out, and the shared expert's row."""
    T, k = s["case"]["T"], s["case"]["k"]
    row = s["slot_to_row"].long().view(T, k)
    w = torch.where(row >= 0, s["topk_w"], torch.zeros_like(s["topk_w"])).to(dt)
    c = (s["y"][row.clamp(min=0)].to(dt) * w[..., None]).sum(1)
    return c + s["y"][s["offsets"][1] + torch.arange(T, device=DEV)].to(dt) if s["case"]["shared"] else c


ALPHA = 0.75          # residual scale of the block's output
DELTA = 0.5           # residual scale of what pre_norm adds


def _plain(s):
    op = s["case"]["op"]
    if op == "quantize":
        return _quantized(s["x"]).to(s["x"].dtype)
    if op == "ffn":
        return _plain_ffn(s)
    if op == "few":
        return _plain_few(s)
    if op == "pre_norm":
        h = s["x"].float()
        if s["delta"] is not None:
            h = h + DELTA * s["delta"].float()
        n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["gain"]
        return dict(h=h.to(s["x"].dtype), n=n.to(s["x"].dtype))
    c = _combined(s, torch.float32)
    n = c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * s["gain"]
    return (s["residual"].float() + ALPHA * s["gate"].float() * n).to(s["residual"].dtype)


# ---------------------------------------------------------------- the library's calls
def _plan(s):
    """What a program makes once for its sizes: buffers, the workspace, the struct of weight pointers."""
    import mixture_experts_layer_select_amd as L
    c = s["case"]
    u8 = dict(dtype=torch.uint8, device=DEV)
    p = dict(L=L)
    if c["op"] == "quantize":
        p["codes"] = torch.empty((c["rows"], c["cols"] // 2), **u8)
        p["scales"] = torch.empty((c["rows"], c["cols"] // BLOCK), **u8)
        p["out"] = torch.empty_like(s["x"])
    elif c["op"] == "pre_norm":
        p["h"], p["n"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    elif c["op"] == "combine_norm":
        p["out"] = torch.empty_like(s["residual"])
    else:
        p["w"] = L.make_weights(L.MXFP4, c["local"], c["H"], c["I"], s["w13"], s["w2"], s["w13_scale"], s["w2_scale"],
                                s.get("ws13"), s.get("ws2"), s.get("ws13_scale"), s.get("ws2_scale"))
        T = s["x"].shape[0]
        if c["op"] == "ffn":
            n = L.moe_expert_ffn_workspace_size(p["w"], s["rows"])
            p["ws"] = torch.empty(max(n, 1), **u8)
            p["codes"] = torch.empty((T, c["H"] // 2), **u8)
            p["scales"] = torch.empty((T, c["H"] // BLOCK), **u8)
            p["y"] = torch.empty((s["rows"], c["H"]), dtype=torch.bfloat16, device=DEV)
        else:
            n = L.moe_layer_few_workspace_size(p["w"], T, c["E"], c["k"])
            p["ws"] = torch.zeros(n, **u8)
            p["ids"] = torch.empty((T, c["k"]), dtype=torch.int32, device=DEV)
            p["weights"] = torch.empty((T, c["k"]), dtype=torch.float32, device=DEV)
            p["out"] = torch.empty_like(s["x"])
    return p


def _own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    p, c = s["plan"], s["case"]
    L = p["L"]
    if c["op"] == "quantize":
        dt = L.dtype_code(s["x"])
        L.moe_quantize_mxfp4(s["x"], dt, c["rows"], c["cols"], p["codes"], p["scales"])
        L.moe_dequantize_mxfp4(p["codes"], p["scales"], c["rows"], c["cols"], p["out"], dt)
        return p["out"]
    if c["op"] == "pre_norm":
        L.moe_pre_norm(s["x"], s["delta"], DELTA, s["gain"], EPS, L.dtype_code(s["x"]), c["T"], c["H"], p["h"], p["n"])
        return dict(h=p["h"], n=p["n"])
    if c["op"] == "combine_norm":
        dt = L.dtype_code(s["y"])
        L.moe_combine_norm(s["y"], dt, s["slot_to_row"], s["topk_w"], c["T"], c["k"], c["H"], s["offsets"],
                           1 if c["shared"] else -1, s["gain"], EPS, s["gate"], c["gate_rows"], ALPHA, s["residual"],
                           p["out"], dt)
        return p["out"]
    if c["op"] == "ffn":
        T, groups = s["T"], len(s["offsets"]) - 1
        L.moe_quantize_mxfp4(s["x"], L.BF16, T, c["H"], p["codes"], p["scales"])
        L.moe_expert_ffn_gate_up_tokens(p["w"], p["codes"], p["scales"], T, c["k"], s["row_to_slot"], s["offsets"],
                                        groups, s["rows"], p["ws"], p["ws"].numel())
        L.moe_expert_ffn_down(p["w"], s["offsets"], groups, s["rows"], p["y"], p["ws"], p["ws"].numel())
        return p["y"]
    L.moe_layer_few(s["x"], s["router"], s["bias"], c["T"], c["E"], c["k"], L.SIGMOID, True, p["w"], 0, p["ids"],
                    p["weights"], p["out"], p["ws"], p["ws"].numel())
    return dict(ids=p["ids"], weights=p["weights"], out=p["out"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work of a pass
def work(case):
    op = case["op"]
    size = 2 if case.get("dtype", "bf16") == "bf16" else 4
    packed = 0.5 + 1 / BLOCK
    if op == "quantize":  # read, packed, read back
        n = case["rows"] * case["cols"]
        return dict(bytes=n * (2 * size + 2 * packed), flops=4 * n)
    if op == "pre_norm":
        n = case["T"] * case["H"]
        return dict(bytes=n * size * (4 if case["delta"] else 3) + 4 * case["H"], flops=6 * n)
    if op == "combine_norm":
        n = case["T"] * case["H"]
        rows = case["k"] * 15 / 16 + (1 if case["shared"] else 0) + 2
        return dict(bytes=size * (n * rows + case["gate_rows"] * case["H"]), flops=2 * n * (rows + 2))
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    T = case["tokens"] if op == "ffn" else case["T"]
    share = case["local"] / E
    hit = case["local"] * (1 - (1 - k / E) ** T) + (1 if case["shared"] else 0)  # distinct experts, in the mean
    if op == "ffn":
        T = T * (1 - (1 - share) ** k)  # tokens that reach this GPU
    rows = (case["tokens"] * k * share if op == "ffn" else T * k) + (T if case["shared"] else 0)
    io = T * H * 2 + (rows * H * 2 if op == "ffn" else T * H * 2 + E * H * 2)
    return dict(bytes=hit * 3 * H * I * packed + io, flops=6 * rows * H * I)


# ---------------------------------------------------------------- 64 bits
def _exact_mx(x):
    """Nearest E2M1 multiple of the block's power of two, ties to the even code, in float64."""
    b = x.double().reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    amax = b.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    e = torch.where(amax > 0, (e - 2).clamp(-127, 127), torch.zeros_like(e))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    m = b.abs() / torch.exp2(e)
    low, high = torch.bucketize(m, middle), torch.bucketize(m, middle, right=True)
    q = grid[torch.where(low % 2 == 0, low, high)]
    return (torch.sign(b) * q * torch.exp2(e)).reshape(x.shape)


def _exact_weight(s, name, j):
    codes, scales = s[name][j].long(), s[name + "_scale"][j].double()
    both = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int64, device=DEV)
    both[:, 0::2], both[:, 1::2] = codes % 16, codes // 16
    v = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[both % 8] * (1 - 2 * (both // 8))
    return v * torch.exp2(scales - 127).repeat_interleave(BLOCK, 1)


def _exact_expert(s, x, j):
    """Rows x (float64, quantised) through expert j, or the shared one (j < 0)."""
    n13, n2, j = ("w13", "w2", j) if j >= 0 else ("ws13", "ws2", 0)
    g, u = torch.split(x @ _exact_weight(s, n13, j).t(), s["case"]["I"], dim=1)
    return _exact_mx(g * torch.sigmoid(g) * u) @ _exact_weight(s, n2, j).t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_mx(s["x"])
    if op == "pre_norm":
        h = s["x"].double() if s["delta"] is None else s["x"].double() + DELTA * s["delta"].double()
        return dict(h=h, n=h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["gain"].double())
    if op == "combine_norm":
        c = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
        for j in range(case["k"]):
            row = s["slot_to_row"][j:: case["k"]].long()
            on = row >= 0
            c[on] += s["topk_w"][on, j, None].double() * s["y"][row[on]].double()
        if case["shared"]:
            a, b = s["offsets"][1:].tolist()
            c += s["y"][a:b].double()
        n = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * s["gain"].double()
        return s["residual"].double() + ALPHA * s["gate"].double() * n
    xq = _exact_mx(s["x"])
    if op == "ffn":
        y = torch.empty((s["rows"], case["H"]), dtype=torch.float64, device=DEV)
        off, n = s["offsets"].tolist(), s["T"] * case["k"]
        for j in range(len(off) - 1):
            if off[j] < off[j + 1]:
                token = [v // case["k"] if v < n else v - n for v in s["row_to_slot"][off[j]:off[j + 1]].tolist()]
                y[off[j]:off[j + 1]] = _exact_expert(s, xq[token], j if j < case["local"] else -1)
        return y
    logits = s["x"].double() @ s["router"].double().t() + s["bias"].double()
    out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
    ids, weights = [], []
    for t in range(case["T"]):
        pick = sorted(range(case["E"]), key=lambda e, row=logits[t].tolist(): (-row[e], e))[: case["k"]]
        w = torch.sigmoid(logits[t, pick])
        ids.append(pick)
        weights.append(w / w.sum())
    for e in sorted({e for pick in ids for e in pick}):
        rows = [t for t in range(case["T"]) if e in ids[t]]
        w = torch.stack([weights[t][ids[t].index(e)] for t in rows])
        out[rows] += w[:, None] * _exact_expert(s, xq[rows], e)
    if case["shared"]:
        out += _exact_expert(s, xq, -1)
    return dict(ids=torch.tensor(ids, dtype=torch.int32), weights=torch.stack(weights), out=out)
