"""Cases of the dense operators beside the MoE layer (the gated block that every
token passes, and products in 8-bit integers), their plain forms in torch, their
definitions in 64 bits, and the calls a program makes of them.

Operators (kind of a case):
  ffn        gated feed-forward block in bf16, added to what the layer gave
  train      the same block, forward and backward
  linear8    tokens quantised to 8-bit integers and multiplied by 8-bit weights
  ffn8       the gated block with both products in 8-bit integers

`own` false: the plain forms run (elementary torch operations in float32,
rounded once at the end).  `own` true: the framework's kernels run.
"""
import torch

own = False

H_V3, I_V3 = 7168, 2048  # hidden and inter of the DeepSeek-V3 layers of moe_inputs


def listed():
    return [
        # one token beside the layer: latency, and a read of the weights
        dict(name="ffn decode 1", kind="ffn", tokens=1, hidden=H_V3, inter=I_V3),
        # the decode workload's batch
        dict(name="ffn decode 64", kind="ffn", tokens=64, hidden=H_V3, inter=I_V3),
        # a ragged batch through a block whose sizes fill no tile
        dict(name="ffn odd 500", kind="ffn", tokens=500, hidden=5128, inter=1368),
        # a long prefill
        dict(name="ffn prefill 16384", kind="ffn", tokens=16384, hidden=H_V3, inter=I_V3),
        # the tiny layer of moe_inputs, trained: latency of the smallest step
        dict(name="train tiny", kind="train", tokens=16, hidden=256, inter=512),
        # a small block on a ragged batch, gradients in bf16
        dict(name="train odd 1003", kind="train", tokens=1003, hidden=1000, inter=2744, grads="bf16"),
        # a packed training batch, one token short of whole tiles three times over
        dict(name="train v3 4093", kind="train", tokens=4093, hidden=H_V3, inter=I_V3),
        # one token through one projection
        dict(name="linear8 decode 1", kind="linear8", tokens=1, k=H_V3, n=I_V3, out="bf16"),
        # float32 results, ragged in every direction
        dict(name="linear8 odd 777", kind="linear8", tokens=777, k=1104, n=5000, out="f32"),
        # a long prefill through a square projection
        dict(name="linear8 prefill 16384", kind="linear8", tokens=16384, k=H_V3, n=H_V3, out="bf16"),
        # the decode workload's batch through the block in 8 bits
        dict(name="ffn8 decode 64", kind="ffn8", tokens=64, hidden=H_V3, inter=I_V3),
        # the prefill workload's batch
        dict(name="ffn8 prefill 4096", kind="ffn8", tokens=4096, hidden=H_V3, inter=I_V3),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["ffn", "train", "linear8", "ffn8"])
    tokens = _log(rng, 1, 4096 if kind == "train" else 16384)
    unit = 16 if kind in ("linear8", "ffn8") else 8  # 16 bytes of a row
    hidden = unit * _log(rng, 128 // unit, H_V3 // unit)
    if kind == "linear8":
        return dict(kind=kind, tokens=tokens, k=hidden, n=8 * _log(rng, 16, H_V3 // 8), out=rng.choice(["f32", "bf16"]))
    c = dict(kind=kind, tokens=tokens, hidden=hidden, inter=unit * _log(rng, 128 // unit, I_V3 // unit))
    if kind == "train":
        c["grads"] = rng.choice(["f32", "bf16"])
    return c


# ---------------------------------------------------------------- inputs
def _quantised(w):
    """8-bit codes and one scale a row, as a program stores its weights."""
    scale = w.abs().amax(dim=1) / 127
    return torch.round(w / scale[:, None]).to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    c, kind, T = case, case["kind"], case["tokens"]
    s = {"case": c, "kept": {}}
    if kind == "linear8":
        # hidden states have a few channels far above the others
        channels = torch.where(torch.rand(c["k"], generator=gen, device="cuda") < 0.01, 8.0, 1.0)
        s["x"] = (randn(T, c["k"]) * channels).bfloat16()
        s["w"], s["w_scales"] = _quantised(randn(c["n"], c["k"]) / c["k"] ** 0.5)
        return s
    H, I = c["hidden"], c["inter"]
    s["x"] = randn(T, H).bfloat16()
    w1 = randn(2 * I, H) / H ** 0.5  # gate rows, then up rows
    w2 = randn(H, I) / I ** 0.5
    s["base"] = randn(T, H).bfloat16()  # the layer's output
    if kind == "ffn8":
        s["w1"], s["w1_scales"] = _quantised(w1)
        s["w2"], s["w2_scales"] = _quantised(w2)
        return s
    s["w1"], s["w2"] = w1.bfloat16(), w2.bfloat16()
    if kind == "train":
        s["dout"] = randn(T, H).bfloat16()
        s["dx_base"] = randn(T, H).bfloat16()  # the input's gradient through the rest of the layer
    return s


# ---------------------------------------------------------------- plain forms
def _codes(x):
    """Codes and scales of the rows of x; the quotients in 64 bits, where a code's
    border may lie within a float32's rounding."""
    scale = x.float().abs().amax(dim=1) / 127
    scale = torch.where(scale > 0, torch.clamp(scale, min=2.0 ** -126), 1.0)
    return torch.round(x.double() / scale.double()[:, None]).float(), scale


def _product8(codes, scale, w, w_scales):
    return (codes @ w.float().T) * scale[:, None] * w_scales


def _plain(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind == "linear8":
        y = _product8(*_codes(s["x"]), s["w"], s["w_scales"])
        return y if c["out"] == "f32" else y.bfloat16()
    I = c["inter"]
    if kind == "ffn8":
        gu = _product8(*_codes(s["x"]), s["w1"], s["w1_scales"])
        g, u = gu[:, :I], gu[:, I:]
        h = g / (1 + torch.exp(-g)) * u
        return (s["base"].float() + _product8(*_codes(h), s["w2"], s["w2_scales"])).bfloat16()
    x, w1, w2 = s["x"].float(), s["w1"].float(), s["w2"].float()
    gu = x @ w1.T
    g, u = gu[:, :I], gu[:, I:]
    sig = 1 / (1 + torch.exp(-g))
    h = g * sig * u
    out = (s["base"].float() + h @ w2.T).bfloat16()
    if kind == "ffn":
        return out
    d = s["dout"].float()
    dh = d @ w2
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=1)
    t = torch.bfloat16 if c.get("grads") == "bf16" else torch.float32
    return {"out": out, "dx": (s["dx_base"].float() + dgu @ w1).bfloat16(), "dw1": (dgu.T @ x).to(t),
            "dw2": (d.T @ h).to(t)}


# ---------------------------------------------------------------- the framework's calls
def _bytes(s, name, size):
    """A workspace the program keeps for its batches of this shape."""
    if name not in s["kept"]:
        s["kept"][name] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["kept"][name]


def _own(s):
    import mixed_precision_moe_topk_amd as M

    c, kind, T, x = s["case"], s["case"]["kind"], s["case"]["tokens"], s["x"]
    if kind == "linear8":
        d = M.Int8Dims(c["k"], c["n"], c["out"])
        ws = _bytes(s, "ws", lambda: M.int8_workspace_query(d, T))
        codes = torch.empty(x.shape, dtype=torch.int8, device="cuda")
        scales = torch.empty(T, dtype=torch.float32, device="cuda")
        out = torch.empty((T, c["n"]), dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
        M.int8_quantize(x, codes, scales)
        M.int8_matmul(d, codes, scales, s["w"], s["w_scales"], None, out, ws)
        return out
    d = M.FfnDims(c["hidden"], c["inter"])
    out = torch.empty_like(x)
    if kind == "ffn8":
        ws = _bytes(s, "ws", lambda: M.ffn_int8_workspace_query(d, T))
        M.ffn_int8_apply(d, x, s["w1"], s["w1_scales"], s["w2"], s["w2_scales"], s["base"], out, ws)
        return out
    ws = _bytes(s, "ws", lambda: M.ffn_workspace_query(d, T))
    if kind == "ffn":
        M.ffn_apply(d, x, s["w1"], s["w2"], s["base"], out, ws)
        return out
    saved = _bytes(s, "saved", lambda: M.ffn_saved_query(d, T))
    M.ffn_apply(d, x, s["w1"], s["w2"], s["base"], out, ws, saved=saved)
    dx = torch.empty_like(x)
    t = torch.bfloat16 if c.get("grads") == "bf16" else torch.float32
    dw1, dw2 = torch.empty_like(s["w1"], dtype=t), torch.empty_like(s["w2"], dtype=t)
    M.ffn_backward(d, s["dout"], x, s["w1"], s["w2"], saved, dw1, dw2, ws, dx=dx, dx_base=s["dx_base"])
    return {"out": out, "dx": dx, "dw1": dw1, "dw2": dw2}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work
def work(case):
    c, kind, T = case, case["kind"], case["tokens"]
    if kind == "linear8":
        K, N = c["k"], c["n"]
        return {"bytes": 2 * T * K + N * K + 4 * N + (4 if c["out"] == "f32" else 2) * T * N, "flops": 2 * T * N * K}
    H, I = c["hidden"], c["inter"]
    weights = 3 * H * I
    if kind == "ffn8":
        return {"bytes": 6 * T * H + weights + 4 * (2 * I + H), "flops": 2 * T * weights}
    if kind == "ffn":
        return {"bytes": 6 * T * H + 2 * weights, "flops": 2 * T * weights}
    # train: dout, dx and its base besides, and the weights' gradients
    grads = 2 if c.get("grads") == "bf16" else 4
    return {"bytes": 12 * T * H + (2 + grads) * weights, "flops": 6 * T * weights}


# ---------------------------------------------------------------- definitions in 64 bits
def _grid(v):
    """v on each row's grid of 127 steps either side of zero."""
    step = (v.abs().max(dim=1, keepdim=True).values.float() / 127).double()
    step[step == 0] = 1
    return (v / step).round() * step


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    x = s["x"].double()
    if kind == "linear8":
        return _grid(x) @ (s["w"].double() * s["w_scales"].double()[:, None]).T
    base = s["base"].double()
    if kind == "ffn8":
        w1 = s["w1"].double() * s["w1_scales"].double()[:, None]
        w2 = s["w2"].double() * s["w2_scales"].double()[:, None]
        gate, up = torch.chunk(_grid(x) @ w1.T, 2, dim=1)
        return base + _grid(torch.nn.functional.silu(gate) * up) @ w2.T
    w1, w2 = s["w1"].double(), s["w2"].double()
    if kind == "ffn":
        gate, up = torch.chunk(x @ w1.T, 2, dim=1)
        return base + (torch.nn.functional.silu(gate) * up) @ w2.T
    # derivatives by automatic differentiation
    x.requires_grad_(True), w1.requires_grad_(True), w2.requires_grad_(True)
    gate, up = torch.chunk(x @ w1.T, 2, dim=1)
    out = base + (torch.nn.functional.silu(gate) * up) @ w2.T
    dx, dw1, dw2 = torch.autograd.grad((out * s["dout"].double()).sum(), (x, w1, w2))
    return {"out": out.detach(), "dx": s["dx_base"].double() + dx, "dw1": dw1, "dw2": dw2}
