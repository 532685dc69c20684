"""Cases of the training and adapter operators beside the MoE layer, their
plain forms in torch, their definitions in 64 bits, and the calls a program
makes of them.

Operators (kind of a case):
  loss       balance loss, z-loss and per-expert counts of the router
  router     gradient of the router's logits: from the two losses and from the
             routing weights (a softmax over the selected logits)
  combine    gradient of the router-weighted sum of the expert rows
  adapter    low-rank adapters of many requests at once beside a projection
  train      the same adapters, forward and backward

`own` false: the plain forms run (elementary torch operations in float32,
rounded once at the end).  `own` true: the framework's kernels run.
"""
import torch

own = False

H_V3 = 7168  # hidden size of the DeepSeek-V3 / V4-Pro MoE layers of moe_inputs


def listed():
    return [
        # the tiny layer of moe_inputs: latency of the smallest loss
        dict(name="loss tiny", kind="loss", tokens=16, experts=8, top_k=2, seqs=1, pad=0.0, bias=0.0),
        # one DeepSeek-V3 prefill batch taken as a whole
        dict(name="loss v3 4096", kind="loss", tokens=4096, experts=256, top_k=8, seqs=1, pad=0.0, bias=0.0),
        # a packed training batch: ragged sequences, padded tokens, skewed experts
        dict(name="loss v4pro 16384 packed", kind="loss", tokens=16384, experts=384, top_k=6, seqs=37, pad=0.1,
             bias=2.0),
        # a micro-batch of the decode workload's size
        dict(name="router v3 64", kind="router", tokens=64, experts=256, top_k=8, seqs=1, pad=0.0, bias=0.0),
        # the packed training batch's backward pass
        dict(name="router v4pro 16384 packed", kind="router", tokens=16384, experts=384, top_k=6, seqs=37, pad=0.1,
             bias=2.0),
        # the weighted sum's backward pass on 64 tokens, float32 rows
        dict(name="combine v3 64 f32", kind="combine", tokens=64, experts=256, top_k=8, hidden=H_V3, rows="f32"),
        # and on the largest prefill batch, row gradients in bf16
        dict(name="combine v4pro 16384 bf16", kind="combine", tokens=16384, experts=384, top_k=6, hidden=H_V3,
             rows="bf16"),
        # one token of one request: latency
        dict(name="adapter decode 1", kind="adapter", tokens=1, adapters=8, rank=16, k=H_V3, n=H_V3, out="bf16",
             none=0.0, runs=0),
        # a decode batch in which most requests bring their own adapter
        dict(name="adapter decode 64", kind="adapter", tokens=64, adapters=64, rank=32, k=H_V3, n=H_V3, out="bf16",
             none=0.1, runs=0),
        # prefill: long runs of tokens with one adapter
        dict(name="adapter prefill 16384", kind="adapter", tokens=16384, adapters=8, rank=64, k=H_V3, n=H_V3,
             out="bf16", none=0.1, runs=1),
        # adapters on the router's float32 logits, trained; an odd batch and rank
        dict(name="train router 4093", kind="train", tokens=4093, adapters=5, rank=12, k=H_V3, n=256, out="f32",
             none=0.05, runs=1),
        # adapters beside the whole layer, trained
        dict(name="train layer 4096", kind="train", tokens=4096, adapters=4, rank=32, k=H_V3, n=H_V3, out="bf16",
             none=0.05, runs=1),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["loss", "router", "combine", "adapter", "train"])
    if kind in ("loss", "router"):
        experts = _log(rng, 4, 1024)
        tokens = _log(rng, 1, 16384)
        return dict(kind=kind, tokens=tokens, experts=experts, top_k=rng.randint(1, min(experts, 16)),
                    seqs=min(_log(rng, 1, 64), tokens), pad=rng.choice([0.0, 0.05, 0.3]),
                    bias=rng.choice([0.0, 1.0, 2.0]))
    if kind == "combine":
        tokens = _log(rng, 1, 8192)
        experts = _log(rng, 8, 1024)
        return dict(kind=kind, tokens=tokens, experts=experts, top_k=rng.randint(1, 8),
                    hidden=128 * rng.randint(1, 56), rows=rng.choice(["f32", "bf16"]))
    tokens = _log(rng, 1, 8192 if kind == "adapter" else 4096)
    router = rng.random() < 0.3  # beside the router's projection, else beside the layer
    return dict(kind=kind, tokens=tokens, adapters=_log(rng, 1, 64 if tokens <= 512 else 8), rank=_log(rng, 1, 128),
                k=8 * _log(rng, 16, 896), n=8 * (_log(rng, 1, 128) if router else _log(rng, 16, 896)),
                out="f32" if router else "bf16", none=rng.choice([0.0, 0.1]), runs=rng.randint(0, 1))


# ---------------------------------------------------------------- inputs
def _routing(c, gen):
    """Logits (with a per-expert bias for skewed loads), the selected experts
    and their softmax weights, as the layer's router gives them."""
    T, E, k = c["tokens"], c["experts"], min(c["top_k"], c["experts"])
    logits = torch.randn(T, E, generator=gen, device="cuda")
    if c.get("bias"):
        logits += c["bias"] * torch.randn(E, generator=gen, device="cuda")
    sel, ids = logits.topk(k, dim=1)
    return logits, ids.to(torch.int32).contiguous(), torch.softmax(sel, dim=1).contiguous()


def _offsets(T, S, gen):
    """S + 1 ragged boundaries from 0 to T."""
    cut = torch.randint(0, T + 1, (S - 1,), generator=gen, device="cuda").sort().values
    zero = cut.new_zeros(1)
    return torch.cat([zero, cut, zero + T]).to(torch.int32)


def _segment(s):
    """Sequence of each token, and whether the token counts."""
    T = s["logits"].shape[0]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["offsets"].long(), t, right=True) - 1
    return seq, s["mask"].bool()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, kind = case, case["kind"]
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    T = c["tokens"]
    s = {"case": c, "kept": {}}
    if kind in ("loss", "router"):
        s["logits"], s["ids"], s["weights"] = _routing(c, gen)
        s["offsets"] = _offsets(T, c["seqs"], gen)
        s["mask"] = (torch.rand(T, generator=gen, device="cuda") >= c["pad"]).to(torch.uint8)
        if kind == "router":
            # what the forward pass and the layers behind the router leave
            seq, on = _segment(s)
            E, S, k = c["experts"], c["seqs"], s["ids"].shape[1]
            slot = (seq[:, None] * E + s["ids"].long())[on].flatten()
            s["counts"] = torch.zeros(S * E, dtype=torch.int64, device="cuda").scatter_add_(
                0, slot, torch.ones_like(slot)).view(S, E).to(torch.int32)
            n = torch.zeros(S, dtype=torch.int64, device="cuda").scatter_add_(0, seq[on], torch.ones_like(seq[on]))
            s["seq_tokens"] = torch.cat([n, n.sum()[None], (n > 0).sum()[None]]).to(torch.int32)
            s["dweights"] = randn(T, k) * 0.1
            # upstream gradients of (balance loss, z-loss): their coefficients
            s["dlosses"] = torch.tensor([0.01, 0.001], device="cuda") * T
    elif kind == "combine":
        _, ids, s["weights"] = _routing(c, gen)
        order = ids.flatten().long().argsort(stable=True)  # rows grouped by expert
        slot_row = torch.empty_like(order)
        slot_row[order] = torch.arange(order.numel(), device="cuda")
        s["slot_row"] = slot_row.view(ids.shape).to(torch.int32)
        s["y2"] = randn(ids.numel(), c["hidden"])
        s["dout"] = randn(T, c["hidden"]).bfloat16()
    else:
        L, R, K, N = c["adapters"], c["rank"], c["k"], c["n"]
        s["x"] = randn(T, K).bfloat16()
        s["a"] = (randn(L, R, K) / K ** 0.5).bfloat16()
        s["b"] = (randn(L, R, N) * 0.2 / R ** 0.5).bfloat16()
        s["scale"] = 1.0 + torch.rand(L, generator=gen, device="cuda")
        ids = torch.randint(0, L, (T,), generator=gen, device="cuda")
        if c["runs"]:
            ids = ids.sort().values  # prompts: each request's tokens together
        off = torch.rand(T, generator=gen, device="cuda") < c["none"]
        s["adapter_ids"] = torch.where(off, -1, ids).to(torch.int32)
        s["base"] = randn(T, N) if c["out"] == "f32" else randn(T, N).bfloat16()
        if kind == "train":
            s["dout"] = randn(T, N) if c["out"] == "f32" else randn(T, N).bfloat16()
            s["dx_base"] = randn(T, K).bfloat16()
    return s


# ---------------------------------------------------------------- plain forms
def _plain_loss(s):
    c, x = s["case"], s["logits"]
    E, S, k = c["experts"], c["seqs"], s["ids"].shape[1]
    seq, on = _segment(s)
    m = x.max(dim=1, keepdim=True).values
    e = torch.exp(x - m)
    z = e.sum(dim=1, keepdim=True)
    p = e / z
    lse = (m + torch.log(z))[:, 0]
    member = ((seq[None, :] == torch.arange(S, device="cuda")[:, None]) & on[None, :]).float()  # [S, T]
    n = member.sum(dim=1)
    per = torch.clamp(n, min=1.0)
    slot = torch.where(on[:, None], seq[:, None] * E + s["ids"].long(), S * E).flatten()
    counts = torch.zeros(S * E + 1, dtype=torch.int64, device="cuda").scatter_add_(
        0, slot, torch.ones_like(slot))[:-1].view(S, E)
    mean = (member @ p) / per[:, None]
    f = counts.float() * (E / (k * per))[:, None]
    live = (n > 0).sum()
    balance = (f * mean).sum() / torch.clamp(live, min=1)
    zl = (torch.where(on, lse, 0.0) ** 2).sum() / torch.clamp(n.sum(), min=1.0)
    tokens = torch.cat([n, n.sum()[None], live[None].float()]).to(torch.int32)
    return {"losses": torch.stack([balance, zl]), "counts": counts.to(torch.int32), "mean_probs": mean,
            "seq_tokens": tokens}


def _plain_router(s):
    c, x = s["case"], s["logits"]
    E, k = c["experts"], s["ids"].shape[1]
    seq, on = _segment(s)
    m = x.max(dim=1, keepdim=True).values
    e = torch.exp(x - m)
    z = e.sum(dim=1, keepdim=True)
    p = e / z
    lse = m + torch.log(z)
    n = s["seq_tokens"][:-2].float()
    f = s["counts"].float() * (E / (k * torch.clamp(n, min=1.0)))[:, None]
    total, live = s["seq_tokens"][-2].float(), s["seq_tokens"][-1].float()
    ft = f[seq]
    g = p * (ft - (p * ft).sum(dim=1, keepdim=True)) * (s["dlosses"][0] / (live * n[seq]))[:, None]
    g = g + p * lse * (2.0 * s["dlosses"][1] / total)
    w, dw = s["weights"], s["dweights"]
    g.scatter_add_(1, s["ids"].long(), w * (dw - (w * dw).sum(dim=1, keepdim=True)))
    return torch.where(on[:, None], g, 0.0)


def _plain_combine(s):
    row, w = s["slot_row"].long(), s["weights"]
    d = s["dout"].float()
    y = s["y2"][row.flatten()].view(*row.shape, -1)  # [T, k, H]
    dweights = (y * d[:, None]).sum(dim=2)
    dy2 = torch.empty_like(s["y2"])
    dy2[row.flatten()] = (w[:, :, None] * d[:, None]).view_as(dy2)
    return {"dweights": dweights, "dy2": dy2.bfloat16() if s["case"]["rows"] == "bf16" else dy2}


def _plain_adapter(s):
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    L, R, _ = a.shape
    # every adapter's product with every token, kept where the token has it
    keep = (s["adapter_ids"][:, None] == torch.arange(L, device="cuda")).float() * s["scale"]
    keep = keep[:, :, None].expand(-1, -1, R).reshape(-1, L * R)
    a, b = a.view(L * R, -1), b.view(L * R, -1)
    u = (x @ a.T) * keep
    out = (s["base"].float() + u @ b).to(s["base"].dtype)
    if s["case"]["kind"] == "adapter":
        return out
    d = s["dout"].float()
    v = (d @ b.T) * keep
    return {"out": out, "dx": (s["dx_base"].float() + v @ a).bfloat16(), "da": (v.T @ x).view(L, R, -1),
            "db": (u.T @ d).view(L, R, -1)}


# ---------------------------------------------------------------- the framework's calls
def _bytes(s, name, size):
    """A workspace the program keeps for its batches of this shape."""
    if name not in s["kept"]:
        s["kept"][name] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["kept"][name]


def _own(s):
    import mixed_precision_moe_topk_amd as M

    c, kind, dev = s["case"], s["case"]["kind"], "cuda"
    T = c["tokens"]
    f32 = torch.float32
    if kind in ("loss", "router"):
        E, S, k = c["experts"], c["seqs"], s["ids"].shape[1]
        d = M.LayerDims(E, H_V3, 2048)
        if kind == "loss":
            ws = _bytes(s, "loss", lambda: M.router_loss_query(d, T, S))
            losses = torch.empty(2, dtype=f32, device=dev)
            counts = torch.empty((S, E), dtype=torch.int32, device=dev)
            mean = torch.empty((S, E), dtype=f32, device=dev)
            tokens = torch.empty(S + 2, dtype=torch.int32, device=dev)
            M.router_loss(d, s["logits"], s["ids"], losses, counts, mean, tokens, ws, seq_offsets=s["offsets"],
                          token_mask=s["mask"])
            return {"losses": losses, "counts": counts, "mean_probs": mean, "seq_tokens": tokens}
        dlogits = torch.empty((T, E), dtype=f32, device=dev)
        M.router_backward(d, s["logits"], s["ids"], dlogits, weights=s["weights"], dweights=s["dweights"],
                          dlosses=s["dlosses"], counts=s["counts"], seq_tokens=s["seq_tokens"],
                          seq_offsets=s["offsets"], token_mask=s["mask"])
        return dlogits
    if kind == "combine":
        d = M.LayerDims(c["experts"], c["hidden"], 2048)
        dweights = torch.empty_like(s["weights"])
        dy2 = torch.empty_like(s["y2"], dtype=torch.bfloat16 if c["rows"] == "bf16" else f32)
        M.finalize_backward(d, s["dout"], s["weights"], s["y2"], s["slot_row"], dweights, dy2)
        return {"dweights": dweights, "dy2": dy2}
    L, R = c["adapters"], c["rank"]
    d = M.AdapterDims(L, R, c["k"], c["n"], c["out"])
    plan = _bytes(s, "plan", lambda: M.adapter_plan_query(L, T))
    ws = _bytes(s, "ws", lambda: M.adapter_workspace_query(d, T))
    M.adapter_plan(L, s["adapter_ids"], plan)
    out = torch.empty_like(s["base"])
    if kind == "adapter":
        M.adapter_apply(d, s["x"], plan, s["a"], s["b"], s["scale"], s["base"], out, ws)
        return out
    u = _bytes(s, "u", lambda: M.adapter_saved_query(d, T))
    M.adapter_apply(d, s["x"], plan, s["a"], s["b"], s["scale"], s["base"], out, ws, saved=u)
    dx = torch.empty_like(s["x"])
    da = torch.empty(s["a"].shape, dtype=f32, device=dev)
    db = torch.empty(s["b"].shape, dtype=f32, device=dev)
    M.adapter_backward(d, s["dout"], s["x"], plan, s["a"], s["b"], s["scale"], u, da, db, ws, dx=dx,
                       dx_base=s["dx_base"])
    return {"out": out, "dx": dx, "da": da, "db": db}


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "loss":
        return _plain_loss(state)
    if kind == "router":
        return _plain_router(state)
    if kind == "combine":
        return _plain_combine(state)
    return _plain_adapter(state)


# ---------------------------------------------------------------- work
def work(case):
    c, kind, T = case, case["kind"], case["tokens"]
    if kind in ("loss", "router"):
        E, S, k = c["experts"], c["seqs"], min(c["top_k"], c["experts"])
        n = 4 * T * E + 4 * T * k + T + 4 * S * (E + 1)  # logits, ids, mask, counts
        if kind == "loss":
            return {"bytes": n + 4 * S * E, "flops": 5 * T * E}
        return {"bytes": n + 4 * T * E + 8 * T * k, "flops": 10 * T * E}
    if kind == "combine":
        H, k = c["hidden"], min(c["top_k"], c["experts"])
        rows = T * k
        return {"bytes": 2 * T * H + rows * H * (4 + (2 if c["rows"] == "bf16" else 4)) + 12 * rows,
                "flops": 3 * rows * H}
    L, R, K, N = c["adapters"], c["rank"], c["k"], c["n"]
    eo = 4 if c["out"] == "f32" else 2
    used = min(L, T)  # adapters a batch can use
    n = 4 * T + 2 * T * K + 2 * eo * T * N + 2 * used * R * (K + N)
    fl = 2 * T * R * (K + N)
    if kind == "train":
        n += eo * T * N + 4 * T * K + 4 * L * R * (K + N)  # dout, dx and its base, da, db
        fl *= 3
    return {"bytes": n, "flops": fl}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind, T = case["kind"], case["tokens"]
    if kind in ("loss", "router"):
        E, S, k = case["experts"], case["seqs"], s["ids"].shape[1]
        edge = s["offsets"].tolist()
        spans = [(i, slice(edge[i], edge[i + 1])) for i in range(S) if edge[i + 1] > edge[i]]
        x, on = s["logits"].double(), s["mask"].bool()
        total = int(on.sum())
        live = sum(int(on[sp].any()) for _, sp in spans)
        if kind == "loss":
            counts = torch.zeros(S, E, dtype=torch.int32, device="cuda")
            mean = torch.zeros(S, E, dtype=torch.float64, device="cuda")
            tokens = torch.zeros(S + 2, dtype=torch.int32, device="cuda")
            balance = x.new_zeros(())
            for i, sp in spans:
                mine = on[sp]
                n = int(mine.sum())
                if n == 0:
                    continue
                counts[i] = torch.bincount(s["ids"][sp][mine].flatten().long(), minlength=E)
                mean[i] = torch.softmax(x[sp][mine], dim=1).mean(dim=0)
                tokens[i] = n
                balance = balance + E * (counts[i].double() / (n * k) * mean[i]).sum() / live
            tokens[S], tokens[S + 1] = total, live
            zl = torch.logsumexp(x[on], dim=1).square().sum() / max(total, 1)
            return {"losses": torch.stack([balance, zl]), "counts": counts, "mean_probs": mean,
                    "seq_tokens": tokens}
        # derivatives by automatic differentiation of the losses and of the
        # softmax over the selected logits
        x.requires_grad_(True)
        goal = x.new_zeros(())
        for i, sp in spans:
            mine = on[sp]
            n = int(mine.sum())
            if n:
                share = s["counts"][i].double() / (n * k)
                goal = goal + s["dlosses"][0].double() * E * (share * torch.softmax(x[sp][mine], 1).mean(0)).sum() / live
        if total:
            goal = goal + s["dlosses"][1].double() * torch.logsumexp(x[on], 1).square().sum() / total
            w = torch.softmax(x[on].gather(1, s["ids"][on].long()), dim=1)
            goal = goal + (w * s["dweights"][on].double()).sum()
            return torch.autograd.grad(goal, x)[0]
        return torch.zeros_like(x)
    if kind == "combine":
        d, w, row = s["dout"].double(), s["weights"].double(), s["slot_row"].long()
        dweights = torch.empty_like(w)
        dy2 = torch.empty(s["y2"].shape, dtype=torch.float64, device="cuda")
        for j in range(row.shape[1]):
            dweights[:, j] = (s["y2"][row[:, j]].double() * d).sum(1)
            dy2[row[:, j]] = w[:, j, None] * d
        return {"dweights": dweights, "dy2": dy2}
    out = s["base"].double()
    train = kind == "train"
    if train:
        dx = s["dx_base"].double()
        da = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
        db = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["adapters"]):
        t = (s["adapter_ids"] == i).nonzero()[:, 0]
        if not t.numel():
            continue
        x, a, b, f = s["x"][t].double(), s["a"][i].double(), s["b"][i].double(), s["scale"][i].double()
        low = x @ a.T
        out[t] += f * (low @ b)
        if train:
            d = s["dout"][t].double()
            back = f * (d @ b.T)
            dx[t] += back @ a
            da[i] = back.T @ x
            db[i] = f * (low.T @ d)
    return {"out": out, "dx": dx, "da": da, "db": db} if train else out
