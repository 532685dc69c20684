"""Low-rank adapters on the GPU against their float64 definition
(oracle/train.py).

Tolerances, element by element, from the absolute products: a contraction of n
terms in float32 is off by at most n 2^-23 of the sum of its absolute terms
(each addition rounds or truncates once); u and v enter the second product as
two bf16 halves, 2^-17 of them; the result is rounded once, half a step."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import train as OT

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23


def bf16(x):
    return F.bf16_to_f32(F.bf16_rne(np.asarray(x, np.float32)))


class Case:
    def __init__(self, T, L, R, K, N, out, ids, seed, pads=(0, 0, 0)):
        rng = np.random.default_rng(seed)
        n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        self.shape = T, L, R, K, N
        self.out = out
        self.pads = pads  # extra elements in the rows of x, base and out
        self.x, self.a, self.b = bf16(n(T, K)), bf16(n(L, R, K) / K ** 0.5), bf16(n(L, R, N))
        self.scale = (0.5 + rng.random(L)).astype(np.float32)
        self.ids = np.asarray(ids(rng, T, L), np.int32)
        self.base, self.dout, self.dxb = n(T, N), n(T, N), bf16(n(T, K))
        if out == "bf16":
            self.base, self.dout = bf16(self.base), bf16(self.dout)

    def dev(self, a, bf, pad=0):
        import torch

        t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
        t = t.bfloat16() if bf else t
        if pad:
            wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, :t.shape[1]] = t
            t = wide[:, :t.shape[1]]
        return t

    def run(self, stale=0xA5, base="given", dx="base", grads=True):
        """-> dict of float32 numpy arrays."""
        import torch

        import mixed_precision_moe_topk_amd as M

        T, L, R, K, N = self.shape
        d = M.AdapterDims(L, R, K, N, self.out)
        lo = self.out == "bf16"
        buf = lambda n: torch.full((n,), stale, dtype=torch.uint8, device="cuda")  # noqa: E731
        plan, ws = buf(M.adapter_plan_query(L, T)), buf(M.adapter_workspace_query(d, T))
        saved = buf(M.adapter_saved_query(d, T))
        x, a, b = self.dev(self.x, True, self.pads[0]), self.dev(self.a, True), self.dev(self.b, True)
        scale, ids = self.dev(self.scale, False), self.dev(self.ids, False)
        bs = self.dev(self.base, lo, self.pads[1])
        out = self.dev(np.full((T, N), np.nan, np.float32), lo, self.pads[2])
        if base == "in place":
            out = bs
        M.adapter_plan(L, ids, plan)
        M.adapter_apply(d, x, plan, a, b, scale, None if base == "none" else bs, out, ws, saved=saved)
        r = {"out": out.float().cpu().numpy()}
        if not grads:
            return r
        ws.fill_(stale ^ 0xFF)
        dout = self.dev(self.dout, lo, self.pads[1])
        da = torch.full((L, R, K), float("nan"), device="cuda")
        db = torch.full((L, R, N), float("nan"), device="cuda")
        dxb = self.dev(self.dxb, True, self.pads[0])
        g = dxb if dx == "in place" else self.dev(np.full((T, K), np.nan, np.float32), True, self.pads[2])
        M.adapter_backward(d, dout, x, plan, a, b, scale, saved, da, db, ws, dx=g,
                           dx_base=None if dx == "none" else dxb)
        r.update(dx=g.float().cpu().numpy(), da=da.cpu().numpy(), db=db.cpu().numpy())
        return r

    def check(self, r, base="given", dx="base"):
        T, L, R, K, N = self.shape
        f = lambda v: v.astype(np.float64)  # noqa: E731
        x, a, b, s, d = f(self.x), f(self.a), f(self.b), f(self.scale), f(self.dout)
        b0 = np.zeros((T, N)) if base == "none" else f(self.base)
        x0 = np.zeros((T, K)) if dx == "none" else f(self.dxb)
        ref = {"out": OT.adapter_apply(x, self.ids, a, b, s, b0)}
        tol = {"out": np.zeros((T, N)), "dx": np.zeros((T, K)), "da": np.zeros(a.shape), "db": np.zeros(b.shape)}
        if "dx" in r:
            ref["dx"], ref["da"], ref["db"] = OT.adapter_backward(d, x, self.ids, a, b, s, x0)
        for i in range(L):
            t = np.nonzero(self.ids == i)[0]
            ax, aa, ab, ad = np.abs(x[t]), np.abs(a[i]), np.abs(b[i]), np.abs(d[t])
            u, v = s[i] * ax @ aa.T, s[i] * ad @ ab.T
            eu, ev = ((K + 34) * STEP + 2.0 ** -17) * u, ((N + 34) * STEP + 2.0 ** -17) * v
            if out_f32 := self.out == "f32":
                ev = ev + 2.0 ** -17 * v  # dout as two halves as well
            tol["out"][t] += (eu + (2 * R + 2) * STEP * u) @ ab
            if "dx" in r:
                tol["dx"][t] += (ev + (2 * R + 2) * STEP * v) @ aa
                n = 3 * len(t) + 40
                tol["da"][i] = (ev + n * STEP * v).T @ ax
                tol["db"][i] = (eu + (n * STEP + (2.0 ** -17 if out_f32 else 0.0)) * u).T @ ad
        half = 2.0 ** -8 if self.out == "bf16" else 2.0 ** -24
        tol["out"] += half * (np.abs(ref["out"]) + tol["out"])
        for k, v in r.items():
            if k == "dx":
                tol[k] += 2.0 ** -8 * (np.abs(ref[k]) + tol[k])
            bad = ~(np.abs(v - ref[k]) <= tol[k])
            assert not bad.any(), (k, np.argwhere(bad)[:4].tolist(), int(bad.sum()),
                                   float(np.nanmax(np.abs(v - ref[k]) / np.maximum(tol[k], 1e-30))))


def scattered(rng, T, L):
    return rng.integers(0, L, T)


def some_without(rng, T, L):
    ids = rng.integers(0, L, T)
    ids[rng.random(T) < 0.3] = -1
    ids[rng.random(T) < 0.1] = L + 5
    return ids


def runs(rng, T, L):
    return np.sort(some_without(rng, T, L))


def one(rng, T, L):
    return np.full(T, L - 1)


def few_of_many(rng, T, L):
    return np.sort(rng.choice([2, 3, 17, 30, -1], T, p=[0.5, 0.01, 0.4, 0.05, 0.04]))


def nobody(rng, T, L):
    return np.full(T, -1)


def each(rng, T, L):
    return np.arange(T) % L


CASES = [  # tokens, adapters, rank, K, N, out, ids
    (1, 1, 1, 8, 8, "bf16", one),
    (1, 8, 16, 512, 384, "bf16", one),
    (1, 3, 128, 264, 72, "f32", one),
    (2, 2, 5, 72, 136, "f32", each),
    (16, 4, 8, 256, 128, "bf16", one),
    (17, 4, 8, 256, 128, "bf16", one),
    (33, 5, 12, 320, 8, "f32", some_without),
    (64, 64, 32, 1032, 520, "bf16", each),
    (64, 4, 64, 512, 1024, "bf16", scattered),
    (65, 1, 17, 200, 264, "f32", one),
    (100, 300, 33, 256, 256, "bf16", scattered),      # more adapters than tokens
    (130, 1023, 3, 64, 64, "f32", scattered),
    (200, 7, 128, 136, 520, "bf16", runs),
    (200, 7, 100, 520, 136, "f32", runs),
    (300, 2, 65, 384, 640, "bf16", scattered),
    (513, 3, 16, 1024, 256, "f32", some_without),     # the router's logits
    (1024, 9, 48, 256, 384, "bf16", some_without),
    (1025, 9, 24, 256, 384, "bf16", some_without),    # past the single-block plan
    (2500, 5, 32, 128, 256, "bf16", runs),
    (40, 3, 16, 128, 128, "bf16", nobody),
    (32, 40, 8, 64, 64, "bf16", each),                # a padded row count without slack, then idle adapters
    (1500, 40, 16, 128, 256, "bf16", few_of_many),    # segments of adapters with idle ones between
    (1500, 40, 70, 136, 64, "f32", few_of_many),
    (2100, 1, 16, 256, 136, "bf16", one),             # one adapter's rows in several segments
    (1100, 1, 128, 128, 128, "f32", one),
    (9000, 3, 8, 64, 64, "bf16", scattered),          # past the plan of one launch
    (33000, 5, 8, 64, 72, "f32", some_without),       # whole tiles for shrink's blocks
    (66000, 2, 4, 16, 8, "bf16", runs),               # a plan of three launches
    (128, 3, 32, 264, 200, "bf16", scattered),
    (129, 3, 32, 264, 200, "f32", scattered),
    (512, 3, 32, 264, 200, "f32", scattered),         # the most sums that expand adds up itself
    (513, 3, 32, 264, 200, "bf16", scattered),
    (1024, 5, 15, 520, 136, "bf16", runs),
    (1030, 5, 16, 520, 136, "f32", runs),
    (128, 9, 128, 136, 264, "f32", each),
]


@pytest.mark.parametrize("T,L,R,K,N,out,ids", CASES)
def test_adapter_forward_and_backward(T, L, R, K, N, out, ids):
    c = Case(T, L, R, K, N, out, ids, T + R)
    r = c.run()
    c.check(r)
    again = c.run(stale=0x00)  # the same bits over other contents of the buffers
    for k in r:
        assert np.array_equal(r[k], again[k]), k


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_strided_rows_and_places(out):
    """Rows of wider tensors, results in place of their bases, and no base."""
    for pads in ((8, 16, 24), (0, 8, 8)):
        c = Case(150, 4, 20, 264, 200, out, some_without, 11, pads)
        c.check(c.run())
        c.check(c.run(base="none", dx="none"), base="none", dx="none")
        c.check(c.run(base="in place", dx="in place"))


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_strided_rows_and_places_of_long_batches(out):
    """The same where the low-rank rows are joined before expand."""
    c = Case(700, 4, 36, 264, 200, out, some_without, 12, (8, 16, 24))
    c.check(c.run())
    c.check(c.run(base="none", dx="none"), base="none", dx="none")
    c.check(c.run(base="in place", dx="in place"))


def test_frozen_factors_and_input_alone_of_long_batches():
    """dx alone, and the factors' gradients alone, where rows are joined."""
    import torch

    import mixed_precision_moe_topk_amd as M

    c = Case(1100, 3, 44, 136, 264, "bf16", some_without, 42)
    r = c.run(dx="none")
    T, L, R, K, N = c.shape
    d = M.AdapterDims(L, R, K, N)
    buf = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    plan, ws, saved = (buf(n) for n in (M.adapter_plan_query(L, T), M.adapter_workspace_query(d, T),
                                        M.adapter_saved_query(d, T)))
    x, a, b, dout = (c.dev(v, True) for v in (c.x, c.a, c.b, c.dout))
    scale = c.dev(c.scale, False)
    M.adapter_plan(L, c.dev(c.ids, False), plan)
    dx = torch.empty_like(x)
    M.adapter_backward(d, dout, None, plan, a, b, scale, None, None, None, ws, dx=dx)
    assert np.array_equal(dx.float().cpu().numpy(), r["dx"])
    M.adapter_apply(d, x, plan, a, b, scale, None, torch.empty_like(dout), ws, saved=saved)
    da, db = torch.empty(L, R, K, device="cuda"), torch.empty(L, R, N, device="cuda")
    M.adapter_backward(d, dout, x, plan, a, b, scale, saved, da, db, ws)
    assert np.array_equal(da.cpu().numpy(), r["da"]) and np.array_equal(db.cpu().numpy(), r["db"])


def test_infinities_pass_as_the_formula_has_them():
    """One infinite element of x: the same infinities and NaN as in float64, and
    no NaN from ranks that only pad, on both ways of the low-rank rows."""
    for T in (40, 700):
        c = Case(T, 2, 1, 64, 136, "bf16", each, 33)
        c.x[4, 9] = np.inf
        r = c.run()
        f = lambda v: v.astype(np.float64)  # noqa: E731
        with np.errstate(invalid="ignore"):
            ref = OT.adapter_apply(f(c.x), c.ids, f(c.a), f(c.b), f(c.scale), f(c.base))
        assert np.isinf(ref[4]).all() and np.isfinite(np.delete(ref, 4, 0)).all()
        assert np.array_equal(r["out"][4], ref[4]) and np.isfinite(np.delete(r["out"], 4, 0)).all()


def test_long_rows_and_many_tokens():
    """The layer's own width; contractions split over several blocks, and an
    adapter with thousands of tokens."""
    c = Case(70, 6, 16, 7168, 2048, "bf16", some_without, 21)
    c.check(c.run())
    c = Case(6000, 2, 40, 256, 128, "f32", runs, 22)
    c.check(c.run())


def test_tokens_of_other_adapters_do_not_reach_each_other():
    """Infinities and NaN in one request's rows and factors stay there."""
    c = Case(90, 3, 16, 128, 256, "bf16", each, 31)
    clean = c.run()
    c.x[1, 5] = np.inf
    c.x[4, 7] = np.nan
    c.dout[7, 3] = np.nan  # tokens of adapter 1
    c.a[1, 2, 3] = np.inf
    r = c.run()
    mine = c.ids == 1
    for k in ("out", "dx"):
        assert np.array_equal(r[k][~mine], clean[k][~mine])
        assert not np.isfinite(r[k][mine]).all()
    for k in ("da", "db"):
        assert np.array_equal(r[k][[0, 2]], clean[k][[0, 2]])
        assert not np.isfinite(r[k][1]).all()


def test_no_tokens_gives_zero_gradients():
    import torch

    import mixed_precision_moe_topk_amd as M

    d = M.AdapterDims(3, 8, 64, 128)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    plan = torch.empty(M.adapter_plan_query(3, 0), dtype=torch.uint8, device="cuda")
    ws = torch.empty(M.adapter_workspace_query(d, 0), dtype=torch.uint8, device="cuda")
    a, b, scale = e(3, 8, 64), e(3, 8, 128), torch.ones(3, device="cuda")
    M.adapter_plan(3, torch.empty(0, dtype=torch.int32, device="cuda"), plan)
    M.adapter_apply(d, e(0, 64), plan, a, b, scale, e(0, 128), e(0, 128), ws)
    da, db = torch.ones(3, 8, 64, device="cuda"), torch.ones(3, 8, 128, device="cuda")
    M.adapter_backward(d, e(0, 128), e(0, 64), plan, a, b, scale, ws, da, db, ws)
    assert not da.any() and not db.any()


def test_frozen_factors_and_input_alone():
    """dx without da and db, and the reverse, are the same as together."""
    import torch

    import mixed_precision_moe_topk_amd as M

    c = Case(77, 3, 12, 136, 264, "bf16", some_without, 41)
    r = c.run(dx="none")
    T, L, R, K, N = c.shape
    d = M.AdapterDims(L, R, K, N)
    buf = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    plan, ws, saved = (buf(n) for n in (M.adapter_plan_query(L, T), M.adapter_workspace_query(d, T),
                                        M.adapter_saved_query(d, T)))
    x, a, b, dout = (c.dev(v, True) for v in (c.x, c.a, c.b, c.dout))
    scale = c.dev(c.scale, False)
    M.adapter_plan(L, c.dev(c.ids, False), plan)
    dx = torch.empty_like(x)
    M.adapter_backward(d, dout, None, plan, a, b, scale, None, None, None, ws, dx=dx)
    assert np.array_equal(dx.float().cpu().numpy(), r["dx"])
    M.adapter_apply(d, x, plan, a, b, scale, None, torch.empty_like(dout), ws, saved=saved)
    da, db = torch.empty(L, R, K, device="cuda"), torch.empty(L, R, N, device="cuda")
    M.adapter_backward(d, dout, x, plan, a, b, scale, saved, da, db, ws)
    assert np.array_equal(da.cpu().numpy(), r["da"]) and np.array_equal(db.cpu().numpy(), r["db"])


def test_two_streams_with_their_own_workspaces():
    import torch

    import mixed_precision_moe_topk_amd as M

    cs = [Case(200, 5, 32, 512, 640, "bf16", scattered, 51 + n) for n in range(2)]
    want = [c.run(grads=False)["out"] for c in cs]
    T, L, R, K, N = cs[0].shape
    d = M.AdapterDims(L, R, K, N)
    buf = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    held = []
    for c in cs:
        held.append(dict(x=c.dev(c.x, True), a=c.dev(c.a, True), b=c.dev(c.b, True), s=c.dev(c.scale, False),
                         ids=c.dev(c.ids, False), base=c.dev(c.base, True), plan=buf(M.adapter_plan_query(L, T)),
                         ws=buf(M.adapter_workspace_query(d, T)), st=torch.cuda.Stream()))
        held[-1]["out"] = torch.empty_like(held[-1]["base"])
    torch.cuda.synchronize()
    for _ in range(5):
        for h in held:
            M.adapter_plan(L, h["ids"], h["plan"], stream=h["st"])
            M.adapter_apply(d, h["x"], h["plan"], h["a"], h["b"], h["s"], h["base"], h["out"], h["ws"],
                            stream=h["st"])
    torch.cuda.synchronize()
    for h, w in zip(held, want):
        assert np.array_equal(h["out"].float().cpu().numpy(), w)


def test_captured_adapters_replay():
    """Plan, forward and backward captured into one graph; the replays take other
    adapter ids and inputs, with eager work between."""
    import torch

    import mixed_precision_moe_topk_amd as M

    cs = [Case(150, 6, 24, 256, 384, "bf16", some_without, 61 + n) for n in range(3)]
    want = [c.run() for c in cs]
    T, L, R, K, N = cs[0].shape
    d = M.AdapterDims(L, R, K, N)
    buf = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    plan, ws, saved = (buf(n) for n in (M.adapter_plan_query(L, T), M.adapter_workspace_query(d, T),
                                        M.adapter_saved_query(d, T)))
    names = ("x", "a", "b", "base", "dout", "dxb")
    st = {n: torch.empty(getattr(cs[0], n).shape, dtype=torch.bfloat16, device="cuda") for n in names}
    st["scale"], st["ids"] = torch.empty(L, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    out, dx = torch.empty_like(st["base"]), torch.empty_like(st["x"])
    da, db = torch.empty(L, R, K, device="cuda"), torch.empty(L, R, N, device="cuda")

    def load(c):
        for n in names:
            st[n].copy_(torch.from_numpy(getattr(c, n)).bfloat16())
        st["scale"].copy_(torch.from_numpy(c.scale))
        st["ids"].copy_(torch.from_numpy(c.ids))

    def step():
        M.adapter_plan(L, st["ids"], plan)
        M.adapter_apply(d, st["x"], plan, st["a"], st["b"], st["scale"], st["base"], out, ws, saved=saved)
        M.adapter_backward(d, st["dout"], st["x"], plan, st["a"], st["b"], st["scale"], saved, da, db, ws, dx=dx,
                           dx_base=st["dxb"])

    load(cs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (1, 0, 2, 2):
        load(cs[n])
        for t in (plan, ws, saved):
            t.fill_(0x6B)
        graph.replay()
        torch.cuda.synchronize()
        for t, k in ((out, "out"), (dx, "dx"), (da, "da"), (db, "db")):
            assert np.array_equal(t.float().cpu().numpy(), want[n][k]), (n, k)
        step()
        cs[n].run(grads=False)  # eager work between replays
    del graph


def test_binding_refuses_wrong_tensors():
    import torch

    import mixed_precision_moe_topk_amd as M

    T, L, R, K, N = 8, 2, 8, 64, 128
    d = M.AdapterDims(L, R, K, N)
    e = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    plan, ws = (e(n, t=torch.uint8) for n in (M.adapter_plan_query(L, T), M.adapter_workspace_query(d, T)))
    f32 = torch.float32
    good = dict(x=e(T, K), plan=plan, a=e(L, R, K), b=e(L, R, N), scale=e(L, t=f32), base=e(T, N), out=e(T, N),
                workspace=ws)

    def status(**kw):
        with pytest.raises(M.MoeError) as ei:
            M.adapter_apply(d, **{**good, **kw})
        return ei.value.status

    M.adapter_plan(L, e(T, t=torch.int32), plan)
    M.adapter_apply(d, **good)
    assert status(x=e(T, K, t=f32)) == 1 and status(x=e(T, K + 8)) == 1 and status(a=e(L, R, N)) == 1
    assert status(b=e(L, N, R)) == 1 and status(scale=e(L)) == 1 and status(base=e(T, N, t=f32)) == 1
    assert status(out=e(N, T).t()) == 1 and status(x=e(T, K + 4)[:, :K]) == 1  # stride of 4 elements over
    assert status(x=e(1, K).expand(T, K)) == 1  # every row the same: no stride
    assert status(plan=plan[:64]) == 3 and status(workspace=ws[:64]) == 3
    assert status(x=e(T, K + 8)[:, 1:K + 1]) == 1  # rows that do not start 16-byte aligned
    with pytest.raises(M.MoeError):
        M.adapter_plan(L, e(T, t=torch.int64), plan)
    torch.cuda.synchronize()


def test_no_tokens_and_frozen_factors():
    """An empty batch asked for dx alone, as a rank without tokens has it."""
    import torch

    import mixed_precision_moe_topk_amd as M

    d = M.AdapterDims(3, 8, 64, 128)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    plan, ws = (torch.empty(n, dtype=torch.uint8, device="cuda")
                for n in (M.adapter_plan_query(3, 0), M.adapter_workspace_query(d, 0)))
    M.adapter_backward(d, e(0, 128), e(0, 64), plan, e(3, 8, 64), e(3, 8, 128), torch.ones(3, device="cuda"), None,
                       None, None, ws, dx=e(0, 64))
    M.adapter_backward(d, e(0, 128), None, plan, e(3, 8, 64), e(3, 8, 128), torch.ones(3, device="cuda"), None,
                       None, None, ws, dx=e(0, 64), dx_base=e(0, 64))
    torch.cuda.synchronize()
