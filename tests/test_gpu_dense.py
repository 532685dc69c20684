"""The gated block in bf16 on the GPU against its float64 definition
(oracle/dense.py), product by product: every product is compared with the float64
product of the operands that the GPU itself rounded (g, u, h in what the forward
pass saves, the gradients of g and u in the workspace), and the roundings with the
formulas, so that no tolerance has to cover a rounding that a later sum hides.
float32 gradients of the weights are compared with the formulas end to end besides.

Tolerances, element by element: a sum of n products of bf16 numbers in float32 is
off by at most (n + 34) 2^-23 of the sum of its absolute terms (each addition
rounds or truncates once, some 34 of them in joins and bases); sigmoid is off by
2^-21 and 2^-23 |g| of itself (the exponential's argument, rounded twice, and a
reciprocal of one step); a bf16 result by half a step, 2^-8 of itself, one in two
bf16 terms by 2^-17 (the first leaves 2^-8 of it at most, and half a step of that
is 2^-9 of its own power of two)."""
import numpy as np
import pytest

from oracle import dense as OD
from oracle import formats as F

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24, "two terms": 2.0 ** -17}


def bf16(x):
    return F.bf16_to_f32(F.bf16_rne(np.asarray(x, np.float32)))


def device(a, pad=0, dtype="bf16"):
    """a on the GPU, with `pad` more elements in every row that hold NaN."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    t = t.bfloat16() if dtype == "bf16" else t
    if pad:
        wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, :t.shape[1]] = t
        t = wide[:, :t.shape[1]]
    return t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def close(name, got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, np.argwhere(bad)[:4].tolist(), int(bad.sum()),
                           float(np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-30))))


def rounded(want, err, kind):
    """Tolerance of a result rounded once, `err` before."""
    return err + HALF[kind] * (np.abs(want) + err)


def product(a, b, base=0.0):
    """a @ b.T + base and the tolerance of its float32 sums."""
    return base + a @ b.T, (a.shape[1] + 34) * STEP * (np.abs(a) @ np.abs(b).T + np.abs(base))


class Block:
    def __init__(self, T, H, I, seed=0, pads=(0, 0, 0, 0)):
        rng = np.random.default_rng([seed, T, H, I])
        n = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.dims, self.pads = (T, H, I), pads  # pads of x, base, out and dout
        self.x, self.base, self.dout, self.dxb = (bf16(n(T, H)) for _ in range(4))
        self.w1, self.w2 = bf16(n(2 * I, H) / H ** 0.5), bf16(n(H, I) / I ** 0.5)

    def buffers(self, M, stale):
        import torch

        T, H, I = self.dims
        d = M.FfnDims(H, I)
        buf = lambda n: torch.full((n,), stale, dtype=torch.uint8, device="cuda")  # noqa: E731
        return d, buf(M.ffn_workspace_query(d, T)), buf(M.ffn_saved_query(d, T))

    def forward(self, base="given", saved=True, stale=0xA5):
        import torch

        import mixed_precision_moe_topk_amd as M

        T, H, I = self.dims
        d, ws, sv = self.buffers(M, stale)
        x, b = device(self.x, self.pads[0]), device(self.base, self.pads[1])
        w1, w2 = device(self.w1), device(self.w2)
        out = b if base == "in place" else device(np.full((T, H), np.nan), self.pads[2])
        M.ffn_apply(d, x, w1, w2, None if base == "none" else b, out, ws, saved=sv if saved else None)
        self.kept = d, x, w1, w2, sv
        r = {"out": host(out)}
        if saved:
            gu = sv[:T * 2 * I * 4].view(torch.float32).view(T, 2 * I)
            at = (T * 2 * I * 4 + 255) // 256 * 256
            h = sv[at:at + T * 2 * I * 2].view(torch.bfloat16).view(2, T, I)
            r.update(g=host(gu[:, :I]), u=host(gu[:, I:]), h=host(h[0]), h2=host(h[0]) + host(h[1]))
        return r

    def check_forward(self, r, base="given"):
        x, w1, w2 = (v.astype(np.float64) for v in (self.x, self.w1, self.w2))
        I = self.dims[2]
        g, eg = product(x, w1[:I])
        u, eu = product(x, w1[I:])
        close("g", r["g"], g, rounded(g, eg, "f32"))
        close("u", r["u"], u, rounded(u, eu, "f32"))
        # |d silu| <= 1.1; |silu(g)| <= |g|
        h = OD.silu_mul(g, u)
        eh = 1.1 * np.abs(u) * eg + np.abs(g) * eu + 1.1 * eg * eu + (2.0 ** -20 + 2 * STEP * np.abs(g)) * np.abs(h)
        close("h", r["h"], h, rounded(h, eh, "bf16"))
        close("h in two terms", r["h2"], h, rounded(h, eh, "two terms"))
        out, eo = product(r["h"], w2, 0.0 if base == "none" else self.base.astype(np.float64))
        close("out", r["out"], out, rounded(out, eo, "bf16"))

    def backward(self, kind="f32", dx="base", weights=True, stale=0x5A):
        import torch

        import mixed_precision_moe_topk_amd as M

        T, H, I = self.dims
        d, x, w1, w2, sv = self.kept
        ws = torch.full((M.ffn_workspace_query(d, T),), stale, dtype=torch.uint8, device="cuda")
        dout, dxb = device(self.dout, self.pads[3]), device(self.dxb, self.pads[1])
        nan = lambda *s: device(np.full(s, np.nan), 0, kind)  # noqa: E731
        dw1, dw2 = (nan(2 * I, H), nan(H, I)) if weights else (None, None)
        out = {"base": device(np.full((T, H), np.nan), self.pads[2]), "in place": dxb, "none": None,
               "no base": device(np.full((T, H), np.nan)), "over x": x, "over dout": dout}[dx]
        M.ffn_backward(d, dout, x, w1, w2, sv, dw1, dw2, ws, dx=out, dx_base=None if dx == "no base" else dxb)
        r = {} if out is None else {"dx": host(out)}
        if weights:
            r.update(dw1=host(dw1), dw2=host(dw2))
        dgu = ws[:T * 8 * I].view(torch.bfloat16).view(2, T, 2 * I)
        r["dgu"] = host(dgu[0])
        if weights and kind == "f32":
            r["dgu2"] = host(dgu[0]) + host(dgu[1])
        return r

    def check_backward(self, f, r, kind="f32", dx="base"):
        x, w1, w2, dout = (v.astype(np.float64) for v in (self.x, self.w1, self.w2, self.dout))
        g, u = f["g"], f["u"]
        dh, ed = product(dout, w2.T)
        dg, du = OD.silu_mul_backward(g, u, dh)
        s = OD.sigmoid(g)
        # (a sigmoid below the smallest normal float, 2^-126, may come out as 0: the
        # reciprocal of 1 + e^-g then is subnormal, and those are flushed)
        es = 2.0 ** -21 + STEP * np.abs(g) + 2.0 ** -126 / np.maximum(s, 2.0 ** -1000)
        part = np.abs(1 + g * (1 - s))
        # sigmoid enters dg three times, once times g; a few products round besides
        eg = np.abs(u) * s * part * ed + np.abs(dh * u) * s * (es * (part + np.abs(g)) + 8 * STEP * (1 + np.abs(g)))
        eu = np.abs(g) * s * (ed + np.abs(dh) * (es + 8 * STEP))
        want, err = np.concatenate([dg, du], axis=1), np.concatenate([eg, eu], axis=1)
        close("dg, du", r["dgu"], want, rounded(want, err, "bf16") + 2.0 ** -126)
        terms = 1
        d, h = r["dgu"], f["h"]
        if "dgu2" in r:
            close("dg, du in two terms", r["dgu2"], want, rounded(want, err, "two terms") + 2.0 ** -126)
            terms, h = 2, f["h2"]
        if "dx" in r:
            want, err = product(d, w1.T, 0.0 if dx == "no base" else self.dxb.astype(np.float64))
            close("dx", r["dx"], want, rounded(want, err, "bf16"))
        if "dw1" in r:
            for name, a, b in (("dw1", r["dgu2"] if terms == 2 else d, x), ("dw2", dout, h)):
                want = a.T @ b
                err = (terms * a.shape[0] + 34) * STEP * (1 + 2.0 ** -7) * (np.abs(a).T @ np.abs(b))
                close(name, r[name], want, rounded(want, err, kind))

    def check_precise(self, r):
        """float32 gradients of the weights against the formulas, end to end: in the
        2-norm, where errors of either sign do not add up, 2^-17 of the operands is
        at most 2^-17 of a result without cancellation; 8 times that is far below what
        one bf16 term (2^-9 and more of the norm) would leave."""
        x, w1, w2, dout = (v.astype(np.float64) for v in (self.x, self.w1, self.w2, self.dout))
        _, dw1, dw2 = OD.ffn_backward(dout, x, w1, w2)
        for name, want in (("dw1", dw1), ("dw2", dw2)):
            assert np.linalg.norm(r[name] - want) <= 2.0 ** -14 * np.linalg.norm(want), name


SMALL = [
    # one token, the smallest block, odd sizes either side of the tiles and K steps
    (1, 8, 8), (1, 256, 512), (2, 72, 136), (3, 1000, 264), (15, 128, 128), (16, 256, 512), (17, 264, 120),
    (31, 520, 72), (32, 64, 64), (33, 136, 392), (48, 512, 256), (63, 1032, 8), (64, 1024, 512), (65, 8, 1032),
    (100, 328, 200), (127, 256, 264), (128, 384, 128), (129, 136, 136), (255, 520, 264), (257, 264, 520),
    (300, 1000, 296),
]


@pytest.mark.parametrize("T, H, I", SMALL)
def test_forward_and_backward(T, H, I):
    b = Block(T, H, I)
    f = b.forward()
    b.check_forward(f)
    r = b.backward()
    b.check_backward(f, r)
    b.check_precise(r)


# few rows with long sums: K in parts, and the kernels of few tokens
@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 32, 33, 49, 64, 65, 130, 200])
def test_long_sums(T):
    b = Block(T, 4104, 1544, seed=1)
    f = b.forward()
    b.check_forward(f)
    b.check_backward(f, b.backward("bf16"), "bf16")
    b.check_precise(b.backward())


# few tokens, short sums and many columns: gates and ups, then the product behind them
@pytest.mark.parametrize("T", [2, 40, 64, 66, 256])
@pytest.mark.parametrize("H, I", [(8, 4104), (64, 4104), (72, 4104), (136, 4104), (256, 4104), (328, 4104), (4104, 8),
                                  (4104, 72), (4104, 192), (4104, 264), (4104, 320)])
def test_few_tokens_and_steps(T, H, I):
    b = Block(T, H, I, seed=6)
    b.check_forward(b.forward())


# enough tiles of 256 x 256 for each product in turn, none of them whole
# (the last three: a last round of tiles that two blocks each take, in every direction)
@pytest.mark.parametrize("T, H, I", [(3589, 72, 3400), (3589, 3400, 72), (2309, 2824, 1416), (77, 4104, 3848),
                                     (6140, 2056, 2040), (6140, 4040, 1032), (4090, 2552, 2048)])
def test_large_tiles(T, H, I):
    b = Block(T, H, I, seed=2)
    f = b.forward()
    b.check_forward(f)
    b.check_backward(f, b.backward())


@pytest.mark.parametrize("T, H, I", [(5, 136, 72), (70, 264, 136), (300, 520, 264)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gradient_types(T, H, I, kind):
    b = Block(T, H, I, seed=3)
    f = b.forward()
    b.check_backward(f, b.backward(kind), kind)


@pytest.mark.parametrize("T, H, I", [(1, 256, 72), (37, 264, 136), (130, 136, 264)])
def test_strides_and_bases(T, H, I):
    b = Block(T, H, I, seed=4, pads=(8, 24, 40, 16))
    for base in ("given", "none", "in place"):
        f = b.forward(base)
        b.check_forward(f, base)
        if base != "in place":
            again = b.forward(base, saved=False)
            assert np.array_equal(again["out"], f["out"])
    f = b.forward()
    for dx in ("base", "no base", "in place", "none"):
        b.check_backward(f, b.backward(dx=dx), dx=dx)
    b.check_backward(f, b.backward(weights=False))


def test_gradient_over_its_inputs():
    """Where the weights are frozen; refused where they are not."""
    import mixed_precision_moe_topk_amd as M

    for dx in ("over x", "over dout"):
        b = Block(150, 264, 136, seed=5)
        f = b.forward()
        with pytest.raises(M.MoeError):
            b.backward(dx=dx)
        b.check_backward(f, b.backward(dx=dx, weights=False), dx=dx)


def test_rows_behind_the_batch_and_padding_stay():
    import torch

    import mixed_precision_moe_topk_amd as M

    b = Block(37, 264, 136, seed=6)
    d, ws, sv = b.buffers(M, 0)
    wide = torch.full((60, 264 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    M.ffn_apply(d, device(b.x), device(b.w1), device(b.w2), None, wide[:37, :264], ws)
    assert (wide[37:] == 3.0).all() and (wide[:, 264:] == 3.0).all() and not (wide[:37, :264] == 3.0).all()


def test_same_bits_on_every_run():
    for T, H, I in ((1, 4104, 1544), (33, 2056, 520), (200, 1000, 296), (2309, 2824, 264)):
        b = Block(T, H, I, seed=7)
        f, g = b.forward(stale=0), b.forward(stale=0xFF)
        assert all(np.array_equal(f[k], g[k]) for k in f)
        r, s = b.backward(stale=0), b.backward(stale=0xFF)
        assert all(np.array_equal(r[k], s[k]) for k in r)


def test_a_token_does_not_depend_on_the_others():
    """NaN and infinities of one token reach no other row, and no row of the gradients
    but its own."""
    for T, at in ((1, 0), (40, 7), (200, 150)):
        b = Block(T, 264, 136, seed=8)
        b.x[at, 3] = np.nan
        b.x[(at + 1) % T, 5] = np.nan if T == 1 else np.inf
        bad = {at, (at + 1) % T}
        f = b.forward()
        rest = [t for t in range(T) if t not in bad]
        clean = Block(T, 264, 136, seed=8)
        want = clean.forward()
        assert np.isnan(f["out"][at]).all() and not np.isfinite(f["out"][list(bad)]).any()
        assert np.array_equal(f["out"][rest], want["out"][rest])
        r, w = b.backward(), clean.backward()
        assert np.array_equal(r["dx"][rest], w["dx"][rest]) and np.isnan(r["dx"][at]).all()
        assert np.isnan(r["dw1"]).all()


def test_large_gates():
    """Gates far out on both sides: silu saturates, nothing overflows."""
    b = Block(20, 64, 72, seed=9)
    b.w1[:72] = bf16(b.w1[:72] * 300.0)
    f = b.forward()
    b.check_forward(f)
    r = b.backward()
    assert all(np.isfinite(v).all() for v in r.values())
    b.check_backward(f, r)


def test_no_tokens():
    import torch

    import mixed_precision_moe_topk_amd as M

    b = Block(0, 264, 136)
    d = M.FfnDims(264, 136)
    e = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    w1, w2 = device(b.w1), device(b.w2)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    M.ffn_apply(d, e, w1, w2, None, e, none)
    dw1, dw2 = (torch.full(s, float("nan"), device="cuda") for s in ((272, 264), (264, 136)))
    M.ffn_backward(d, e, e, w1, w2, none, dw1, dw2, none, dx=e)
    assert (dw1 == 0).all() and (dw2 == 0).all()
