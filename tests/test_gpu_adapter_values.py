"""Low-rank adapters on the GPU at values where the bf16 parts of a float32 could
show: full mantissas, infinities, the largest floats, signed zeros."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import train as OT
from tests.test_gpu_adapter import Case, each, one

pytestmark = pytest.mark.gpu

PATHS = [24, 1032]  # tokens: expand adds up the blocks' sums itself, or takes joined rows (rank 16 at most)


def rest_of_two(v):
    """What two bf16 parts leave of v, relative."""
    v = np.asarray(v, np.float32)
    p = [F.bf16_to_f32(F.bf16_rne(v))]
    p.append(F.bf16_to_f32(F.bf16_rne((v - p[0]).astype(np.float32))))
    return np.abs(v.astype(np.float64) - p[0] - p[1]) / np.abs(v)


def full(rng, n):
    """n floats in +-[1, 2) of which two bf16 parts leave 2^-19 or more."""
    v = (1 + rng.random(64 * n)).astype(np.float32)
    v = v[rest_of_two(v) >= 2.0 ** -19][:n]
    assert len(v) == n
    return v * rng.choice([-1, 1], n).astype(np.float32)


class Diagonal(Case):
    """Rank 1, x = 1 and A = 1: u = scale of the adapter; dout a diagonal.  One
    term in every sum, so that the float32 result is the term."""

    def __init__(self, T, out, scale, diagonal):
        super().__init__(T, len(scale), 1, T, T, out, each, T)
        self.x = np.eye(T, dtype=np.float32)
        self.a = np.ones((len(scale), 1, T), np.float32)
        n = np.arange(T)
        self.b = np.broadcast_to((np.where(n % 2, -1, 1) * 2.0 ** (n % 5 - 2)).astype(np.float32),
                                 (len(scale), 1, T)).copy()
        self.scale = np.asarray(scale, np.float32)
        self.dout = np.diag(np.asarray(diagonal, np.float32))
        self.dxb = np.zeros((T, T), np.float32)

    def wants(self):
        """u B, the diagonal's part of dA and of dB; zero elsewhere."""
        T = self.shape[0]
        t = np.arange(T)
        s, b, d = self.scale.astype(np.float64)[self.ids], self.b[0, 0].astype(np.float64), np.diag(self.dout).astype(np.float64)
        da, db = np.zeros(self.a.shape), np.zeros(self.b.shape)
        da[self.ids, 0, t] = s * d * b
        db[self.ids, 0, t] = s * d
        return s[:, None] * b, da, db


@pytest.mark.parametrize("T", PATHS)
@pytest.mark.parametrize("which,out", [("rows", "bf16"), ("rows", "f32"), ("dout", "f32"), ("both", "f32")])
def test_float32_results_keep_24_bits(T, which, out):
    """Three bf16 parts of the low-rank rows, and of a float32 dout, hold the
    float32 value.  With one of them a power of two every product and every sum
    of parts fits 24 bits: one step (2^-23) is granted.  With both full, v is
    rounded once, the products of parts that are left out are two of 2^-25 and
    one of 2^-34, and six additions are off by a step each: 8 steps, 2^-20.  Two
    parts would leave 2^-19 or more of the values used here."""
    rng = np.random.default_rng(T)
    scale = np.float32([2.0, -0.5, 4.0]) if which == "dout" else full(rng, 3)
    c = Diagonal(T, out, scale, np.ones(T) if which == "rows" else full(rng, T))
    r = c.run(base="none", dx="none")
    o, da, db = c.wants()
    tol = 8 * 2.0 ** -23 if which == "both" else 2.0 ** -23
    if out == "f32":
        assert np.all(np.abs(r["out"] - o) <= 2.0 ** -23 * np.abs(o))
    assert np.all(np.abs(r["da"] - da) <= tol * np.abs(da))
    assert np.all(np.abs(r["db"] - db) <= tol * np.abs(db))


@pytest.mark.parametrize("T", PATHS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_rows_without_an_adapter_are_their_base(T, out):
    """The same bits: negative zeros, the smallest numbers, infinities; NaN stays
    NaN; 0 without a base."""
    K, N = 72, 136
    c = Case(T, 2, 3, K, N, out, lambda rng, T, L: np.where(np.arange(T) % 3 == 1, -1, np.arange(T) % 2), 5)
    tiny = np.float32(2.0 ** -133)  # the smallest bf16
    special = np.float32([-0.0, 0.0, tiny, -tiny, np.inf, -np.inf, np.nan, np.finfo(np.float32).tiny])
    off = c.ids < 0
    c.base[off, :8] = special
    c.dxb[off, 8:16] = special
    for place in ("given", "in place"):
        r = c.run(base=place, dx="base" if place == "given" else place)
        for got, want in ((r["out"][off], c.base[off]), (r["dx"][off], c.dxb[off])):
            nan = np.isnan(want)
            assert np.all(np.isnan(got[nan])) and nan.any()
            other = got[~nan].view(np.uint32) != want[~nan].view(np.uint32)
            assert not other.any(), int(other.sum())
    r = c.run(base="none", dx="none")
    assert not r["out"][off].view(np.uint32).any() and not r["dx"][off].view(np.uint32).any()


@pytest.mark.parametrize("T", PATHS)
def test_the_largest_floats_stay_finite(T):
    """Values that round up to an infinite bf16 (from 511 / 512 of 2^128 on): as a
    scale, hence a low-rank row, and as elements of dout."""
    top = np.finfo(np.float32).max
    c = Diagonal(T, "f32", [top, -top, np.float32(3.397e38)], np.ones(T))
    c.b *= np.float32(2.0 ** -30)
    r = c.run(base="none", dx="none")
    o, da, db = c.wants()
    assert np.all(np.abs(r["out"] - o) <= 2.0 ** -23 * np.abs(o))
    assert np.all(np.abs(r["da"] - da) <= 2.0 ** -23 * np.abs(da))
    assert np.all(np.abs(r["db"] - db) <= 2.0 ** -23 * np.abs(db))
    c = Diagonal(T, "f32", [0.25, -0.25, 0.125], np.where(np.arange(T) % 2, top, -top))
    c.b *= np.float32(0.25)
    r = c.run(base="none", dx="none")
    o, da, db = c.wants()
    assert np.all(np.abs(r["da"] - da) <= 2.0 ** -23 * np.abs(da))
    assert np.all(np.abs(r["db"] - db) <= 2.0 ** -23 * np.abs(db))
    dx = np.zeros((T, T))
    dx += (c.scale.astype(np.float64)[c.ids] * np.diag(c.dout).astype(np.float64) * c.b[0, 0])[:, None]
    assert np.all(np.abs(r["dx"] - dx) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(dx))


INFINITE = ["x", "a", "b", "dout"]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,L,R", [(40, 3, 2), (40, 3, 70), (700, 2, 20), (700, 3, 100), (1100, 1, 40), (3, 3, 1)])
@pytest.mark.parametrize("where", INFINITE)
def test_infinities_in_every_operand(where, T, L, R, out):
    """An infinite element of x, of a factor or of dout: infinities and NaN where
    the float64 definition has them, with its signs, in the results and in all
    gradients; everything else the same bits as without it."""
    K, N = 264, 200
    c = Case(T, L, R, K, N, out, one if L == 1 else each, 77)
    clean = c.run()
    last = L - 1
    t = int(np.nonzero(c.ids == last)[0][-1])
    if where == "x":
        c.x[t, 9] = np.inf
    elif where == "a":
        c.a[last, R // 2, 130] = -np.inf
    elif where == "b":
        c.b[last, R - 1, 17] = np.inf
        c.b[last, 0, 199] = -np.inf
    else:
        c.dout[t, 63] = -np.inf
    r = c.run()
    f = lambda v: v.astype(np.float64)  # noqa: E731
    with np.errstate(invalid="ignore"):
        x, a, b, s, d = f(c.x), f(c.a), f(c.b), f(c.scale), f(c.dout)
        ref = {"out": OT.adapter_apply(x, c.ids, a, b, s, f(c.base))}
        ref["dx"], ref["da"], ref["db"] = OT.adapter_backward(d, x, c.ids, a, b, s, f(c.dxb))
    assert any(np.isinf(v).any() for v in ref.values())
    for k in r:
        fin = np.isfinite(ref[k])
        other = ~((r[k] == ref[k]) | np.isnan(r[k]) & np.isnan(ref[k]))[~fin]
        assert not other.any(), (k, int(other.sum()), int((~fin).sum()))
        changed = (r[k] != clean[k])[fin]
        assert not changed.any(), (k, int(changed.sum()))
