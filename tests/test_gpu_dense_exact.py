"""The gated block on operands whose float32 sums are exact, whatever their order: every
result has to be equal, element by element, so that a step of K, a part, a tile or
the second bf16 term of an operand that is lost or taken twice shows however
long the sums are (an error bound grows with their length and may hide one).

The operands: a token has one feature (1), so that its gates and ups are entries of
w1, whole numbers; gates are 18 or more, where sigmoid is 1 in float32; a token
has one gradient at most.  "twelve bits": products of two odd numbers from 33 to 63,
which take both bf16 terms (8 bits each); "powers": powers of two, with w2 full
of ones of either sign.  A sum is exact when the magnitudes of its terms, in units
of the largest power of two that divides them all, add up to less than 2^24; `total`
asserts it of every sum."""
import pytest

pytestmark = pytest.mark.gpu


class Exact:
    def __init__(self, T, H, I, values, seed):
        import torch

        self.dims, self.values = (T, H, I), values
        gen = torch.Generator(device="cuda").manual_seed(seed)
        ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
        sign = lambda *s: 2 * ints(0, 2, *s) - 1  # noqa: E731
        row = lambda: torch.randint(0, H, (T,), generator=gen, device="cuda")  # noqa: E731
        bf16 = torch.bfloat16
        self.feature, self.result = row(), row()
        self.x = torch.zeros((T, H), dtype=bf16, device="cuda")
        self.x[torch.arange(T, device="cuda"), self.feature] = 1
        if values == "powers":
            self.unit = 32
            gate = lambda *s: 32 * ints(1, 3, *s)  # noqa: E731
            up = lambda *s: ints(1, 3, *s) * sign(*s)  # noqa: E731
            given = sign(T)
            self.w2 = sign(H, I).to(bf16)
        else:
            self.unit = 1
            odd = lambda *s: 33 + 2 * ints(0, 16, *s)  # noqa: E731
            gate, up = odd, lambda *s: odd(*s) * sign(*s)
            # some 16 of a row of w2 and at most some 30 tokens of a result
            given = odd(T) * sign(T) * (torch.rand(T, generator=gen, device="cuda") < 30 * H / T)
            self.w2 = (sign(H, I) * (torch.rand((H, I), generator=gen, device="cuda") < 16 / I)).to(bf16)
        self.dout = torch.zeros((T, H), dtype=bf16, device="cuda")
        self.dout[torch.arange(T, device="cuda"), self.result] = given.to(bf16)
        self.w1 = torch.empty((2 * I, H), dtype=bf16, device="cuda")
        self.w1[:I], self.w1[I:] = gate(I, H), up(I, H)

    def total(self, a, b):
        """a @ b in float64, in slices of its terms."""
        out, most = 0.0, 0.0
        for k in range(0, a.shape[1], 1 << 16):
            p, q = a[:, k:k + (1 << 16)].double(), b[k:k + (1 << 16)].double()
            out, most = out + p @ q, most + p.abs() @ q.abs()
        assert most.max() < self.unit * 2 ** 24
        return out

    def run(self, kind="f32", dx=True, weights=True):
        import torch

        import mixed_precision_moe_topk_amd as M

        T, H, I = self.dims
        d, bf16 = M.FfnDims(H, I), torch.bfloat16
        buf = lambda n: torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")  # noqa: E731
        nan = lambda t, *s: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        ws, saved, out = buf(M.ffn_workspace_query(d, T)), buf(M.ffn_saved_query(d, T)), nan(bf16, T, H)
        M.ffn_apply(d, self.x, self.w1, self.w2, None, out, ws, saved=saved)
        gu = saved[:T * 8 * I].view(torch.float32).view(T, 2, I)
        h = saved[(T * 8 * I + 255) // 256 * 256:][:T * 4 * I].view(bf16).view(2, T, I)
        g, u = (self.w1[r * I:(r + 1) * I].T[self.feature].double() for r in (0, 1))
        assert torch.equal(gu[:, 0].double(), g) and torch.equal(gu[:, 1].double(), u)
        want = g * u
        first = want.to(bf16)
        assert torch.equal(h[0], first) and torch.equal(h[1].double(), want - first.double())
        assert torch.equal(out, self.total(first, self.w2.T).to(bf16))

        t = torch.float32 if kind == "f32" else bf16
        dw1, dw2 = (nan(t, 2 * I, H), nan(t, H, I)) if weights else (None, None)
        got = nan(bf16, T, H) if dx else None
        ws.fill_(0x5A)
        M.ffn_backward(d, self.dout, self.x, self.w1, self.w2, saved, dw1, dw2, ws, dx=got)
        dh = self.total(self.dout, self.w2)
        both = torch.cat([dh * u, dh * g], dim=1)
        hi = both.to(bf16)
        dgu = ws[:T * 8 * I].view(bf16).view(2, T, 2 * I)
        assert torch.equal(dgu[0], hi)
        if weights and kind == "f32":
            assert torch.equal(dgu[1].double(), both - hi.double())
            hi_w, h_w = both, want
        else:
            hi_w, h_w = hi, first
        if self.values != "powers":  # (both terms are at work)
            assert (both != hi.double()).any() and (want != first.double()).any()
        if dx:
            assert torch.equal(got, self.total(hi, self.w1).to(bf16))
        if weights:
            for name, grad, a, b in (("dw1", dw1, hi_w, self.x), ("dw2", dw2, self.dout, h_w)):
                for r in range(0, grad.shape[0], 1 << 16):
                    part = self.total(a[:, r:r + (1 << 16)].T, b)
                    assert torch.equal(grad[r:r + (1 << 16)], part.to(t)), name


# What the choice of tiles (tests/test_dense_choice.py holds it to that) makes of them:
# products in parts, tiles of 256 x 256 and of 128 x 128, and last rounds of tiles that two
# blocks share, of each product with an operand across k
ALL = [(70001, 136, 72), (5000, 64, 264), (2309, 2824, 1416), (6140, 2056, 2040), (6140, 4040, 1032),
       (5248, 264, 3104), (3994, 520, 4112), (5309, 144, 136)]


@pytest.mark.parametrize("T, H, I", ALL)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gradients(T, H, I, kind):
    Exact(T, H, I, "twelve bits", 1).run(kind)


INPUT = [(8820, 1800, 136), (3385, 4752, 64), (70001, 136, 72), (643, 3576, 2352)]


@pytest.mark.parametrize("T, H, I", INPUT)
def test_gradient_of_the_input_alone(T, H, I):
    Exact(T, H, I, "twelve bits", 2).run(weights=False)


WEIGHTS = [(70001, 136, 72), (130, 5752, 904), (3413, 408, 1736), (1033, 1816, 3616)]


@pytest.mark.parametrize("T, H, I", WEIGHTS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gradients_of_the_weights_alone(T, H, I, kind):
    Exact(T, H, I, "twelve bits", 3).run(kind, dx=False)


@pytest.mark.parametrize("T, kind", [(1, "f32"), (3, "bf16")])
def test_largest_weights(T, kind):
    """2^30 weights a matrix: every row of w1 (2^33 bytes of float32 gradients) and of w2
    counts."""
    Exact(T, 4096, 1 << 18, "powers", 4).run(kind)


@pytest.mark.parametrize("H", [2048, 6144, 6152, 8200])
def test_one_token(H):
    """Either side of where a wave takes one row of weights or two."""
    Exact(1, H, 136, "twelve bits", 5).run()


@pytest.mark.parametrize("N", [6144, 6152, 8200])
@pytest.mark.parametrize("K", [16, 1040, 9232])
def test_one_token_int8(N, K):
    import torch

    import mixed_precision_moe_topk_amd as M

    gen = torch.Generator(device="cuda").manual_seed(N + K)
    rand = lambda *s: torch.randint(-128, 128, s, generator=gen, device="cuda").to(torch.int8)  # noqa: E731
    codes, w, d = rand(1, K), rand(N, K), M.Int8Dims(K, N, "f32")
    one, out = torch.ones(N, device="cuda"), torch.full((1, N), float("nan"), device="cuda")
    ws = torch.empty(max(M.int8_workspace_query(d, 1), 16), dtype=torch.uint8, device="cuda")
    M.int8_matmul(d, codes, one[:1], w, one, None, out, ws)
    assert torch.equal(out.double(), (codes.double() @ w.double().T).float().double())
