"""The gated block at the ends of the float range: values next to the largest, and
infinities.  Tolerances as in tests/test_gpu_dense.py, where results are finite; an
infinity or NaN of the formulas (in float64, from the operands that the GPU saved) has to
come out as that infinity or NaN."""
import numpy as np
import pytest

from tests.test_gpu_dense import HALF, STEP, Block, close, product, rounded

pytestmark = pytest.mark.gpu
HUGE = 2.0 ** 127


def large(T, H, I):
    """One token whose h, dg and du lie next to 2^128 (1 - 2^-11): bf16 has no number
    between 2^128 (1 - 2^-8) and 2^128, and rounds up from 2^128 (1 - 2^-9) on."""
    b, at = Block(T, H, I, seed=60), T // 2
    units = np.arange(I) % 3 == 0  # so large there, 0 elsewhere
    sign = np.where(np.arange(I) % 2, -1.0, 1.0)
    b.x[:, :2], b.x[at] = 0, 0
    b.x[at, :2] = 1
    near = np.array([2.0 ** 64, -2.0 ** 52])  # adds up to 2^64 (1 - 2^-12)
    b.w1[:, :2] = 0
    b.w1[:I, :2] = units[:, None] * near
    b.w1[I:, :2] = (units * sign)[:, None] * near
    b.w1[:, 2:] *= 2.0 ** -30
    b.w2 *= 2.0 ** -30
    b.w2[:2] = 2.0 ** -30 * np.where(np.arange(I) % 5, 1.0, -1.0)
    b.dout[at] *= 2.0 ** -20
    b.dout[at, :2] = 2.0 ** 94, -2.0 ** 82
    return b, at


@pytest.mark.parametrize("T, H, I", [(1, 72, 40), (3, 264, 136), (40, 4104, 72), (300, 264, 136), (2309, 1032, 1416)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_finite_values_stay_finite(T, H, I, kind):
    b, at = large(T, H, I)
    f = b.forward()
    assert np.abs(f["h2"][at]).max() > HUGE and np.isfinite(f["h"]).all()
    b.check_forward(f)
    r = b.backward(kind)
    assert np.isfinite(r["dgu"]).all()
    x, w1, w2, dout = (v.astype(np.float64) for v in (b.x, b.w1, b.w2, b.dout))
    # the gradients of the large units, from what was saved: sigmoid is 1, 1 - sigmoid 0
    dh = dout[at] @ w2
    big = np.abs(f["g"][at]) > 0
    want = np.concatenate([(dh * f["u"][at])[big], (dh * f["g"][at])[big]])
    assert np.abs(want).max() > HUGE
    both = np.concatenate([big, big])
    err = (H + 40) * STEP * np.abs(want)
    close("dg, du", r["dgu"][at][both], want, rounded(want, err, "bf16"))
    if kind == "f32":
        close("dg, du in two terms", r["dgu2"][at][both], want, rounded(want, err, "two terms"))
    d, h = (r["dgu2"], f["h2"]) if kind == "f32" else (r["dgu"], f["h"])
    for name, a, c, k in (("dx", r["dgu"], w1.T, "bf16"), ("dw1", d.T, x.T, kind), ("dw2", dout.T, h.T, kind)):
        base = b.dxb.astype(np.float64) if name == "dx" else 0.0
        want, err = product(a, c, base)
        tol = rounded(want, 2 * err, k)
        fits = np.abs(a) @ np.abs(c).T < 2 * HUGE * (1 - 2.0 ** -12)  # no sum on the way may overflow
        assert fits.mean() > (0.5 if name == "dx" else 0.9)
        close(name, np.where(fits, r[name], 0), np.where(fits, want, 0), tol)


@pytest.mark.parametrize("T, H, I, dx", [(1, 72, 40, "base"), (5, 136, 72, "base"), (40, 264, 136, "base"),
                                         (300, 520, 264, "base"), (5000, 64, 72, "base"), (2309, 1032, 1416, "base"),
                                         (2309, 2824, 1416, "none"), (130, 5752, 904, "none")])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_infinities(T, H, I, dx, kind):
    b = Block(T, H, I, seed=61)
    b.dout[0, 3], b.dout[T // 2, 5], b.dout[T - 1, 6] = np.inf, -np.inf, np.inf
    b.x[T // 3, 4], b.x[2 * T // 3, 2] = np.inf, -np.inf
    f = b.forward()
    r = b.backward(kind, dx=dx)
    x, dout = b.x.astype(np.float64), b.dout.astype(np.float64)
    d, h = (r["dgu2"], f["h2"]) if kind == "f32" else (r["dgu"], f["h"])
    seen = 0
    with np.errstate(invalid="ignore", over="ignore"):
        for name, a, c in (("dw1", d, x), ("dw2", dout, h)):
            want = a.T @ c
            odd = ~np.isfinite(want)
            seen += int(np.isinf(want).sum())
            assert np.array_equal(r[name][odd], want[odd], equal_nan=True), name
            err = (2 * T + 34) * STEP * (1 + 2.0 ** -7) * (np.abs(a).T @ np.abs(c))
            tol = err + HALF[kind] * (np.abs(want) + err)
            close(name, np.where(odd, 0, r[name]), np.where(odd, 0, want), np.where(odd, 0, tol))
    assert seen > 0


@pytest.mark.parametrize("T, H, I", [(5, 136, 72), (300, 520, 264), (5000, 64, 72), (130, 5752, 904)])
def test_infinities_leave_the_other_rows(T, H, I):
    """A tile that is taken again keeps the bits of its finite sums."""
    got = []
    for value in (1.0, np.inf):
        b = Block(T, H, I, seed=62)
        b.dout[T // 2, 7] = value
        b.forward()
        got.append(b.backward(dx="none")["dw2"])
    rest = np.arange(H) != 7
    assert np.array_equal(got[0][rest], got[1][rest]) and np.isfinite(got[0]).all()
    assert not np.isfinite(got[1][7]).any()


def test_infinities_captured():
    """The second round of such tiles in a graph, between replays over finite inputs."""
    import torch

    import mixed_precision_moe_topk_amd as M

    T, H, I = 700, 264, 136
    b = Block(T, H, I, seed=63)
    f = b.forward()
    d, x, w1, w2, saved = b.kept
    dout = torch.from_numpy(b.dout).cuda().bfloat16()
    new = lambda: (torch.empty(2 * I, H, device="cuda"), torch.empty(H, I, device="cuda"),  # noqa: E731
                   torch.empty(M.ffn_workspace_query(d, T), dtype=torch.uint8, device="cuda"))
    one, two = new(), new()
    M.ffn_backward(d, dout, x, w1, w2, saved, *one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.ffn_backward(d, dout, x, w1, w2, saved, *one)
    for turn in range(6):
        dout[T // 2, 7] = float("inf") if turn % 2 else 1.0
        graph.replay()
        M.ffn_backward(d, dout, x, w1, w2, saved, *two)
        torch.cuda.synchronize()
        for a, c in zip(one[:2], two[:2]):
            assert torch.equal(a.nan_to_num(5.0, 6.0, 7.0), c.nan_to_num(5.0, 6.0, 7.0)), turn
        assert bool(two[1].isfinite().all()) == (turn % 2 == 0)
    assert np.isfinite(f["h2"]).all()
    del graph
