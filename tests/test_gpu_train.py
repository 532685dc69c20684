"""The router's losses and gradients and the weighted sum's gradient on the
GPU against their float64 definitions (oracle/train.py).

Tolerances count float32 roundings (u = 2^-24).  With logits at most R below a
row's largest, exp(x - m) is off by at most (3 R + 4) u relative: the
difference, its product with the rounded log2 e and the exp2 (2 u); a row's
sum of E terms adds (E/64 + 6) u <= 22 u, its reciprocal and the product 4 u.
So p is off by (6 R + 34) u relative, below."""
import numpy as np
import pytest

import moe_inputs as MI
from oracle import train as OT
from oracle import formats as F

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dev(a):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _routing(seed, T, E, k, bias=0.0):
    logits = MI.router_logits(seed, T, E, bias)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    w = OT.softmax(np.take_along_axis(logits, ids, axis=1))[0].astype(np.float32)
    return logits, ids, w


def _spread(logits, mask):
    z = np.where(np.isfinite(logits), logits, np.nan)
    z = z if mask is None else z[mask != 0]
    with np.errstate(all="ignore"):
        import warnings

        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            r = np.nanmax(np.nanmax(z, axis=1) - np.nanmin(z, axis=1)) if z.size else 0.0
    return 0.0 if np.isnan(r) else float(r)


class Buffers:
    def __init__(self, T, E, S):
        import torch

        import mixed_precision_moe_topk_amd as M

        self.d = M.LayerDims(E, 256, 512)
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.losses, self.mean = e(2), e(S, E)
        self.counts, self.tokens = e(S, E, t=torch.int32), e(S + 2, t=torch.int32)
        self.ws = torch.full((M.router_loss_query(self.d, T, S),), 0xA5, dtype=torch.uint8, device="cuda")

    def run(self, logits, ids, offs, mask):
        import mixed_precision_moe_topk_amd as M

        M.router_loss(self.d, logits, ids, self.losses, self.counts, self.mean, self.tokens, self.ws,
                      seq_offsets=offs, token_mask=mask)

    def host(self):
        return (self.losses.cpu().numpy(), self.counts.cpu().numpy(), self.mean.cpu().numpy(),
                self.tokens.cpu().numpy())


def check_loss(got, ref, logits, mask):
    losses, counts, mean, tokens = got
    T, E = logits.shape
    assert np.array_equal(counts, ref["counts"]) and np.array_equal(tokens, ref["seq_tokens"])
    R = _spread(logits, mask)
    depth = 16 + 4 + T / 1024 + 17  # additions one probability sum passes through, and its division
    eta = (6 * R + 34 + depth) * U
    assert np.all(np.abs(mean - ref["mean_probs"]) <= eta * ref["mean_probs"] + 2.0 ** -126)
    assert abs(losses[0] - ref["losses"][0]) <= (eta + (8 + 6 + E / 64 + 26) * U) * ref["losses"][0]
    # lse: the sum's relative error, the logarithm's and one rounding at the size of m and of log E
    _, lse = OT.softmax(logits)
    spans, _ = OT.sequences(T, None, mask)
    big = np.nanmax(np.where(np.isfinite(logits), np.abs(logits), 0.0)) if logits.size else 0.0
    delta = (3 * R + 26 + 3 * (big + np.log(E))) * U
    worst = 2 * np.abs(lse).max(initial=0.0) * delta + delta ** 2
    assert abs(losses[1] - ref["losses"][1]) <= worst + (depth + 32) * U * ref["losses"][1]


LOSS_CASES = [  # tokens, experts, top_k, boundaries, masked share, bias, seed
    (1, 1, 1, None, 0.0, 0.0, 1),
    (1, 8, 2, None, 0.0, 0.0, 2),
    (15, 3, 3, None, 0.2, 0.0, 3),
    (64, 64, 6, None, 0.0, 0.0, 4),
    (65, 65, 8, None, 0.0, 2.0, 5),
    (300, 384, 6, [0, 300], 0.1, 2.0, 6),
    (300, 129, 5, [0, 1, 1, 17, 64, 128, 130, 299, 300], 0.2, 1.0, 7),
    (1000, 256, 8, [3, 400, 400, 900], 0.1, 0.0, 8),         # tokens before and behind the sequences
    (257, 1024, 16, [0, 256, 257], 0.0, 0.0, 9),
    (200, 16, 2, list(range(0, 201)), 0.3, 0.0, 10),         # one token a sequence
    (4096, 256, 8, None, 0.0, 0.0, 11),
    (5000, 500, 4, [0, 64, 128, 4000, 5000], 0.5, 2.0, 12),
    (128, 700, 3, [0, 0, 0, 128, 128], 1.0, 0.0, 13),        # every token masked, empty sequences
]


@pytest.mark.parametrize("T,E,k,offs,share,bias,seed", LOSS_CASES)
def test_router_loss_and_gradient(T, E, k, offs, share, bias, seed):
    import torch

    import mixed_precision_moe_topk_amd as M

    rng = np.random.default_rng(seed)
    logits, ids, w = _routing(seed, T, E, k, bias)
    mask = (rng.random(T) >= share).astype(np.uint8) if share else None
    if mask is not None:  # what padded tokens hold must not matter
        logits[mask == 0] = np.nan
        w[mask == 0] = np.inf
    ref = OT.router_loss(logits, ids, offs, mask)
    S = 1 if offs is None else len(offs) - 1
    o = _dev(None if offs is None else np.asarray(offs, np.int32))
    b = Buffers(T, E, S)
    zl, zi, zm = _dev(logits), _dev(ids), _dev(mask)
    b.run(zl, zi, o, zm)
    got = b.host()
    check_loss(got, ref, logits, mask)
    b.ws.fill_(0xFF)
    b.run(zl, zi, o, zm)  # the same bits again, over another workspace content
    for x, y in zip(got, b.host()):
        assert np.array_equal(x.view(np.uint32), y.view(np.uint32))

    dw, dl = rng.standard_normal((T, k)).astype(np.float32), np.array([0.7, -0.3], np.float32) * T
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        kw = dict(weights=_dev(w), dweights=_dev(dw)) if use_w else {}
        if use_l:
            kw.update(dlosses=_dev(dl), counts=b.counts, seq_tokens=b.tokens)
        out = torch.full((T, E), 7.25, device="cuda")
        M.router_backward(b.d, zl, zi, out, seq_offsets=o, token_mask=zm, **kw)
        w64 = np.where(np.isfinite(w), w, 0.0).astype(np.float64)
        g, mag = OT.router_backward(logits, ids, offs, mask, w64, dw.astype(np.float64) if use_w else None,
                                    dl.astype(np.float64) if use_l else None, ref["counts"], ref["seq_tokens"])
        x = out.cpu().numpy()
        outside = np.isnan(g)
        assert np.all(x[outside] == 7.25)  # rows in no sequence
        # p's error three times (p, p in the sum, the sum), the factors and k + 10 roundings of each term
        eta = (3 * (6 * _spread(logits, mask) + 34) + 2 * k + 30) * U
        assert np.all(np.abs(x - g)[~outside] <= eta * mag[~outside] + 2.0 ** -126)


def test_rows_that_masked_experts_leave_empty():
    """Masked experts: -inf, the type's lowest value and NaN; rows in which
    nothing is left have no part and no gradient, and +inf makes NaN."""
    import torch

    import mixed_precision_moe_topk_amd as M

    T, E, k = 70, 40, 4
    logits, ids, w = _routing(31, T, E, k)
    low = np.finfo(np.float32).min
    logits[3, 5:] = -np.inf
    logits[4, 5:] = low
    logits[5, :] = -np.inf
    logits[6, :] = np.nan
    logits[7, 1::2] = np.nan
    logits[8, :] = low
    ids = np.argsort(-np.where(np.isnan(logits), -np.inf, logits), axis=1, kind="stable")[:, :k].astype(np.int32)
    sel = np.take_along_axis(logits, ids, axis=1)
    w = OT.softmax(sel)[0].astype(np.float32)
    w[5:7] = np.nan  # as the router leaves them
    ref = OT.router_loss(logits, ids)
    b = Buffers(T, E, 1)
    zl, zi = _dev(logits), _dev(ids)
    b.run(zl, zi, None, None)
    losses, counts, mean, tokens = b.host()
    assert np.array_equal(counts, ref["counts"]) and np.array_equal(tokens, ref["seq_tokens"])
    eta = (6 * 10 + 34 + 40) * U  # terms more than 10 below their row's largest are under 5e-5 of it
    assert np.all(np.abs(mean - ref["mean_probs"]) <= eta)
    assert abs(losses[0] - ref["losses"][0]) <= 2 * eta * ref["losses"][0] * E
    assert np.isinf(losses[1]) or losses[1] > 1e38  # the lowest value's square leaves float32
    dw = np.ones((T, k), np.float32)
    out = torch.empty((T, E), device="cuda")
    M.router_backward(b.d, zl, zi, out, weights=_dev(w), dweights=_dev(dw * np.arange(k, dtype=np.float32)),
                      dlosses=_dev(np.array([1.0, 0.0], np.float32)), counts=b.counts, seq_tokens=b.tokens)
    x = out.cpu().numpy()
    assert np.all(x[5:7] == 0) and np.all(x[7, 1::2] == 0) and np.all(x[3, 5:] == 0)
    g, mag = OT.router_backward(logits, ids, None, None, np.nan_to_num(w.astype(np.float64)),
                                dw * np.arange(k, dtype=np.float64), np.array([1.0, 0.0]), ref["counts"],
                                ref["seq_tokens"])
    keep = np.ones(T, bool)
    keep[8] = False  # every lse there is of the lowest value's size
    assert np.all(np.abs(x - g)[keep] <= (3 * (6 * 10 + 34) + 40) * U * (mag[keep] + 1.0 / T))
    logits[9, 2] = np.inf
    b.run(_dev(logits), zi, None, None)
    assert np.isnan(b.losses.cpu().numpy()).all()


def test_ids_out_of_range_and_repeated_ids():
    import torch

    import mixed_precision_moe_topk_amd as M

    T, E, k = 33, 12, 3
    logits, ids, w = _routing(41, T, E, k)
    ids[0] = [5, 5, 5]
    ids[1] = [-1, 12, 1 << 30]
    b = Buffers(T, E, 1)
    b.run(_dev(logits), _dev(ids), None, None)
    good = ids[(ids >= 0) & (ids < E)]
    assert np.array_equal(b.counts.cpu().numpy()[0], np.bincount(good, minlength=E))
    dw = np.random.default_rng(3).standard_normal((T, k)).astype(np.float32)
    out = torch.empty((T, E), device="cuda")
    M.router_backward(b.d, _dev(logits), _dev(ids), out, weights=_dev(w), dweights=_dev(dw))
    x = out.cpu().numpy()
    wd = w[0].astype(np.float64) * dw[0]
    term = wd - w[0] * wd.sum()
    assert abs(x[0, 5] - term.sum()) <= 30 * U * np.abs(wd).sum() * 2 and np.count_nonzero(x[0]) <= 1
    assert np.all(x[1] == 0)


def test_gradient_in_place_of_the_logits():
    import mixed_precision_moe_topk_amd as M

    T, E, k = 203, 130, 5
    logits, ids, w = _routing(71, T, E, k)
    b = Buffers(T, E, 2)
    offs = _dev(np.array([0, 101, 203], np.int32))
    z, i = _dev(logits), _dev(ids)
    b.run(z, i, offs, None)
    kw = dict(weights=_dev(w), dweights=_dev(w), dlosses=_dev(np.array([1.0, 1.0], np.float32)), counts=b.counts,
              seq_tokens=b.tokens, seq_offsets=offs)
    import torch

    out = torch.empty_like(z)
    M.router_backward(b.d, z, i, out, **kw)
    M.router_backward(b.d, z, i, z, **kw)
    assert torch.equal(out, z)


def test_no_tokens():
    import mixed_precision_moe_topk_amd as M
    import torch

    b = Buffers(0, 8, 1)
    b.losses.fill_(3.0)
    z, i = torch.empty((0, 8), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    b.run(z, i, None, None)
    losses, counts, mean, tokens = b.host()
    assert not losses.any() and not counts.any() and not mean.any() and not tokens.any()
    M.router_backward(b.d, z, i, z, weights=torch.empty((0, 2), device="cuda"),
                      dweights=torch.empty((0, 2), device="cuda"))
    b = Buffers(0, 8, 3)
    b.run(z, i, torch.zeros(4, dtype=torch.int32, device="cuda"), None)
    assert not any(x.any() for x in b.host())


COMBINE_CASES = [(1, 1, 128), (1, 16, 7168), (7, 3, 384), (64, 8, 7168), (1023, 2, 256), (1024, 1, 256),
                 (1100, 6, 640), (1030, 3, 128), (1025, 8, 2176), (1024, 11, 256), (1024, 16, 128)]


@pytest.mark.parametrize("T,k,H", COMBINE_CASES)
def test_finalize_backward(T, k, H):
    import torch

    import mixed_precision_moe_topk_amd as M

    rng = np.random.default_rng(T + k)
    dout = F.bf16_rne(rng.standard_normal((T, H)).astype(np.float32))
    d64 = F.bf16_to_f32(dout)
    w = rng.random((T, k)).astype(np.float32)
    y2 = rng.standard_normal((T * k, H)).astype(np.float32)
    rows = rng.permutation(T * k).reshape(T, k).astype(np.int32)
    d = M.LayerDims(16, H, 512)
    rw, mag, _ = OT.finalize_backward(d64, w, y2, rows)
    dd, dy, dr, dwt = _dev(dout.view(np.int16)), _dev(y2), _dev(rows), _dev(w)
    want = (w[:, :, None] * d64[:, None, :]).astype(np.float32)  # one rounding: the same bits
    for kind in (None, torch.float32, torch.bfloat16, "in place"):
        dw = torch.full((T, k), np.nan, device="cuda")
        g = dy.clone() if kind == "in place" else None if kind is None else torch.empty(
            (T * k, H), dtype=kind, device="cuda")
        M.finalize_backward(d, dd, dwt, g if kind == "in place" else dy, dr, dw, g)
        # a thread adds H / 256 products in a row, then 6 + 2 joins
        assert np.all(np.abs(dw.cpu().numpy() - rw) <= (H / 256 + 10) * U * mag)
        if kind is None:
            continue
        if kind is torch.bfloat16:
            x = g.view(torch.int16).cpu().numpy().view(np.uint16)[rows]
            assert np.array_equal(x, F.bf16_rne(want))
        else:
            assert np.array_equal(g.cpu().numpy()[rows], want)


def test_finalize_backward_leaves_out_rows_outside_the_batch():
    import torch

    import mixed_precision_moe_topk_amd as M

    for T in (5, 1200):
        k, H = 3, 256
        rng = np.random.default_rng(T)
        dout = F.bf16_rne(rng.standard_normal((T, H)).astype(np.float32))
        rows = np.arange(T * k, dtype=np.int32).reshape(T, k)
        rows[2] = [-1, T * k, 1 << 30]
        dw = torch.empty((T, k), device="cuda")
        dy2 = torch.full((T * k, H), 5.0, device="cuda")
        y2 = torch.ones((T * k, H), device="cuda")
        M.finalize_backward(M.LayerDims(4, H, 512), _dev(dout.view(np.int16)), torch.ones((T, k), device="cuda"),
                            y2, _dev(rows), dw, dy2)
        assert not dw[2].any() and bool(dw[3].all())
        assert bool((dy2[6:9] == 5.0).all()) and not bool((dy2[9:12] == 5.0).all())


def test_binding_refuses_wrong_tensors():
    import torch

    import mixed_precision_moe_topk_amd as M

    T, E, k = 8, 8, 2
    b = Buffers(T, E, 1)
    z, i = torch.zeros((T, E), device="cuda"), torch.zeros((T, k), dtype=torch.int32, device="cuda")

    def refused(f, *a, **kw):
        with pytest.raises(M.MoeError) as ei:
            f(*a, **kw)
        return ei.value.status

    args = (b.losses, b.counts, b.mean, b.tokens)
    assert refused(M.router_loss, b.d, z.half(), i, *args, b.ws) == 1
    assert refused(M.router_loss, b.d, z[:, :4], i, *args, b.ws) == 1
    assert refused(M.router_loss, b.d, z.t(), i, *args, b.ws) == 1  # not contiguous
    assert refused(M.router_loss, b.d, z, i.long(), *args, b.ws) == 1
    assert refused(M.router_loss, b.d, z, i, *args, b.ws.cpu()) == 1
    assert refused(M.router_loss, b.d, z, i, *args, b.ws[:16]) == 3
    assert refused(M.router_loss, b.d, z, i, *args, b.ws, token_mask=z[:, 0]) == 1
    assert refused(M.router_loss, b.d, z, i, *args, b.ws, seq_offsets=i[0, :1]) == 1
    assert refused(M.router_backward, b.d, z, i, z) == 1
    assert refused(M.router_backward, b.d, z, i, z, dlosses=b.losses) == 1  # its counts are missing
    assert refused(M.finalize_backward, b.d, z, z[:, :2], z, i, z[:, :2]) == 1


def test_captured_training_step_replays():
    """Losses and gradients captured into a graph, replayed over other contents
    with eager work between, each time the eager bits."""
    import torch

    import mixed_precision_moe_topk_amd as M

    T, E, k, H = 300, 96, 6, 256
    offs = torch.tensor([0, 10, 170, 300], dtype=torch.int32, device="cuda")
    sets = [_routing(50 + n, T, E, k, 1.0) for n in range(3)]
    b = Buffers(T, E, 3)
    d = M.LayerDims(E, H, 512)
    z, i, w = (_dev(x) for x in sets[0])
    y2, dout = torch.randn(T * k, H, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    rows = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    dl = torch.tensor([0.5, 0.25], device="cuda")
    dw, dz = torch.empty_like(w), torch.empty_like(z)

    def step():
        b.run(z, i, offs, None)
        M.finalize_backward(d, dout, w, y2, rows, dw)
        M.router_backward(b.d, z, i, dz, weights=w, dweights=dw, dlosses=dl, counts=b.counts, seq_tokens=b.tokens,
                          seq_offsets=offs)

    def take():
        torch.cuda.synchronize()
        return [t.cpu().numpy().copy() for t in (b.losses, b.counts, b.mean, b.tokens, dw, dz)]

    eager = []
    for s in sets:
        for dst, src in zip((z, i, w), s):
            dst.copy_(torch.from_numpy(src))
        step()
        eager.append(take())
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for n in (1, 0, 2, 1):
        for dst, src in zip((z, i, w), sets[n]):
            dst.copy_(torch.from_numpy(src))
        b.ws.fill_(0x7F)
        graph.replay()
        for x, y in zip(take(), eager[n]):
            assert np.array_equal(x, y)
        step()  # eager work between replays
    del graph


@pytest.mark.parametrize("E,k", [(16, 6), (300, 16), (1024, 3)])
def test_repeated_ids_are_summed_in_slot_order(E, k):
    """A token that selects one expert in several slots: their terms, added in the
    slots' order, bit for bit.  A slot's term is what it gives with other ids."""
    import torch

    import mixed_precision_moe_topk_amd as M

    T = 203
    rng = np.random.default_rng(E)
    logits, ids, w = _routing(81, T, E, k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    d = M.LayerDims(E, 256, 512)

    def grad(ids):
        out = torch.full((T, E), np.nan, device="cuda")
        M.router_backward(d, _dev(logits), _dev(ids), out, weights=_dev(w), dweights=_dev(dw))
        return out.cpu().numpy()

    term = np.take_along_axis(grad(ids), ids, axis=1)
    same = rng.integers(0, 3, (T, k)).astype(np.int32) * 5 % E
    want = np.zeros((T, E), np.float32)
    for t in range(T):
        for e in set(same[t].tolist()):
            slots = np.nonzero(same[t] == e)[0]
            want[t, e] = term[t, slots[0]]
            for j in slots[1:]:
                want[t, e] = np.float32(want[t, e] + term[t, j])
    other = grad(same) != want
    assert not other.any(), int(other.sum())
