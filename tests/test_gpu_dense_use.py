"""The dense operators as a program uses them: beside the layer, captured into graphs,
on several streams, with workspaces of longer batches, far apart rows, and what
the binding refuses."""
import numpy as np
import pytest

import moe_inputs as MI
from oracle import dense as OD
from oracle import formats as F
from tests.harness import Problem
from tests.test_gpu_dense import STEP, Block, close, device, host, product, rounded
from tests.test_gpu_int8 import Block8

pytestmark = pytest.mark.gpu


def bits(t):
    """bf16 of int16 bits on the GPU, as float64."""
    return F.bf16_to_f32(t.cpu().numpy().view(np.uint16)).astype(np.float64)


@pytest.mark.parametrize("T", [1, 24, 150])
def test_beside_the_layer(T):
    """A training step and a serving step of layer and shared expert: the block adds to
    the layer's output in place, and its gradient to the one of the layer's input."""
    import torch

    import mixed_precision_moe_topk_amd as M

    E, k, H, I = 8, 2, 256, 256
    p = Problem(MI.small_workload(T, E, k, H, I, "mxfp4", "bf16", 17, 1.0), experts_for_oracle=[])
    b = Block(T, H, 136, seed=11)
    b.x = F.bf16_to_f32(p.hidden)
    d, ws, saved = b.buffers(M, 0xA5)
    lay = M.workspace_layout(p.dims, T, k)
    layer_ws = torch.full((lay.total,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.empty((T, H), dtype=torch.int16, device="cuda")
    w1, w2 = device(b.w1), device(b.w2)
    M.run_ws(p.dims, p.h_dev, p.l_dev, p.weights, p.scales, k, out, layer_ws)
    routed = bits(out)
    M.ffn_apply(d, p.h_dev, w1, w2, out, out, ws, saved=saved)
    h = host(saved[(T * 8 * 136 + 255) // 256 * 256:][:T * 2 * 136].view(torch.bfloat16).view(T, 136))
    want, err = product(h, b.w2.astype(np.float64), routed)
    close("out", bits(out), want, rounded(want, err, "bf16"))

    # backward: the router's weights from the layer's rows, the block into dx_base
    dout = device(b.dout)
    y2 = layer_ws[lay.y2:lay.y2 + 4 * T * k * H].view(torch.float32).view(T * k, H)
    topk_w = layer_ws[lay.topk_w:lay.topk_w + 4 * T * k].view(torch.float32).view(T, k)
    slot_row = layer_ws[lay.slot_row:lay.slot_row + 4 * T * k].view(torch.int32).view(T, k)
    dweights = torch.empty((T, k), device="cuda")
    M.finalize_backward(p.dims, dout, topk_w, y2, slot_row, dweights)
    rows = host(y2)[slot_row.cpu().numpy()]
    want = (rows * b.dout[:, None].astype(np.float64)).sum(2)
    assert np.abs(host(dweights) - want).max() <= (H + 34) * STEP * np.abs(rows * b.dout[:, None]).sum(2).max()
    dx = device(b.dxb)
    dw1, dw2 = torch.empty(w1.shape, device="cuda"), torch.empty(w2.shape, device="cuda")
    M.ffn_backward(d, dout, p.h_dev, w1, w2, saved, dw1, dw2, ws, dx=dx, dx_base=dx)
    dgu, rest = host(ws[:T * 8 * 136].view(torch.bfloat16).view(2, T, 272))
    want, err = product(dgu, b.w1.T.astype(np.float64), b.dxb.astype(np.float64))
    close("dx", host(dx), want, rounded(want, err, "bf16"))
    want, err = product((dgu + rest).T, b.x.T.astype(np.float64))
    close("dw1", host(dw1), want, rounded(want, 2 * err, "f32"))

    # serving: the same weights in 8 bits
    e = Block8(T, H, 144, seed=12)
    e.x = b.x
    codes, scales = torch.empty((288, H), dtype=torch.int8, device="cuda"), torch.empty(288, device="cuda")
    master = device(np.random.default_rng(3).standard_normal((288, H)), 0, "f32")
    M.int8_quantize(master, codes, scales)
    e.w1, e.s1 = codes.cpu().numpy(), scales.cpu().numpy()
    M.run_ws(p.dims, p.h_dev, p.l_dev, p.weights, p.scales, k, out, layer_ws)
    e.base = bits(out).astype(np.float32)
    d8 = M.FfnDims(H, 144)
    ws8 = torch.empty(M.ffn_int8_workspace_query(d8, T), dtype=torch.uint8, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    M.ffn_int8_apply(d8, p.h_dev, codes, scales, dev(e.w2), dev(e.s2), out, out, ws8)
    e.check(bits(out))


@pytest.mark.parametrize("T, H, I", [(1, 4096, 528), (40, 2048, 272), (300, 272, 528)])
def test_captured_and_replayed(T, H, I):
    """Forward and backward in bf16 and the block in int8 in one graph; replays over
    other inputs, stale workspaces and eager work in between."""
    import torch

    import mixed_precision_moe_topk_amd as M

    d = M.FfnDims(H, I)
    gen = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    w1, w2 = (rand(2 * I, H) / H ** 0.5).bfloat16(), (rand(H, I) / I ** 0.5).bfloat16()
    q1, q2 = torch.empty(w1.shape, dtype=torch.int8, device="cuda"), torch.empty(w2.shape, dtype=torch.int8, device="cuda")
    s1, s2 = torch.empty(2 * I, device="cuda"), torch.empty(H, device="cuda")
    M.int8_quantize(w1, q1, s1)
    M.int8_quantize(w2, q2, s2)

    def buffers():
        e = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        return dict(x=rand(T, H).bfloat16(), base=rand(T, H).bfloat16(), dout=rand(T, H).bfloat16(),
                    out=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"),
                    out8=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"),
                    dx=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"),
                    dw1=torch.empty(2 * I, H, device="cuda"), dw2=torch.empty(H, I, device="cuda"),
                    ws=e(M.ffn_workspace_query(d, T)), saved=e(M.ffn_saved_query(d, T)),
                    ws8=e(M.ffn_int8_workspace_query(d, T)))

    def step(c):
        M.ffn_apply(d, c["x"], w1, w2, c["base"], c["out"], c["ws"], saved=c["saved"])
        M.ffn_backward(d, c["dout"], c["x"], w1, w2, c["saved"], c["dw1"], c["dw2"], c["ws"], dx=c["dx"])
        M.ffn_int8_apply(d, c["x"], q1, s1, q2, s2, c["base"], c["out8"], c["ws8"])

    outs = ("out", "out8", "dx", "dw1", "dw2")
    eager, kept = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kept)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kept)
    for turn in range(4):
        for name in ("x", "base", "dout"):
            kept[name].copy_(rand(T, H))
            eager[name].copy_(kept[name])
        for name in ("ws", "saved", "ws8"):
            kept[name].fill_(0xFF if turn % 2 else 0x7E)
        for name in outs:
            kept[name].zero_()
        step(eager)  # eager work between replays
        graph.replay()
        torch.cuda.synchronize()
        for name in outs:
            assert torch.equal(kept[name], eager[name]), (turn, name)
    del graph


def test_two_streams_with_their_own_workspaces():
    import torch

    import mixed_precision_moe_topk_amd as M

    H, I = 1032, 520
    d = M.FfnDims(H, I)
    halves = []
    for i, T in enumerate((64, 300)):
        b = Block(T, H, I, seed=20 + i)
        c = dict(b=b, st=torch.cuda.Stream(), x=device(b.x), base=device(b.base), w1=device(b.w1), w2=device(b.w2),
                 dout=device(b.dout), out=device(np.full((T, H), np.nan)), dx=device(np.full((T, H), np.nan)),
                 dw1=torch.empty(2 * I, H, device="cuda"), dw2=torch.empty(H, I, device="cuda"))
        c["d"], c["ws"], c["saved"] = b.buffers(M, 0xA5)
        halves.append(c)
    torch.cuda.synchronize()
    for _ in range(3):
        for c in halves:
            M.ffn_apply(d, c["x"], c["w1"], c["w2"], c["base"], c["out"], c["ws"], saved=c["saved"], stream=c["st"])
        for c in halves:
            M.ffn_backward(d, c["dout"], c["x"], c["w1"], c["w2"], c["saved"], c["dw1"], c["dw2"], c["ws"],
                           dx=c["dx"], stream=c["st"])
    torch.cuda.synchronize()
    for c in halves:
        b = c["b"]
        f = b.forward()
        assert np.array_equal(host(c["out"]), f["out"])
        r = b.backward(dx="no base")
        assert all(np.array_equal(host(c[k]), r[k]) for k in ("dx", "dw1", "dw2"))


def test_a_workspace_of_a_longer_batch():
    import torch

    import mixed_precision_moe_topk_amd as M

    H, I = 4096, 528
    d = M.FfnDims(H, I)
    ws = torch.full((M.ffn_workspace_query(d, 700),), 0xA5, dtype=torch.uint8, device="cuda")
    saved = torch.full((M.ffn_saved_query(d, 700),), 0xA5, dtype=torch.uint8, device="cuda")
    ws8 = torch.full((M.ffn_int8_workspace_query(d, 700),), 0xA5, dtype=torch.uint8, device="cuda")
    for T in (1, 3, 64, 65, 250, 700):
        b = Block(T, H, I, seed=30)
        out = device(np.full((T, H), np.nan))
        M.ffn_apply(d, device(b.x), device(b.w1), device(b.w2), device(b.base), out, ws, saved=saved)
        f = b.forward()
        assert np.array_equal(host(out), f["out"])
        dw1, dw2 = torch.empty(2 * I, H, device="cuda"), torch.empty(H, I, device="cuda")
        M.ffn_backward(d, device(b.dout), device(b.x), device(b.w1), device(b.w2), saved, dw1, dw2, ws)
        r = b.backward(dx="none")
        assert np.array_equal(host(dw1), r["dw1"]) and np.array_equal(host(dw2), r["dw2"])
        e = Block8(T, H, I, seed=31)
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        M.ffn_int8_apply(d, device(e.x), dev(e.w1), dev(e.s1), dev(e.w2), dev(e.s2), device(e.base), out, ws8)
        assert np.array_equal(host(out), e.run())


@pytest.mark.parametrize("T", [1, 50, 300])
def test_output_over_the_input(T):
    """out may be x, and base x as well: a residual in place."""
    import torch

    import mixed_precision_moe_topk_amd as M

    b = Block(T, 272, 144, seed=35)
    b.base = b.x
    d, ws, _ = b.buffers(M, 0xA5)
    w1, w2 = device(b.w1), device(b.w2)
    for base in ("none", "given"):
        want = b.forward(base)["out"]
        x = device(b.x)
        M.ffn_apply(d, x, w1, w2, None if base == "none" else x, x, ws)
        assert np.array_equal(host(x), want)
        e = Block8(T, 272, 144, seed=36)
        e.base = e.x
        want = e.run(base)
        x = device(e.x)
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        ws8 = torch.empty(M.ffn_int8_workspace_query(d, T), dtype=torch.uint8, device="cuda")
        M.ffn_int8_apply(d, x, dev(e.w1), dev(e.s1), dev(e.w2), dev(e.s2), None if base == "none" else x, x, ws8)
        assert np.array_equal(host(x), want)


def test_rows_far_apart():
    """Rows that lie more than 2^32 bytes behind the first."""
    import torch

    import mixed_precision_moe_topk_amd as M

    T, H, I, stride = 600, 64, 72, 1 << 22
    b = Block(T, H, I, seed=40)
    room = torch.empty((T - 1) * stride + 2 * H, dtype=torch.bfloat16, device="cuda")
    view = lambda at: room[at:].as_strided((T, H), (stride, 1))  # noqa: E731
    x, out = view(0), view(H)
    x.copy_(device(b.x))
    d, ws, saved = b.buffers(M, 0)
    M.ffn_apply(d, x, device(b.w1), device(b.w2), device(b.base), out, ws, saved=saved)
    assert np.array_equal(host(out), b.forward()["out"])
    dw1, dw2 = torch.empty(2 * I, H, device="cuda"), torch.empty(H, I, device="cuda")
    out.copy_(device(b.dout))
    M.ffn_backward(d, out, x, device(b.w1), device(b.w2), saved, dw1, dw2, ws)
    r = b.backward(dx="none")
    assert np.array_equal(host(dw1), r["dw1"]) and np.array_equal(host(dw2), r["dw2"])
    codes, scales = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    M.int8_quantize(x, codes, scales)
    want, ws_ = OD.int8_quantize(b.x)
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), ws_)


@pytest.mark.parametrize("T", [1, 3])
def test_largest_weights(T):
    """2^30 weights a matrix: gates and ups lie 2^31 bytes apart, w1 ends behind 2^32."""
    import torch

    import mixed_precision_moe_topk_amd as M

    H, I, last = 4096, 1 << 18, 512
    d = M.FfnDims(H, I)
    gen = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda scale, *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=gen)  # noqa: E731
    x, dout = rand(1, T, H), rand(1, T, H)
    w1, w2 = rand(H ** -0.5, 2 * I, H), rand(I ** -0.5, H, I)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(M.ffn_workspace_query(d, T), dtype=torch.uint8, device="cuda")
    saved = torch.empty(M.ffn_saved_query(d, T), dtype=torch.uint8, device="cuda")
    dw1, dw2 = torch.empty_like(w1), torch.empty_like(w2)
    M.ffn_apply(d, x, w1, w2, None, out, ws, saved=saved)
    M.ffn_backward(d, dout, x, w1, w2, saved, dw1, dw2, ws, dx=dx)
    gu = saved[:T * 8 * I].view(torch.float32).view(T, 2, I)
    h = saved[(T * 8 * I + 255) // 256 * 256:][:T * 2 * I].view(torch.bfloat16).view(T, I)
    dgu = ws[:T * 4 * I].view(torch.bfloat16).view(T, 2 * I)
    f = lambda t: t.double()  # noqa: E731
    half = 2.0 ** -8
    for name, got, a, c, kind in (
            ("g", gu[:, 0, -last:], f(x), f(w1[I - last:I]).T, 0.0), ("u", gu[:, 1, -last:], f(x), f(w1[-last:]).T, 0.0),
            ("out", out, f(h), f(w2).T, half), ("dx", dx[:, -last:], f(dgu), f(w1[:, -last:]), half),
            ("dw1", dw1[-last:], f(dgu[:, -last:]).T, f(x), half), ("dw2", dw2[-last:], f(dout[:, -last:]).T, f(h), half)):
        want, bound = a @ c, a.abs() @ c.abs()
        err = (2 * a.shape[1] + 34) * STEP * bound
        assert ((f(got) - want).abs() <= err + kind * (want.abs() + err)).all(), name
    w1 = torch.randint(-127, 128, w1.shape, generator=gen, dtype=torch.int8, device="cuda")
    d8 = M.Int8Dims(H, 1 << 18, "f32")
    codes, scales = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    M.int8_quantize(x, codes, scales)
    got = torch.empty((T, 1 << 18), device="cuda")
    ws8 = torch.empty(M.int8_workspace_query(d8, T), dtype=torch.uint8, device="cuda")
    one = torch.ones(1 << 18, device="cuda")
    M.int8_matmul(d8, codes, torch.ones(T, device="cuda"), w1[-(1 << 18):], one, None, got, ws8)
    assert (f(got[:, -last:]) == f(codes) @ f(w1[-last:]).T).all()


def test_long_batches():
    """More than 2^16 tokens, odd: the weights' gradients sum over all of them."""
    import torch

    import mixed_precision_moe_topk_amd as M

    T, H, I = 70001, 136, 72
    d = M.FfnDims(H, I)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dout = rand(T, H).bfloat16(), rand(T, H).bfloat16()
    w1, w2 = (rand(2 * I, H) / H ** 0.5).bfloat16(), (rand(H, I) / I ** 0.5).bfloat16()
    out, dx = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(M.ffn_workspace_query(d, T), dtype=torch.uint8, device="cuda")
    saved = torch.empty(M.ffn_saved_query(d, T), dtype=torch.uint8, device="cuda")
    dw1, dw2 = torch.empty(w1.shape, device="cuda"), torch.empty(w2.shape, device="cuda")
    M.ffn_apply(d, x, w1, w2, None, out, ws, saved=saved)
    M.ffn_backward(d, dout, x, w1, w2, saved, dw1, dw2, ws, dx=dx)
    h = saved[(T * 8 * I + 255) // 256 * 256:][:T * 4 * I].view(torch.bfloat16).view(2, T, I).double()
    dgu = ws[:T * 8 * I].view(torch.bfloat16).view(2, T, 2 * I).double()
    f = lambda t: t.double()  # noqa: E731
    for name, got, a, c, kind in (("out", out, h[0], f(w2).T, 2.0 ** -8), ("dx", dx, dgu[0], f(w1), 2.0 ** -8),
                                  ("dw1", dw1, dgu.sum(0).T, f(x), 2.0 ** -24),
                                  ("dw2", dw2, f(dout).T, h.sum(0), 2.0 ** -24)):
        want, bound = a @ c, a.abs() @ c.abs()
        err = (2 * a.shape[1] + 34) * STEP * bound
        assert ((f(got) - want).abs() <= err + kind * (want.abs() + err)).all(), name


def test_binding_refuses():
    import torch

    import mixed_precision_moe_topk_amd as M

    b = Block(4, 64, 72, seed=50)
    d, ws, saved = b.buffers(M, 0)
    x, w1, w2, out = device(b.x), device(b.w1), device(b.w2), device(b.base)
    codes, scales = torch.empty((4, 64), dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")

    def refused(fn, *args, status=1, **kw):
        with pytest.raises(M.MoeError) as e:
            fn(*args, **kw)
        assert e.value.status == status

    refused(M.ffn_apply, d, x.float(), w1, w2, None, out, ws)
    refused(M.ffn_apply, d, x, w1[:, :56], w2, None, out, ws)
    refused(M.ffn_apply, d, x, w1, w2.T, None, out, ws)
    refused(M.ffn_apply, d, x, w1, w2.T.contiguous().T, None, out, ws)
    refused(M.ffn_apply, d, x, w1, w2, out[:3], out, ws)
    refused(M.ffn_apply, d, x.T.contiguous().T, w1, w2, None, out, ws)
    refused(M.ffn_apply, d, x, w1, w2, None, out, ws.cpu())
    refused(M.ffn_apply, d, x, w1, w2, None, out, ws[:16], status=3)
    refused(M.ffn_apply, d, x, w1, w2, None, out, ws, saved=saved[:64], status=3)
    refused(M.ffn_apply, d, x, w1, w2, None, out.cpu(), ws)
    dw1, dw2 = torch.empty(w1.shape, device="cuda"), torch.empty(w2.shape, device="cuda")
    refused(M.ffn_backward, d, out, x, w1, w2, saved, dw1, dw2.bfloat16(), ws)
    refused(M.ffn_backward, d, out, x, w1, w2, saved, dw1, None, ws)
    refused(M.ffn_backward, d, out, x, w1, w2, saved, None, None, ws)
    refused(M.ffn_backward, d, out, x, w1, w2, None, dw1, dw2, ws)
    refused(M.int8_quantize, x.half(), codes, scales)
    refused(M.int8_quantize, x, codes.view(torch.uint8), scales)
    refused(M.int8_quantize, x, codes, scales[:3])
    refused(M.int8_quantize, x[0], codes, scales)
    d8 = M.Int8Dims(64, 72, "f32")
    w, ws8 = torch.zeros((72, 64), dtype=torch.int8, device="cuda"), torch.empty(16, dtype=torch.uint8, device="cuda")
    y = torch.empty((4, 72), device="cuda")
    refused(M.int8_matmul, d8, codes, scales, w, torch.ones(71, device="cuda"), None, y, ws8)
    refused(M.int8_matmul, d8, codes, scales, w, torch.ones(72, device="cuda"), None, y.bfloat16(), ws8)
    refused(M.int8_matmul, d8, codes, scales, w, torch.ones(72, device="cuda"), y.bfloat16(), y, ws8)
    M.int8_matmul(d8, codes, scales, w, torch.ones(72, device="cuda"), None, y, ws8)
    torch.cuda.synchronize()
