"""The training and adapter operators around the layer, run together as a
fine-tuning step does: adapters on the router's logits and beside the layer, the
layer itself (moe_run_ws, its intermediates taken from the workspace), the
router's losses, and the whole way back."""
import numpy as np
import pytest

import moe_inputs as MI
from oracle import formats as F
from oracle import train as OT
from tests.harness import Problem

pytestmark = pytest.mark.gpu

T, E, k, H, I, L, R = 120, 16, 4, 256, 256, 3, 8
OFFS = [0, 50, 50, 113]  # the tokens behind 113 are padding
MIX = np.array([0.9, 0.05])  # coefficients of (balance, z)


def _bf16(x):
    return F.bf16_to_f32(F.bf16_rne(np.asarray(x, np.float32)))


def _dev(a, bf=False):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.bfloat16() if bf else t


@pytest.mark.parametrize("wf,af", [("mxfp4", "fp8"), ("mxfp4", "bf16"), ("int4", "fp8")])
def test_fine_tuning_step(wf, af):
    import torch

    import mixed_precision_moe_topk_amd as M

    rng = np.random.default_rng(3)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    p = Problem(MI.small_workload(T, E, k, H, I, wf, af, 91, 1.0), experts_for_oracle=[])
    x = F.bf16_to_f32(p.hidden)
    ids_a = rng.integers(-1, L, T).astype(np.int32)
    fa = {s: (_bf16(n(L, R, H) / 16), _bf16(n(L, R, c) / 4)) for s, c in (("router", E), ("layer", H))}
    scale = np.array([0.5, 1.0, 2.0], np.float32)
    dout, empty = _bf16(n(T, H)), lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    dout[OFFS[-1]:] = 0.0

    # ---- forward on the GPU
    d = p.dims
    dr, dl = M.AdapterDims(L, R, H, E, "f32"), M.AdapterDims(L, R, H, H, "bf16")
    buf = lambda size: torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")  # noqa: E731
    plan = buf(M.adapter_plan_query(L, T))
    xd, sd = p.h_dev, _dev(scale)
    ab = {s: tuple(_dev(f, True) for f in fa[s]) for s in fa}
    ws_r, ws_l = buf(M.adapter_workspace_query(dr, T)), buf(M.adapter_workspace_query(dl, T))
    saved_r, saved_l = buf(M.adapter_saved_query(dr, T)), buf(M.adapter_saved_query(dl, T))
    z, out = empty(T, E), torch.empty((T, H), dtype=torch.int16, device="cuda")
    lay = M.workspace_layout(d, T, k)
    ws = buf(lay.total)
    M.adapter_plan(L, _dev(ids_a), plan)
    M.adapter_apply(dr, xd, plan, *ab["router"], sd, p.l_dev, z, ws_r, saved=saved_r)
    M.run_ws(d, xd, z, p.weights, p.scales, k, out, ws)
    part = lambda off, t, *s: ws[off:off + 4 * int(np.prod(s))].view(t).view(s)  # noqa: E731
    ids, w = part(lay.ids, torch.int32, T, k), part(lay.topk_w, torch.float32, T, k)
    rows, y2 = part(lay.slot_row, torch.int32, T, k), part(lay.y2, torch.float32, T * k, H)
    layer_out = out.clone()
    M.adapter_apply(dl, xd, plan, *ab["layer"], sd, out, out, ws_l, saved=saved_l)
    offs = _dev(np.array(OFFS, np.int32))
    S = len(OFFS) - 1
    losses, mean = empty(2), empty(S, E)
    counts = torch.empty((S, E), dtype=torch.int32, device="cuda")
    tokens = torch.empty(S + 2, dtype=torch.int32, device="cuda")
    M.router_loss(d, z, ids, losses, counts, mean, tokens, buf(M.router_loss_query(d, T, S)), seq_offsets=offs)

    # ---- and back
    do, mix = _dev(dout, True), _dev(MIX.astype(np.float32))
    dw, dz = empty(T, k), torch.zeros((T, E), device="cuda")
    M.finalize_backward(d, do, w, y2, rows, dw)
    M.router_backward(d, z, ids, dz, weights=w, dweights=dw, dlosses=mix, counts=counts, seq_tokens=tokens,
                      seq_offsets=offs)
    da_r, db_r, da_l, db_l = (empty(*f.shape) for s in ("router", "layer") for f in fa[s])
    dx = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    M.adapter_backward(dl, do, xd, plan, *ab["layer"], sd, saved_l, da_l, db_l, ws_l, dx=dx)
    M.adapter_backward(dr, dz, xd, plan, *ab["router"], sd, saved_r, da_r, db_r, ws_r, dx=dx, dx_base=dx)
    torch.cuda.synchronize()

    # ---- the same in float64, on the layer's own experts' rows
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    ids_h, rows_h, y2_h = ids.cpu().numpy(), rows.cpu().numpy(), f(y2)
    ref = OT.router_loss(f(z), ids_h, OFFS)
    assert np.array_equal(counts.cpu().numpy(), ref["counts"])

    def logits(a, b):
        return OT.adapter_apply(x, ids_a, a, b, scale, p.logits)

    def weights(zz):
        return OT.softmax(np.take_along_axis(zz, ids_h, axis=1))[0]

    def goal(ar, br, al, bl):
        zz = logits(ar, br)
        y = (weights(zz)[:, :, None] * y2_h[rows_h]).sum(1)
        y = OT.adapter_apply(x, ids_a, al, bl, scale, y)
        return (dout * y).sum() + MIX @ OT.router_loss(zz, ids_h, OFFS)["losses"]

    f64 = [np.asarray(v, np.float64) for s in ("router", "layer") for v in fa[s]]
    z64 = logits(*f64[:2])
    w64 = weights(z64)
    dw64, dwm, _ = OT.finalize_backward(dout, w64, y2_h, rows_h)
    g, _ = OT.router_backward(z64, ids_h, OFFS, None, w64, dw64, MIX, ref["counts"], ref["seq_tokens"])
    _, gm = OT.router_backward(z64, ids_h, OFFS, None, w64, dwm, MIX, ref["counts"], ref["seq_tokens"])
    g, zeros = np.nan_to_num(g), np.zeros((T, H))
    dx_r, *want_r = OT.adapter_backward(g, x, ids_a, *f64[:2], scale, zeros)
    dx_l, *want_l = OT.adapter_backward(dout, x, ids_a, *f64[2:], scale, zeros)
    # the gradient is that of the whole step: along a random direction, by differences
    way = [n(*v.shape) for v in f64]
    step = 1e-5
    diff = (goal(*[v + step * u for v, u in zip(f64, way)]) - goal(*[v - step * u for v, u in zip(f64, way)])) / (2 * step)
    along = sum((a * b).sum() for a, b in zip(want_r + want_l, way))
    # third derivatives enter at step^2, the goal's own rounding at 2^-52 / step
    assert abs(diff - along) <= 1e-6 * sum(np.abs(a * b).sum() for a, b in zip(want_r + want_l, way))

    # Rounding: z differs by 2^-17 of the adapter's terms and 2^-24 of itself, which moves a softmax by
    # as much (below 2^-12 here); every later stage adds at most 2^-15 of its absolute terms.
    absf = [np.abs(v) for v in f64]
    ab_r = OT.adapter_backward(gm, np.abs(x), ids_a, *absf[:2], scale, zeros)
    ab_l = OT.adapter_backward(np.abs(dout), np.abs(x), ids_a, *absf[2:], scale, zeros)
    tol = 2.0 ** -11
    for got, want, size in ((da_r, want_r[0], ab_r[1]), (db_r, want_r[1], ab_r[2]),
                            (da_l, want_l[0], ab_l[1]), (db_l, want_l[1], ab_l[2])):
        assert np.all(np.abs(f(got) - want) <= tol * size + 1e-30)
    # dx passes bf16 twice
    first = 2.0 ** -8 * (np.abs(dx_l) + tol * ab_l[0])
    second = 2.0 ** -8 * (np.abs(dx_l + dx_r) + first + tol * (ab_l[0] + ab_r[0]))
    assert np.all(np.abs(f(dx) - dx_l - dx_r) <= first + second + tol * (ab_l[0] + ab_r[0]))
    # beside the layer: its own output plus the adapters', rounded once
    base = F.bf16_to_f32(layer_out.cpu().numpy().view(np.uint16))
    y = OT.adapter_apply(x, ids_a, *f64[2:], scale, base)
    mag = OT.adapter_apply(np.abs(x), ids_a, *absf[2:], scale, np.zeros((T, H)))
    got = F.bf16_to_f32(out.cpu().numpy().view(np.uint16))
    assert np.all(np.abs(got - y) <= 2.0 ** -8 * (np.abs(y) + 2.0 ** -13 * mag) + 2.0 ** -13 * mag)
