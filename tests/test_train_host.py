"""Host-side checks of the training and adapter entry points (CPU only): sizes
and refusals before any launch."""
import ctypes
import os

import pytest

import mixed_precision_moe_topk_amd as M

OK, BAD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1000 + 8)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    return M.lib()


def _d(experts=8, hidden=256):
    return ctypes.byref(M.LayerDims(experts, hidden, 512).c())


def _status(fn, *args):
    with pytest.raises(M.MoeError) as ei:
        fn(*args)
    return ei.value.status


def test_router_loss_query(L):
    d = M.LayerDims(8, 256, 512)
    # a slot of 2 E + 2 words per run of 16 tokens and per sequence
    assert M.router_loss_query(d, 64, 1) >= (4 + 1) * 18 * 4
    assert M.router_loss_query(d, 4096, 9) >= (256 + 9) * 18 * 4
    assert M.router_loss_query(d, 0, 1) > 0
    for tokens, seqs in ((-1, 1), ((1 << 26) + 1, 1), (4, 0), (4, 65536)):
        assert _status(M.router_loss_query, d, tokens, seqs) == 1
    assert L.moe_router_loss_query(_d(), 4, 1, None) == 1


def test_router_loss_refuses(L):
    f = lambda **kw: _loss(L, **kw)  # noqa: E731
    for name in ("logits", "ids", "losses", "counts", "mean", "tokens", "ws"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(offs=BAD) == 1 and f(mask=BAD) == 1
    assert f(k=9) == 1 and f(k=0) == 1 and f(T=-1) == 1
    assert f(S=0, offs=OK) == 1 and f(S=3) == 1  # several sequences need boundaries
    assert f(room=64) == 3 and b"workspace" in L.moe_last_error()


def _loss(L, logits=OK, ids=OK, T=4, k=2, offs=None, S=1, mask=None, losses=OK, counts=OK, mean=OK, tokens=OK,
          ws=OK, room=BIG):
    return L.moe_router_loss(_d(), logits, ids, T, k, offs, S, mask, losses, counts, mean, tokens, ws, room, None)


def test_router_backward_refuses(L):
    def f(logits=OK, ids=OK, T=4, k=2, offs=None, S=1, mask=None, w=OK, dw=OK, dl=OK, c=OK, n=OK, out=OK):
        return L.moe_router_backward(_d(), logits, ids, T, k, offs, S, mask, w, dw, dl, c, n, out, None)

    assert f(T=0, logits=None, ids=None, out=None) == 0
    for name in ("logits", "ids", "out", "w", "c", "n"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(dw=None, dl=None) == 1 and b"gradient" in L.moe_last_error()
    assert f(dw=BAD) == 1 and f(dl=BAD) == 1 and f(mask=BAD) == 1 and f(S=2) == 1 and f(k=17) == 1


def test_finalize_backward_refuses(L):
    def f(dout=OK, T=4, k=2, w=OK, y2=OK, rows=OK, dw=OK, dy2=OK, kind=0):
        return L.moe_finalize_backward(_d(), dout, T, k, w, y2, rows, dw, dy2, kind, None)

    assert f(T=0, dout=None) == 0
    for name in ("dout", "w", "y2", "rows", "dw"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(dy2=BAD) == 1 and f(kind=2) == 1 and f(k=9) == 1 and f(T=-1) == 1
    assert f(T=1 << 26) == 1 and b"threads" in L.moe_last_error()  # 64 threads a token


def test_adapter_queries(L):
    assert M.adapter_plan_query(1, 1) > 0 and M.adapter_plan_query(1023, 1 << 20) > 4 << 20
    for n, t in ((0, 4), (1024, 4), (4, -1), (4, (1 << 26) + 1)):
        assert _status(M.adapter_plan_query, n, t) == 1
    d = M.AdapterDims(4, 20, 256, 512)
    # partial sums and halves of 32 ranks for 100 tokens at least
    assert M.adapter_workspace_query(d, 100) >= 2 * 100 * 32 * 4
    assert M.adapter_saved_query(d, 100) >= 100 * 32 * 4
    for bad in (dict(rank=0), dict(rank=129), dict(in_features=12), dict(out_features=0), dict(num_adapters=0),
                dict(in_features=(1 << 18) + 8)):
        kw = dict(num_adapters=4, rank=20, in_features=256, out_features=512)
        kw.update(bad)
        assert _status(M.adapter_workspace_query, M.AdapterDims(**kw), 4) == 1, bad
        assert _status(M.adapter_saved_query, M.AdapterDims(**kw), 4) == 1, bad
    with pytest.raises(KeyError):
        M.AdapterDims(4, 20, 256, 512, "fp8").c()
    dims = M.AdapterDims(4, 20, 256, 512).c()
    dims.out_type = 5
    assert L.moe_adapter_workspace_query(ctypes.byref(dims), 4, ctypes.byref(ctypes.c_size_t())) == 1
    assert L.moe_adapter_plan_query(4, 4, None) == 1


def test_adapter_plan_refuses(L):
    assert L.moe_adapter_plan(4, None, 0, None, 0, None) == 0
    assert L.moe_adapter_plan(4, None, 4, OK, BIG, None) == 1
    assert L.moe_adapter_plan(4, OK, 4, BAD, BIG, None) == 1
    assert L.moe_adapter_plan(0, OK, 4, OK, BIG, None) == 1
    assert L.moe_adapter_plan(4, OK, 4, OK, 16, None) == 3


def test_adapter_apply_refuses(L):
    dims = M.AdapterDims(4, 20, 256, 512).c()

    def f(x=OK, xs=256, T=4, plan=OK, pb=BIG, a=OK, b=OK, scale=OK, base=OK, bs=512, out=OK, os_=512, saved=OK,
          sb=BIG, ws=OK, wb=BIG):
        return L.moe_adapter_apply(ctypes.byref(dims), x, xs, T, plan, pb, a, b, scale, base, bs, out, os_, saved,
                                   sb, ws, wb, None)

    assert f(T=0, x=None, plan=None, out=None, ws=None) == 0
    for name in ("x", "plan", "a", "b", "scale", "out", "ws"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(base=BAD) == 1 and f(saved=BAD) == 1
    assert f(xs=248) == 1 and f(xs=260) == 1 and f(os_=504) == 1 and f(bs=516) == 1
    assert f(bs=520) == 1  # base is out, with another stride
    assert f(pb=16) == 3 and f(wb=16) == 3 and f(sb=16) == 3


def test_adapter_backward_refuses(L):
    dims = M.AdapterDims(4, 20, 256, 512).c()

    def f(dout=OK, ds=512, x=OK, xs=256, T=4, plan=OK, pb=BIG, a=OK, b=OK, scale=OK, saved=OK, sb=BIG, da=OK,
          db=OK, base=None, bs=256, dx=OK, dxs=256, ws=OK, wb=BIG):
        return L.moe_adapter_backward(ctypes.byref(dims), dout, ds, x, xs, T, plan, pb, a, b, scale, saved, sb, da,
                                      db, base, bs, dx, dxs, ws, wb, None)

    for name in ("dout", "x", "plan", "a", "b", "scale", "saved", "ws"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(da=None) == 1 and f(db=None) == 1 and f(da=None, db=None, dx=None) == 1
    assert f(da=BAD) == 1 and f(dx=BAD) == 1 and f(base=BAD) == 1
    assert f(ds=504) == 1 and f(xs=250) == 1 and f(dxs=264, base=OK) == 1 and f(bs=100, base=OK) == 1
    assert f(pb=16) == 3 and f(wb=16) == 3 and f(sb=16) == 3
    assert f(T=0, da=None, db=None) == 0


def test_binding_refuses_cpu_tensors(L):
    import torch

    z, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    d = M.LayerDims(8, 256, 512)
    assert _status(M.router_loss, d, z, i, z[0, :2], i, z, i[0], z) == 1
    assert _status(M.router_backward, d, z, i, z) == 1
    assert _status(M.finalize_backward, d, z, z, z, i, z) == 1
    assert _status(M.adapter_plan, 4, i[:, 0], z) == 1
    a = M.AdapterDims(4, 8, 8, 8)
    assert _status(M.adapter_apply, a, z, z, z, z, z, z, z, z) == 1
    assert _status(M.adapter_backward, a, z, z, z, z, z, z, z, z, z, z) == 1


def test_outputs_over_inputs_that_are_still_read_are_refused(L):
    """bf16 row gradients over the float rows they come from; dx over what the
    factors' gradients read after it."""
    X = [ctypes.c_void_p(0x10000 * i) for i in range(1, 16)]

    assert L.moe_finalize_backward(_d(), X[0], 4, 2, X[1], X[4], X[2], X[3], X[4], M.T_BF16, None) == 1
    assert b"y2" in L.moe_last_error()

    dims = M.AdapterDims(4, 20, 256, 256).c()

    def back(dx, da=X[9], db=X[10]):
        return L.moe_adapter_backward(ctypes.byref(dims), X[0], 256, X[1], 256, 4, X[2], BIG, X[3], X[4], X[5], X[6],
                                      BIG, da, db, None, 256, dx, 256, X[8], BIG, None)

    for dx in (X[0], X[1]):
        assert back(dx) == 1 and b"dx" in L.moe_last_error()


def test_an_empty_batch_with_frozen_factors_is_accepted(L):
    """No token and no factors' gradients: nothing to write, whatever dx is (an
    empty tensor has no address)."""
    import torch

    dims = M.AdapterDims(4, 20, 256, 512).c()
    for dx in (None, OK):
        assert L.moe_adapter_backward(ctypes.byref(dims), None, 512, None, 256, 0, None, 0, None, None, None, None, 0,
                                      None, None, None, 256, dx, 256, None, 0, None) == 0
    # one factor without the other stays refused, and so does no gradient of some tokens
    for da, db, tokens in ((OK, None, 0), (None, OK, 0), (None, None, 4)):
        assert L.moe_adapter_backward(ctypes.byref(dims), OK, 512, OK, 256, tokens, OK, BIG, OK, OK, OK, OK, BIG, da,
                                      db, None, 256, None, 256, OK, BIG, None) == 1
    assert torch.empty(0, 256).data_ptr() == 0


def test_router_loss_workspace_holds_every_slot(L):
    """2 E + 2 words for each run of 8 tokens (whole blocks of 8 runs) and for each
    sequence, then the sequences' parts."""
    for experts, tokens, seqs in ((8, 64, 1), (8, 65, 1), (8, 4096, 9), (384, 16384, 37), (1024, 1, 65535)):
        runs = -(-tokens // 64) * 8
        parts = seqs * (-(-experts // 64) + 1)
        need = 4 * ((runs + seqs) * (2 * experts + 2) + parts)
        assert need < M.router_loss_query(M.LayerDims(experts, 256, 512), tokens, seqs) <= need + 1024
