"""Host-side checks of the dense entry points (CPU only): sizes and refusals before
any launch."""
import ctypes
import os

import pytest

import mixed_precision_moe_topk_amd as M

OK, BAD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1000 + 8)
OTHER = ctypes.c_void_p(0x2000)
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    return M.lib()


def _status(fn, *args):
    with pytest.raises(M.MoeError) as ei:
        fn(*args)
    return ei.value.status


def _ffn(hidden=256, inter=512):
    return ctypes.byref(M.FfnDims(hidden, inter).c())


def test_sizes(L):
    d = M.FfnDims(256, 512)
    assert M.ffn_saved_query(d, 100) >= 100 * 512 * 12
    assert M.ffn_workspace_query(d, 100) >= 100 * 2 * 512 * 4
    assert M.ffn_int8_workspace_query(d, 100) >= 100 * (256 + 4 + 5 * 512 + 4)
    assert M.ffn_workspace_query(d, 0) == M.ffn_saved_query(d, 0) == 0
    assert M.ffn_int8_workspace_query(d, 0) == M.int8_workspace_query(M.Int8Dims(256, 512), 0) == 0
    for q in (M.ffn_workspace_query, M.ffn_saved_query, M.ffn_int8_workspace_query):
        assert _status(q, d, -1) == 1 and _status(q, d, (1 << 26) + 1) == 1
        assert q(d, 1 << 26) > 0
        for H, I in ((0, 512), (252, 512), (256, -8), ((1 << 18) + 16, 512), (1 << 16, 1 << 15)):
            assert _status(q, M.FfnDims(H, I), 4) == 1, (q, H, I)
    assert _status(M.ffn_int8_workspace_query, M.FfnDims(264, 512), 4) == 1  # 16 bytes of codes
    assert M.ffn_workspace_query(M.FfnDims(264, 512), 4) > 0
    assert _status(M.ffn_workspace_query, M.FfnDims(4096, 512), 1 << 26) == 1  # 2^38 results
    assert _status(M.int8_workspace_query, M.Int8Dims(256, 4096), 1 << 26) == 1
    for K, N, t in ((8, 512, "bf16"), (131072, 512, "bf16"), (256, 4, "f32"), (256, (1 << 18) + 8, "f32")):
        assert _status(M.int8_workspace_query, M.Int8Dims(K, N, t), 4) == 1
    bad = M.CInt8Dims(256, 512, 7)
    n = ctypes.c_size_t()
    assert L.moe_int8_workspace_query(ctypes.byref(bad), 4, ctypes.byref(n)) == 1
    for f in (L.moe_ffn_workspace_query, L.moe_ffn_saved_query, L.moe_ffn_int8_workspace_query):
        assert f(_ffn(), 4, None) == 1 and f(None, 4, ctypes.byref(n)) == 1
    assert L.moe_int8_workspace_query(None, 4, ctypes.byref(n)) == 1


@pytest.mark.parametrize("H, I", [(256, 512), (7168, 2048), (1000, 2744), (8, 8), (4096, 16)])
def test_a_workspace_serves_fewer_tokens(L, H, I):
    d, e = M.FfnDims(H, I), M.FfnDims((H + 15) // 16 * 16, (I + 15) // 16 * 16)
    f = M.Int8Dims(e.hidden, e.inter)
    last = (0, 0, 0, 0)
    for T in [1, 2, 15, 16, 17, 63, 64, 65, 100, 127, 128, 129, 200, 256, 257, 500, 511, 512, 513, 1000, 1024, 1500,
              2048, 3000, 4093, 4096, 5000, 8192, 16384, 65536]:
        now = (M.ffn_workspace_query(d, T), M.ffn_saved_query(d, T), M.ffn_int8_workspace_query(e, T),
               M.int8_workspace_query(f, T))
        assert all(a >= b for a, b in zip(now, last)), T
        last = now


def test_apply_refuses(L):
    def f(d=_ffn(), x=OK, xs=256, T=4, w1=OK, w2=OK, base=OK, bs=256, out=OK, os=256, saved=None, sr=0, ws=OK,
          room=BIG):
        return L.moe_ffn_apply(d, x, xs, T, w1, w2, base, bs, out, os, saved, sr, ws, room, None)

    assert f(T=0, x=None, out=None) == 0
    for name in ("x", "w1", "w2", "out", "ws"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(d=None) == 1 and f(T=-1) == 1 and f(base=BAD) == 1 and f(saved=BAD) == 1
    for name in ("xs", "bs", "os"):
        for s in (248, 260, -256, (1 << 22) + 8):
            assert f(**{name: s}) == 1, (name, s)
    assert f(bs=264) == 1 and b"another row stride" in L.moe_last_error()
    assert f(room=16) == 3 and b"workspace" in L.moe_last_error()
    assert f(saved=OK, sr=16) == 3 and b"saved" in L.moe_last_error()


def test_backward_refuses(L):
    def f(d=_ffn(), dout=OK, ds=256, x=OK, xs=256, T=4, w1=OK, w2=OK, saved=OK, sr=BIG, dw1=OK, dw2=OK, kind=1,
          dxb=OTHER, dxbs=256, dx=OTHER, dxs=256, ws=OK, room=BIG):
        return L.moe_ffn_backward(d, dout, ds, x, xs, T, w1, w2, saved, sr, dw1, dw2, kind, dxb, dxbs, dx, dxs, ws,
                                  room, None)

    assert f(T=0, dw1=None, dw2=None, dout=None, dx=None) == 0
    for name in ("dout", "x", "w1", "w2", "saved", "ws", "dw1", "dw2"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(dx=None, dw1=None, dw2=None) == 1 and b"gradient" in L.moe_last_error()
    assert f(dx=BAD) == 1 and f(dxb=BAD) == 1 and f(kind=2) == 1 and f(kind=-1) == 1
    for name in ("ds", "xs", "dxs", "dxbs"):
        for s in (248, 260, -256, (1 << 22) + 8):
            assert f(**{name: s}) == 1, (name, s)
    assert f(dxbs=264) == 1 and b"another row stride" in L.moe_last_error()
    assert f(dx=OK, dxb=None) == 1 and b"x or dout" in L.moe_last_error()
    assert f(room=16) == 3 and b"workspace" in L.moe_last_error()
    assert f(sr=16) == 3 and b"saved" in L.moe_last_error()


def test_int8_refuses(L):
    def q(x=OK, kind=0, xs=256, R=4, K=256, codes=OK, scales=OK):
        return L.moe_int8_quantize(x, kind, xs, R, K, codes, scales, None)

    assert q(R=0, x=None) == 0
    for name in ("x", "codes", "scales"):
        assert q(**{name: None}) == 1 and q(**{name: BAD}) == 1, name
    assert q(kind=2) == 1 and q(R=-1) == 1 and q(K=0) == 1 and q(K=264) == 1 and q(K=131072, xs=131072) == 1
    assert q(xs=248) == 1 and q(xs=260) == 1

    d = ctypes.byref(M.Int8Dims(256, 512).c())

    def m(d=d, codes=OK, scales=OK, T=4, w=OK, wsc=OK, base=OK, bs=512, out=OK, os=512, ws=OK, room=BIG):
        return L.moe_int8_matmul(d, codes, scales, T, w, wsc, base, bs, out, os, ws, room, None)

    assert m(T=0, codes=None) == 0
    for name in ("codes", "scales", "w", "wsc", "out"):
        assert m(**{name: None}) == 1 and m(**{name: BAD}) == 1, name
    assert m(d=None) == 1 and m(T=-1) == 1 and m(base=BAD) == 1 and m(ws=BAD) == 1
    assert m(os=504) == 1 and m(bs=516) == 1 and m(bs=520) == 1
    deep = ctypes.byref(M.Int8Dims(7168, 512).c())
    assert m(d=deep, room=16) == 3 and m(d=deep, ws=None, room=0) == 1

    def f(x=OK, xs=256, T=4, w1=OK, s1=OK, w2=OK, s2=OK, base=OK, bs=256, out=OK, os=256, ws=OK, room=BIG):
        return L.moe_ffn_int8_apply(_ffn(), x, xs, T, w1, s1, w2, s2, base, bs, out, os, ws, room, None)

    assert f(T=0, x=None) == 0
    for name in ("x", "w1", "s1", "w2", "s2", "out", "ws"):
        assert f(**{name: None}) == 1 and f(**{name: BAD}) == 1, name
    assert f(base=BAD) == 1 and f(xs=248) == 1 and f(os=260) == 1 and f(bs=264) == 1 and f(room=16) == 3


def test_binding_refuses_cpu_tensors(L):
    import torch

    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    d = M.FfnDims(256, 512)
    assert _status(M.ffn_apply, d, t, t, t, None, t, None) == 1
    assert _status(M.ffn_backward, d, t, t, t, t, None, None, None, None) == 1
    assert _status(M.int8_quantize, t, t, t) == 1
    assert _status(M.int8_matmul, M.Int8Dims(256, 512), t, t, t, t, None, t, None) == 1
    assert _status(M.ffn_int8_apply, d, t, t, t, t, t, None, t, None) == 1
