"""Python binding of the MI355X fused mixed-precision MoE library (libmoe_amd.so).

Argument marshalling only: every step of the layer runs in the HIP kernels of
the library; PyTorch provides device memory and the current stream.  The C
ABI is declared in include/moe.h.  If the library is missing every call raises
(there is no CPU fallback).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_amd.so")

W_MXFP4, W_INT4_G128 = 0, 1
A_FP8_TOKEN, A_BF16, A_MXFP8, A_MXFP4 = 0, 1, 2, 3
WFMT = {"mxfp4": W_MXFP4, "int4": W_INT4_G128}
AFMT = {"fp8": A_FP8_TOKEN, "bf16": A_BF16, "mxfp8": A_MXFP8, "mxfp4": A_MXFP4}

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_HIP", 5: "MOE_ERR_INTERNAL"}

EXPORTS = ("moe_abi_version", "moe_last_error", "moe_weights_query", "moe_prepare_weights",
           "moe_unpack_weights", "moe_workspace_query", "moe_workspace_layout", "moe_run_ws",
           "moe_run", "moe_route", "moe_quantize_tokens", "moe_tune_set", "moe_tune_clear",
           "moe_autotune", "moe_trace_enable", "moe_trace_read", "moe_release_arenas",
           "moe_set_fc2_fused", "moe_run_noalloc", "moe_router_loss_query", "moe_router_loss",
           "moe_router_backward", "moe_finalize_backward", "moe_adapter_plan_query",
           "moe_adapter_plan", "moe_adapter_workspace_query", "moe_adapter_saved_query",
           "moe_adapter_apply", "moe_adapter_backward")
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES
T_BF16, T_F32 = 0, 1
OUT_TYPE = {"bf16": T_BF16, "f32": T_F32}
STAGES = ("route", "quant", "gemm1", "requant", "gemm2", "finalize")


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("wfmt", ctypes.c_int32), ("afmt", ctypes.c_int32)]


class CAdapterDims(ctypes.Structure):
    _fields_ = [("num_adapters", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("out_type", ctypes.c_int32)]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "total", "ids", "topk_w", "chunk_counts", "offsets", "row_token", "slot_row", "tiles",
        "num_tiles", "tok_codes", "tok_scales", "h", "fc2_codes", "fc2_scales", "y2")] + [
        ("tile_m", ctypes.c_int32), ("gemm_cfg", ctypes.c_int32), ("max_tiles", ctypes.c_int64),
        ("tok_bscales", ctypes.c_size_t), ("fc2_bscales", ctypes.c_size_t),
        ("fc2_fused", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mixed_precision_moe_topk_amd.build`")
        # torch ships its own HIP runtime (soname libamdhip64.so.7, loaded by
        # torch under the file name libamdhip64.so).  Loaded first, it also
        # satisfies the library's libamdhip64.so.7 dependency, so the process
        # has one runtime; the library loaded first would bring the system
        # runtime and torch a second one, and one of the two would find no
        # device.
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        DP, AP = ctypes.POINTER(Dims), ctypes.POINTER(CAdapterDims)
        L.moe_abi_version.restype = I32
        L.moe_last_error.restype = ctypes.c_char_p
        sig = {
            "moe_weights_query": [DP, ctypes.POINTER(SZ), ctypes.POINTER(SZ)],
            "moe_prepare_weights": [DP, P, P, I32, I32, P, P, P],
            "moe_unpack_weights": [DP, P, P, I32, I32, P, P, P, P, P],
            "moe_workspace_query": [DP, I64, I32, ctypes.POINTER(SZ)],
            "moe_workspace_layout": [DP, I64, I32, ctypes.POINTER(WsLayout)],
            "moe_run_ws": [DP, P, I64, P, P, P, I32, P, P, SZ, P],
            "moe_run": [DP, P, I64, P, P, P, I32, P, P],
            "moe_run_noalloc": [DP, P, I64, P, P, P, I32, P, P],
            "moe_route": [DP, P, I64, I32, P, P, P, P, P, P, SZ, P],
            "moe_quantize_tokens": [DP, P, I64, P, P, P, P],
            "moe_tune_set": [DP, I64, I32, I32],
            "moe_tune_clear": [],
            "moe_autotune": [DP, P, I64, P, P, P, I32, I32, ctypes.POINTER(I32),
                             ctypes.POINTER(ctypes.c_float), P],
            "moe_trace_enable": [I32],
            "moe_release_arenas": [],
            "moe_set_fc2_fused": [I32],
            "moe_trace_read": [ctypes.POINTER(ctypes.c_float), I32, ctypes.POINTER(I32)],
            "moe_router_loss_query": [DP, I64, I32, ctypes.POINTER(SZ)],
            "moe_router_loss": [DP, P, P, I64, I32, P, I32, P, P, P, P, P, P, SZ, P],
            "moe_router_backward": [DP, P, P, I64, I32, P, I32, P, P, P, P, P, P, P, P],
            "moe_finalize_backward": [DP, P, I64, I32, P, P, P, P, P, I32, P],
            "moe_adapter_plan_query": [I32, I64, ctypes.POINTER(SZ)],
            "moe_adapter_plan": [I32, P, I64, P, SZ, P],
            "moe_adapter_workspace_query": [AP, I64, ctypes.POINTER(SZ)],
            "moe_adapter_saved_query": [AP, I64, ctypes.POINTER(SZ)],
            "moe_adapter_apply": [AP, P, I64, I64, P, SZ, P, P, P, P, I64, P, I64, P, SZ, P, SZ, P],
            "moe_adapter_backward": [AP, P, I64, P, I64, I64, P, SZ, P, P, P, P, SZ, P, P, P, I64,
                                     P, I64, P, SZ, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise MoeError(status, lib().moe_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


@dataclass(frozen=True)
class LayerDims:
    num_experts: int
    hidden: int
    inter: int
    wfmt: str = "mxfp4"
    afmt: str = "fp8"

    def c(self) -> Dims:
        return Dims(self.num_experts, self.hidden, self.inter, WFMT[self.wfmt], AFMT[self.afmt])

    @functools.cache
    def ref(self):
        return ctypes.byref(self.c())


def abi_version() -> int:
    return lib().moe_abi_version()


def weights_query(d: LayerDims):
    w, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_weights_query(ctypes.byref(d.c()), ctypes.byref(w), ctypes.byref(s)))
    return w.value, s.value


def prepare_weights(d: LayerDims, w1, w2, expert_begin: int, weights, scales, stream=None):
    """w1: float32 cuda [n, 2I, H]; w2: float32 cuda [n, H, I] for experts
    [expert_begin, expert_begin + n); weights/scales: uint8 cuda buffers."""
    n = 0 if w1 is None else int(w1.shape[0])
    _check(lib().moe_prepare_weights(ctypes.byref(d.c()), _ptr(w1), _ptr(w2), expert_begin, n,
                                     _ptr(weights), _ptr(scales), _stream(stream)))


def unpack_weights(d: LayerDims, weights, scales, expert_begin: int, w1q, w1s, w2q, w2s,
                   stream=None):
    n = int(w1q.shape[0])
    _check(lib().moe_unpack_weights(ctypes.byref(d.c()), _ptr(weights), _ptr(scales),
                                    expert_begin, n, _ptr(w1q), _ptr(w1s), _ptr(w2q), _ptr(w2s),
                                    _stream(stream)))


def workspace_query(d: LayerDims, num_tokens: int, top_k: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().moe_workspace_query(ctypes.byref(d.c()), num_tokens, top_k, ctypes.byref(b)))
    return b.value


def workspace_layout(d: LayerDims, num_tokens: int, top_k: int) -> WsLayout:
    L = WsLayout()
    _check(lib().moe_workspace_layout(ctypes.byref(d.c()), num_tokens, top_k, ctypes.byref(L)))
    return L


def run_ws(d: LayerDims, hidden, logits, weights, scales, top_k: int, out, workspace,
           stream=None):
    """hidden: bf16 (or int16 bits) cuda [T, H]; logits: float32 cuda [T, E];
    out: bf16 cuda [T, H]; workspace: uint8 cuda of workspace_query bytes."""
    T = int(hidden.shape[0])
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().moe_run_ws(ctypes.byref(d.c()), _ptr(hidden), T, _ptr(logits), _ptr(weights),
                            _ptr(scales), top_k, _ptr(out), _ptr(workspace), nbytes,
                            _stream(stream)))


def run(d: LayerDims, hidden, logits, weights, scales, top_k: int, out, stream=None):
    T = int(hidden.shape[0])
    _check(lib().moe_run(ctypes.byref(d.c()), _ptr(hidden), T, _ptr(logits), _ptr(weights),
                         _ptr(scales), top_k, _ptr(out), _stream(stream)))


def run_noalloc(d: LayerDims, hidden, logits, weights, scales, top_k: int, out, stream=None):
    """The layer with the library's static device workspace (allocates
    nothing; workspaces above NOALLOC_SCRATCH_BYTES are refused)."""
    T = int(hidden.shape[0])
    _check(lib().moe_run_noalloc(ctypes.byref(d.c()), _ptr(hidden), T, _ptr(logits),
                                 _ptr(weights), _ptr(scales), top_k, _ptr(out), _stream(stream)))


def route(d: LayerDims, logits, top_k: int, ids, weights, expert_offsets, row_token,
          slot_row, workspace, stream=None):
    """The routing step alone.  logits: float32 cuda [T, E]; outputs int32/
    float32 cuda: ids [T, k], weights [T, k], expert_offsets [E + 1],
    row_token [T*k], slot_row [T, k]; workspace: uint8 cuda of
    workspace_query bytes."""
    T = int(logits.shape[0])
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().moe_route(ctypes.byref(d.c()), _ptr(logits), T, top_k, _ptr(ids), _ptr(weights),
                           _ptr(expert_offsets), _ptr(row_token), _ptr(slot_row),
                           _ptr(workspace), nbytes, _stream(stream)))


def quantize_tokens(d: LayerDims, hidden, codes, scales, block_scales=None, stream=None):
    """The token quantisation step alone.  hidden: bf16 bits cuda [T, H];
    codes: uint8 cuda [T, H] (E4M3) or [T, H/2] (E2M1); scales: float32 cuda
    [T]; block_scales: uint8 cuda [T, 16*ceil(H/512)] for the MX formats."""
    T = int(hidden.shape[0])
    _check(lib().moe_quantize_tokens(ctypes.byref(d.c()), _ptr(hidden), T, _ptr(codes),
                                     _ptr(scales), _ptr(block_scales), _stream(stream)))


NUM_GEMM_CFG = 3


def tune_set(d: LayerDims, num_tokens: int, top_k: int, gemm_cfg: int):
    """Tile configuration for this shape and token bucket (-1 removes it)."""
    _check(lib().moe_tune_set(ctypes.byref(d.c()), num_tokens, top_k, gemm_cfg))


def tune_clear():
    _check(lib().moe_tune_clear())


def autotune(d: LayerDims, hidden, logits, weights, scales, top_k: int, iters: int = 5,
             stream=None):
    """Validates and times every tile configuration on these inputs, keeps the
    fastest for the shape and token bucket; -> (chosen, [ms per call or -1])."""
    T = int(hidden.shape[0])
    chosen = ctypes.c_int32()
    ms = (ctypes.c_float * NUM_GEMM_CFG)()
    _check(lib().moe_autotune(ctypes.byref(d.c()), _ptr(hidden), T, _ptr(logits), _ptr(weights),
                              _ptr(scales), top_k, iters, ctypes.byref(chosen), ms,
                              _stream(stream)))
    return chosen.value, [float(v) for v in ms]


TRACE_OFF, TRACE_ALL, TRACE_GEMM1 = 0, 1, 2


def trace_enable(mode=TRACE_ALL):
    """Stage timing: TRACE_ALL (every stage), TRACE_GEMM1 (GEMM1 only, two
    events per call) or TRACE_OFF; True / False mean TRACE_ALL / TRACE_OFF."""
    if mode is True:
        mode = TRACE_ALL
    elif mode is False:
        mode = TRACE_OFF
    _check(lib().moe_trace_enable(int(mode)))


def trace_read():
    """-> (calls, {stage: summed ms}) of the calls recorded since the last read."""
    n = len(STAGES)
    arr = (ctypes.c_float * n)()
    calls = ctypes.c_int32()
    _check(lib().moe_trace_read(arr, n, ctypes.byref(calls)))
    return calls.value, {s: float(arr[i]) for i, s in enumerate(STAGES)}


def release_arenas():
    """Frees the workspaces moe_run keeps per device and stream."""
    _check(lib().moe_release_arenas())


def set_fc2_fused(enable: bool):
    """Test hook: False makes GEMM1 store float32 h and the separate FC2
    quantiser run for every format (process-wide; changes the workspace
    layout)."""
    _check(lib().moe_set_fc2_fused(1 if enable else 0))


# ---------------------------------------------------------------- training and adapters
# These calls check their tensors before the library sees a pointer: a wrong
# element type, shape, stride or device raises MoeError (MOE_ERR_INVALID_ARG).
# They are short calls in a decode step's loop, so the checks pass one tensor
# in a few attribute reads and spell out what is wrong only when something is.

def _refuse(msg: str):
    raise MoeError(1, msg)


def _tensor(name, t, dtypes, shape, index, rows=False):
    """Address of tensor t, None for None; t has to have one of the dtypes, the
    shape and the device index; rows: any stride between rows, else contiguous."""
    if t is None:
        return None
    if (t.dtype in dtypes and t.shape == shape and t.get_device() == index
            and (t.is_contiguous() or (rows and (shape[1] == 1 or t.stride(1) == 1)))):
        return t.data_ptr()
    if t.dtype not in dtypes:
        _refuse(f"{name} is {t.dtype}, {' or '.join(map(str, dtypes))} is needed")
    if t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, {shape} is needed")
    if t.get_device() != index:
        _refuse(f"{name} is on {t.device}, the call runs on cuda:{index}")
    _refuse(f"{name} is not contiguous")


def _buffer(name, t, index):
    """(address, bytes) of a workspace; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.get_device() != index or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous buffer on cuda:{index}")
    return t.data_ptr(), t.nbytes


def _types():
    """Element types by name (torch is imported when first needed)."""
    global _dtypes
    if _dtypes is None:
        import torch

        _dtypes = dict(f32=(torch.float32,), i32=(torch.int32,), u8=(torch.uint8,),
                       bf16=(torch.bfloat16, torch.int16),
                       row=(torch.float32, torch.bfloat16, torch.int16))
    return _dtypes


_dtypes = None


@functools.cache
def _queries():
    """(current device, handle of a device's current stream), each without the
    wrappers around it where torch has them (0.2 and 2.6 us a call)."""
    import torch

    device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return device, raw or (lambda _: torch.cuda.current_stream().cuda_stream)


def _current(t, stream):
    """(index of tensor t's device, stream handle): the device has to be the
    current one (the library launches on it) and the stream's."""
    index = t.get_device()
    device, raw = _queries()
    if index < 0 or index != device():
        _refuse(f"tensors on {t.device}, but the current device is another one")
    if stream is None:
        return index, raw(index)
    if stream.device_index != index:
        _refuse(f"stream of {stream.device} for tensors on {t.device}")
    return index, stream.cuda_stream


def _stride(t, features):
    """Elements between rows; a single row (or none, or no tensor) has no stride
    of its own."""
    return t.stride(0) if t is not None and t.shape[0] > 1 else (features + 7) // 8 * 8


def _size(query, *args) -> int:
    b = ctypes.c_size_t()
    _check(query(*args, ctypes.byref(b)))
    return b.value


def _seqs(seq_offsets, index):
    """(sequences, address of their boundaries)."""
    if seq_offsets is None:
        return 1, None
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
        _refuse("seq_offsets must hold at least two boundaries")
    n = seq_offsets.shape[0]
    return n - 1, _tensor("seq_offsets", seq_offsets, _types()["i32"], (n,), index)


def router_loss_query(d: LayerDims, num_tokens: int, num_seqs: int = 1) -> int:
    return _size(lib().moe_router_loss_query, d.ref(), num_tokens, num_seqs)


def router_loss(d: LayerDims, logits, ids, losses, counts, mean_probs, seq_tokens, workspace,
                seq_offsets=None, token_mask=None, stream=None):
    """Balance loss, z-loss and per-expert counts.  logits: float32 cuda [T, E];
    ids: int32 [T, k]; seq_offsets: int32 [S + 1] (None: one sequence);
    token_mask: uint8 [T], 0 for padding; outputs losses float32 [2], counts
    int32 [S, E], mean_probs float32 [S, E], seq_tokens int32 [S + 2];
    workspace: uint8 of router_loss_query bytes."""
    dev, st = _current(logits, stream)
    ty = _types()
    f32, i32 = ty["f32"], ty["i32"]
    T, E, k = logits.shape[0], d.num_experts, ids.shape[-1]
    S, offs = _seqs(seq_offsets, dev)
    ws, room = _buffer("workspace", workspace, dev)
    _check(lib().moe_router_loss(
        d.ref(), _tensor("logits", logits, f32, (T, E), dev), _tensor("ids", ids, i32, (T, k), dev),
        T, k, offs, S, _tensor("token_mask", token_mask, ty["u8"], (T,), dev),
        _tensor("losses", losses, f32, (2,), dev), _tensor("counts", counts, i32, (S, E), dev),
        _tensor("mean_probs", mean_probs, f32, (S, E), dev),
        _tensor("seq_tokens", seq_tokens, i32, (S + 2,), dev), ws, room, st))


def router_backward(d: LayerDims, logits, ids, dlogits, weights=None, dweights=None, dlosses=None,
                    counts=None, seq_tokens=None, seq_offsets=None, token_mask=None, stream=None):
    """dlogits float32 [T, E] from the routing weights' gradient (weights and
    dweights float32 [T, k]) and the losses' (dlosses float32 [2], with the
    counts and seq_tokens of router_loss)."""
    dev, st = _current(logits, stream)
    ty = _types()
    f32, i32 = ty["f32"], ty["i32"]
    T, E, k = logits.shape[0], d.num_experts, ids.shape[-1]
    S, offs = _seqs(seq_offsets, dev)
    _check(lib().moe_router_backward(
        d.ref(), _tensor("logits", logits, f32, (T, E), dev), _tensor("ids", ids, i32, (T, k), dev),
        T, k, offs, S, _tensor("token_mask", token_mask, ty["u8"], (T,), dev),
        _tensor("weights", weights, f32, (T, k), dev),
        _tensor("dweights", dweights, f32, (T, k), dev), _tensor("dlosses", dlosses, f32, (2,), dev),
        _tensor("counts", counts, i32, (S, E), dev),
        _tensor("seq_tokens", seq_tokens, i32, (S + 2,), dev),
        _tensor("dlogits", dlogits, f32, (T, E), dev), st))


def finalize_backward(d: LayerDims, dout, weights, y2, slot_row, dweights, dy2=None, stream=None):
    """Gradient of the weighted sum.  dout: bf16 (or int16 bits) [T, H]; weights
    float32 [T, k]; y2 float32 [T*k, H]; slot_row int32 [T, k]; outputs dweights
    float32 [T, k] and dy2 [T*k, H], float32 or bf16 (int16 bits), or None."""
    dev, st = _current(dout, stream)
    ty = _types()
    f32 = ty["f32"]
    T, H, k = dout.shape[0], d.hidden, weights.shape[-1]
    kind = T_F32 if dy2 is not None and dy2.dtype in f32 else T_BF16
    _check(lib().moe_finalize_backward(
        d.ref(), _tensor("dout", dout, ty["bf16"], (T, H), dev), T, k,
        _tensor("weights", weights, f32, (T, k), dev), _tensor("y2", y2, f32, (T * k, H), dev),
        _tensor("slot_row", slot_row, ty["i32"], (T, k), dev),
        _tensor("dweights", dweights, f32, (T, k), dev),
        _tensor("dy2", dy2, ty["row"], (T * k, H), dev), kind, st))


@dataclass(frozen=True)
class AdapterDims:
    """num_adapters factors A bf16 [rank, in_features] and B bf16 [rank,
    out_features]; out_type: "bf16" or "f32" (base, out and dout)."""

    num_adapters: int
    rank: int
    in_features: int
    out_features: int
    out_type: str = "bf16"

    def c(self) -> CAdapterDims:
        return CAdapterDims(self.num_adapters, self.rank, self.in_features, self.out_features,
                            OUT_TYPE[self.out_type])

    @functools.cache
    def ref(self):
        return ctypes.byref(self.c())


def adapter_plan_query(num_adapters: int, num_tokens: int) -> int:
    return _size(lib().moe_adapter_plan_query, num_adapters, num_tokens)


def adapter_plan(num_adapters: int, adapter_ids, plan, stream=None):
    """Groups the tokens of a batch by adapter.  adapter_ids: int32 cuda [T], ids
    outside [0, num_adapters) mean no adapter; plan: uint8 of
    adapter_plan_query bytes."""
    dev, st = _current(adapter_ids, stream)
    T = adapter_ids.shape[0]
    pl, room = _buffer("plan", plan, dev)
    _check(lib().moe_adapter_plan(
        num_adapters, _tensor("adapter_ids", adapter_ids, _types()["i32"], (T,), dev), T, pl, room,
        st))


def adapter_workspace_query(d: AdapterDims, num_tokens: int) -> int:
    return _size(lib().moe_adapter_workspace_query, d.ref(), num_tokens)


def adapter_saved_query(d: AdapterDims, num_tokens: int) -> int:
    return _size(lib().moe_adapter_saved_query, d.ref(), num_tokens)


def _factors(d: AdapterDims, a, b, scale, dev, ty):
    """Addresses of the adapters' factors and scales."""
    L, R = d.num_adapters, d.rank
    return (_tensor("a", a, ty["bf16"], (L, R, d.in_features), dev),
            _tensor("b", b, ty["bf16"], (L, R, d.out_features), dev),
            _tensor("scale", scale, ty["f32"], (L,), dev))


def adapter_apply(d: AdapterDims, x, plan, a, b, scale, base, out, workspace, saved=None,
                  stream=None):
    """out = base + scale * (x A^T) B of each token's adapter.  x: bf16 cuda
    [T, K]; a bf16 [L, R, K]; b bf16 [L, R, N]; scale float32 [L]; base (or None)
    and out [T, N] of the dims' type; x, base and out may have a row stride;
    saved: uint8 of adapter_saved_query bytes for adapter_backward."""
    dev, st = _current(x, stream)
    ty = _types()
    T, K, N = x.shape[0], d.in_features, d.out_features
    ot = ty[d.out_type]
    pl, plan_room = _buffer("plan", plan, dev)
    sv, saved_room = _buffer("saved", saved, dev)
    ws, room = _buffer("workspace", workspace, dev)
    _check(lib().moe_adapter_apply(
        d.ref(), _tensor("x", x, ty["bf16"], (T, K), dev, True), _stride(x, K), T, pl, plan_room,
        *_factors(d, a, b, scale, dev, ty), _tensor("base", base, ot, (T, N), dev, True),
        _stride(base, N), _tensor("out", out, ot, (T, N), dev, True), _stride(out, N), sv,
        saved_room, ws, room, st))


def adapter_backward(d: AdapterDims, dout, x, plan, a, b, scale, saved, da, db, workspace, dx=None,
                     dx_base=None, stream=None):
    """Gradients of adapter_apply: da, db float32 of the factors' shapes (or both
    None) and dx = dx_base + ... bf16 [T, K] (or None).  saved: as
    adapter_apply left it for the same plan."""
    dev, st = _current(dout, stream)
    ty = _types()
    bits = ty["bf16"]
    T, K, N = dout.shape[0], d.in_features, d.out_features
    L, R = d.num_adapters, d.rank
    pl, plan_room = _buffer("plan", plan, dev)
    sv, saved_room = _buffer("saved", saved, dev)
    ws, room = _buffer("workspace", workspace, dev)
    _check(lib().moe_adapter_backward(
        d.ref(), _tensor("dout", dout, ty[d.out_type], (T, N), dev, True), _stride(dout, N),
        _tensor("x", x, bits, (T, K), dev, True), _stride(x, K), T, pl, plan_room,
        *_factors(d, a, b, scale, dev, ty), sv, saved_room,
        _tensor("da", da, ty["f32"], (L, R, K), dev), _tensor("db", db, ty["f32"], (L, R, N), dev),
        _tensor("dx_base", dx_base, bits, (T, K), dev, True), _stride(dx_base, K),
        _tensor("dx", dx, bits, (T, K), dev, True), _stride(dx, K), ws, room, st))
