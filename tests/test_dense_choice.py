"""Which tiles the dense products take, and into how many parts their sums are cut
(CPU only): the host side of the library, compiled with launches that only note what
they are asked for."""
import ctypes
import os
import random
import subprocess

import pytest

import mixed_precision_moe_topk_amd as M
from mixed_precision_moe_topk_amd import build as B
from tests.test_gpu_dense_exact import ALL, INPUT, WEIGHTS

BIG, MID, LOW, FEW = range(4)
NOTES = """
#include "%s/moe_dense_api.cpp"
#include <vector>
static std::vector<int64_t> notes;
static hipError_t note(int what, const moe::DenseGemm& p) {
  if (p.M > 0) notes.insert(notes.end(), {what, p.M, p.N, p.K, p.shape, p.split, p.steps, p.halves});
  return hipSuccess;
}
namespace moe {
moe_status set_error(moe_status s, const char*) { return s; }
moe_status set_errorf(moe_status s, const char*, ...) { return s; }
moe_status set_ok() { return MOE_OK; }
moe_status check_hip(hipError_t, const char*, hipStream_t) { return MOE_OK; }
moe_status check_gfx950() { return MOE_OK; }
hipError_t launch_dense_gemm_bf16(int mode, const DenseGemm& p, hipStream_t) { return note(mode == kDenseGate ? 0 : 1, p); }
hipError_t launch_dense_gemm_int8(int mode, const DenseGemm& p, hipStream_t) { return note(mode == kDenseGate ? 0 : 1, p); }
hipError_t launch_dense_one(bool, int, const DenseGemm&, hipStream_t) { return hipSuccess; }
hipError_t launch_dense_dgate(const DenseGemm& p, hipStream_t) { return note(2, p); }
hipError_t launch_dense_grads(const DenseGemm (&p)[3], hipStream_t) {
  for (int q = 0; q < 3; ++q) (void)note(3 + q, p[q]);
  return hipSuccess;
}
hipError_t launch_dense_join(bool, int, const DenseGemm&, hipStream_t) { return hipSuccess; }
hipError_t launch_dense_join_quant(const DenseGemm&, int8_t*, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_int8_quant(const void*, bool, int64_t, int64_t, int32_t, int8_t*, float*, hipStream_t) {
  return hipSuccess;
}
}  // namespace moe
extern "C" int64_t taken(int64_t* out, int64_t room) {
  const int64_t n = (int64_t)notes.size();
  for (int64_t i = 0; i < n && i < room; ++i) out[i] = notes[i];
  notes.clear();
  return n;
}
"""
WHAT = ("gate", "down", "dgate", "dw1", "dw2", "dx")


class Choice:
    def __init__(self, folder):
        src, lib = os.path.join(folder, "notes.cpp"), os.path.join(folder, "notes.so")
        with open(src, "w") as f:
            f.write(NOTES % B.CSRC)
        subprocess.run([B.HIPCC, "--offload-arch=gfx950", "-O1", "-fPIC", "-std=c++17", "-shared", src, "-o", lib],
                       check=True, capture_output=True)
        self.lib = ctypes.CDLL(lib)
        self.at = lambda i: ctypes.c_void_p(0x1000 * i)

    def taken(self):
        room = (ctypes.c_int64 * 64)()
        n = self.lib.taken(room, ctypes.c_int64(64))
        assert n <= 64
        rows = [dict(zip(("what", "M", "N", "K", "shape", "split", "steps", "halves"), room[i:i + 8]))
                for i in range(0, n, 8)]
        return {WHAT[r.pop("what")]: r for r in rows}

    def forward(self, T, H, I):
        a, n, room = self.at, ctypes.c_int64, ctypes.c_size_t(1 << 50)
        assert self.lib.moe_ffn_apply(M.FfnDims(H, I).ref(), a(1), n(H), n(T), a(2), a(3), None, n(0), a(4), n(H),
                                      a(5), room, a(6), room, None) == 0
        return self.taken()

    def backward(self, T, H, I, kind="f32", dx=True, weights=True):
        a, n, room = self.at, ctypes.c_int64, ctypes.c_size_t(1 << 50)
        dw = (a(6), a(7)) if weights else (None, None)
        assert self.lib.moe_ffn_backward(
            M.FfnDims(H, I).ref(), a(1), n(H), a(2), n(H), n(T), a(3), a(4), a(5), room, *dw, M.OUT_TYPE[kind], None,
            n(0), a(8) if dx else None, n(H), a(9), room, None) == 0
        return self.taken()


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    return Choice(str(tmp_path_factory.mktemp("choice")))


def test_exact_cases_reach_every_kernel(choice):
    """What tests/test_gpu_dense_exact.py is there for: each product with an operand across
    k in large tiles, in medium ones, in parts, and with tiles that two blocks share, with
    one term and with two where it has both."""
    seen = set()

    def add(chosen, kind):
        for name, c in chosen.items():
            key = (name, kind) if name in ("dw1", "dw2") else (name,)
            seen.add(key + (c["shape"],))
            if c["halves"]:
                seen.add(key + ("halves",))
            if c["split"] > 1:
                seen.add(key + ("parts",))

    for sizes in ALL:
        for kind in ("f32", "bf16"):
            add(choice.backward(*sizes, kind), kind)
    for sizes in INPUT:
        add(choice.backward(*sizes, weights=False), "f32")
    for sizes in WEIGHTS:
        for kind in ("f32", "bf16"):
            add(choice.backward(*sizes, kind, dx=False), kind)
    for key in [("dgate",), ("dx",), ("dw2", "f32"), ("dw2", "bf16")]:
        for form in (BIG, MID, "parts", "halves"):
            assert key + (form,) in seen, (key, form)
    for kind in ("f32", "bf16"):
        for form in (BIG, MID, "parts"):
            assert ("dw1", kind, form) in seen, (kind, form)
    assert ("dgate", LOW) in seen
    # the loop that the long training steps run: many steps of large tiles, two terms
    c = choice.backward(6140, 4040, 1032)
    assert c["dw1"]["shape"] == c["dw2"]["shape"] == BIG and min(c["dw1"]["steps"], c["dw2"]["steps"]) > 100


def test_halves_and_room(choice):
    """dw1 has no tiles in halves (its kernel has no code for them), and the parts of a
    launch fit into the workspace behind the operands."""
    rng = random.Random(0)
    for _ in range(300):
        T, H, I = (int(2 ** rng.uniform(lo, hi)) for lo, hi in ((0, 14), (0, 10), (0, 9)))
        d = M.FfnDims(8 * H, 8 * I)
        chosen = [choice.forward(T, d.hidden, d.inter)]
        for kind in ("f32", "bf16"):
            for dx, weights in ((True, True), (False, True), (True, False)):
                chosen.append(choice.backward(T, d.hidden, d.inter, kind, dx, weights))
        room = M.ffn_workspace_query(d, T) - (T * 8 * d.inter + 255) // 256 * 256
        for c in chosen:
            assert c.get("dw1", {}).get("halves", 0) == 0, (T, d)
            part = {n: (p["split"] * p["M"] * p["N"] * 4 + 255) // 256 * 256 if p["split"] > 1 else 0 for n, p in c.items()}
            together = sum(part.get(n, 0) for n in ("dw1", "dw2", "dx"))
            assert max([together] + [part.get(n, 0) for n in ("gate", "down", "dgate")]) <= room, (T, d)


def test_long_sums_are_cut(choice):
    """A few long sums among very many short ones: 16 blocks of 8192 steps ran four times as
    long as all the others together when the estimate left the longest block out."""
    for T in (1, 3, 64):
        c = choice.backward(T, 4096, 1 << 18)
        assert c["dx"]["split"] > 1 and c["dx"]["steps"] <= 2048, (T, c["dx"])


def test_tiles_of_few_tokens(choice):
    """Tiles of 64 x 64 up to 128 tokens, and up to 256 for sums of at most 32 steps."""
    assert choice.forward(128, 2744, 1000)["gate"]["shape"] == FEW
    assert choice.forward(129, 2744, 1000)["gate"]["shape"] != FEW
    assert choice.forward(256, 2048, 1024)["gate"]["shape"] == FEW
    assert choice.forward(256, 2056, 1024)["gate"]["shape"] != FEW
    assert choice.forward(257, 2048, 1024)["gate"]["shape"] != FEW
