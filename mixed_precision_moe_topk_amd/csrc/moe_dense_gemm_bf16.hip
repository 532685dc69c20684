// Products of the gated block in bf16, and the joins of all dense products.
#include "moe_dense_gemm.h"

namespace moe {

hipError_t launch_dense_gemm_bf16(int mode, const DenseGemm& p, hipStream_t st) {
  if (mode == kDenseGate) return dense::launch<false, false, false, kDenseGate>(p, st);
  if (mode == kDenseStore) return dense::launch<false, false, false, kDenseStore>(p, st);
  return hipErrorInvalidValue;
}

// Sums of the parts in their order, eight columns a thread; eight parts' reads are
// under way at a time.
template <bool I8, int MODE>
__global__ __launch_bounds__(64) void k_dense_join(DenseGemm p) {
  constexpr bool GATE = MODE == kDenseGate;
  constexpr int kReads = 8;
  const int64_t units = GATE ? p.N / 2 : p.N;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x, m = id / (units / 8);
  const int64_t n = id % (units / 8) * 8;
  if (m >= p.M) return;
  auto sum = [&](int64_t col, float (&v)[8]) __attribute__((always_inline)) {
    const uint32_t* first = static_cast<const uint32_t*>(p.part) + m * p.N + col;
    uint32_t t[8] = {};
    for (int s = 0; s < p.split; s += kReads) {
      Bytes32 b[kReads];
#pragma unroll
      for (int r = 0; r < kReads; ++r) b[r] = load32(first + min(s + r, p.split - 1) * (p.M * p.N));
#pragma unroll
      for (int r = 0; r < kReads; ++r) {
        const uint32_t w[8] = {b[r].lo.x, b[r].lo.y, b[r].lo.z, b[r].lo.w, b[r].hi.x, b[r].hi.y, b[r].hi.z, b[r].hi.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (I8) t[j] += s + r < p.split ? w[j] : 0u;
          else t[j] = s + r < p.split ? __float_as_uint(__uint_as_float(t[j]) + __uint_as_float(w[j])) : t[j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = I8 ? (float)(int32_t)t[j] : __uint_as_float(t[j]);
  };
  float v[8], u[8];
  Ahead<I8, MODE> ahead;
  ahead.load(p.e, m, n);
  sum(n, v);
  if constexpr (I8) scale8(p.e.row_scale[m], load32(p.e.col_scale + n), v);
  if constexpr (GATE) {
    sum(units + n, u);
    if constexpr (I8) scale8(p.e.row_scale[m], load32(p.e.col_scale + units + n), u);
    finish_gate<I8>(p.e, m, n, v, u);
  } else {
    finish<I8, MODE>(p.e, m, n, v, ahead);
  }
}

hipError_t launch_dense_join(bool int8, int mode, const DenseGemm& p, hipStream_t st) {
  const int64_t threads = p.M * ((mode == kDenseGate ? p.N / 2 : p.N) / 8);
  const int64_t blocks = (threads + 63) / 64;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  const unsigned g = (unsigned)blocks;
  if (int8 && mode == kDenseGate) k_dense_join<true, kDenseGate><<<g, 64, 0, st>>>(p);
  else if (int8 && mode == kDenseStore) k_dense_join<true, kDenseStore><<<g, 64, 0, st>>>(p);
  else if (int8) return hipErrorInvalidValue;
  else if (mode == kDenseGate) k_dense_join<false, kDenseGate><<<g, 64, 0, st>>>(p);
  else if (mode == kDenseDgate) k_dense_join<false, kDenseDgate><<<g, 64, 0, st>>>(p);
  else k_dense_join<false, kDenseStore><<<g, 64, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
