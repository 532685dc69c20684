// Products of the gated block in bf16, and the joins of all dense products.
#include "moe_dense_gemm.h"

namespace moe {

hipError_t launch_dense_gemm_bf16(int mode, bool big, const DenseGemm& p, hipStream_t st) {
  if (mode == kDenseGate) return dense::launch<false, false, false, kDenseGate>(big, p, st);
  if (mode == kDenseStore) return dense::launch<false, false, false, kDenseStore>(big, p, st);
  return hipErrorInvalidValue;
}

// Sums of the parts in their order, eight columns a thread.
template <bool I8, int MODE>
__global__ __launch_bounds__(256) void k_dense_join(DenseGemm p) {
  constexpr bool GATE = MODE == kDenseGate;
  const int64_t units = GATE ? p.N / 2 : p.N;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, m = id / (units / 8);
  const int64_t n = id % (units / 8) * 8;
  if (m >= p.M) return;
  auto sum = [&](int64_t col, float (&v)[8]) __attribute__((always_inline)) {
    const uint32_t* at = static_cast<const uint32_t*>(p.part) + m * p.N + col;
    uint4 lo = reinterpret_cast<const uint4*>(at)[0], hi = reinterpret_cast<const uint4*>(at)[1];
    float f[8];
    sums_to_float(false, lo, hi, v);
    for (int s = 1; s < p.split; ++s) {
      at += p.M * p.N;
      const uint4 l2 = reinterpret_cast<const uint4*>(at)[0], h2 = reinterpret_cast<const uint4*>(at)[1];
      if constexpr (I8) {
        lo = make_uint4(lo.x + l2.x, lo.y + l2.y, lo.z + l2.z, lo.w + l2.w);
        hi = make_uint4(hi.x + h2.x, hi.y + h2.y, hi.z + h2.z, hi.w + h2.w);
      } else {
        sums_to_float(false, l2, h2, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[j];
      }
    }
    if constexpr (I8) sums_to_float(true, lo, hi, v);
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
  const int64_t blocks = (threads + 255) / 256;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  const unsigned g = (unsigned)blocks;
  if (int8 && mode == kDenseGate) k_dense_join<true, kDenseGate><<<g, 256, 0, st>>>(p);
  else if (int8 && mode == kDenseStore) k_dense_join<true, kDenseStore><<<g, 256, 0, st>>>(p);
  else if (int8) return hipErrorInvalidValue;
  else if (mode == kDenseGate) k_dense_join<false, kDenseGate><<<g, 256, 0, st>>>(p);
  else if (mode == kDenseDgate) k_dense_join<false, kDenseDgate><<<g, 256, 0, st>>>(p);
  else k_dense_join<false, kDenseStore><<<g, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
