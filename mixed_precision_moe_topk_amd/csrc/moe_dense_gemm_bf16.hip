// Products of the gated block in bf16, and the joins of all dense products.
#include "moe_dense_gemm.h"

namespace moe {

hipError_t launch_dense_gemm_bf16(int mode, const DenseGemm& p, hipStream_t st) {
  if (mode == kDenseGate) return dense::launch<false, false, false, kDenseGate>(p, st);
  if (mode == kDenseStore) return dense::launch<false, false, false, kDenseStore>(p, st);
  return hipErrorInvalidValue;
}

// Adds up the parts, eight columns a thread; bound by latency (64 tokens x 7168, 4
// parts: 3.7 us; one part's reads after another's took 10).
template <bool I8, int MODE>
__global__ __launch_bounds__(64) void k_dense_join(DenseGemm p) {
  constexpr bool GATE = MODE == kDenseGate;
  const int64_t units = GATE ? p.N / 2 : p.N;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x, m = id / (units / 8);
  const int64_t n = id % (units / 8) * 8;
  if (m >= p.M) return;
  float v[8], u[8];
  Ahead<I8, MODE> ahead;
  ahead.load(p.e, m, n);
  join_sums<I8>(p, m, n, v);
  if constexpr (I8) scale8(p.e.row_scale[m], load32(p.e.col_scale + n), v);
  if constexpr (GATE) {
    join_sums<I8>(p, m, units + n, u);
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
