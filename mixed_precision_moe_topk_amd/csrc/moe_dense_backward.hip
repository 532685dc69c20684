// Gradients of the gated block: of gate and up, then of the weights and of the
// input in one launch.
#include "moe_dense_gemm.h"

namespace moe {

hipError_t launch_dense_dgate(const DenseGemm& p, hipStream_t st) {
  return dense::launch<false, false, true, kDenseDgate>(p, st);
}

// dw1 and dw2 (both operands across k) and dx (b across k) need the same and not
// one another: one launch leaves fewer CUs idle at the end than three, and a short
// one costs 5 us less each.  first[q]: first block of product q, multiples of 8 so
// that blocks keep their XCD.
struct DenseGrads {
  DenseGemm w[2], x;
  int64_t first[4];
  int64_t blocks[3];
};
template <class S>
__global__ __launch_bounds__(S::NW* kWave, 2) void k_dense_grads(DenseGrads g) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  const int64_t b = blockIdx.x;
  if (b < g.first[2]) {
    const int q = b >= g.first[1];
    const int64_t c = b - g.first[q];
    if (c < g.blocks[q]) dense::dense_block<false, true, true, kDenseStore, S>(g.w[q], c, g.blocks[q], lds);
  } else {
    const int64_t c = b - g.first[2];
    if (c < g.blocks[2]) dense::dense_block<false, false, true, kDenseStore, S>(g.x, c, g.blocks[2], lds);
  }
}

hipError_t launch_dense_grads(const DenseGemm& dw1, const DenseGemm& dw2, const DenseGemm& dx, hipStream_t st) {
  DenseGrads g = {{dw1, dw2}, dx, {}, {}};
  for (int q = 0; q < 3; ++q) {
    const DenseGemm& p = q < 2 ? g.w[q] : g.x;
    if (p.shape != dw1.shape) return hipErrorInvalidValue;
    g.blocks[q] = dense_tiles(p) * p.split;
    g.first[q + 1] = g.first[q] + (g.blocks[q] + 7) / 8 * 8;
  }
  if (g.first[3] == 0) return hipSuccess;
  if (g.first[3] > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  const unsigned n = (unsigned)g.first[3];
  if (dw1.shape == kDenseBig) k_dense_grads<dense::Big><<<n, dense::Big::NW * kWave, 0, st>>>(g);
  else if (dw1.shape == kDenseMid) k_dense_grads<dense::Mid><<<n, dense::Mid::NW * kWave, 0, st>>>(g);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace moe
