// Gradients of the gated block: of gate and up, then of the weights and of the
// input in one launch.

#include "moe_dense_gemm.h"

namespace moe {

hipError_t launch_dense_dgate(const DenseGemm& p, hipStream_t st) {
  return dense::launch<false, false, true, kDenseDgate>(p, st);
}

// dw1, dw2 (both operands across k) and dx (columns across k) do not need one another:
// in one launch fewer CUs are idle at its end than in three, and a short one costs 5
// us less each.  first[q]: first block of product q, multiples of 8 so that blocks
// keep their XCD; the products with the longer sums come first (4096 tokens of 7168 x
// 2048, float32 gradients: dw2 beside the gradients of gate and up, then dw1 beside dx,
// took 1098 us; the gradients of gate and up, then these three, 957, and 851 since
// operands with one term are loaded once).  Bound by power and LDS as in
// moe_dense_gemm.h: 701 us at 4093 tokens on one card, 759 on another, 1.37 and 1.27
// PFLOP/s with both terms counted.
struct DenseGrads {
  DenseGemm p[3];  // dw1, dw2, dx
  int64_t first[3], blocks[3];
};

// TERMS: the weights' gradients are float32, of operands in two terms.
template <class S, bool TERMS>
__global__ __launch_bounds__(S::NW* kWave, 2) void k_dense_grads(DenseGrads g) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  const int64_t b = blockIdx.x;
  const int64_t cx = b - g.first[2], c1 = b - g.first[1], c0 = b - g.first[0];
  using namespace dense;
  if (cx >= 0 && cx < g.blocks[2]) {
    dense_block<false, false, true, kDenseStore, S>(g.p[2], cx, lds);
  } else if (c1 >= 0 && c1 < g.blocks[1]) {
    dense_block<false, true, true, kDenseStore, S, TERMS ? kColumnTerms : kPlain>(g.p[1], c1, lds);
  } else if (c0 >= 0 && c0 < g.blocks[0]) {
    // (dw2, whose sums are as long, comes behind it: its tiles are the ones in halves)
    dense_block<false, true, true, kDenseStore, S, TERMS ? kRowTerms : kPlain, false>(g.p[0], c0, lds);
  }
}

hipError_t launch_dense_grads(const DenseGemm (&p)[3], hipStream_t st) {
  DenseGrads g = {{p[0], p[1], p[2]}, {}, {}};
  int order[3];
  dense_order(p, order);
  int64_t blocks = 0;
  for (const int q : order) {
    if (p[q].shape != p[0].shape) return hipErrorInvalidValue;
    g.first[q] = blocks;
    g.blocks[q] = dense_blocks(p[q]);
    blocks += (g.blocks[q] + 7) / 8 * 8;
  }
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFFLL || p[0].halves != 0) return hipErrorInvalidValue;
  const unsigned n = (unsigned)blocks;
  using dense::Big;
  using dense::Mid;
  const bool two = p[0].terms != 0;
  if (two != (p[1].terms != 0)) return hipErrorInvalidValue;
  if (p[0].shape == kDenseBig && two) k_dense_grads<Big, true><<<n, Big::NW * kWave, 0, st>>>(g);
  else if (p[0].shape == kDenseBig) k_dense_grads<Big, false><<<n, Big::NW * kWave, 0, st>>>(g);
  else if (p[0].shape == kDenseMid && two) k_dense_grads<Mid, true><<<n, Mid::NW * kWave, 0, st>>>(g);
  else if (p[0].shape == kDenseMid) k_dense_grads<Mid, false><<<n, Mid::NW * kWave, 0, st>>>(g);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace moe
