// Gradients of the gated block in two launches of two products each.
#include "moe_dense_gemm.h"

namespace moe {

// Products that do not need one another share a launch: fewer CUs are idle at its
// end, and a short one costs 5 us less.  4096 tokens of 7168 x 2048: the gradients of
// gate and up alone left half of the CUs without a tile of 256 x 256.  The blocks of
// y start at a multiple of 8, so that they keep their XCD; those of x, which has
// the longer K, come first.
struct DensePair {
  DenseGemm x, y;
  int64_t blocks_x, first_y;
};

// XT, XMODE: layout of x's rows and its mode; y's rows alike (columns across k).
// XTERMS, YTERMS: float32 gradients of weights take both terms of their operand.
template <bool XT, int XMODE, bool YT, class S, int XTERMS, int YTERMS>
__global__ __launch_bounds__(S::NW* kWave, 2) void k_dense_pair(DensePair g) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  const int64_t b = blockIdx.x;
  if (b < g.first_y) {
    if (b < g.blocks_x) dense::dense_block<false, XT, true, XMODE, S, XTERMS>(g.x, b, lds);
  } else {
    dense::dense_block<false, YT, true, kDenseStore, S, YTERMS>(g.y, b - g.first_y, lds);
  }
}

template <bool XT, int XMODE, bool YT, int XTERMS, int YTERMS>
hipError_t launch_pair(const DenseGemm& x, const DenseGemm& y, hipStream_t st) {
  if (x.shape != y.shape) return hipErrorInvalidValue;
  DensePair g = {x, y, dense_blocks(x), 0};
  g.first_y = (g.blocks_x + 7) / 8 * 8;
  const int64_t blocks = g.first_y + dense_blocks(y);
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  const unsigned n = (unsigned)blocks;
  using dense::Big;
  using dense::Mid;
  if (x.shape == kDenseBig) k_dense_pair<XT, XMODE, YT, Big, XTERMS, YTERMS><<<n, Big::NW * kWave, 0, st>>>(g);
  else if (x.shape == kDenseMid) k_dense_pair<XT, XMODE, YT, Mid, XTERMS, YTERMS><<<n, Mid::NW * kWave, 0, st>>>(g);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_dense_dgate_dw2(const DenseGemm& dgate, const DenseGemm& dw2, hipStream_t st) {
  return dw2.terms == 2 ? launch_pair<false, kDenseDgate, true, 1, 2>(dgate, dw2, st)
                        : launch_pair<false, kDenseDgate, true, 1, 1>(dgate, dw2, st);
}
hipError_t launch_dense_dw1_dx(const DenseGemm& dw1, const DenseGemm& dx, hipStream_t st) {
  return dw1.terms == 2 ? launch_pair<true, kDenseStore, false, 2, 1>(dw1, dx, st)
                        : launch_pair<true, kDenseStore, false, 1, 1>(dw1, dx, st);
}

}  // namespace moe
