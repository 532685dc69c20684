// Launch parameters of the dense operators beside the layer: the gated block in
// bf16 and its gradients, products in 8-bit integers, and their quantiser.
#pragma once

#include "moe_common.h"

namespace moe {

// What becomes of the sums of a product.
enum DenseMode : int {
  kDenseStore = 0,  // out = base + sum
  kDenseGate = 1,   // columns are gate and up: out = silu(gate) * up
  kDenseDgate = 2,  // sum is the gradient of silu(gate) * up: out = its gradients
};

struct DenseEpilogue {
  const float* row_scale;  // int8: scale of each row (token)
  const float* col_scale;  // int8: scale of each column (channel)
  const void* base;        // kDenseStore: of out's type, or null
  int64_t base_stride;     // elements between rows, as all strides here
  void* out;               // kDenseGate: [M, inter]; kDenseDgate: bf16 [M, 2 inter]
  int64_t out_stride;
  int32_t out_f32;         // float32 or bf16 out
  int32_t inter;
  float* gu_out;           // kDenseGate: gate and up [M, 2 inter], or null
  const float* gu_in;      // kDenseDgate: the same
  uint16_t* out_lo;        // bf16 of kDenseGate and kDenseDgate: what out's rounding left, or null
};

// Tiles of a block.
enum DenseShape : int {
  kDenseBig = 0,  // 256 x 256, 8 waves; see dense_halves
  kDenseMid = 1,  // 128 x 128, 4 waves, two blocks a CU
  kDenseLow = 2,  // 64 x 128, 4 waves, two blocks a CU; not for rows across k
  kDenseFew = 3,  // 64 x 64, 4 waves, two blocks a CU, four steps under way; both
                  // operands along k, few rows (see few_rows in moe_dense_api.cpp)
};
constexpr int dense_rows(int shape) { return shape == kDenseBig ? 256 : shape == kDenseMid ? 128 : 64; }
constexpr int dense_columns(int shape) { return shape == kDenseBig ? 256 : shape == kDenseFew ? 64 : 128; }

// Product of rows and columns over k: sum_k a(m, k) b(n, k).  An operand lies
// either along k (element (m, k) at m * stride + k) or across it (k * stride + m).
struct DenseGemm {
  const uint8_t* a;
  int64_t a_stride;  // bytes, as b_stride
  const uint8_t* b;
  int64_t b_stride;
  // not 0: an operand (1: of the rows, 2: of the columns) is the sum of two bf16
  // matrices, the second so many bytes behind the first
  int32_t terms;
  int64_t lo;
  int64_t M;         // rows
  int32_t N;         // columns; kDenseGate: 2 inter
  int64_t K;
  int32_t shape;     // DenseShape
  int32_t split;     // parts of K, each summed by blocks of their own
  int32_t steps;     // K steps (see dense_step) of a part
  int32_t halves;    // kDenseBig: so many tiles, the last, by two blocks each
  void* part;        // split > 1: sums [split, M, N], float32 or int32
  DenseEpilogue e;
};

constexpr int kDenseStepBytes = 128;  // K step of an operand row
constexpr int dense_step(bool int8, int terms) { return int8 ? 128 : terms ? 32 : 64; }

inline int64_t dense_tiles(const DenseGemm& p) {
  return (p.M + dense_rows(p.shape) - 1) / dense_rows(p.shape) *
         ((p.N + dense_columns(p.shape) - 1) / dense_columns(p.shape));
}
// Big tiles of a launch that two blocks of 256 x 128 each take: those of the last
// round of 256 (one block a CU) when they are at most half of one, which then takes
// little more than half as long.
constexpr int64_t kCus = 256;
inline int64_t dense_halves(int shape, int64_t tiles) {
  const int64_t rest = tiles % kCus;
  return shape == kDenseBig && rest <= kCus / 2 ? rest : 0;
}
// The order of a launch of three products: the longer sums first.
inline void dense_order(const DenseGemm (&p)[3], int (&order)[3]) {
  for (int q = 0; q < 3; ++q) {
    int at = q;
    for (; at > 0 && p[order[at - 1]].steps < p[q].steps; --at) order[at] = order[at - 1];
    order[at] = q;
  }
}
inline int64_t dense_blocks(const DenseGemm& p) { return dense_tiles(p) * p.split + p.halves; }

// Both operands along k: kDenseStore or kDenseGate.
hipError_t launch_dense_gemm_bf16(int mode, const DenseGemm& p, hipStream_t st);
hipError_t launch_dense_gemm_int8(int mode, const DenseGemm& p, hipStream_t st);
// The same for M = 1, without parts.
hipError_t launch_dense_one(bool int8, int mode, const DenseGemm& p, hipStream_t st);
// The gradients of gate and up (columns across k).
hipError_t launch_dense_dgate(const DenseGemm& p, hipStream_t st);
// dw1, dw2 (both operands across k) and dx (columns) in one launch, all of one shape
// (kDenseBig or kDenseMid); one with M = 0 is left out.
hipError_t launch_dense_grads(const DenseGemm (&p)[3], hipStream_t st);
// Adds up the parts (split > 1) and finishes them.
hipError_t launch_dense_join(bool int8, int mode, const DenseGemm& p, hipStream_t st);

// The same for an int8 kDenseGate and the quantiser behind it: codes [M, N / 2] and
// scales [M] of the rows of the gated sums (e.out is not written).
hipError_t launch_dense_join_quant(const DenseGemm& p, int8_t* codes, float* scales, hipStream_t st);

// Codes int8 [rows, cols] and scales [rows] of x, bf16 or float32, stride elements
// between rows.
hipError_t launch_int8_quant(const void* x, bool x_f32, int64_t x_stride, int64_t rows, int32_t cols,
                             int8_t* codes, float* scales, hipStream_t st);

}  // namespace moe
