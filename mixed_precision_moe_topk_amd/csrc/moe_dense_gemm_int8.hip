// Products of 8-bit integers with scales of tokens and channels, and the
// quantiser of their rows.
#include <algorithm>

#include "moe_dense_gemm.h"

namespace moe {

hipError_t launch_dense_gemm_int8(int mode, const DenseGemm& p, hipStream_t st) {
  if (mode == kDenseGate) return dense::launch<true, false, false, kDenseGate>(p, st);
  if (mode == kDenseStore) return dense::launch<true, false, false, kDenseStore>(p, st);
  return hipErrorInvalidValue;
}

// round(v / s) to the nearest integer, ties to even, of the exact quotient.  With
// inv = fl32(1 / s) the product v * inv is within 2^-23 of v / s relative to it,
// 2^-16 for the codes' range; only where that could cross a half are the half and
// v compared, by the sign of the fused v - half * s, which is exact where v and s are
// far above the smallest numbers.
__device__ __forceinline__ int int8_near_half(float v, float s, float q) {
  const float n = floorf(fabsf(q)), up = s < 0x1p-60f ? 0x1p64f : 1.0f;
  const float past = fmaf(-(n + 0.5f), s * up, fabsf(v) * up);
  const int c = (int)n + (past > 0.0f || (past == 0.0f && ((int)n & 1)) ? 1 : 0);
  return v < 0.0f ? -c : c;
}
// Eight codes in two words.
__device__ __forceinline__ uint2 int8_codes(const float (&v)[8], float s, float inv) {
  int code[8];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = v[j] * inv, r = rintf(q);
    code[j] = (int)r;
    near |= fabsf(q - r) > 0.5f - 0x1p-15f;
  }
  if (__builtin_expect(near, 0)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = v[j] * inv;
      if (fabsf(q - rintf(q)) > 0.5f - 0x1p-15f) code[j] = int8_near_half(v[j], s, q);
    }
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j / 4] |= ((uint32_t)code[j] & 0xFFu) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

// Largest magnitude's bits (NaN above infinity above all others) over the block.
__device__ __forceinline__ uint32_t magnitude8(const float (&v)[8], uint32_t top) {
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return top;
}
template <int NT>
__device__ __forceinline__ uint32_t block_top(uint32_t top) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if constexpr (NT > kWave) {
    __shared__ uint32_t red[NT / kWave];
    if (lane_id() == 0) red[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) top = max(top, red[w]);
  }
  return top;
}
// Scale of a row, amax times fl32(1 / 127): a zero row has 1, a row that is not finite NaN (and codes 0).
__device__ __forceinline__ float int8_scale(uint32_t top) {
  if (top >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return top == 0 ? 1.0f : fmaxf(__uint_as_float(top) * (1.0f / 127.0f), 0x1p-126f);
}

// A block a row: eight values a thread and round, kept in registers for up to KEEP
// rounds, computed again behind that.  values(c, v): columns c .. c + 7.
template <int NT, int KEEP, class F>
__device__ __forceinline__ void quant_row(int32_t cols, F values, int8_t* __restrict__ codes,
                                          float* __restrict__ scale) {
  float keep[KEEP][8];
  uint32_t top = 0;
  // (all reads first, the row's last values again behind its end: a branch would wait
  // for each; 64 rows of 7168: 6.5 -> 5.2 us)
#pragma unroll
  for (int i = 0; i < KEEP; ++i) values(min((i * NT + (int)threadIdx.x) * 8, cols - 8), keep[i]);
#pragma unroll
  for (int i = 0; i < KEEP; ++i) top = magnitude8(keep[i], top);
  for (int c = (KEEP * NT + threadIdx.x) * 8; c < cols; c += NT * 8) {
    float v[8];
    values(c, v);
    top = magnitude8(v, top);
  }
  top = block_top<NT>(top);
  const bool finite = top < 0x7F800000u;
  const float s = int8_scale(top), inv = __fdiv_rn(1.0f, s);
  if (threadIdx.x == 0) *scale = s;
  auto store = [&](int c, const float (&v)[8]) __attribute__((always_inline)) {
    *reinterpret_cast<uint2*>(codes + c) = finite ? int8_codes(v, s, inv) : make_uint2(0, 0);
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int c = (i * NT + threadIdx.x) * 8;
    if (c < cols) store(c, keep[i]);
  }
  for (int c = (KEEP * NT + threadIdx.x) * 8; c < cols; c += NT * 8) {
    float v[8];
    values(c, v);
    store(c, v);
  }
}

// A read of x and a write of half as many bytes: 16384 rows of 7168 bf16 take 63 us,
// 5.6 TB/s; one row 2.6 us.  A wave a row up to 2048 columns (one round of registers),
// four beyond.
template <bool F32, int NT>
__global__ __launch_bounds__(NT) void k_int8_quant(const void* __restrict__ x, int64_t stride, int64_t rows,
                                                   int32_t cols, int8_t* __restrict__ codes,
                                                   float* __restrict__ scales) {
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= rows) return;
  quant_row<NT, 4>(
      cols,
      [&](int c, float (&v)[8]) __attribute__((always_inline)) {
        if constexpr (F32) load8(static_cast<const float*>(x) + row * stride + c, v);
        else bf16_unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + row * stride + c), v);
      },
      codes + row * cols, scales + row);
}

// A block a token: sums the parts of gate and up in their order (as k_dense_join
// does), and quantises silu(gate) * up.  64 tokens of 7168 x 2048, 4 parts: 6.4 us in
// place of a join (3.9) and a launch of the quantiser (5.2).  Bound by latency.
template <int NT>
__global__ __launch_bounds__(NT) void k_dense_join_quant(DenseGemm p, int8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  const int64_t m = blockIdx.x;
  const int32_t units = p.N / 2;
  const float rs = p.e.row_scale[m];
  quant_row<NT, 2>(
      units,
      [&](int c, float (&v)[8]) __attribute__((always_inline)) {
        float u[8];
        join_sums<true>(p, m, c, v);
        join_sums<true>(p, m, units + c, u);
        scale8(rs, load32(p.e.col_scale + c), v);
        scale8(rs, load32(p.e.col_scale + units + c), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * sigmoid(v[j]) * u[j];
      },
      codes + m * units, scales + m);
}

hipError_t launch_dense_join_quant(const DenseGemm& p, int8_t* codes, float* scales, hipStream_t st) {
  if (p.M == 0) return hipSuccess;
  if (p.M > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  k_dense_join_quant<256><<<(unsigned)p.M, 256, 0, st>>>(p, codes, scales);
  return hipGetLastError();
}

hipError_t launch_int8_quant(const void* x, bool x_f32, int64_t x_stride, int64_t rows, int32_t cols,
                             int8_t* codes, float* scales, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  // (a dimension of a grid holds fewer than 2^32 threads)
  constexpr int64_t kRow = 1 << 20;
  const dim3 g((unsigned)std::min(rows, kRow), (unsigned)((rows + kRow - 1) / kRow));
  if (g.y > 65535) return hipErrorInvalidValue;
  const bool wide = cols > 2048;
  if (x_f32 && wide) k_int8_quant<true, 256><<<g, 256, 0, st>>>(x, x_stride, rows, cols, codes, scales);
  else if (x_f32) k_int8_quant<true, 64><<<g, 64, 0, st>>>(x, x_stride, rows, cols, codes, scales);
  else if (wide) k_int8_quant<false, 256><<<g, 256, 0, st>>>(x, x_stride, rows, cols, codes, scales);
  else k_int8_quant<false, 64><<<g, 64, 0, st>>>(x, x_stride, rows, cols, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
