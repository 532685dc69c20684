// Products of 8-bit integers with scales of tokens and channels, and the
// quantiser of their rows.
#include "moe_dense_gemm.h"

namespace moe {

hipError_t launch_dense_gemm_int8(int mode, const DenseGemm& p, hipStream_t st) {
  if (mode == kDenseGate) return dense::launch<true, false, false, kDenseGate>(p, st);
  if (mode == kDenseStore) return dense::launch<true, false, false, kDenseStore>(p, st);
  return hipErrorInvalidValue;
}

// round(v / s) to the nearest integer, ties to even, of the exact quotient.  With
// inv = fl32(1 / s) the product v * inv is within 2^-23 of v / s relative to it,
// 2^-16 for the codes' range; only where that could cross a half is the half
// compared with v exactly (doubles hold the 24 + 9 bits of its product).
__device__ __forceinline__ int int8_code(float v, float s, float inv) {
  const float q = v * inv;
  const float r = rintf(q);
  int code = (int)r;
  if (__builtin_expect(fabsf(q - r) > 0.5f - 0x1p-14f, 0)) {
    const float n = floorf(fabsf(q));
    const double half = ((double)n + 0.5) * (double)s, mag = fabs((double)v);
    const int c = (int)n + (mag > half || (mag == half && ((int)n & 1)) ? 1 : 0);
    code = v < 0.0f ? -c : c;
  }
  return code;
}

// A block a row of x: eight values a thread, in registers up to kKeep rounds,
// read again behind that.
template <bool F32, int NT>
__global__ __launch_bounds__(NT) void k_int8_quant(const void* __restrict__ x, int64_t stride, int32_t cols,
                                                   int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int kKeep = 4;
  const int64_t row = blockIdx.x;
  auto load = [&](int c, float (&v)[8]) __attribute__((always_inline)) {
    if constexpr (F32) load8(static_cast<const float*>(x) + row * stride + c, v);
    else bf16_unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + row * stride + c), v);
  };
  float keep[kKeep][8];
  uint32_t top = 0;  // largest magnitude's bits: NaN above infinity above all others
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int c = (i * NT + threadIdx.x) * 8;
    if (c < cols) {
      load(c, keep[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(keep[i][j]) & 0x7FFFFFFFu);
    }
  }
  for (int c = (kKeep * NT + threadIdx.x) * 8; c < cols; c += NT * 8) {
    float v[8];
    load(c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if constexpr (NT > kWave) {
    __shared__ uint32_t red[NT / kWave];
    if (lane_id() == 0) red[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) top = max(top, red[w]);
  }
  // a zero row has scale 1, a row that is not finite scale NaN and codes 0
  const bool finite = top < 0x7F800000u;
  const float amax = __uint_as_float(top);
  const float s = !finite ? __uint_as_float(0x7FC00000u)
                  : top == 0 ? 1.0f : fmaxf(__fdiv_rn(amax, 127.0f), 0x1p-126f);
  const float inv = __fdiv_rn(1.0f, s);
  if (threadIdx.x == 0) scales[row] = s;
  auto store = [&](int c, const float (&v)[8]) __attribute__((always_inline)) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j / 4] |= ((uint32_t)(finite ? int8_code(v[j], s, inv) : 0) & 0xFFu) << (8 * (j & 3));
    *reinterpret_cast<uint2*>(codes + row * cols + c) = make_uint2(w[0], w[1]);
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int c = (i * NT + threadIdx.x) * 8;
    if (c < cols) store(c, keep[i]);
  }
  for (int c = (kKeep * NT + threadIdx.x) * 8; c < cols; c += NT * 8) {
    float v[8];
    load(c, v);
    store(c, v);
  }
}

hipError_t launch_int8_quant(const void* x, bool x_f32, int64_t x_stride, int64_t rows, int32_t cols,
                             int8_t* codes, float* scales, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  if (rows > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  const unsigned g = (unsigned)rows;
  const bool wide = cols > 2048;
  if (x_f32 && wide) k_int8_quant<true, 256><<<g, 256, 0, st>>>(x, x_stride, cols, codes, scales);
  else if (x_f32) k_int8_quant<true, 64><<<g, 64, 0, st>>>(x, x_stride, cols, codes, scales);
  else if (wide) k_int8_quant<false, 256><<<g, 256, 0, st>>>(x, x_stride, cols, codes, scales);
  else k_int8_quant<false, 64><<<g, 64, 0, st>>>(x, x_stride, cols, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
