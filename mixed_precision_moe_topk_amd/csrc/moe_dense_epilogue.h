// What the dense products do with a row's eight consecutive sums (device code
// shared by the tile kernels, the joins and the kernels of few rows).
#pragma once

#include "moe_dense.h"

namespace moe {

// float32 -> two bf16 in a word, to nearest even, NaN and infinities kept.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint4 bf16_pack8(const float (&v)[8]) {
  return make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                    bf16_pair(v[6], v[7]));
}
// The same of operands of further products: a finite value stays finite.  From
// 2^128 - 2^119 on it would round up to infinity and takes the largest bf16, 2^128 -
// 2^120, which is within 2^-8 of it as any rounding is.  (One test of eight.)
__device__ __forceinline__ uint4 bf16_operand8(const float (&v)[8]) {
  constexpr float kUp = 0x1.FFp127f;
  const uint4 u = bf16_pack8(v);
  float top = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
  if (__builtin_expect(!(top >= kUp), 1)) return u;
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 8; ++j)  // (the bits before infinity's)
    if (fabsf(v[j]) >= kUp && fabsf(v[j]) < __builtin_inff()) w[j / 2] -= j & 1 ? 0x10000u : 1u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// What the rounding of v to bf16 (packed in `hi`) left, rounded in turn: together
// within 2^-17 of v.  0 where that is not finite.
__device__ __forceinline__ uint4 bf16_rest8(const float (&v)[8], const uint4& hi) {
  const uint32_t w[4] = {hi.x, hi.y, hi.z, hi.w};
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float h = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    r[j] = fabsf(h) < __builtin_inff() ? v[j] - h : 0.0f;
  }
  return bf16_pack8(r);
}
__device__ __forceinline__ void bf16_unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
// Eight sums as they left the matrix cores.
__device__ __forceinline__ void sums_to_float(bool int8, const uint4& lo, const uint4& hi, float (&v)[8]) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = int8 ? (float)(int32_t)w[j] : __uint_as_float(w[j]);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 lo = reinterpret_cast<const float4*>(p)[0], hi = reinterpret_cast<const float4*>(p)[1];
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
  v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// 1 / (1 + e^-g): within 4 ulp and, from the exponential's argument, 2^-24 |g|; 0 where
// it lies below 2^-126 (the reciprocal flushes what is subnormal).
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// What finishing eight sums reads from memory.  Read ahead (`Ahead::load`), with
// clamped rows and columns, so that no sum waits for its own reads.
struct Bytes32 {
  uint4 lo, hi;
};
__device__ __forceinline__ Bytes32 load32(const void* p) {
  return {static_cast<const uint4*>(p)[0], static_cast<const uint4*>(p)[1]};
}
__device__ __forceinline__ void floats(const Bytes32& b, float (&v)[8]) {
  sums_to_float(false, b.lo, b.hi, v);
}

template <bool I8, int MODE>
struct Ahead;

// kDenseStore: the base of columns n .. n + 7 of row m.
template <bool I8>
struct Ahead<I8, kDenseStore> {
  Bytes32 base;
  __device__ __forceinline__ void load(const DenseEpilogue& e, int64_t m, int64_t n) {
    base = {};
    if (!e.base) return;
    const int64_t at = m * e.base_stride + n;
    if (e.out_f32) base = load32(static_cast<const float*>(e.base) + at);
    else base.lo = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.base) + at);
  }
};
template <bool I8>
struct Ahead<I8, kDenseGate> {
  __device__ __forceinline__ void load(const DenseEpilogue&, int64_t, int64_t) {}
};
// kDenseDgate: gates and ups of hidden units n .. n + 7 of row m.
template <>
struct Ahead<false, kDenseDgate> {
  Bytes32 g, u;
  __device__ __forceinline__ void load(const DenseEpilogue& e, int64_t m, int64_t n) {
    const float* in = e.gu_in + m * 2 * e.inter + n;
    g = load32(in);
    u = load32(in + e.inter);
  }
};

// Scales of eight int8 sums: the token's, then the channels'.
__device__ __forceinline__ void scale8(float row, const Bytes32& columns, float (&v)[8]) {
  float cs[8];
  floats(columns, cs);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = v[j] * row * cs[j];
}

// kDenseStore: out = base + v, columns n .. n + 7 of row m.
__device__ __forceinline__ void finish_store(const DenseEpilogue& e, int64_t m, int64_t n, float (&v)[8],
                                             const Bytes32& base) {
  const int64_t at = m * e.out_stride + n;
  float b[8];
  if (e.out_f32) {
    if (e.base) {
      floats(base, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    store8(static_cast<float*>(e.out) + at, v);
  } else {
    if (e.base) {
      bf16_unpack8(base.lo, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.out) + at) = bf16_pack8(v);
  }
}

// kDenseGate: gates and ups of hidden units n .. n + 7 of row m.  bf16: gate and
// up stay float32 for the backward pass; h is rounded to bf16 for the second
// product (as the layer's bf16 experts do), and what that leaves is kept for w2's
// gradient in float32.
template <bool I8>
__device__ __forceinline__ void finish_gate(const DenseEpilogue& e, int64_t m, int64_t n, float (&g)[8],
                                            float (&u)[8]) {
  if (!I8 && e.gu_out) {
    float* row = e.gu_out + m * 2 * e.inter + n;
    store8(row, g);
    store8(row + e.inter, u);
  }
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = g[j] * sigmoid(g[j]) * u[j];
  const int64_t at = m * e.out_stride + n;
  if constexpr (I8) {
    store8(static_cast<float*>(e.out) + at, h);
  } else {
    const uint4 hi = bf16_operand8(h);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.out) + at) = hi;
    if (e.out_lo) *reinterpret_cast<uint4*>(e.out_lo + at) = bf16_rest8(h, hi);
  }
}

// kDenseDgate: v is the gradient of h = silu(gate) * up.  With s = sigmoid(gate),
// dgate = v up s (1 + gate (1 - s)) and dup = v gate s, rounded to bf16 for the
// products behind; what that leaves is kept for float32 gradients of w1.
__device__ __forceinline__ void finish_dgate(const DenseEpilogue& e, int64_t m, int64_t n, float (&v)[8],
                                             const Bytes32& gate, const Bytes32& up) {
  const int64_t at = m * 2 * e.inter + n;
  float g[8], u[8];
  floats(gate, g);
  floats(up, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = sigmoid(g[j]);
    const float du = v[j] * (g[j] * s);
    g[j] = v[j] * u[j] * s * (1.0f + g[j] * (1.0f - s));
    u[j] = du;
  }
  uint16_t* out = static_cast<uint16_t*>(e.out) + at;
  const uint4 dg = bf16_operand8(g), du = bf16_operand8(u);
  *reinterpret_cast<uint4*>(out) = dg;
  *reinterpret_cast<uint4*>(out + e.inter) = du;
  if (e.out_lo) {
    *reinterpret_cast<uint4*>(e.out_lo + at) = bf16_rest8(g, dg);
    *reinterpret_cast<uint4*>(e.out_lo + at + e.inter) = bf16_rest8(u, du);
  }
}

template <bool I8, int MODE>
__device__ __forceinline__ void finish(const DenseEpilogue& e, int64_t m, int64_t n, float (&v)[8],
                                       const Ahead<I8, MODE>& ahead) {
  static_assert(MODE != kDenseGate, "gate and up are finished together");
  if constexpr (MODE == kDenseDgate) finish_dgate(e, m, n, v, ahead.g, ahead.u);
  else finish_store(e, m, n, v, ahead.base);
}

// Sums of the parts of columns col .. col + 7 of row m, in the parts' order, eight
// parts' reads under way at a time.
template <bool I8>
__device__ __forceinline__ void join_sums(const DenseGemm& p, int64_t m, int64_t col, float (&v)[8]) {
  constexpr int kReads = 8;
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
}

}  // namespace moe
