// Dense products of few rows (up to 64 tokens), both operands along k: a read of the
// weights.
//
// A block takes 16 NT weight rows, its eight waves an eighth of k each, so that the
// sums of a result meet in LDS and need no second launch.  Operands go from memory
// straight into registers, kAhead steps (128 bytes of every row) under way: a
// lane holds 16 bytes of row lane % 16, pieces lane / 16 and lane / 16 + 4 of a
// step, for two matrix instructions.
#include <type_traits>

#include "moe_dense_epilogue.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 8;

template <bool I8>
__device__ __forceinline__ v4i mma(v4i a, v4i b, v4i c) {
  if constexpr (I8) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  } else {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), __builtin_bit_cast(v4f, c), 0, 0, 0));
  }
}

// MT: tiles of 16 tokens; NT: tiles of 16 weight rows.
template <bool I8, int MODE, int MT, int NT, int AHEAD>
__global__ __launch_bounds__(kFewWaves* kWave) void k_dense_few(DenseGemm p) {
  constexpr bool GATE = MODE == kDenseGate;
  constexpr int kPitch = 16 * NT + 4;  // words of a token's sums
  __shared__ __attribute__((aligned(16))) uint32_t sums[kFewWaves][16 * MT * kPitch];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = lane_id();
  const int r = lane & 15, q = lane >> 4;
  const int bytes = (int)(p.K * (I8 ? 1 : 2));  // of a row
  const int steps = (bytes + 127) / 128, per = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);

  // a gate block has 8 NT gates, then the ups of the same units
  const int64_t units = GATE ? p.N / 2 : p.N;
  const int64_t n0 = (int64_t)blockIdx.x * (GATE ? 8 * NT : 16 * NT);
  const uint8_t* wrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = 16 * t + r;
    int64_t row;
    if (GATE) row = min(n0 + c % (8 * NT), units - 1) + (c >= 8 * NT ? units : 0);
    else row = min(n0 + c, units - 1);
    wrow[t] = p.b + row * p.b_stride;
  }
  const uint8_t* xrow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) xrow[t] = p.a + min((int64_t)(16 * t + r), p.M - 1) * p.a_stride;

  // the eight results that this thread finishes, and what it reads for them
  constexpr int kGroups = GATE ? NT : 2 * NT;  // eights of finished columns of a token
  const int m = threadIdx.x / kGroups, c = threadIdx.x % kGroups * 8;
  const int64_t unit = n0 + c;
  Ahead<I8, MODE> ahead;
  ahead.load(p.e, min((int64_t)m, p.M - 1), min(unit, units - 8));

  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  v4i w[AHEAD][NT][2], x[AHEAD][MT][2];
  // (pieces behind the end of a row: its last piece, taken as zeros in `multiply`)
  auto load = [&](int slot, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = min(s * 128 + 64 * h + 16 * q, bytes - 16);
#pragma unroll
      for (int t = 0; t < NT; ++t) w[slot][t][h] = *reinterpret_cast<const v4i*>(wrow[t] + at);
#pragma unroll
      for (int t = 0; t < MT; ++t) x[slot][t][h] = *reinterpret_cast<const v4i*>(xrow[t] + at);
    }
  };
  auto multiply = [&](auto ends, int slot, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = !decltype(ends)::value || (s < s1 && s * 128 + 64 * h + 16 * q < bytes);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v4i b = in ? w[slot][j][h] : v4i{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const v4i a = in ? x[slot][i][h] : v4i{0, 0, 0, 0};
          acc[i][j] = mma<I8>(b, a, acc[i][j]);
        }
      }
    }
  };
  // kAhead steps; the last ones load nothing and may lie behind the end
  auto chunk = [&](auto last, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      multiply(last, u, s + u);
      if (!decltype(last)::value) load(u, min(s + u + AHEAD, s1 - 1));
      __builtin_amdgcn_sched_barrier(0);  // (the compiler would move the reads to their use)
    }
  };
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    load(u, min(s0 + u, max(s1, 1) - 1));
    __builtin_amdgcn_sched_barrier(0);
  }
  int s = s0;
  for (; s + AHEAD < s1; s += AHEAD) chunk(std::false_type(), s);
  chunk(std::true_type(), s);

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<v4i*>(&sums[wave][(16 * i + r) * kPitch + 16 * j + 4 * q]) = acc[i][j];
  __syncthreads();
  if (threadIdx.x >= 16 * MT * kGroups || m >= p.M || unit >= units) return;
  auto sum = [&](int col, float (&v)[8]) __attribute__((always_inline)) {
    v4i lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
    float f[8];
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) {
      const uint4* at = reinterpret_cast<const uint4*>(&sums[k][m * kPitch + col]);
      const uint4 a = at[0], b = at[1];
      if constexpr (I8) {
        lo += __builtin_bit_cast(v4i, a);
        hi += __builtin_bit_cast(v4i, b);
      } else if (k == 0) {
        sums_to_float(false, a, b, v);
      } else {
        sums_to_float(false, a, b, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[j];
      }
    }
    if constexpr (I8) sums_to_float(true, __builtin_bit_cast(uint4, lo), __builtin_bit_cast(uint4, hi), v);
  };
  float v[8], up[8];
  sum(c, v);
  if constexpr (I8) scale8(p.e.row_scale[m], load32(p.e.col_scale + unit), v);
  if constexpr (GATE) {
    sum(8 * NT + c, up);
    if constexpr (I8) scale8(p.e.row_scale[m], load32(p.e.col_scale + units + unit), up);
    finish_gate<I8>(p.e, m, unit, v, up);
  } else {
    finish<I8, MODE>(p.e, m, unit, v, ahead);
  }
}

template <bool I8, int MODE>
hipError_t launch_few(const DenseGemm& p, hipStream_t st) {
  const int64_t units = MODE == kDenseGate ? p.N / 2 : p.N, per = MODE == kDenseGate ? 8 : 16;
  const unsigned blocks = (unsigned)((units + per - 1) / per);
  if (p.M <= 16) k_dense_few<I8, MODE, 1, 1, 6><<<blocks, kFewWaves * kWave, 0, st>>>(p);
  else if (p.M <= 32) k_dense_few<I8, MODE, 2, 1, 4><<<blocks, kFewWaves * kWave, 0, st>>>(p);
  else k_dense_few<I8, MODE, 4, 1, 4><<<blocks, kFewWaves * kWave, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_few(bool int8, int mode, const DenseGemm& p, hipStream_t st) {
  if (p.M < 1 || p.M > kDenseFew) return hipErrorInvalidValue;
  if (mode == kDenseGate) return int8 ? launch_few<true, kDenseGate>(p, st) : launch_few<false, kDenseGate>(p, st);
  if (mode == kDenseStore) return int8 ? launch_few<true, kDenseStore>(p, st) : launch_few<false, kDenseStore>(p, st);
  return hipErrorInvalidValue;
}

}  // namespace moe
