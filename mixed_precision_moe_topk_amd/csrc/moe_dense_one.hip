// Dense products of one row (a token alone), both operands along k: a read of the
// weights.
//
// A wave takes ROWS weight rows whole, a kilobyte of a row at a time (16 bytes a
// lane), AHEAD of them under way, so that all lanes of a read lie in one row and no
// sums meet in memory: the lanes' sums meet by shuffles.  Products are float32
// fused multiply-adds (int8: four products to an int32).  Memory bounds it: 7168 x 4096
// gates and ups 11.9 us (58.7 MB, 4.9 TB/s), down 2048 x 7168 7.2 us, of which some 3
// are the launch and the first reads.  With matrix instructions, whose lanes gather 16
// rows a read, they took 13.9 and 10.2.
#include <type_traits>

#include "moe_dense_epilogue.h"

namespace moe {
namespace {

constexpr int kOneWaves = 8;

template <bool I8>
struct Sum {
  using type = float;
};
template <>
struct Sum<true> {
  using type = int32_t;
};

// kDenseGate: ROWS / 2 gates and the ups of the same units.
template <bool I8, int MODE, int ROWS>
__global__ __launch_bounds__(kOneWaves* kWave) void k_dense_one(DenseGemm p) {
  constexpr bool GATE = MODE == kDenseGate;
  constexpr int kPer = GATE ? ROWS / 2 : ROWS, kUnits = kOneWaves * kPer;  // finished columns of a wave, a block
  constexpr int AHEAD = 8;
  using T = typename Sum<I8>::type;
  __shared__ __attribute__((aligned(16))) T sums[GATE ? 2 : 1][kUnits];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), lane = lane_id();
  const int bytes = (int)(p.K * (I8 ? 1 : 2));  // of a row
  const int chunks = (bytes + 1023) / 1024;
  const int64_t units = GATE ? p.N / 2 : p.N, n0 = (int64_t)blockIdx.x * kUnits;

  // what the threads that finish eight results read for them
  const int c = threadIdx.x * 8;
  Ahead<I8, MODE> ahead;
  if (c < kUnits) ahead.load(p.e, 0, min(n0 + c, units - 8));

  const uint8_t* w[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    w[r] = p.b + (min(n0 + wave * kPer + r % kPer, units - 1) + (r >= kPer ? units : 0)) * p.b_stride;

  T acc[ROWS] = {};
  uint4 wr[AHEAD][ROWS], xr[AHEAD];
  // (behind the end of a row: its last piece, taken as zeros below)
  auto load = [&](int slot, int k) __attribute__((always_inline)) {
    const int at = min(k * 1024 + lane * 16, bytes - 16);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) wr[slot][r] = *reinterpret_cast<const uint4*>(w[r] + at);
    xr[slot] = *reinterpret_cast<const uint4*>(p.a + at);
  };
  auto multiply = [&](auto ends, int slot, int k) __attribute__((always_inline)) {
    const bool in = !decltype(ends)::value || (k < chunks && k * 1024 + lane * 16 < bytes);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 a = in ? xr[slot] : zero;
    if constexpr (I8) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const uint4 b = wr[slot][r];
        T s = acc[r];
        s = __builtin_amdgcn_sdot4((int)a.x, (int)b.x, s, false);
        s = __builtin_amdgcn_sdot4((int)a.y, (int)b.y, s, false);
        s = __builtin_amdgcn_sdot4((int)a.z, (int)b.z, s, false);
        acc[r] = __builtin_amdgcn_sdot4((int)a.w, (int)b.w, s, false);
      }
    } else {
      float x[8], y[8];
      bf16_unpack8(a, x);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        bf16_unpack8(in ? wr[slot][r] : zero, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[r] = fmaf(x[j], y[j], acc[r]);
      }
    }
  };
  // AHEAD kilobytes; the last ones load nothing and may lie behind the end
  auto run = [&](auto last, int k) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      multiply(last, u, k + u);
      if (!decltype(last)::value) load(u, min(k + u + AHEAD, chunks - 1));
      __builtin_amdgcn_sched_barrier(0);  // (the compiler would move the reads to their use)
    }
  };
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    load(u, min(u, chunks - 1));
    __builtin_amdgcn_sched_barrier(0);
  }
  int k = 0;
  for (; k + AHEAD < chunks; k += AHEAD) run(std::false_type(), k);
  run(std::true_type(), k);

#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[r] += __shfl_xor(acc[r], o);
    if (lane == 0) sums[r / kPer][wave * kPer + r % kPer] = acc[r];
  }
  __syncthreads();
  const int64_t unit = n0 + c;
  if (c >= kUnits || unit >= units) return;
  float v[8], up[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = (float)sums[0][c + j];
    if constexpr (GATE) up[j] = (float)sums[1][c + j];
  }
  if constexpr (I8) {
    scale8(p.e.row_scale[0], load32(p.e.col_scale + unit), v);
    if constexpr (GATE) scale8(p.e.row_scale[0], load32(p.e.col_scale + units + unit), up);
  }
  if constexpr (GATE) finish_gate<I8>(p.e, 0, unit, v, up);
  else finish<I8, MODE>(p.e, 0, unit, v, ahead);
}

template <bool I8, int MODE, int ROWS>
hipError_t launch_rows(const DenseGemm& p, hipStream_t st) {
  constexpr int kUnits = kOneWaves * (MODE == kDenseGate ? ROWS / 2 : ROWS);
  const int64_t units = MODE == kDenseGate ? p.N / 2 : p.N;
  const unsigned blocks = (unsigned)((units + kUnits - 1) / kUnits);
  k_dense_one<I8, MODE, ROWS><<<blocks, kOneWaves * kWave, 0, st>>>(p);
  return hipGetLastError();
}

// Rows of weights a wave, where several copies of the weights are read in turn, us by 1
// and by 2 rows:
//   columns           2048       4096       6144  |    6400       8192       9216
//   int8, 1024 long   3.3  3.9   4.6  4.3   6.2  6.3 |  6.9  6.3   7.6  6.4   9.3  8.3
//   int8, 7168 long   4.9  5.9   7.3  7.6   9.7 10.7 | 10.9 10.9  11.9 12.3  14.6 14.8
//   bf16, 1024 long (the block, gate and up included)
//                     9.5 10.6  11.9 11.9  16.0 16.4 | 16.8 16.4  17.9 17.4  21.3 21.7
//   bf16, 7168 long  22.7 24.6  34.4 35.0  51.3 53.4 | 53.7 53.6  63.0 63.5  73.4 76.1
// One row up to three blocks of 8 rows a CU, which are all at work at once; from there on
// two, which win by up to 15 % for short rows and lose up to 4 % for long ones.  Four rows
// were not faster at any size.  Gates and ups take one unit's two rows: two units a wave
// gained 2 to 8 % for 2304 to 2560 units of 7168 and longer, and lost 4 to 25 % elsewhere.
template <bool I8>
hipError_t launch_one(int mode, const DenseGemm& p, hipStream_t st) {
  if (mode == kDenseGate) return launch_rows<I8, kDenseGate, 2>(p, st);
  return p.N <= 3 * kCus * kOneWaves ? launch_rows<I8, kDenseStore, 1>(p, st) : launch_rows<I8, kDenseStore, 2>(p, st);
}

}  // namespace

hipError_t launch_dense_one(bool int8, int mode, const DenseGemm& p, hipStream_t st) {
  if (p.M != 1 || (mode != kDenseGate && mode != kDenseStore)) return hipErrorInvalidValue;
  return int8 ? launch_one<true>(mode, p, st) : launch_one<false>(mode, p, st);
}

}  // namespace moe
