// Tile kernel of the dense products.
//
// A block takes BM rows and BN columns; a K step is 128 bytes of every operand
// row.  Both operands' tiles go straight into LDS, two stages: the loads of step
// s + 1 are in flight under the products of step s, one barrier a step.  The
// columns are the matrix instruction's first operand, so that a lane holds four
// consecutive columns of one row.
//
// An operand along k lies in LDS as [row][128 bytes], its 16-byte pieces at
// piece ^ (row % 8): eight lanes that read one piece of eight rows touch all
// banks.  An operand across k lies as [k][columns] and is read transposed
// (ds_read_b64_tr_b16: 16 lanes read 4 k x 16 columns and get a column's four k
// each); its 32-byte pairs of pieces are permuted by bits of k.
#pragma once

#include "moe_dense_epilogue.h"
#include "moe_lds_dma.h"

namespace moe {
namespace dense {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

// 16 bytes of zeros: the source of pieces behind the end of k.
__device__ const uint4 g_zero = {0, 0, 0, 0};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// One operand's tile of ROWS rows (or columns) in LDS, loaded by NW waves.
template <int ROWS, bool ACROSS, int NW>
struct Tile {
  static constexpr int kBytes = ROWS * kDenseStepBytes;
  static constexpr int kLoads = kBytes / 1024 / NW;  // 1-KB loads of a wave and step
  static constexpr int kPieces = ROWS / 8;           // across k: 16-byte pieces of a k row
  static constexpr int kRowsPerLoad = ACROSS ? 64 / kPieces : 8;

  int64_t next;          // address of the K step to load next
  int64_t advance;       // bytes of a K step
  uint32_t off[kLoads];  // this lane's piece of each load
  int first;             // this lane's row (k row when across) of load 0

  // Bits of k that permute the pairs of pieces: a transposed read of one wave
  // touches k, k + 1, k + 2, k + 3 of two groups 8 apart at a time.
  static __device__ __forceinline__ int swizzle(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

  // rows: what is left of the operand from the tile on (the last one is repeated).
  // source(r): which row of the operand the tile's row r is.
  template <class F>
  __device__ __forceinline__ void init(const uint8_t* p, int64_t stride, int64_t rows, int64_t step,
                                       int wave, F source) {
    const int lane = lane_id();
    advance = uniform(ACROSS ? stride * 64 : (int64_t)kDenseStepBytes);
    next = uniform((int64_t)p + step * advance);
    if constexpr (ACROSS) {
      first = wave * kRowsPerLoad + lane / kPieces;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int k = first + u * NW * kRowsPerLoad;
        const int piece = (lane % kPieces) ^ (swizzle(k) << 1);
        off[u] = (uint32_t)(k * stride + min((int64_t)piece, rows / 8 - 1) * 16);
      }
    } else {
      first = wave * 8 + lane / 8;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int r = first + u * NW * 8;
        off[u] = (uint32_t)(source(r) * stride + ((lane ^ r) & 7) * 16);
      }
    }
  }
  __device__ __forceinline__ void issue(uint32_t lds, int wave) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      lds_dma16_s(reinterpret_cast<const uint8_t*>(next), off[u], lds + (u * NW + wave) * 1024);
    next += advance;
  }
  // The last step: `left` bytes of each row (along k) or k rows (across).
  __device__ __forceinline__ void issue_tail(int left, uint32_t lds, int wave) const {
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int r = first + u * NW * kRowsPerLoad;
      const bool in = ACROSS ? r < left : ((lane_id() ^ r) & 7) * 16 < left;
      lds_dma16(in ? reinterpret_cast<const uint8_t*>(next) + off[u] : zero, lds + (u * NW + wave) * 1024);
    }
  }
};

// Reads of a wave's operand fragments: W rows from `row0` of the tile on.
template <int ROWS, bool ACROSS, int W>
struct Fragments {
  static constexpr int kN = W / 16;
  int at[ACROSS ? kN : 2];

  __device__ __forceinline__ void init(int row0) {
    const int lane = lane_id();
    if constexpr (ACROSS) {
      const int q = (lane & 15) >> 2, g = lane >> 4;  // k = 8 g + q of a half step's 32
      const int f = q | (g & 1) << 2;                 // Tile::swizzle of that k
      const int c = row0 / 8 + ((lane & 3) >> 1);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        at[i] = (8 * g + q) * (ROWS * 2) + ((c + 2 * i) ^ (f << 1)) * 16 + (lane & 1) * 8;
    } else {
      at[0] = (row0 + (lane & 15)) * 128 + (((lane >> 4) ^ lane) & 7) * 16;
      at[1] = at[0] ^ 64;
    }
  }
  // Fragment i of half step h: 16 bytes of a lane, row lane % 16, k from
  // 16 bytes * (lane / 16) on.
  __device__ __forceinline__ v4i read(const uint8_t* tile, int i, int h) const {
    if constexpr (ACROSS) {
      using P = __attribute__((address_space(3))) v4s*;
      const uint8_t* p = tile + at[i] + h * 32 * (ROWS * 2);
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * (ROWS * 2)));
      const v8s v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(v4i, v);
    } else {
      return *reinterpret_cast<const v4i*>(tile + at[h] + i * 2048);
    }
  }
};

template <bool I8>
__device__ __forceinline__ v4i mma(v4i a, v4i b, v4i c) {
  if constexpr (I8) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  } else {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), __builtin_bit_cast(v4f, c), 0, 0, 0));
  }
}

// Orders a wave's own LDS writes and reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <bool I8, bool AT, bool BT, int MODE, int WAVES_M, int WAVES_N, int WM, int WN>
__global__ __launch_bounds__(WAVES_M* WAVES_N* kWave, 2) void k_dense(DenseGemm p) {
  constexpr int NW = WAVES_M * WAVES_N, BM = WAVES_M * WM, BN = WAVES_N * WN;
  constexpr bool GATE = MODE == kDenseGate;
  using TA = Tile<BM, AT, NW>;
  using TB = Tile<BN, BT, NW>;
  constexpr int kStage = TA::kBytes + TB::kBytes;
  constexpr int kPitch = WN * 4 + 16;  // bytes of a row in the epilogue's staging
  static_assert(NW * 16 * kPitch <= 2 * kStage, "the epilogue stages in the operands' place");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];

  // Blocks go round the 8 XCDs: each takes a contiguous range of the tiles, in
  // groups of 8 rows of tiles, so that the blocks at work on one XCD share their
  // operands in its L2.
  const int64_t tiles_m = (p.M + BM - 1) / BM;
  const int tiles_n = (p.N + BN - 1) / BN;
  const int64_t total = (int64_t)gridDim.x, b = blockIdx.x, x = b & 7;
  int64_t t = x * (total >> 3) + min(x, total & 7) + (b >> 3);
  const int64_t tiles = tiles_m * tiles_n;
  const int part = uniform((int)(t / tiles));
  t -= part * tiles;
  const int64_t group = t / (8 * tiles_n), first_m = group * 8;
  const int gm = (int)min((int64_t)8, tiles_m - first_m);
  const int r = (int)(t - group * 8 * tiles_n);
  const int64_t m0 = (first_m + r % gm) * BM;
  const int nt = r / gm;
  const int64_t n0 = (int64_t)nt * BN;

  const int wave = uniform((int)threadIdx.x / kWave), lane = lane_id();
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  constexpr int kStep = I8 ? 128 : 64;
  const int all = uniform((int)((p.K + kStep - 1) / kStep));
  const int s0 = part * p.steps, s1 = min(all, s0 + p.steps);
  const int rest = (int)(p.K % kStep);  // of the last step, 0: whole
  TA ta;
  TB tb;
  const int64_t left_m = p.M - m0, left_n = p.N - n0;
  ta.init(p.a + m0 * (AT ? 2 : p.a_stride), p.a_stride, left_m, s0, wave,
          [&](int row) { return min((int64_t)row, left_m - 1); });
  if constexpr (GATE) {
    // a wave's columns are as many gates, then the ups of the same hidden units
    const int64_t inter = p.N / 2, c0 = (int64_t)nt * (BN / 2);
    tb.init(p.b + c0 * p.b_stride, p.b_stride, left_n, s0, wave, [&](int row) {
      const int64_t unit = min(c0 + row / WN * (WN / 2) + row % (WN / 2), inter - 1);
      return unit - c0 + (row % WN >= WN / 2 ? inter : 0);
    });
  } else {
    tb.init(p.b + n0 * (BT ? 2 : p.b_stride), p.b_stride, left_n, s0, wave,
            [&](int row) { return min((int64_t)row, left_n - 1); });
  }
  Fragments<BM, AT, WM> fa;
  Fragments<BN, BT, WN> fb;
  fa.init(wm * WM);
  fb.init(wn * WN);

  v4i acc[WM / 16][WN / 16];
#pragma unroll
  for (int i = 0; i < WM / 16; ++i)
#pragma unroll
    for (int j = 0; j < WN / 16; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  auto issue = [&](int s) __attribute__((always_inline)) {
    const uint32_t at = lds0 + (uint32_t)((s - s0) & 1) * kStage;
    if (rest != 0 && s == all - 1) {
      ta.issue_tail(AT ? rest : rest * (I8 ? 1 : 2), at, wave);
      tb.issue_tail(BT ? rest : rest * (I8 ? 1 : 2), at + TA::kBytes, wave);
    } else {
      ta.issue(at, wave);
      tb.issue(at + TA::kBytes, wave);
    }
  };
  if (s0 < s1) issue(s0);
  for (int s = s0; s < s1; ++s) {
    wait_barrier<0>();
    if (s + 1 < s1) issue(s + 1);
    const uint8_t* la = lds + ((s - s0) & 1) * kStage;
    const uint8_t* lb = la + TA::kBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4i bf[WN / 16];
#pragma unroll
      for (int j = 0; j < WN / 16; ++j) bf[j] = fb.read(lb, j, h);
#pragma unroll
      for (int i = 0; i < WM / 16; ++i) {
        const v4i af = fa.read(la, i, h);
#pragma unroll
        for (int j = 0; j < WN / 16; ++j) acc[i][j] = mma<I8>(bf[j], af, acc[i][j]);
      }
    }
  }
  // all waves are done with the operands; each stages its sums in a place of its
  // own, 16 rows at a time, and takes them back eight columns a lane
  wait_barrier<0>();
  uint8_t* mine = lds + wave * 16 * kPitch;
  constexpr int kUnits = GATE ? WN / 2 : WN;  // finished columns of a row
  constexpr int kLanes = kUnits / 8;          // lanes of a row
  const int row = lane / kLanes, c = lane % kLanes * 8;
  const int64_t unit = (int64_t)nt * (GATE ? BN / 2 : BN) + wn * kUnits + c;
  const int64_t units = GATE ? p.N / 2 : p.N;
#pragma unroll
  for (int i = 0; i < WM / 16; ++i) {
#pragma unroll
    for (int j = 0; j < WN / 16; ++j)
      *reinterpret_cast<v4i*>(mine + (lane & 15) * kPitch + (16 * j + 4 * (lane >> 4)) * 4) = acc[i][j];
    wave_sync();
#pragma unroll
    for (int pass = 0; pass < 16 * kLanes / 64; ++pass) {
      const int rr = pass * (64 / kLanes) + row;
      const int64_t m = m0 + wm * WM + 16 * i + rr;
      const uint4* src = reinterpret_cast<const uint4*>(mine + rr * kPitch + c * 4);
      const uint4 lo = src[0], hi = src[1];
      uint4 lo2, hi2;
      if constexpr (GATE) {
        const uint4* up = reinterpret_cast<const uint4*>(mine + rr * kPitch + (WN / 2 + c) * 4);
        lo2 = up[0], hi2 = up[1];
      }
      if (m < p.M && unit < units) {
        if (p.split > 1) {
          uint32_t* at = static_cast<uint32_t*>(p.part) + ((int64_t)part * p.M + m) * p.N + unit;
          reinterpret_cast<uint4*>(at)[0] = lo;
          reinterpret_cast<uint4*>(at)[1] = hi;
          if constexpr (GATE) {
            reinterpret_cast<uint4*>(at + units)[0] = lo2;
            reinterpret_cast<uint4*>(at + units)[1] = hi2;
          }
        } else {
          float v[8];
          sums_to_float(I8, lo, hi, v);
          if constexpr (GATE) {
            float up[8];
            sums_to_float(I8, lo2, hi2, up);
            finish_gate<I8>(p.e, m, unit, v, up);
          } else {
            finish<I8, MODE>(p.e, m, unit, v);
          }
        }
      }
    }
    wave_sync();
  }
}

template <bool I8, bool AT, bool BT, int MODE>
hipError_t launch(bool big, const DenseGemm& p, hipStream_t st) {
  const int t = dense_tile(big);
  const int64_t blocks = (p.M + t - 1) / t * ((p.N + t - 1) / t) * p.split;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  if (big) k_dense<I8, AT, BT, MODE, 4, 2, 64, 128><<<(unsigned)blocks, 512, 0, st>>>(p);
  else k_dense<I8, AT, BT, MODE, 2, 2, 64, 64><<<(unsigned)blocks, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace dense
}  // namespace moe
