// Tile kernel of the dense products.
//
// A block takes BM rows and BN columns; a K step is 128 bytes of every operand
// row.  Both operands' tiles go straight into LDS, up to two steps ahead; one barrier a
// step.  The columns are the matrix instruction's first operand, so that a lane holds
// four consecutive columns of one row.
//
// An operand along k lies in LDS as [row][128 bytes], its 16-byte pieces at
// piece ^ (row % 8): eight lanes that read one piece of eight rows touch all
// banks.  An operand across k lies as [k][columns] and is read transposed
// (ds_read_b64_tr_b16: 16 lanes read 4 k x 16 columns and get a column's four k
// each); its 32-byte pairs of pieces are permuted by bits of k.  No bank conflicts
// were counted either way.
//
// What bounds it: a 256 x 256 step is 2048 clocks of matrix instructions and moves 64
// KB into LDS and 196 out of it, 2030 clocks at 128 bytes a clock; it takes 2250, and in
// long launches the part lowers its clock to 1.7 GHz.  16384 tokens: gate and up of
// 7168 x 4096 1.41 PFLOP/s, down of 2048 x 7168 1.09 (each tile's 256 KB of base and
// result in one burst, 13 of 60 us), int8 7168 x 7168 2.5 POP/s; the library's bf16
// product of 8192^3 takes 1.35 PFLOP/s, its int8 one 2.05.  Tried and not kept: one half
// step's fragments at a time (1237 us for the block in place of 1070), 32 x 32 x 16
// instructions (5 % slower, int8 10), tiles of 128 x 256 and 192 x 128 by four waves, two
// K groups of waves in a block, four steps ahead for 128 x 128.
#pragma once

#include "moe_dense_epilogue.h"
#include "moe_lds_dma.h"

namespace moe {
namespace dense {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

template <int V>
struct Int {
  static constexpr int value = V;
};

// 16 bytes of zeros: the source of pieces behind the end of k.
__device__ const uint4 g_zero = {0, 0, 0, 0};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// An operand that is the sum of two bf16 terms: a K step is then 32 k of it, the first
// term's in the place of a plain step's first half, the second's in the other's, and
// as many k of the other operand, whose fragments serve both halves.
enum Terms : int { kPlain = 0, kRowTerms = 1, kColumnTerms = 2 };

// One operand's tile of ROWS rows (or columns) in LDS, loaded by NW waves.  STEP: what
// a K step takes of it, 128 bytes of every row (kWholeStep), half of that
// (kHalfStep), or half of that of each of its two terms (kTwoTerms).
enum StepKind : int { kWholeStep = 0, kHalfStep = 1, kTwoTerms = 2 };
template <int ROWS, bool ACROSS, int NW, int STEP>
struct Tile {
  static_assert(ACROSS || STEP == kWholeStep, "halves of steps across k");
  static constexpr int kBytes = ROWS * kDenseStepBytes / (STEP == kHalfStep ? 2 : 1);
  static constexpr int kLoads = kBytes / 1024 / NW;  // 1-KB loads of a wave and step
  static constexpr int kPieces = ROWS / 8;           // across k: 16-byte pieces of a k row
  static constexpr int kRowsPerLoad = ACROSS ? 64 / kPieces : 8;
  static_assert(STEP != kTwoTerms || 32 % (NW * kRowsPerLoad) == 0, "a load is of one term");

  int64_t next;          // address of the K step to load next
  int64_t advance;       // bytes to the one behind it
  int64_t lo;            // kTwoTerms: bytes to the second term
  uint32_t off[kLoads];  // this lane's piece of each load
  int first;             // this lane's row (k row when across) of load 0

  // Bits of k that permute the pairs of pieces: a transposed read of one wave
  // touches k, k + 1, k + 2, k + 3 of two groups 8 apart at a time.
  static __device__ __forceinline__ int swizzle(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

  // rows: what is left of the operand from the tile on (the last one is repeated).
  // source(r): which row of the operand the tile's row r is.
  template <class F>
  __device__ __forceinline__ void init(const uint8_t* p, int64_t stride, int64_t rows, int64_t step, int64_t second,
                                       int wave, F source) {
    const int lane = lane_id();
    advance = uniform(ACROSS ? stride * (STEP == kWholeStep ? 64 : 32) : (int64_t)kDenseStepBytes);
    next = uniform((int64_t)p + step * advance);
    if constexpr (STEP == kTwoTerms) lo = uniform(second);
    if constexpr (ACROSS) {
      first = wave * kRowsPerLoad + lane / kPieces;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int k = first + u * NW * kRowsPerLoad;
        const int piece = (lane % kPieces) ^ (swizzle(k) << 1);
        off[u] = (uint32_t)((STEP == kTwoTerms ? k % 32 : k) * stride + min((int64_t)piece, rows / 8 - 1) * 16);
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
  // Where load u of the step at `next` reads from.
  __device__ __forceinline__ const uint8_t* source_of(int u) const {
    return reinterpret_cast<const uint8_t*>(STEP == kTwoTerms && u >= kLoads / 2 ? next + lo : next);
  }
  // Load u of the step at `next`; the last one moves on.
  __device__ __forceinline__ void issue(int u, uint32_t lds, int wave) {
    lds_dma16_s(source_of(u), off[u], lds + (u * NW + wave) * 1024);
    if (u == kLoads - 1) next += advance;
  }
  // The same for the last step: `left` bytes of each row (along k) or k rows (across).
  __device__ __forceinline__ void issue_tail(int u, int left, uint32_t lds, int wave) const {
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero);
    const int r = first + u * NW * kRowsPerLoad;
    const bool in = ACROSS ? (STEP == kTwoTerms ? r % 32 : r) < left : ((lane_id() ^ r) & 7) * 16 < left;
    lds_dma16(in ? source_of(u) + off[u] : zero, lds + (u * NW + wave) * 1024);
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

// Waves and their tiles of a block; what the block takes of LDS.
// A block holds two steps' rows and three steps' columns.
template <int WAVES_M_, int WAVES_N_, int WM_, int WN_>
struct Shape {
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WM = WM_, WN = WN_;
  static constexpr int NW = WAVES_M * WAVES_N, BM = WAVES_M * WM, BN = WAVES_N * WN;
  static constexpr int kLds = (2 * BM + 3 * BN) * kDenseStepBytes;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
};
using Big = Shape<4, 2, 64, 128>;  // 256 x 256, 160 KB of LDS
using Half = Shape<4, 2, 64, 64>;  // 256 x 128: half of a Big one, by as many waves
using Mid = Shape<2, 2, 64, 64>;   // 128 x 128, 80 KB: two blocks a CU
using Low = Shape<2, 2, 32, 64>;   // 64 x 128, 64 KB: two blocks a CU
// Few rows: steps of both operands in a ring of STAGES.
template <int WAVES_M_, int WAVES_N_, int WM_, int WN_, int STAGES>
struct Ring {
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WM = WM_, WN = WN_, kStages = STAGES;
  static constexpr int NW = WAVES_M * WAVES_N, BM = WAVES_M * WM, BN = WAVES_N * WN;
  static constexpr int kLds = STAGES * (BM + BN) * kDenseStepBytes;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
};
using Few = Ring<4, 1, 16, 64, 5>;  // 64 x 64, 80 KB: two blocks a CU

// Gates and ups: a wave's WN columns are as many gates, then the ups of the same hidden
// units.  Row of the weights, from c0 on, that column `row` of a tile is.
template <int WN>
__device__ __forceinline__ int64_t gate_row(int row, int64_t c0, int64_t inter) {
  const int64_t unit = min(c0 + row / WN * (WN / 2) + row % (WN / 2), inter - 1);
  return unit - c0 + (row % WN >= WN / 2 ? inter : 0);
}

// A lane holds columns 4 (lane / 16) + 0 .. 3 of each 16 x 16 sums.  Of two
// neighbours, the odd quarters of the wave give theirs of the first for the even
// quarters' of the second: every lane then has eight consecutive columns.
__device__ __forceinline__ void eight_columns(const v4i& first, const v4i& second, uint4& lo, uint4& hi) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const auto x = __builtin_amdgcn_permlane16_swap((uint32_t)first[r], (uint32_t)second[r], false, false);
    a[r] = x[0], b[r] = x[1];
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// What becomes of a block's sums: parts of them, or results.
template <bool I8, int MODE, class S>
__device__ __forceinline__ void dense_sums(const DenseGemm& p, int part, int64_t m0, int nt, int wm, int wn,
                                           v4i (&acc)[S::WM / 16][S::WN / 16]) {
  constexpr int BN = S::BN, WM = S::WM, WN = S::WN, FM = WM / 16;
  constexpr bool GATE = MODE == kDenseGate;
  const int lane = lane_id();
  constexpr int kUnits = GATE ? WN / 2 : WN;  // finished columns of a row
  const int64_t units = GATE ? p.N / 2 : p.N;
  const int64_t unit0 = (int64_t)nt * (GATE ? BN / 2 : BN) + wn * kUnits + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  auto eight = [&](int i, int j, uint4& lo, uint4& hi) __attribute__((always_inline)) {
    eight_columns(acc[i][j], acc[i][j + 1], lo, hi);
  };
  constexpr int kPairs = kUnits / 32;
  const int64_t row0 = m0 + wm * WM + (lane & 15);
  if (p.split > 1) {
    uint32_t* sums = static_cast<uint32_t*>(p.part) + (int64_t)part * p.M * p.N;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = row0 + 16 * i;
#pragma unroll
      for (int j = 0; j < (GATE ? 2 : 1) * kPairs; ++j) {
        uint4 lo, hi;
        eight(i, 2 * j, lo, hi);
        const int64_t unit = unit0 + 32 * (j % kPairs);
        if (m < p.M && unit < units) {
          uint4* at = reinterpret_cast<uint4*>(sums + m * p.N + (j / kPairs) * units + unit);
          at[0] = lo, at[1] = hi;
        }
      }
    }
    return;
  }
  // reads of a group of rows are under way while the one before is finished (int8:
  // the columns' scales take the registers; float32 gates and ups are too many)
  constexpr int kDeep = I8 || MODE == kDenseDgate ? 1 : 2;
  Ahead<I8, MODE> ahead[kDeep][kPairs];
  float row_scale = 1.0f;
  Bytes32 col_scale[I8 ? (GATE ? 2 : 1) * kPairs : 1];
  auto load = [&](int i) __attribute__((always_inline)) {
    const int64_t m = min(row0 + 16 * i, p.M - 1);
    if constexpr (I8) row_scale = p.e.row_scale[m];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) ahead[i % kDeep][j].load(p.e, m, min(unit0 + 32 * j, units - 8));
  };
  if constexpr (kDeep == 2) load(0);
  if constexpr (I8) {
#pragma unroll
    for (int j = 0; j < (GATE ? 2 : 1) * kPairs; ++j)
      col_scale[j] = load32(p.e.col_scale + (j / kPairs) * units + min(unit0 + 32 * (j % kPairs), units - 8));
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = row0 + 16 * i;
    if (kDeep == 1 || i + 1 < FM) load(i + kDeep - 1);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int64_t unit = unit0 + 32 * j;
      uint4 lo, hi;
      float v[8], up[8];
      eight(i, 2 * j, lo, hi);
      sums_to_float(I8, lo, hi, v);
      if constexpr (I8) scale8(row_scale, col_scale[j], v);
      if constexpr (GATE) {
        eight(i, 2 * (j + kPairs), lo, hi);
        sums_to_float(I8, lo, hi, up);
        if constexpr (I8) scale8(row_scale, col_scale[j + kPairs], up);
      }
      if (m < p.M && unit < units) {
        if constexpr (GATE) finish_gate<I8>(p.e, m, unit, v, up);
        else finish<I8, MODE>(p.e, m, unit, v, ahead[i % kDeep][j]);
      }
    }
  }
}

// The same for an operand in two terms, whose sums (or parts) are float32 without a
// base: whether one of this lane's is not finite.  again: the sums are twice those of
// the first terms (see dense_tile_terms); where they are not finite and neither is what the
// lane stored before, they take its place.
template <class S>
__device__ __forceinline__ bool sums_of_terms(const DenseGemm& p, int part, int64_t m0, int nt, int wm, int wn,
                                              v4i (&acc)[S::WM / 16][S::WN / 16], bool again) {
  const int lane = lane_id();
  const bool parts = p.split > 1;
  float* const to = parts ? static_cast<float*>(p.part) + (int64_t)part * p.M * p.N : static_cast<float*>(p.e.out);
  const int64_t stride = parts ? p.N : p.e.out_stride;
  const int64_t column = (int64_t)nt * S::BN + wn * S::WN + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  const int64_t row = m0 + wm * S::WM + (lane & 15);
  constexpr float inf = __builtin_inff();
  float odd = 0.0f;  // 0 as long as all are finite
#pragma unroll
  for (int i = 0; i < S::WM / 16; ++i) {
#pragma unroll
    for (int j = 0; j < S::WN / 32; ++j) {
      uint4 lo, hi;
      float v[8];
      eight_columns(acc[i][2 * j], acc[i][2 * j + 1], lo, hi);
      sums_to_float(false, lo, hi, v);
      if (row + 16 * i >= p.M || column + 32 * j >= p.N) continue;
      float* at = to + (row + 16 * i) * stride + column + 32 * j;
      if (again) {
        float before[8];
        load8(at, before);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fabsf(v[k]) < inf || fabsf(before[k]) < inf ? before[k] : v[k];
      }
      store8(at, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) odd = fmaf(v[k], 0.0f, odd);
    }
  }
  return odd != 0.0f;
}

// Tile (mt, nt) of part `part` of the product p.  Of an operand in two terms the first is
// taken in the place of both when `again`; returns whether a sum of this lane is then
// not finite.
template <bool I8, bool AT, bool BT, int MODE, class S, int TERMS = kPlain>
__device__ __forceinline__ bool dense_tile(const DenseGemm& p, int part, int64_t mt, int nt, uint8_t* lds,
                                           bool again = false) {
  constexpr int NW = S::NW, BM = S::BM, BN = S::BN, WAVES_N = S::WAVES_N, WM = S::WM, WN = S::WN;
  constexpr bool GATE = MODE == kDenseGate;
  using TA = Tile<BM, AT, NW, TERMS == kPlain ? kWholeStep : TERMS == kRowTerms ? kTwoTerms : kHalfStep>;
  using TB = Tile<BN, BT, NW, TERMS == kPlain ? kWholeStep : TERMS == kColumnTerms ? kTwoTerms : kHalfStep>;
  const int64_t m0 = mt * BM, n0 = (int64_t)nt * BN;
  if (n0 >= p.N) return false;  // (a half behind the last column)
  const int wave = uniform((int)threadIdx.x / kWave), lane = lane_id();
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  constexpr int kStep = I8 ? 128 : TERMS == kPlain ? 64 : 32;
  const int all = uniform((int)((p.K + kStep - 1) / kStep));
  const int s0 = min(all, part * p.steps), s1 = min(all, s0 + p.steps);
  const int rest = (int)(p.K % kStep);  // of the last step, 0: whole
  TA ta;
  TB tb;
  const int64_t second = again ? 0 : p.lo;  // bytes to the second term
  const int64_t left_m = p.M - m0, left_n = p.N - n0;
  ta.init(p.a + m0 * (AT ? 2 : p.a_stride), p.a_stride, left_m, s0, second, wave,
          [&](int row) { return min((int64_t)row, left_m - 1); });
  if constexpr (GATE) {
    const int64_t inter = p.N / 2, c0 = n0 / 2;
    tb.init(p.b + c0 * p.b_stride, p.b_stride, left_n, s0, second, wave,
            [&](int row) { return gate_row<WN>(row, c0, inter); });
  } else {
    tb.init(p.b + n0 * (BT ? 2 : p.b_stride), p.b_stride, left_n, s0, second, wave,
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

  auto tail = [&](int s) __attribute__((always_inline)) { return rest != 0 && s == all - 1; };
  // rows: stages s % 2; columns: stages s % 3
  int a_cur = 0, b_cur = 0;  // stages of the step at work, relative to the first
  auto a_stage = [&](int d) __attribute__((always_inline)) { return (uint32_t)((a_cur + d) & 1) * TA::kBytes; };
  auto b_stage = [&](int d) __attribute__((always_inline)) {
    const int b = b_cur + d;
    return 2 * TA::kBytes + (uint32_t)(b >= 3 ? b - 3 : b) * TB::kBytes;
  };
  // load u of the rows (columns) of the step d behind the one at work; `last`: the
  // end of k lies in it
  auto issue_a = [&](bool last, int d, int u) __attribute__((always_inline)) {
    if (last) ta.issue_tail(u, AT ? rest : rest * (I8 ? 1 : 2), lds0 + a_stage(d), wave);
    else ta.issue(u, lds0 + a_stage(d), wave);
  };
  auto issue_b = [&](bool last, int d, int u) __attribute__((always_inline)) {
    if (last) tb.issue_tail(u, BT ? rest : rest * (I8 ? 1 : 2), lds0 + b_stage(d), wave);
    else tb.issue(u, lds0 + b_stage(d), wave);
  };
  // Fragments of the two half steps: those of the next half are read under the
  // products of this one, a group of products (one fragment of rows with all
  // fragments of columns) at a time, and the loads go out between the products of
  // a group: the columns of step s + 2 in the first half of step s, in the place
  // of those of step s - 1, its rows in the second, as soon as all waves hold the
  // last fragments of step s, whose place they take.
  constexpr int FM = WM / 16, FN = WN / 16, kPerGroup = FN / FM;
  constexpr int LA = TA::kLoads, LB = TB::kLoads;
  v4i af[2][FM], bf[2][FN];
  auto read_a = [&](int buf, int d, int h, int i) __attribute__((always_inline)) {
    af[buf][i] = fa.read(lds + a_stage(d), i, h);
  };
  auto read_b = [&](int buf, int d, int h, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int j = i * FN / FM; j < (i + 1) * FN / FM; ++j) bf[buf][j] = fb.read(lds + b_stage(d), j, h);
  };
  // Group i of the second half's fragments, and of the next step's first half's (those
  // of the operand with one term wait in the other buffer, see below)
  auto read_second = [&](int i) __attribute__((always_inline)) {
    if constexpr (TERMS != kRowTerms) read_b(1, 0, 1, i);
    if constexpr (TERMS != kColumnTerms) read_a(1, 0, 1, i);
  };
  auto read_first = [&](int d, int i) __attribute__((always_inline)) {
    read_b(TERMS == kRowTerms && d == 1, d, 0, i);
    read_a(TERMS == kColumnTerms && d == 1, d, 0, i);
  };
  auto multiply = [&](int h, int i, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int j = half * FN / 2; j < (half + 1) * FN / 2; ++j)
      acc[i][j] = mma<I8>(bf[TERMS == kRowTerms ? 0 : h][j], af[TERMS == kColumnTerms ? 0 : h][i], acc[i][j]);
  };
  // Of the two waves of a SIMD the older one is served first, and the other falls
  // behind by half a step until the barrier, where the first waits for it alone:
  // behind the barrier the younger one goes first (16384 x 4096 x 7168: 732 -> 701 us).
  const bool late = NW == 8 && wave >= 4;
  // One step.  LOAD: step s + 2 is loaded, 0 not, 1 whole, 2 with the end of k;
  // MORE: step s + 1 follows.  No branches in a step: behind one the
  // compiler waits for every fragment.
  auto step = [&](auto load_c, auto more_c) __attribute__((always_inline)) {
    constexpr int LOAD = decltype(load_c)::value;
    constexpr bool MORE = decltype(more_c)::value;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      read_second(i);
      multiply(0, i, 0);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (LOAD != 0)
#pragma unroll
        for (int u = i * LB / FM; u < (i + 1) * LB / FM; ++u) issue_b(LOAD == 2, 2, u);
      multiply(0, i, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    // step s + 1 has landed (what was issued behind its rows may be under way), and
    // no wave reads the rows of step s any more
    wait_barrier<LOAD != 0 ? LB : 0>();
    if (late) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (MORE) read_first(1, i);
      multiply(1, i, 0);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (LOAD != 0)
#pragma unroll
        for (int u = i * LA / FM; u < (i + 1) * LA / FM; ++u) issue_a(LOAD == 2, 2, u);
      multiply(1, i, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (late) __builtin_amdgcn_s_setprio(0);
    if constexpr (MORE && TERMS == kRowTerms)
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[0][j] = bf[1][j];
    if constexpr (MORE && TERMS == kColumnTerms)
#pragma unroll
      for (int i = 0; i < FM; ++i) af[0][i] = af[1][i];
    a_cur ^= 1;
    b_cur = b_cur == 2 ? 0 : b_cur + 1;
  };
  const int n = s1 - s0;
  if (n > 0) {
    for (int d = 0; d < min(n, 2); ++d) {
      const bool last = tail(s0 + d);
#pragma unroll
      for (int u = 0; u < LB; ++u) issue_b(last, d, u);
#pragma unroll
      for (int u = 0; u < LA; ++u) issue_a(last, d, u);
    }
    if (n > 1) wait_barrier<LA + LB>();
    else wait_barrier<0>();
#pragma unroll
    for (int i = 0; i < FM; ++i) read_first(0, i);
    const bool ends = n > 2 && tail(s1 - 1);
    for (int s = ends ? 3 : 2; s < n; ++s) step(Int<1>(), Int<1>());
    if (ends) step(Int<2>(), Int<1>());
    if (n > 1) step(Int<0>(), Int<1>());
    step(Int<0>(), Int<0>());
  }
  if constexpr (TERMS != kPlain) return sums_of_terms<S>(p, part, m0, nt, wm, wn, acc, again);
  dense_sums<I8, MODE, S>(p, part, m0, nt, wm, wn, acc);
  return false;
}

// The same of an operand in two terms.  An infinity of the other operand, times terms of
// opposite signs or one of them 0, makes NaN of what the formula has as an infinity.  So
// where a sum of the block is not finite its tile is taken again, from the first terms
// in both terms' place: they have the operand's signs, infinities and NaN, and twice
// their sums has the infinities and NaN of the formula.  (4093 tokens of 7168 x 2048,
// trained: 1112 -> 1121 us for the test alone.)
template <bool AT, bool BT, class S, int TERMS>
__device__ __forceinline__ void dense_tile_terms(const DenseGemm& p, int part, int64_t mt, int nt, uint8_t* lds) {
  const int wave = uniform((int)threadIdx.x / kWave);
  int* odd = reinterpret_cast<int*>(lds);  // (no wave reads its operands any more)
  for (bool again = false;; again = true) {
    const bool mine = dense_tile<false, AT, BT, kDenseStore, S, TERMS>(p, part, mt, nt, lds, again);
    if (again) return;
    const bool any = __any(mine);
    if (lane_id() == 0) odd[wave] = any;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < S::NW; ++w) all |= odd[w];
    if (uniform(all) == 0) return;
    __syncthreads();
  }
}


// Tile (mt, nt) of a product of few rows, both operands along k.  All steps but one of a
// ring of S::kStages are under way; one barrier a step, behind which the place of the
// step before is loaded anew.  Narrower than Low, so that more of the CUs work without
// parts and a join: 64 tokens of 2048 x 7168 take 11.4 us (Low in 4 parts 10.2, and 4.0
// for the join), in int8 8.5 (Low 11.8); the block of 7168 x 2048 in int8 with 2
// tokens 27.0 -> 23.2 us, with 64 31.4 -> 26.7.  What a CU takes in of a step's 16 KB
// bounds it, 0.27 us alone and 0.22 by two blocks, also with 64 blocks in all.  Not
// better: rings of 9 steps (28.0 us in place of 26.6 for the block in bf16, 64 tokens, the
// same weights in every call; 4 steps as 5), the fragments read a step ahead with halves
// of a step to a wave (8.6 -> 10.9), blocks that begin at k of their own.
template <bool I8, int MODE, class S>
__device__ __forceinline__ void few_tile(const DenseGemm& p, int part, int64_t mt, int nt, uint8_t* lds) {
  constexpr int NW = S::NW, BM = S::BM, BN = S::BN, WM = S::WM, WN = S::WN, ST = S::kStages;
  using TA = Tile<BM, false, NW, kWholeStep>;
  using TB = Tile<BN, false, NW, kWholeStep>;
  constexpr int kStage = TA::kBytes + TB::kBytes, L = TA::kLoads + TB::kLoads;
  static_assert(L * (ST - 1) < 64, "loads a wave can count");
  static_assert(S::WAVES_N == 1 && ST == 5, "a wave takes all columns; the waits below");
  const int64_t m0 = mt * BM, n0 = (int64_t)nt * BN;
  const int wave = uniform((int)threadIdx.x / kWave);
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  constexpr int kStep = I8 ? 128 : 64;
  const int all = uniform((int)((p.K + kStep - 1) / kStep));
  const int s0 = min(all, part * p.steps), s1 = min(all, s0 + p.steps), n = s1 - s0;
  const int rest = (int)(p.K % kStep) * (I8 ? 1 : 2);  // bytes of the last step, 0: whole
  TA ta;
  TB tb;
  const int64_t left_m = p.M - m0, left_n = p.N - n0;
  ta.init(p.a + m0 * p.a_stride, p.a_stride, left_m, s0, 0, wave,
          [&](int row) { return min((int64_t)row, left_m - 1); });
  if constexpr (MODE == kDenseGate) {
    const int64_t inter = p.N / 2, c0 = n0 / 2;
    tb.init(p.b + c0 * p.b_stride, p.b_stride, left_n, s0, 0, wave,
            [&](int row) { return gate_row<WN>(row, c0, inter); });
  } else {
    tb.init(p.b + n0 * p.b_stride, p.b_stride, left_n, s0, 0, wave,
            [&](int row) { return min((int64_t)row, left_n - 1); });
  }
  Fragments<BM, false, WM> fa;
  Fragments<BN, false, WN> fb;
  fa.init(wave * WM);
  fb.init(0);
  v4i acc[WM / 16][WN / 16];
#pragma unroll
  for (int i = 0; i < WM / 16; ++i)
#pragma unroll
    for (int j = 0; j < WN / 16; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  // step s into place `at` of the ring
  auto issue = [&](int s, int at) __attribute__((always_inline)) {
    const uint32_t to = lds0 + at * kStage;
    if (rest != 0 && s0 + s == all - 1) {
#pragma unroll
      for (int u = 0; u < TB::kLoads; ++u) tb.issue_tail(u, rest, to + TA::kBytes, wave);
#pragma unroll
      for (int u = 0; u < TA::kLoads; ++u) ta.issue_tail(u, rest, to, wave);
    } else {
#pragma unroll
      for (int u = 0; u < TB::kLoads; ++u) tb.issue(u, to + TA::kBytes, wave);
#pragma unroll
      for (int u = 0; u < TA::kLoads; ++u) ta.issue(u, to, wave);
    }
  };
  for (int s = 0; s < min(n, ST - 1); ++s) issue(s, s);
  int at = 0;
  for (int s = 0; s < n; ++s) {
    const int behind = n - 1 - s;  // steps that may be under way, as many as a ring holds
    if (behind >= 3) wait_barrier<3 * L>();
    else if (behind == 2) wait_barrier<2 * L>();
    else if (behind == 1) wait_barrier<L>();
    else wait_barrier<0>();
    const uint8_t* a = lds + at * kStage;
    const uint8_t* b = a + TA::kBytes;
    v4i af[2][WM / 16], bf[2][WN / 16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < WM / 16; ++i) af[h][i] = fa.read(a, i, h);
#pragma unroll
      for (int j = 0; j < WN / 16; ++j) bf[h][j] = fb.read(b, j, h);
    }
    if (s + ST - 1 < n) issue(s + ST - 1, at == 0 ? ST - 1 : at - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < WM / 16; ++i)
#pragma unroll
        for (int j = 0; j < WN / 16; ++j) acc[i][j] = mma<I8>(bf[h][j], af[h][i], acc[i][j]);
    at = at == ST - 1 ? 0 : at + 1;
  }
  dense_sums<I8, MODE, S>(p, part, m0, nt, wave, 0, acc);
}

// The blocks of an XCD take parts and columns next to one another; rows' tiles go last.
template <bool I8, int MODE, class S>
__global__ __launch_bounds__(S::NW* kWave, 2) void k_dense_few(DenseGemm p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  const int tiles_n = (p.N + S::BN - 1) / S::BN;
  const int64_t total = gridDim.x, c = blockIdx.x, x = c & 7;
  const int64_t t = x * (total >> 3) + min(x, total & 7) + (c >> 3);
  const int64_t tiles = total / p.split;
  const int part = uniform((int)(t / tiles));
  const int64_t tile = t - part * tiles;
  few_tile<I8, MODE, S>(p, part, tile / tiles_n, (int)(tile % tiles_n), lds);
}

// Block b of those that share the product p (dense_blocks of them).  Blocks go round
// the 8 XCDs: each takes a contiguous range of the tiles, in groups of 4 rows of
// tiles, so that the blocks at work on one XCD share their operands in its L2.
// HALVES: the last tiles may be those of two blocks each.
template <bool I8, bool AT, bool BT, int MODE, class S, int TERMS = kPlain, bool HALVES = S::BN == Big::BN>
__device__ __forceinline__ void dense_block(const DenseGemm& p, int64_t b, uint8_t* lds) {
  const int64_t tiles_m = (p.M + S::BM - 1) / S::BM;
  const int tiles_n = (p.N + S::BN - 1) / S::BN;
  const int64_t tiles = tiles_m * tiles_n, all = tiles * p.split;
  const int64_t halves = p.halves, whole = all - halves;
  const bool half = b >= whole;
  const int64_t total = half ? 2 * halves : whole, c = half ? b - whole : b, x = c & 7;
  int64_t t = x * (total >> 3) + min(x, total & 7) + (c >> 3);
  const int side = half ? (int)(t & 1) : 0;
  if (half) t = whole + (t >> 1);
  const int part = uniform((int)(t / tiles));
  t -= part * tiles;
  const int64_t group = t / (4 * tiles_n), first_m = group * 4;
  const int gm = (int)min((int64_t)4, tiles_m - first_m);
  const int r = (int)(t - group * 4 * tiles_n);
  const int64_t mt = first_m + r % gm;
  const int nt = r / gm;
  if constexpr (HALVES) {
    if (half) {
      if constexpr (TERMS != kPlain) dense_tile_terms<AT, BT, Half, TERMS>(p, part, mt, 2 * nt + side, lds);
      else dense_tile<I8, AT, BT, MODE, Half>(p, part, mt, 2 * nt + side, lds);
      return;
    }
  }
  if constexpr (TERMS != kPlain) dense_tile_terms<AT, BT, S, TERMS>(p, part, mt, nt, lds);
  else dense_tile<I8, AT, BT, MODE, S>(p, part, mt, nt, lds);
}

template <bool I8, bool AT, bool BT, int MODE, class S>
__global__ __launch_bounds__(S::NW* kWave, 2) void k_dense(DenseGemm p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  dense_block<I8, AT, BT, MODE, S>(p, blockIdx.x, lds);
}

template <bool I8, bool AT, bool BT, int MODE, class S>
hipError_t launch_shape(const DenseGemm& p, hipStream_t st) {
  const int64_t blocks = dense_blocks(p);
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
  k_dense<I8, AT, BT, MODE, S><<<(unsigned)blocks, S::NW * kWave, 0, st>>>(p);
  return hipGetLastError();
}
template <bool I8, bool AT, bool BT, int MODE>
hipError_t launch(const DenseGemm& p, hipStream_t st) {
  switch (p.shape) {
    case kDenseBig: return launch_shape<I8, AT, BT, MODE, Big>(p, st);
    case kDenseMid: return launch_shape<I8, AT, BT, MODE, Mid>(p, st);
    case kDenseLow:
      if constexpr (!AT) return launch_shape<I8, AT, BT, MODE, Low>(p, st);
      return hipErrorInvalidValue;
    case kDenseFew:
      if constexpr (!AT && !BT) {
        const int64_t blocks = dense_blocks(p);
        if (blocks == 0) return hipSuccess;
        if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
        k_dense_few<I8, MODE, Few><<<(unsigned)blocks, Few::NW * kWave, 0, st>>>(p);
        return hipGetLastError();
      }
      return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
  }
}

static_assert(Big::BM == dense_rows(kDenseBig) && Big::BN == dense_columns(kDenseBig), "tiles");
static_assert(Half::BM == Big::BM && 2 * Half::BN == Big::BN && Half::NW == Big::NW && Half::kLds <= Big::kLds, "halves");
static_assert(Mid::BM == dense_rows(kDenseMid) && Mid::BN == dense_columns(kDenseMid), "tiles");
static_assert(Few::BM == dense_rows(kDenseFew) && Few::BN == dense_columns(kDenseFew), "tiles");
static_assert(Low::BM == dense_rows(kDenseLow) && Low::BN == dense_columns(kDenseLow), "tiles");

}  // namespace dense
}  // namespace moe
