// Low-rank adapters of many requests beside one projection.
//
// Token t with adapter a (rank R, factors A_a [R, K] and B_a [R, N], both
// stored with the rank first, scale s_a):
//   u[t]   = s_a x[t] A_a^T                 (shrink: contraction over K)
//   out[t] = base[t] + u[t] B_a             (expand: contraction over R)
// and backwards, with v[t] = s_a dout[t] B_a^T:
//   dx[t] = dx_base[t] + v[t] A_a
//   dA_a  = sum over the adapter's tokens of v[t]^T x[t]
//   dB_a  = sum over the adapter's tokens of u[t]^T dout[t]
// So three kernels serve both directions: shrink, expand and the sum of outer
// products (and a join of shrink's partial sums between them).  With the rank
// first in both factors, shrink reads its operands as the matrix cores take
// them, through LDS where a tile is full; expand and outer transpose theirs in
// registers (8 rows of 2 W columns a lane, one byte permute for two elements).
//
// Bound by memory but for the smallest batches: x, base and out pass once, and
// the products, 2 R (K + N) a token, are a few percent of the matrix cores' rate.
// The factors' gradients take three times the products of theirs (parts, below):
// above rank 64 the matrix cores bound them (4096 tokens, rank 128: 45 GFLOP, 37 us
// at the 1214 TFLOP/s of a large product, against 23 us of reads).
// What is measured below is one launch beside a projection of 7168 x 7168
// features; a copy of 1 GiB moves 5.16 TB/s on this card.
//
// x and the factors are bf16, u and v float32.  Where float32 values enter a
// matrix instruction they are split into bf16 parts, v = v0 + v1 (+ v2): two
// parts hold v to 2^-17 and serve bf16 results, three hold all of a float32 and
// serve float32 results (the factors' gradients, float32 out).  A single bf16
// part would cost 2^-8.
//
// An infinity in the operand opposite the parts would meet parts of both signs
// and zeros, whose sum is NaN where v times the infinity is infinite.  The first
// part alone has v's sign and zeros (but for v below 2^-126, which may count as 0
// there).  So where a wave's sums are not all finite they are taken again: expand
// lets only the first parts meet a factor's infinities, shrink of float32 rows
// and outer take the sums of the first parts alone where both are not finite.
// Looking at the sums costs at most 1 us of a launch; a batch trained on an
// infinity or on NaN throughout takes two to four times as long.
#include <type_traits>

#include "moe_train.h"

namespace moe {

// ---------------------------------------------------------------- plan
// The tokens of a group in their order, groups padded to 16 rows (a matrix
// block never spans two adapters) and cut into tiles of 64.  Latency is all of
// it: ids are read once, counted in LDS and scanned; 1024 tokens or fewer 3.0 us.
__device__ __forceinline__ int32_t plan_id(const PlanParams& p, int64_t t) {
  return p.adapter_ids[min(t, p.tokens - 1)];
}
__device__ __forceinline__ int plan_group(const PlanParams& p, int32_t id) {
  return (uint32_t)id < (uint32_t)p.adapters ? id : p.adapters;
}

constexpr int kPlanChunks = kPlanGroup / kPlanChunk;

// Per chunk of 64 tokens and group, the mask of the chunk's tokens in it
// (atomic ORs: the order does not matter).
__device__ __forceinline__ int plan_masks(const PlanParams& p, int64_t block,
                                          uint64_t (*mask)[kMaxAdapters + 1]) {
  const int G = p.adapters + 1;
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int64_t t = block * kPlanGroup + threadIdx.x;
  const int32_t id = plan_id(p, t);  // under the masks' clearing
  for (int e = lane; e < G; e += kWave) mask[w][e] = 0;
  __syncthreads();
  int g = -1;
  if (t < p.tokens) {
    g = plan_group(p, id);
    atomicOr(reinterpret_cast<unsigned long long*>(&mask[w][g]), 1ull << lane);
  }
  __syncthreads();
  return g;
}

// Rank of this thread's token among its group's tokens of the block.
__device__ __forceinline__ int plan_rank(const uint64_t (*mask)[kMaxAdapters + 1], int g) {
  const int lane = lane_id(), w = threadIdx.x / kWave;
  int r = __popcll(mask[w][g] & ((1ull << lane) - 1ull));
  for (int u = 0; u < w; ++u) r += __popcll(mask[u][g]);
  return r;
}

// Thread e holds the tokens n of group e: first rows, padding and tiles.
// Returns the first row of group e; the block that has to write fills the
// plan's lists.
__device__ int32_t plan_scan(const PlanParams& p, const PlanLayout& l, int32_t n,
                             int32_t (*wsum)[16], bool write) {
  const int G = p.adapters + 1, e = threadIdx.x;
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int32_t pad = (n + kAdapterPad - 1) / kAdapterPad * kAdapterPad;
  const int32_t nt = (n + kAdapterTile - 1) / kAdapterTile;
  int32_t a = pad, b = nt;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int32_t ya = __shfl_up(a, o), yb = __shfl_up(b, o);
    if (lane >= o) {
      a += ya;
      b += yb;
    }
  }
  if (lane == kWave - 1) {
    wsum[0][w] = a;
    wsum[1][w] = b;
  }
  __syncthreads();
  int32_t pa = 0, pb = 0;
  for (int i = 0; i < w; ++i) {
    pa += wsum[0][i];
    pb += wsum[1][i];
  }
  const int32_t row0 = pa + a - pad, tile0 = pb + b - nt;
  if (e < G && write) {
    p.plan[l.first + e] = row0;
    for (int32_t i = n; i < pad; ++i) p.plan[l.rows + row0 + i] = -1;
    Tile* tiles = reinterpret_cast<Tile*>(p.plan + l.tiles);
    for (int32_t i = 0; i < nt; ++i) {
      Tile t;
      t.expert = e;
      t.row0 = row0 + i * kAdapterTile;
      t.nrows = min(kAdapterTile, n - i * kAdapterTile);
      t.pad = 0;
      tiles[tile0 + i] = t;
    }
    if (e == G - 1) {  // the group without an adapter comes last
      p.plan[l.first + G] = row0 + pad;
      p.plan[0] = tile0 + nt;
      p.plan[1] = tile0;
    }
  }
  return row0;
}

// Adds a wave's tokens to counters in LDS: the first groups met with one add
// each (prompts hold few), the lanes that are left one by one.
__device__ __forceinline__ void plan_add(int32_t* count, int g) {
  uint64_t left = __ballot(g >= 0);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (left == 0) return;
    const int first = __ffsll((unsigned long long)left) - 1;
    const int lead = __builtin_amdgcn_readlane(g, first);
    const uint64_t same = __ballot(g == lead);
    if (lane_id() == first) atomicAdd(&count[lead], (int32_t)__popcll(same));
    left &= ~same;
  }
  if (left >> lane_id() & 1) atomicAdd(&count[g], 1);
}

// A batch of up to kPlanOne tokens in one launch: every block counts all the
// tokens for itself (integer counts in LDS), those before its own apart, and so
// knows where its rows go; block 0 writes the rest of the plan.  4096 tokens: 6.3
// us against 13.4 in three launches; 16384: 16.6 against 11 in two.
__global__ __launch_bounds__(kPlanGroup) void k_plan_one(PlanParams p, PlanLayout l) {
  __shared__ uint64_t mask[kPlanChunks][kMaxAdapters + 1];
  __shared__ int32_t before[kMaxAdapters + 1], after[kMaxAdapters + 1];
  __shared__ int32_t wsum[2][16];
  const int G = p.adapters + 1, e = threadIdx.x;
  constexpr int kB = kPlanOne / kPlanGroup;
  int32_t id[kB];  // of all blocks' tokens, read at once
  if (l.nblocks > 1) {
#pragma unroll
    for (int u = 0; u < kB; ++u) id[u] = plan_id(p, (int64_t)u * kPlanGroup + threadIdx.x);
  }
  if (e < G) before[e] = after[e] = 0;
  const int g = plan_masks(p, blockIdx.x, mask);  // (its barriers cover the counters)
  if (l.nblocks > 1) {
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const bool other = u != (int)blockIdx.x && u * kPlanGroup + (int)threadIdx.x < p.tokens;
      plan_add(u < (int)blockIdx.x ? before : after, other ? plan_group(p, id[u]) : -1);
    }
  }
  __syncthreads();
  int32_t n = 0;
  if (e < G) {
    for (int u = 0; u < kPlanChunks; ++u) n += __popcll(mask[u][e]);
    n += before[e] + after[e];
  }
  const int32_t row0 = plan_scan(p, l, n, wsum, blockIdx.x == 0);
  if (e < G) before[e] += row0;
  __syncthreads();
  if (g >= 0) p.plan[l.rows + before[g] + plan_rank(mask, g)] = (int32_t)(blockIdx.x * kPlanGroup + threadIdx.x);
}

__global__ __launch_bounds__(kPlanGroup) void k_plan_count(PlanParams p, PlanLayout l) {
  __shared__ int32_t count[kMaxAdapters + 1];
  const int G = p.adapters + 1, e = threadIdx.x;
  const int64_t t = (int64_t)blockIdx.x * kPlanGroup + threadIdx.x;
  const int g = t < p.tokens ? plan_group(p, plan_id(p, t)) : -1;
  if (e < G) count[e] = 0;
  __syncthreads();
  plan_add(count, g);
  __syncthreads();
  if (e < G) p.plan[l.counts + (int64_t)blockIdx.x * G + e] = count[e];
}

// Tokens of group e in all blocks, and (before) in the first `upto`; `store`
// puts the prefixes in the counts' place.
__device__ __forceinline__ int32_t plan_total(const PlanParams& p, const PlanLayout& l, int e, int64_t upto,
                                              int32_t* before, bool store) {
  const int G = p.adapters + 1;
  int32_t n = 0;
  constexpr int kB = 16;  // independent loads in flight
  for (int64_t b0 = 0; b0 < l.nblocks; b0 += kB) {
    int32_t v[kB];
#pragma unroll
    for (int u = 0; u < kB; ++u) v[u] = b0 + u < l.nblocks ? p.plan[l.counts + (b0 + u) * G + e] : 0;
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      if (store && b0 + u < l.nblocks) p.plan[l.counts + (b0 + u) * G + e] = n;
      if (b0 + u == upto) *before = n;
      n += v[u];
    }
  }
  return n;
}

__global__ __launch_bounds__(kPlanGroup) void k_plan_scan(PlanParams p, PlanLayout l) {
  __shared__ int32_t wsum[2][16];
  const int e = threadIdx.x;
  int32_t n = 0, before;
  if (e <= p.adapters) n = plan_total(p, l, e, -1, &before, true);
  plan_scan(p, l, n, wsum, true);
}

// SCAN: every block adds up the counts for itself, which saves the scan's launch
// while they are few.
template <bool SCAN>
__global__ __launch_bounds__(kPlanGroup) void k_plan_scatter(PlanParams p, PlanLayout l) {
  __shared__ uint64_t mask[kPlanChunks][kMaxAdapters + 1];
  __shared__ int32_t first[kMaxAdapters + 1];
  __shared__ int32_t wsum[2][16];
  const int G = p.adapters + 1, e = threadIdx.x;
  const int g = plan_masks(p, blockIdx.x, mask);
  if (SCAN) {
    int32_t n = 0, before = 0;
    if (e < G) n = plan_total(p, l, e, blockIdx.x, &before, false);
    const int32_t row0 = plan_scan(p, l, n, wsum, blockIdx.x == 0);
    if (e < G) first[e] = row0 + before;
    __syncthreads();
  }
  if (g < 0) return;
  const int32_t row = (SCAN ? first[g] : p.plan[l.first + g] + p.plan[l.counts + (int64_t)blockIdx.x * G + g]) +
                      plan_rank(mask, g);
  p.plan[l.rows + row] = (int32_t)(blockIdx.x * (int64_t)kPlanGroup + threadIdx.x);
}

hipError_t launch_adapter_plan(const PlanParams& p, const PlanLayout& l, hipStream_t st) {
  if (p.tokens <= kPlanOne) {
    k_plan_one<<<(unsigned)l.nblocks, kPlanGroup, 0, st>>>(p, l);
    return hipGetLastError();
  }
  k_plan_count<<<(unsigned)l.nblocks, kPlanGroup, 0, st>>>(p, l);
  if (l.nblocks <= 64) {
    k_plan_scatter<true><<<(unsigned)l.nblocks, kPlanGroup, 0, st>>>(p, l);
  } else {
    k_plan_scan<<<1, kPlanGroup, 0, st>>>(p, l);
    k_plan_scatter<false><<<(unsigned)l.nblocks, kPlanGroup, 0, st>>>(p, l);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------- operands
// Tile i of the plan; false behind the last one, and for one that the plan
// cannot hold.
__device__ __forceinline__ bool plan_tile(const PlanView& v, int64_t i, Tile* t) {
  if (i >= v.max_tiles || i >= v.head[0]) return false;
  *t = v.tiles[i];
  return plan_tile_fits(*t, v.adapters, v.max_rows);
}
// Token of a row, -1 for padding.
__device__ __forceinline__ int64_t plan_token(const PlanView& v, int64_t row) {
  const int64_t t = v.rows[row];
  return t < v.tokens ? t : -1;
}

// v as a sum of N bf16 parts; the first part of an infinity or NaN is all of it,
// and that of a finite v stays finite (from 2^128 - 2^119 on the nearest bf16 is
// infinite).  No product is fused into the differences: the parts are those of
// the rounded v wherever they are made.
template <int N>
__device__ __forceinline__ void split_bf16(float v, __bf16 (&part)[N]) {
#pragma clang fp contract(off)
  constexpr float kTop = 0x1.FEp127f;  // the largest bf16
  const bool finite = __builtin_isfinite(v);
  part[0] = (__bf16)(finite ? __builtin_amdgcn_fmed3f(v, -kTop, kTop) : v);
#pragma unroll
  for (int i = 1; i < N; ++i) {
    v = finite ? v - (float)part[i - 1] : 0.0f;
    part[i] = (__bf16)v;
  }
}
template <int N>
__device__ __forceinline__ void split8(const float (&v)[8], v8bf (&part)[N]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __bf16 q[N];
    split_bf16<N>(v[i], q);
#pragma unroll
    for (int n = 0; n < N; ++n) part[n][i] = q[n];
  }
}

// 8 rows x 2 W columns of bf16, row i in raw[i][0 .. W) -> per column its 8
// rows: one byte permute for two elements.
template <int W>
__device__ __forceinline__ void transpose8(const uint32_t (&raw)[8][W], v8bf (&col)[2 * W]) {
#pragma unroll
  for (int j = 0; j < 2 * W; ++j) {
    v4u q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = __builtin_amdgcn_perm(raw[2 * i + 1][j / 2], raw[2 * i][j / 2],
                                   j & 1 ? 0x07060302u : 0x05040100u);
    col[j] = __builtin_bit_cast(v8bf, q);
  }
}

template <int W>
__device__ __forceinline__ void load_words(const void* p, bool in, uint32_t (&w)[W]) {
  typedef uint32_t vec __attribute__((ext_vector_type(W)));
  vec v = {};
  if (in) v = *static_cast<const vec*>(p);
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = v[i];
}
__device__ __forceinline__ v8bf load_bf16x8(const void* p, bool in) {
  uint32_t w[4];
  load_words<4>(p, in, w);
  return __builtin_bit_cast(v8bf, v4u{w[0], w[1], w[2], w[3]});
}
__device__ __forceinline__ void load_f32x8(const float* p, bool in, float (&v)[8]) {
  uint32_t a[4], b[4];
  load_words<4>(p, in, a);
  load_words<4>(p + 4, in, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(a[i]);
    v[4 + i] = __uint_as_float(b[i]);
  }
}

__device__ __forceinline__ v4f mfma_bf16(const v8bf& a, const v8bf& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Infinities and NaN as 0.
__device__ __forceinline__ v8bf clear_infinite(const v8bf& v) {
  v4u w = __builtin_bit_cast(v4u, v);
#pragma unroll
  for (int i = 0; i < 4; ++i)  // an exponent of ones carries into the sign's place
    w[i] &= ~(((w[i] & 0x7F807F80u) + 0x00800080u >> 15 & 0x00010001u) * 0xFFFFu);
  return __builtin_bit_cast(v8bf, w);
}

// Whether any of this lane's sums is infinite or NaN (or their total is beyond
// the floats: then a second look finds nothing).
template <int N>
__device__ __forceinline__ bool any_infinite(const v4f (&acc)[N]) {
  v4f t = acc[0];
#pragma unroll
  for (int i = 1; i < N; ++i) t += acc[i];
  return !__builtin_isfinite(t[0] + t[1] + (t[2] + t[3]));
}
// A sum of all parts' products, given that of the first parts'.
__device__ __forceinline__ float or_first(float all, float first) {
  return __builtin_isfinite(all) || __builtin_isfinite(first) ? all : first;
}

// Sums the accumulators of a block's WAVES waves into wave 0's: the upper half
// of the waves hands its sums to the lower half until one is left.  red holds
// WAVES / 2 x N x 64 entries.
template <int WAVES, int N>
__device__ __forceinline__ void join_waves(v4f (&acc)[N], v4f* red) {
  const int w = threadIdx.x / kWave, lane = lane_id();
#pragma unroll
  for (int h = WAVES / 2; h > 0; h /= 2) {
    if (w >= h && w < 2 * h) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[((w - h) * N + i) * kWave + lane] = acc[i];
    }
    __syncthreads();
    if (w < h) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += red[(w * N + i) * kWave + lane];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- low-rank rows
// Where the low-rank rows go.  frag: operands of expand, per 16 rows and 32
// ranks one 1-KB block for each part, lane (l16, g) holding ranks [8 g, 8 g + 8)
// of row l16.  saved: operands of outer, part n of rank r and row i at
// saved[(n rank_pad + r) max_rows + i].  Both optional.
__device__ __forceinline__ int64_t frag_block(int64_t row16, int rank_pad32, int r32, int parts, int n) {
  return ((row16 * (rank_pad32 / 32) + r32) * parts + n) * 512;
}

// Ranks [16 r + 4 g, + 4) of row row0 + l16 (row0 a multiple of 16), scaled; 0
// behind the adapter's last row and rank.
template <int PARTS>
__device__ __forceinline__ void put_low(const LowRows& o, int64_t row0, int r, const v4f& v) {
  typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
  const int l16 = lane_id() & 15, g = lane_id() >> 4;
  v4bf part[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __bf16 q[3];
    split_bf16<3>(v[i], q);
#pragma unroll
    for (int n = 0; n < 3; ++n) part[n][i] = q[n];
  }
  if (o.frag) {
    const int at = (l16 + 16 * (2 * (r & 1) + (g >> 1))) * 8 + 4 * (g & 1);
#pragma unroll
    for (int n = 0; n < PARTS; ++n) {
      __bf16* dst = reinterpret_cast<__bf16*>(o.frag) + frag_block(row0 / 16, o.rank_pad32, r / 2, PARTS, n);
      *reinterpret_cast<v4bf*>(dst + at) = part[n];
      if (16 * (r + 1) == o.rank_pad && o.rank_pad != o.rank_pad32)  // no rank in the block's other half
        *reinterpret_cast<v4bf*>(dst + at + 256) = v4bf{};
    }
  }
  if (o.saved) {
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<__bf16*>(o.saved)[((int64_t)n * o.rank_pad + 16 * r + 4 * g + i) * o.max_rows + row0 + l16] =
            part[n][i];
  }
}

// ---------------------------------------------------------------- shrink
// The work is cut into units, kShrinkK elements of K of one tile, and every
// block takes an equal run of them, which ends inside a tile: as many tiles as
// CUs, or a few more, would leave most CUs waiting for those with two.  A tile
// is then summed by several blocks (`slots`, at most kMaxSlots), whose float32
// sums meet in the join or in expand.
// Measured: 4096 tokens, rank 32: 13.7 us (58.7 MB of x, 4.3 TB/s); 16384,
// rank 64: 55 us (4.3 TB/s: every 64 rows of x read as many of the factor, from
// L2); 64 tokens of 64 adapters, rank 32: 9.4 us (29 MB of factors, 3.1 TB/s, of
// which 3.8 us are the launch's, as one token takes).
// Blocks a CU: two with two LDS buffers; four with one buffer took 22 and 62 us.
__device__ __forceinline__ int64_t quotient(int64_t a, int32_t b) {  // a >= 0, b > 0
  // the usual sizes fit the 32-bit division, a fraction of the 64-bit one's steps
  return a >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
struct ShrinkRuns {
  int32_t units;  // of a tile
  int32_t run;    // units of a block
  int64_t total;
};
__device__ __forceinline__ ShrinkRuns shrink_runs(const PlanView& v, const ShrinkShape& s) {
  ShrinkRuns r;
  r.units = s.units;
  const int64_t tiles = max(0, min(v.head[1], (int32_t)v.max_tiles));
  r.total = tiles * s.units;
  const int64_t each = (r.total + kShrinkBlocks - 1) / kShrinkBlocks;
  r.run = (int32_t)max((int64_t)s.min_run, each);
  return r;
}
// First of the blocks that sum tile i, and how many they are.
__device__ __forceinline__ int shrink_first(const ShrinkRuns& r, int64_t i) { return (int)quotient(i * r.units, r.run); }
__device__ __forceinline__ int shrink_slots(const ShrinkRuns& r, int64_t i) {
  return (int)quotient(i * r.units + r.units - 1, r.run) - shrink_first(r, i) + 1;
}

template <int RT>
struct ShrinkLds {
  static constexpr int KC = RT <= 4 ? 128 : 64;  // elements of K staged at once
  static constexpr int P = KC + 8;               // row pitch: 16-byte reads of 16 rows meet all banks
  static constexpr int kWords = 2 * (kAdapterTile + 16 * RT) * P;
};

// Operands straight from memory: up to 16 rows, the waves taking the 64-wide
// steps of [k0, ke) in turn (FEW; their sums are joined), or float32 rows (the
// gradient of the router's logits: few columns), 16 a wave.
template <int RT, bool F32, bool FEW>
__device__ __forceinline__ void shrink_direct(const ShrinkParams& p, const Tile& tile, int k0, int ke, v4f (&acc)[RT],
                                              v4f* red) {
  typedef std::conditional_t<F32, float, uint16_t> X;
  const int lane = lane_id(), w = threadIdx.x / kWave, l16 = lane & 15, g = lane >> 4;
  // rows behind the tile's last repeat it; their sums are dropped
  const int64_t t = plan_token(p.plan, tile.row0 + min((FEW ? 0 : 16 * w) + l16, tile.nrows - 1));
  const X* xp = static_cast<const X*>(p.x) + (t < 0 ? 0 : t) * p.x_stride + 8 * g;
  const uint16_t* wp[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    wp[r] = p.w + ((int64_t)tile.expert * p.rank + min(16 * r + l16, p.rank - 1)) * p.K + 8 * g;
  // U steps' reads at once, without a branch around any (a step behind the end
  // repeats the last 8 elements and counts as 0): with so few rows a block's life
  // is the memory's latency, a few times over
  constexpr int U = FEW && !F32 && RT <= 2 ? 4 : FEW && !F32 && RT <= 4 ? 2 : 1;
  constexpr int STEP = FEW ? 256 : 64;
  const auto add = [&](auto parts, v4f (&sum)[RT]) {
    constexpr int PARTS = decltype(parts)::value;
    for (int k = k0 + (FEW ? 64 * w : 0); k < ke; k += U * STEP) {
      v8bf a[U][2][RT], x[U][2][PARTS];
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = k + q * STEP + 32 * h;  // (x and w point at the lane's 8 elements)
          const bool in = at + 8 * g < ke;
          const int from = in ? at : ke - 8 - 8 * g;
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            a[q][h][r] = load_bf16x8(wp[r] + from, true);
            a[q][h][r] = in ? a[q][h][r] : v8bf{};
          }
          if constexpr (F32) {
            float v[8];
            load_f32x8(xp + from, true, v);
            split8<PARTS>(v, x[q][h]);
          } else {
            x[q][h][0] = load_bf16x8(xp + from, true);
          }
#pragma unroll
          for (int n = 0; n < PARTS; ++n) x[q][h][n] = in ? x[q][h][n] : v8bf{};
        }
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = PARTS - 1; n >= 0; --n) sum[r] = mfma_bf16(a[q][h][r], x[q][h][n], sum[r]);
    }
  };
  add(std::integral_constant<int, F32 ? 3 : 1>(), acc);
  if constexpr (F32) {
    if (__any(any_infinite(acc))) {
      v4f first[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) first[r] = v4f{0.f, 0.f, 0.f, 0.f};
      add(std::integral_constant<int, 1>(), first);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = or_first(acc[r][c], first[r][c]);
    }
  }
  if constexpr (FEW) join_waves<4>(acc, red);
}

// A whole tile: KC elements of K of its rows and of the factor pass through
// LDS, read from memory in whole row pieces (256 bytes at RT <= 4; 16 rows of 64
// bytes, as the matrix operands lie, ran at two thirds of the speed), the next
// piece under this one's products.  Wave w sums rows [16 w, 16 w + 16), or from
// rank 64 on 32 rows and half of the ranks (acc: rows, then ranks), which reads a
// fifth (rank 64) or a third less from LDS.
template <int RT>
constexpr int shrink_row_blocks() { return RT >= 4 ? 2 : 1; }  // of a wave
template <int RT>
__device__ __forceinline__ void shrink_staged(const ShrinkParams& p, const Tile& tile, int k0, int ke, v4f (&acc)[RT],
                                              uint16_t* lds) {
  constexpr int KC = ShrinkLds<RT>::KC, P = ShrinkLds<RT>::P;
  constexpr int VR = KC / 8, ROWS = 256 / VR;               // vectors of a row, rows a pass
  constexpr int NX = kAdapterTile / ROWS, NA = (16 * RT + ROWS - 1) / ROWS;
  const int lane = lane_id(), w = threadIdx.x / kWave, l16 = lane & 15, g = lane >> 4;
  const int row = threadIdx.x / VR, col = threadIdx.x % VR * 8;
  constexpr int RB = shrink_row_blocks<RT>(), RW = RT / RB;
  const int m0 = RB * (w % (4 / RB)), r0 = RW * (w / (4 / RB));  // the wave's row and rank blocks
  uint16_t* sx = lds;
  uint16_t* sa = lds + 2 * kAdapterTile * P;
  const uint16_t *xp[NX], *wp[NA];
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int64_t t = plan_token(p.plan, tile.row0 + min(i * ROWS + row, tile.nrows - 1));
    xp[i] = static_cast<const uint16_t*>(p.x) + (t < 0 ? 0 : t) * p.x_stride + col;
  }
#pragma unroll
  for (int i = 0; i < NA; ++i)
    wp[i] = p.w + ((int64_t)tile.expert * p.rank + min(i * ROWS + row, p.rank - 1)) * p.K + col;
  v4u rx[NX], ra[NA];
  const auto load = [&](int k) {
    const bool in = k + col < ke;
#pragma unroll
    for (int i = 0; i < NX; ++i)
      rx[i] = in ? __builtin_nontemporal_load(reinterpret_cast<const v4u*>(xp[i] + k)) : v4u{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NA; ++i) ra[i] = in ? *reinterpret_cast<const v4u*>(wp[i] + k) : v4u{0, 0, 0, 0};
  };
  const auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
      *reinterpret_cast<v4u*>(sx + (b * kAdapterTile + i * ROWS + row) * P + col) = rx[i];
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (NA * ROWS == 16 * RT || i * ROWS + row < 16 * RT)
        *reinterpret_cast<v4u*>(sa + (b * 16 * RT + i * ROWS + row) * P + col) = ra[i];
  };
  load(k0);
  put(0);
  __syncthreads();
  int b = 0;
  for (int k = k0; k < ke; k += KC, b ^= 1) {
    const bool more = k + KC < ke;
    if (more) load(k + KC);
    const uint16_t* x = sx + (b * kAdapterTile + 16 * m0 + l16) * P + 8 * g;
    const uint16_t* a = sa + (b * 16 * RT + 16 * r0 + l16) * P + 8 * g;
#pragma unroll
    for (int s = 0; s < KC; s += 32) {
      v8bf xs[RB];
#pragma unroll
      for (int m = 0; m < RB; ++m) xs[m] = *reinterpret_cast<const v8bf*>(x + 16 * m * P + s);
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const v8bf as = *reinterpret_cast<const v8bf*>(a + 16 * r * P + s);
#pragma unroll
        for (int m = 0; m < RB; ++m) acc[m * RW + r] = mfma_bf16(as, xs[m], acc[m * RW + r]);
      }
    }
    if (more) put(b ^ 1);
    __syncthreads();
  }
}

// kShrinkBlocks blocks, two a CU; block b runs on XCD b % 8, and neighbouring
// runs, mostly of one adapter, go to one XCD, whose L2 then holds its factor.
template <int RT, bool F32>
__global__ __launch_bounds__(256, 2) void k_adapter_shrink(ShrinkParams p) {
  constexpr int kLds = F32 ? 16 : ShrinkLds<RT>::kWords;
  __shared__ uint4 lds[(kLds * 2 > 2 * RT * kWave * 16 ? kLds * 2 : 2 * RT * kWave * 16) / 16];
  const int lane = lane_id(), w = threadIdx.x / kWave, l16 = lane & 15, g = lane >> 4;
  const ShrinkRuns runs = shrink_runs(p.plan, p.shape);
  const int me = (int)(blockIdx.x % 8 * (kShrinkBlocks / 8) + blockIdx.x / 8);
  int64_t u = (int64_t)me * runs.run;
  const int64_t end = min(u + runs.run, runs.total);
  while (u < end) {
    const int64_t i = quotient(u, runs.units);
    const int c0 = (int)(u - i * runs.units), c1 = (int)min((int64_t)runs.units, c0 + end - u);
    u += c1 - c0;
    Tile tile;
    if (!plan_tile(p.plan, i, &tile) || tile.expert == p.plan.adapters) return;
    const int k0 = c0 * kShrinkK, ke = min(p.K, c1 * kShrinkK);
    const bool few = tile.nrows <= 16;
    v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
    if (few) shrink_direct<RT, F32, true>(p, tile, k0, ke, acc, reinterpret_cast<v4f*>(lds));
    else if constexpr (F32) {
      if (16 * w < tile.nrows) shrink_direct<RT, F32, false>(p, tile, k0, ke, acc, nullptr);
    } else {
      shrink_staged<RT>(p, tile, k0, ke, acc, reinterpret_cast<uint16_t*>(lds));
    }
    if (few && w > 0) continue;
    // lane: row l16 of a row block, ranks [4 g, 4 g + 4) of a rank block
    constexpr int RB = F32 ? 1 : shrink_row_blocks<RT>(), RW = RT / RB;
    float* part = p.part + (me - shrink_first(runs, i)) * p.plan.max_rows * p.rank_pad +
                  tile.row0 * (int64_t)p.rank_pad + 4 * g;
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      // acc[q]: its row and rank block
      const int m = few ? 0 : RB * (w % (4 / RB)) + q / RW;
      const int r = few ? q : RW * (w / (4 / RB)) + q % RW;
      const int row = 16 * m + l16;
      if (16 * m >= tile.nrows || 16 * r >= p.rank_pad) continue;
      v4f v = acc[q];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = row < tile.nrows && 16 * r + 4 * g + c < p.rank ? v[c] : 0.0f;
      *reinterpret_cast<v4f*>(part + row * (int64_t)p.rank_pad + 16 * r) = v;
    }
  }
}

template <bool F32>
static void launch_shrink(const ShrinkParams& p, hipStream_t st) {
  if (p.rank_pad <= 16) k_adapter_shrink<1, F32><<<kShrinkBlocks, 256, 0, st>>>(p);
  else if (p.rank_pad <= 32) k_adapter_shrink<2, F32><<<kShrinkBlocks, 256, 0, st>>>(p);
  else if (p.rank_pad <= 64) k_adapter_shrink<4, F32><<<kShrinkBlocks, 256, 0, st>>>(p);
  else k_adapter_shrink<8, F32><<<kShrinkBlocks, 256, 0, st>>>(p);
}
hipError_t launch_adapter_shrink(const ShrinkParams& p, bool x_f32, hipStream_t st) {
  if (x_f32) launch_shrink<true>(p, st);
  else launch_shrink<false>(p, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------- join
// The blocks' sums of a tile, scaled, into frag and saved: a wave for 16 rows
// and 16 ranks, once, so that expand's 56 column blocks and outer's take finished
// operands.  Bound by the latency of its reads: 4096 tokens, rank 32: 4.9 us;
// 16384, rank 64: 5.8.
__global__ __launch_bounds__(256) void k_adapter_join(JoinParams p) {
  Tile tile;
  if (!plan_tile(p.plan, blockIdx.x, &tile) || tile.expert == p.plan.adapters) return;
  const int lane = lane_id(), l16 = lane & 15, g = lane >> 4, ranks = p.rank_pad / 16;
  const int64_t step = p.plan.max_rows * (int64_t)p.rank_pad;
  const float scale = p.scale[tile.expert];
  const int slots = min(shrink_slots(shrink_runs(p.plan, p.shape), blockIdx.x), kMaxSlots);
  const int blocks = (tile.nrows + 15) / 16 * ranks;
  for (int i = blockIdx.y * 4 + threadIdx.x / kWave; i < blocks; i += 4 * gridDim.y) {
    const int64_t row0 = tile.row0 + 16 * (i / ranks);
    const int r = i % ranks;
    const float* s = p.part + (row0 + l16) * p.rank_pad + 16 * r + 4 * g;
    v4f x[kMaxSlots], v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kMaxSlots; ++q)
      x[q] = q < slots ? *reinterpret_cast<const v4f*>(s + q * step) : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kMaxSlots; ++q) v += x[q];
    v *= scale;
    if (p.low.parts == 3) put_low<3>(p.low, row0, r, v);
    else put_low<2>(p.low, row0, r, v);
  }
}

hipError_t launch_adapter_join(const JoinParams& p, hipStream_t st) {
  k_adapter_join<<<dim3((unsigned)p.plan.max_tiles, (unsigned)(p.rank_pad / 16)), 256, 0, st>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------- expand
constexpr int kExpandCols = 128;  // columns of a wave

// 8 elements of a row.  bf16 rows pass the caches by (read once, written once);
// float32 ones take two accesses to a line, which must not leave in between.
struct Row8Bf16 {
  v4u w;
  __device__ __forceinline__ void load(const uint16_t* p) {
    w = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    v8bf o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (__bf16)v[j];
    w = __builtin_bit_cast(v4u, o);
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(p));
  }
};
struct Row8F32 {
  v4f w[2];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = reinterpret_cast<const v4f*>(p)[0];
    w[1] = reinterpret_cast<const v4f*>(p)[1];
  }
  __device__ __forceinline__ float get(int j) const { return w[j / 4][j % 4]; }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    w[0] = v4f{v[0], v[1], v[2], v[3]};
    w[1] = v4f{v[4], v[5], v[6], v[7]};
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<v4f*>(p)[0] = w[0];
    reinterpret_cast<v4f*>(p)[1] = w[1];
  }
};

// Ranks [r0, r0 + 8) of a tile's row as operands of outer, 0 behind the last row.
__device__ __forceinline__ void put_saved(const ExpandParams& p, const Tile& tile, int row, int r0, const float (&u)[8]) {
  const int64_t M = p.plan.max_rows, part = (int64_t)p.rank_pad * M;
  __bf16* dst = reinterpret_cast<__bf16*>(p.saved) + r0 * M + tile.row0 + row;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __bf16 q[3];
    split_bf16<3>(row < tile.nrows ? u[i] : 0.0f, q);
#pragma unroll
    for (int n = 0; n < 3; ++n) dst[n * part + i * M] = q[n];
  }
}

// The steps of a wave's columns whose sums are not finite (bits of steps): as in
// expand, but only the first parts of the rows meet a factor's infinities.  It
// reads everything anew: rarely run, it must not hold registers where it is not.
template <typename T, bool JOINED, typename Row8, int PARTS>
__device__ __forceinline__ void expand_again(const ExpandParams& p, const Tile& tile, uint32_t steps, int n0, int slots,
                                             float scale) {
  int lane = lane_id();
  asm volatile("" : "+v"(lane));  // nothing of this is computed ahead
  const int l16 = lane & 15, g = lane >> 4;
  const bool in = n0 + 8 * l16 < p.N;
  const int n = in ? n0 + 8 * l16 : 0;
#pragma unroll 1
  for (int m = 0; m < kAdapterTile / 16; ++m) {
    if (!(steps >> m & 1)) continue;
    v4f acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int r = 0; 32 * r < p.rank_pad; ++r) {
      const int rank = 32 * r + 8 * g;
      v8bf row[PARTS], col[8];
      if constexpr (JOINED) {
        const uint16_t* f = p.frag + frag_block(tile.row0 / 16 + m, p.rank_pad32, r, PARTS, 0) + lane * 8;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) row[q] = load_bf16x8(f + 512 * q, true);
      } else {
        const float* s = p.part + (int64_t)(tile.row0 + min(16 * m + l16, tile.nrows - 1)) * p.rank_pad + rank;
        float u[8] = {}, x[8];
#pragma unroll 1
        for (int q = 0; q < slots; ++q) {
          load_f32x8(s + q * (p.plan.max_rows * p.rank_pad), rank < p.rank_pad, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] += x[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] *= scale;
        split8<PARTS>(u, row);
      }
      uint32_t raw[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        load_words<4>(p.w + ((int64_t)tile.expert * p.rank + rank + i) * p.N + n, rank + i < p.rank, raw[i]);
      transpose8<4>(raw, col);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const v8bf rest = clear_infinite(col[j]);
#pragma unroll
        for (int q = PARTS - 1; q >= 0; --q) acc[j] = mfma_bf16(row[q], q > 0 ? rest : col[j], acc[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 16 * m + 4 * g + i;
      if (!in || at >= tile.nrows) continue;
      const int64_t t = max((int64_t)0, plan_token(p.plan, tile.row0 + at));
      float f[8];
      Row8 v;
      if (p.base) v.load(static_cast<const T*>(p.base) + t * p.base_stride + n);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = p.base ? v.get(j) + acc[j][i] : acc[j][i];
      v.set(f);
      v.store(static_cast<T*>(p.out) + t * p.out_stride + n);
    }
  }
}

// A wave's 128 columns of a tile.  The factor's columns stay in registers, as
// matrix operands of all its ranks, while the tile's row blocks pass: lane
// (l16, g) holds columns 8 l16 + j, which are column l16 of matrix j, and of
// the sums rows 4 g + i, so it reads and writes 8 consecutive elements of a
// row.  RT: blocks of 32 ranks.  JOINED: the low-rank rows come as operands
// (frag); else as the float32 sums of shrink's blocks, which every wave adds up
// for itself, and the first columns' writes to `saved` when it is wanted: less
// time than a launch that does it once, where rows are few.
// Measured: 4096 tokens, rank 32: 27 us (117 MB of base and out, 4.3 TB/s);
// 16384, rank 64: 98 us (470 MB, 4.8 TB/s; 109 us with each step's reads behind
// the last one's stores); 64 tokens of 64 adapters, rank 32: 7.2 us (32 MB; 2 us
// more with registers for two waves a SIMD in place of three), one token 5.1.
template <int RT, typename T, bool JOINED>
__global__ __launch_bounds__(256, JOINED ? (RT == 1 && sizeof(T) == 2 ? 4 : RT <= 2 ? 3 : 2) : RT == 1 && sizeof(T) == 2 ? 3 : 1) void k_adapter_expand(ExpandParams p) {
  constexpr int PARTS = sizeof(T) == 4 ? 3 : 2;
  typedef std::conditional_t<sizeof(T) == 4, Row8F32, Row8Bf16> Row8;
  // neighbouring blocks on one XCD (block b runs on XCD b % 8), columns first:
  // its blocks cover whole rows of one tile and share a factor
  const int32_t per_tile = p.col_blocks * p.row_blocks;
  const uint32_t total = (uint32_t)max(0, min(p.plan.head[0], (int32_t)p.plan.max_tiles)) * per_tile;  // <= the grid
  const uint32_t each = (total + 7) / 8, id = blockIdx.x % 8 * each + blockIdx.x / 8;
  if (blockIdx.x / 8 >= each || id >= total) return;
  const uint32_t ti = id / (uint32_t)per_tile, at = id - ti * per_tile;
  Tile tile;
  if (!plan_tile(p.plan, ti, &tile)) return;
  const int m0 = (int)(at / (uint32_t)p.col_blocks);
  if (16 * m0 >= tile.nrows) return;
  const int n0 = (int)((at - m0 * p.col_blocks) * (blockDim.x / kWave) + threadIdx.x / kWave) * kExpandCols;
  if (n0 >= p.N) return;
  const int lane = lane_id(), l16 = lane & 15, g = lane >> 4;
  const bool in = n0 + 8 * l16 < p.N;
  const int n = in ? n0 + 8 * l16 : 0;  // columns behind the last read the first and store nothing
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  const bool low = tile.expert != p.plan.adapters;
  if (!low && p.base == p.out && p.base) return;  // no adapter, and the base is in place

  // Row 16 m + 4 g + i of the tile is the lane's i-th of step m; rows behind the
  // last read the last one's base and store nothing.
  const int tok = max(0, (int)plan_token(p.plan, tile.row0 + min(lane, tile.nrows - 1)));
  int t[4], tn[4];  // of this step and of the rows in v
  Row8 v[4];
  const auto load_base = [&](int m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tn[i] = __shfl(tok, 16 * m + 4 * g + i);
    if (base) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i].load(base + tn[i] * (int64_t)p.base_stride + n);
    }
  };
  v8bf a[RT][PARTS];  // the rows as operands
  const auto load_rows = [&](int m, int r) {
    const uint16_t* f =
        p.frag + frag_block(tile.row0 / 16 + m, p.rank_pad32, 32 * r < p.rank_pad ? r : 0, PARTS, 0) + lane * 8;
#pragma unroll
    for (int q = 0; q < PARTS; ++q) a[r][q] = load_bf16x8(f + 512 * q, true);
  };
  // AHEAD: a step's reads go out before the last one's stores, and the first
  // under the factor's (float32 rows do not leave the registers for it)
  constexpr bool AHEAD = JOINED && sizeof(T) == 2;
  const auto ahead = [&](int m) {
    if (!low) return;
#pragma unroll
    for (int r = 0; r < RT; ++r) load_rows(m, r);
  };
  if (AHEAD) {
    ahead(m0);
    load_base(m0);
  }
  v8bf b[RT][8];
  if (low) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      uint32_t raw[8][4];
      const uint16_t* w = p.w + ((int64_t)tile.expert * p.rank + 32 * r + 8 * g) * p.N + n;
      const int left = p.rank - 32 * r - 8 * g;  // ranks of this lane's 8
      if (32 * (r + 1) <= p.rank) {
#pragma unroll
        for (int i = 0; i < 8; ++i) load_words<4>(w + (int64_t)i * p.N, true, raw[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) load_words<4>(w + (int64_t)i * p.N, i < left, raw[i]);
      }
      transpose8<4>(raw, b[r]);
    }
  }
  const int64_t step = p.plan.max_rows * (int64_t)p.rank_pad;
  const float scale = low && !JOINED ? p.scale[tile.expert] : 0.0f;
  const int slots = low && !JOINED
                        ? min(shrink_slots(shrink_runs(p.plan, p.shape), ti), kMaxSlots) : 0;
  uint32_t again = 0;  // bit m: a step with sums that are not finite, which is left for expand_again
#pragma unroll 1
  for (int m = m0; 16 * m < tile.nrows; m += p.row_blocks) {
    if (!AHEAD) load_base(m);
    v4f acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    if (low) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (32 * r >= p.rank_pad) break;
        if constexpr (JOINED && !AHEAD) load_rows(m, r);
        if constexpr (!JOINED) {
          const int row = min(16 * m + l16, tile.nrows - 1);
          const float* s = p.part + (int64_t)(tile.row0 + row) * p.rank_pad + 32 * r + 8 * g;
          const bool some = 32 * r + 8 * g < p.rank_pad;
          float u[8], x[kMaxSlots][8];
#pragma unroll
          for (int q = 0; q < kMaxSlots; ++q) load_f32x8(s + q * step, some && q < slots, x[q]);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = 0.0f;
#pragma unroll
          for (int q = 0; q < kMaxSlots; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] += x[q][i];
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] *= scale;
          if (p.saved && n0 == 0 && some) put_saved(p, tile, 16 * m + l16, 32 * r + 8 * g, u);
          split8<PARTS>(u, a[r]);
        }
#pragma unroll
        for (int q = PARTS - 1; q >= 0; --q)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = mfma_bf16(a[r][q], b[r][j], acc[j]);
      }
    }
    const bool odd = low && __any(any_infinite(acc));
    again |= odd << m;
    const int next = m + p.row_blocks;
    const bool more = AHEAD && 16 * next < tile.nrows;
    if (more) ahead(next);
    Row8 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = base ? v[i].get(j) + acc[j][i] : acc[j][i];
      o[i].set(f);
      if (!low && base) o[i] = v[i];  // as it is: -0 + 0 would be 0
      t[i] = tn[i];
    }
    // (a wait for reads waits for the stores issued before them as well)
    if (more) load_base(next);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (in && !odd && 16 * m + 4 * g + i < tile.nrows) o[i].store(out + t[i] * (int64_t)p.out_stride + n);
  }
  if (again) expand_again<T, JOINED, Row8, PARTS>(p, tile, again, n0, slots, scale);
}

template <typename T, bool JOINED>
static void launch_expand(ExpandParams p, hipStream_t st) {
  const int64_t cols = (p.N + kExpandCols - 1) / kExpandCols;
  const int waves = cols >= 4 ? 4 : (int)cols;
  p.col_blocks = (int32_t)((cols + waves - 1) / waves);
  // few waves (a narrow result): a block for each 16 rows of a tile, else the
  // waves take them one after another and read their columns once
  p.row_blocks = p.plan.max_tiles * cols < 2048 && p.plan.tokens > p.plan.max_tiles ? kAdapterTile / 16 : 1;
  const unsigned grid = (unsigned)((p.plan.max_tiles * p.col_blocks * p.row_blocks + 7) / 8 * 8);
  const unsigned block = waves * kWave;
  if (p.rank_pad <= 32) k_adapter_expand<1, T, JOINED><<<grid, block, 0, st>>>(p);
  else if (p.rank_pad <= 64) k_adapter_expand<2, T, JOINED><<<grid, block, 0, st>>>(p);
  else k_adapter_expand<4, T, JOINED><<<grid, block, 0, st>>>(p);
}
hipError_t launch_adapter_expand(const ExpandParams& p, bool out_f32, hipStream_t st) {
  if (out_f32 && p.frag) launch_expand<float, true>(p, st);
  else if (out_f32) launch_expand<float, false>(p, st);
  else if (p.frag) launch_expand<uint16_t, true>(p, st);
  else launch_expand<uint16_t, false>(p, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------- outer
constexpr int kOuterRows = 64;  // rows of an adapter staged at once

// A staged line holds 64 rows of one column (or rank) as 8 pieces of 8 rows;
// piece i lies at place i ^ swizzle, so that the 16 lines a matrix operand
// reads, and the lines a wave writes, meet all banks.
__device__ __forceinline__ int outer_at(int line, int piece) {
  return line * kOuterRows + (piece ^ ((line >> 2 ^ (line >> 1 & 1) << 2) & 7)) * 8;
}

// Line of column c in a block whose waves take TW matrix blocks each: column l16
// of a wave's block t is its column TW l16 + t, so that a lane ends with TW
// neighbouring columns and a wave stores whole 256-byte pieces at TW = 4.
template <int TW>
__device__ __forceinline__ int outer_line(int c) {
  return c / (16 * TW) * (16 * TW) + c % TW * 16 + c / TW % 16;
}

// An adapter of n rows is summed in m = max(1, ceil(n / p.chunk)) segments of
// equal length (one where p.chunks is 1), so that few adapters, or one that has
// most tokens, still fill the CUs, in one round of blocks: a block's steps follow
// one another at the memory's latency, and the longest segment sets the time.
// Segments are numbered along the adapters.  A single one is summed into the
// gradient at once, several into partial sums (slots, numbered among themselves),
// which k_adapter_outer_join adds up.
struct OuterSegment {
  int a, m;
  int64_t row, end;  // its rows
  int64_t slot;      // of the partial sums; -1: the gradient itself
};
// Segment j, or (JOIN) the j-th adapter of several segments, with its first
// slot; false behind the last.  By the whole wave, 64 adapters at a time.
template <bool JOIN>
__device__ __forceinline__ bool outer_segment(const OuterParams& p, int64_t j, OuterSegment* s) {
  const int L = p.plan.adapters;
  if (p.plan.tokens == 0) {
    *s = {(int)j, 1, 0, 0, -1};
    return !JOIN && j < L;
  }
  const int64_t M = p.plan.max_rows;
  int64_t segs = 0, slots = 0, several = 0;  // of the adapters before
  for (int a0 = 0; a0 < L; a0 += kWave) {
    const int a = a0 + lane_id();
    const int64_t b = min(max((int64_t)p.plan.first[min(a, L)], (int64_t)0), M) / kAdapterPad * kAdapterPad;
    const int64_t e = min(max((int64_t)p.plan.first[min(a + 1, L)], b), M) / kAdapterPad * kAdapterPad;
    const int m = a < L ? p.chunks > 1 ? max(1, (int)((e - b + p.chunk - 1) / p.chunk)) : 1 : 0;
    const int q = m > 1 ? m : 0;
    int sm = m, sq = q;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int ym = __shfl_up(sm, o), yq = __shfl_up(sq, o);
      if (lane_id() >= o) {
        sm += ym;
        sq += yq;
      }
    }
    const uint64_t many = __ballot(m > 1);
    const uint64_t hit = JOIN ? __ballot(m > 1 && several + __popcll(many & ((1ull << lane_id()) - 1ull)) == j)
                              : __ballot(a < L && segs + sm > j);
    if (hit) {
      const int f = __ffsll((unsigned long long)hit) - 1;
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, f); };
      const int64_t row = of((int)b), end = of((int)e);
      s->a = a0 + f;
      s->m = of(m);
      const int64_t k = JOIN ? 0 : j - (segs + of(sm) - s->m);
      const int64_t len = ((end - row + s->m - 1) / s->m + kOuterRows - 1) / kOuterRows * kOuterRows;
      s->row = row + k * len;
      s->end = min(end, s->row + len);
      s->slot = s->m > 1 ? slots + of(sq) - s->m + k : -1;
      return s->slot < 2 * (int64_t)p.chunks;  // a plan of these sizes has no more
    }
    segs += __builtin_amdgcn_readlane(sm, kWave - 1);
    slots += __builtin_amdgcn_readlane(sq, kWave - 1);
    several += __popcll(many);
  }
  return false;
}

// A wave's sums again, from the first parts alone and straight from memory: where
// neither is finite the first parts' takes the stored one's place.
template <bool F32, int TW, int RW>
__device__ __forceinline__ void outer_again(const OuterParams& p, const OuterSide& s, const OuterSegment& seg, float* grad,
                                            int c0) {
  typedef std::conditional_t<F32, float, uint16_t> X;
  int thread = threadIdx.x;
  asm volatile("" : "+v"(thread));  // nothing of this is computed ahead, where it would hold registers
  const int l16 = thread & 15, g = thread / 16 % 4, r0 = thread / 256 * RW;
  c0 += thread / kWave % 4 * 16 * TW;
  const int64_t M = p.plan.max_rows;
#pragma unroll 1
  for (int i = 0; i < TW * RW; ++i) {
    const int c = c0 + l16 * TW + i % TW, r = 16 * (r0 + i / TW);
    float all[4];
    bool odd = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int rank = r + 4 * g + k;
      all[k] = c < s.C && rank < p.rank ? grad[(int64_t)rank * s.C + c] : 0.0f;
      odd |= !__builtin_isfinite(all[k]);
    }
    if (!__any(odd)) continue;
    const X* x = static_cast<const X*>(s.x) + min(c, s.C - 1);
    const uint16_t* saved = s.saved + min(r + l16, p.rank_pad - 1) * M;
    v4f first = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int64_t row = seg.row + 8 * g; row - 8 * g < seg.end; row += 32) {
      const bool in = row < seg.end;  // (segments are whole pieces of 16 rows)
      v8bf q;
      int64_t t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = in ? plan_token(p.plan, row + k) : -1;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const X v = x[max(t[k], (int64_t)0) * s.x_stride];
        __bf16 part[1];
        if constexpr (F32) split_bf16<1>(v, part);
        else part[0] = __builtin_bit_cast(__bf16, v);
        q[k] = t[k] < 0 ? (__bf16)0.0f : part[0];
      }
      first = mfma_bf16(load_bf16x8(saved + row, in), q, first);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!__builtin_isfinite(all[k])) grad[(int64_t)(r + 4 * g + k) * s.C + c] = or_first(all[k], first[k]);
  }
}

// Sums of one block's columns [c0, c0 + CB) of a factor.  Each thread reads W
// columns of 8 rows (a wave whole row pieces of 256 or 512 bytes), turns them in
// registers into lines of 8 rows, and hands them to the block through LDS; the
// saved values already lie so.  The waves then sum a quarter of the columns
// each, over all rows: no partial sums to join.  F32: X is float32,
// three bf16 parts like the saved values; the products of a second with a third
// part (2^-25 of the term, twice) and of the third parts (2^-34) are left out.
// Measured: 4096 tokens, rank 32, both factors: 32 us (117 MB of x and dout, 3.7
// TB/s; rank 64: 45, 128: 72 us), beside the router (7168 and 256 float32
// columns, rank 12) 19.8 us.  Bound by memory up to rank 64: without the products 3 us less, without
// the sums' stores 3.7, a launch without rows 6.5.  Four waves that split the rows
// and transpose straight into operands, without LDS, took 36 us: each reads the
// saved values for 128 columns in place of 256.  Rank 64 by eight waves, 256
// columns: 49 us.
// RT > 4: eight waves, two for each quarter, half of the ranks each.
template <int RT>
constexpr int outer_threads() { return RT <= 4 ? 256 : 512; }
template <int RT, bool F32>
constexpr int outer_cols() { return F32 ? 64 : RT <= 2 ? 256 : 128; }  // columns of a block
template <int RT, bool F32>
__device__ __forceinline__ void outer_block(const OuterParams& p, const OuterSide& s, const OuterSegment& seg, int c0,
                                            __bf16* lds) {
  constexpr int XP = F32 ? 3 : 1;       // parts of X
  constexpr int CB = outer_cols<RT, F32>();
  constexpr int TW = CB / 64;           // matrix column blocks of a wave
  constexpr int NT = outer_threads<RT>(), PT = NT / 8;  // threads, and those of 8 rows
  constexpr int RW = RT * 256 / NT;     // rank blocks of a wave
  constexpr int W = CB / PT;            // columns of a thread
  constexpr int WORDS = F32 ? W : W / 2;
  constexpr int NV = (3 * 16 * RT * 8 + NT - 1) / NT;
  typedef std::conditional_t<F32, float, uint16_t> X;
  __bf16* xs = lds;
  __bf16* vs = lds + XP * CB * kOuterRows;
  const int lane = lane_id(), l16 = lane & 15, g = lane >> 4;
  const int w = threadIdx.x / kWave % 4, r0 = threadIdx.x / 256 * RW;  // the wave's columns and rank blocks
  const int piece = threadIdx.x / PT, col = threadIdx.x % PT * W;
  const bool in = c0 + col < s.C;
  const X* x = static_cast<const X*>(s.x) + (in ? c0 + col : 0);
  const int64_t M = p.plan.max_rows;
  const uint32_t last = (uint32_t)max((int64_t)1, p.plan.tokens) - 1;
  int64_t row = seg.row;
  const int64_t end = seg.end;
  // The next step's tokens, as they lie in the plan: read without a condition
  // and looked at when they are used (a test at the read would wait for it, and
  // for all reads before it).
  int4 tok[2];
  uint32_t raw[8][WORDS];
  v4u rv[NV];
  const auto tokens = [&](int64_t r) {
    const int4* t = reinterpret_cast<const int4*>(p.plan.rows + min(r + 8 * piece, M - 8));
    tok[0] = t[0];
    tok[1] = t[1];
  };
  uint32_t drop;  // bit 7 - i: row i of this thread's 8 is padding, or behind the end
  const auto load = [&](int64_t r) {
    const int32_t t[8] = {tok[0].x, tok[0].y, tok[0].z, tok[0].w, tok[1].x, tok[1].y, tok[1].z, tok[1].w};
    drop = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      drop = __builtin_amdgcn_alignbit(drop, (uint32_t)t[i], 31);  // drop << 1 | sign of t
      load_words<WORDS>(x + (int64_t)min((uint32_t)t[i], last) * s.x_stride, true, raw[i]);
    }
    drop = in && r + 8 * piece < end ? drop : 0xFF;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * NT + threadIdx.x, line = min(v / 8, 3 * 16 * RT - 1);  // line: part, then rank
      const int rank = min(line % (16 * RT), p.rank_pad - 1), part = line / (16 * RT);
      rv[i] = *reinterpret_cast<const v4u*>(s.saved + ((int64_t)part * p.rank_pad + rank) * M +
                                            min(r + 8 * (v % 8), M - 8));
    }
  };
  const auto put = [&](int64_t r) {
    if (__any((int)drop)) {  // mostly none is
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < WORDS; ++j) raw[i][j] = drop >> (7 - i) & 1 ? 0 : raw[i][j];
    }
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float v[8];
        v8bf q[3];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(raw[i][j]);
        split8<3>(v, q);
#pragma unroll
        for (int n = 0; n < 3; ++n)
          *reinterpret_cast<v8bf*>(xs + n * CB * kOuterRows + outer_at(outer_line<TW>(col + j), piece)) = q[n];
      }
    } else {
      v8bf q[W];
      transpose8<WORDS>(raw, q);
#pragma unroll
      for (int j = 0; j < W; ++j) *reinterpret_cast<v8bf*>(xs + outer_at(outer_line<TW>(col + j), piece)) = q[j];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * NT + threadIdx.x;
      const bool ok = r + 8 * (v % 8) < end;  // (ranks behind the last repeat it, and are not stored)
      if (3 * 16 * RT * 8 % NT == 0 || v < 3 * 16 * RT * 8)
        *reinterpret_cast<v4u*>(vs + outer_at(v / 8, v % 8)) = ok ? rv[i] : v4u{0, 0, 0, 0};
    }
  };
  v4f acc[TW][RW];
#pragma unroll
  for (int t = 0; t < TW; ++t)
#pragma unroll
    for (int r = 0; r < RW; ++r) acc[t][r] = v4f{0.f, 0.f, 0.f, 0.f};
  if (row < end) {
    tokens(row);
    load(row);
    tokens(row + kOuterRows);
  }
  for (; row < end; row += kOuterRows) {
    put(row);
    __syncthreads();
    if (row + kOuterRows < end) {  // under this step's products
      load(row + kOuterRows);
      tokens(row + 2 * kOuterRows);
    }
#pragma unroll
    for (int k = 0; k < kOuterRows / 32; ++k) {
      v8bf q[TW][XP];
#pragma unroll
      for (int t = 0; t < TW; ++t)
#pragma unroll
        for (int m = 0; m < XP; ++m)
          q[t][m] = *reinterpret_cast<const v8bf*>(
              xs + m * CB * kOuterRows + outer_at((w * TW + t) * 16 + l16, 4 * k + g));
#pragma unroll
      for (int n = 2; n >= 0; --n)
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const v8bf u =
              *reinterpret_cast<const v8bf*>(vs + outer_at((n * RT + r0 + r) * 16 + l16, 4 * k + g));
#pragma unroll
          for (int m = min(XP - 1, 2 - n); m >= 0; --m)
#pragma unroll
            for (int t = 0; t < TW; ++t) acc[t][r] = mfma_bf16(u, q[t][m], acc[t][r]);
        }
    }
    __syncthreads();
  }
  float* grad = seg.slot < 0 ? s.grad + (int64_t)seg.a * p.rank * s.C
                             : p.part + (seg.slot * (p.x.C + p.dout.C) + s.part_at) * p.rank;
  // lane: TW columns of ranks 4 g .. 4 g + 3 of a rank block
  typedef float vec __attribute__((ext_vector_type(TW)));
  const int c = c0 + (w * 16 + l16) * TW;
  if (c < s.C) {
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = 16 * (r0 + r) + 4 * g + i;
        vec v;
#pragma unroll
        for (int t = 0; t < TW; ++t) v[t] = acc[t][r][i];
        if (q < p.rank) *reinterpret_cast<vec*>(grad + (int64_t)q * s.C + c) = v;
      }
  }
  bool odd = false;
#pragma unroll
  for (int t = 0; t < TW; ++t) odd |= any_infinite(acc[t]);
  if (__any(odd)) outer_again<F32, TW, RW>(p, s, seg, grad, c0);
}

// Block (columns of either factor, segment).  Both factors in one launch: the
// second's blocks fill the CUs the first leaves.
template <int RT, bool F32>
__global__ __launch_bounds__(outer_threads<RT>(), RT <= 4 ? 3 : 4) void k_adapter_outer(OuterParams p) {
  constexpr int kX = outer_cols<RT, false>();
  constexpr int kLds = (F32 && 3 * 64 > kX ? 3 * 64 : kX) * kOuterRows + 3 * 16 * RT * kOuterRows;
  __shared__ __align__(16) __bf16 lds[kLds];
  // columns first, over all XCDs: segments differ in length, and a run of them on
  // one XCD (its L2 would hold their saved values) left others idle
  const uint32_t at = blockIdx.x / (uint32_t)p.cols;
  OuterSegment seg;
  if (!outer_segment<false>(p, at, &seg)) return;
  const int col = (int)(blockIdx.x - at * p.cols), second = col - p.cols0;
  if (second < 0) outer_block<RT, false>(p, p.x, seg, col * kX, lds);
  else outer_block<RT, F32>(p, p.dout, seg, second * outer_cols<RT, F32>(), lds);
}

// Block (elements, j): the partial sums of the j-th adapter of several
// segments, added in the rows' order.  5.8 us for 4 adapters of 4096 tokens.
__global__ __launch_bounds__(256) void k_adapter_outer_join(OuterParams p) {
  OuterSegment seg;
  if (!outer_segment<true>(p, blockIdx.y, &seg)) return;
  const int64_t CA = (int64_t)p.x.C * p.rank, both = CA + (int64_t)p.dout.C * p.rank;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= both) return;
  const int64_t step = both / 4, last = min((int64_t)seg.m, 2 * (int64_t)p.chunks - seg.slot);
  const v4f* src = reinterpret_cast<const v4f*>(p.part + i) + seg.slot * step;
  v4f v = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k = 0; k < last; k += 4) {  // four segments' reads together
    v4f x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = k + q < last ? src[(k + q) * step] : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q) v += x[q];
  }
  float* dst = i < CA ? p.x.grad + seg.a * CA + i : p.dout.grad + (int64_t)seg.a * (both - CA) + (i - CA);
  *reinterpret_cast<v4f*>(dst) = v;
}

template <int RT, bool F32>
static void launch_outer(OuterParams p, hipStream_t st) {
  constexpr int X = outer_cols<RT, false>(), D = outer_cols<RT, F32>();
  p.cols0 = (p.x.C + X - 1) / X;
  p.cols = p.cols0 + (p.dout.C + D - 1) / D;
  // at most one segment an adapter and one a chunk
  k_adapter_outer<RT, F32><<<(unsigned)(p.cols * ((int64_t)p.plan.adapters + p.chunks)), outer_threads<RT>(), 0, st>>>(p);
}
hipError_t launch_adapter_outer(const OuterParams& p, bool dout_f32, hipStream_t st) {
  const int rt = p.rank_pad / 16;
  if (dout_f32) {
    if (rt <= 1) launch_outer<1, true>(p, st);
    else if (rt <= 2) launch_outer<2, true>(p, st);
    else if (rt <= 4) launch_outer<4, true>(p, st);
    else launch_outer<8, true>(p, st);
  } else {
    if (rt <= 1) launch_outer<1, false>(p, st);
    else if (rt <= 2) launch_outer<2, false>(p, st);
    else if (rt <= 4) launch_outer<4, false>(p, st);
    else launch_outer<8, false>(p, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.chunks <= 1) return e;
  const int64_t both = (int64_t)p.rank * (p.x.C + p.dout.C);
  k_adapter_outer_join<<<dim3((unsigned)((both + 1023) / 1024), (unsigned)min(p.chunks, p.plan.adapters)), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
