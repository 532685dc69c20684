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
// products.  With the rank first in both factors, shrink reads its operands as
// the matrix cores take them; expand and outer transpose theirs in registers
// (8 rows x 8 columns a lane, one byte permute for two elements), so nothing
// passes through LDS but the low-rank rows and the waves' partial sums.
//
// x and the factors are bf16, u and v float32.  Where u and v enter a matrix
// instruction they are split into a high and a low bf16 half (relative error
// at most 2^-18), which fill the two halves of a 32-long contraction: a bf16 u
// would cost the float32 outputs 2^-9.  Float32 dout is split likewise.
#include "moe_train.h"

namespace moe {

// ---------------------------------------------------------------- plan
__device__ __forceinline__ int plan_group(const PlanParams& p, int64_t t) {
  const int32_t id = p.adapter_ids[t];
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
  for (int e = lane; e < G; e += kWave) mask[w][e] = 0;
  __syncthreads();
  int g = -1;
  if (t < p.tokens) {
    g = plan_group(p, t);
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
// Returns the first row of group e.
__device__ int32_t plan_scan(const PlanParams& p, const PlanLayout& l, int32_t n,
                             int32_t (*wsum)[16]) {
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
  if (e < G) {
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
    if (e == G - 1) {
      p.plan[l.first + G] = row0 + pad;
      p.plan[0] = tile0 + nt;
      p.plan[1] = row0 + pad;
    }
  }
  return row0;
}

// A batch of at most 1024 tokens in one launch.
__global__ __launch_bounds__(kPlanGroup) void k_plan_small(PlanParams p, PlanLayout l) {
  __shared__ uint64_t mask[kPlanChunks][kMaxAdapters + 1];
  __shared__ int32_t first[kMaxAdapters + 1];
  __shared__ int32_t wsum[2][16];
  const int g = plan_masks(p, 0, mask);
  int32_t n = 0;
  if ((int)threadIdx.x <= p.adapters)
    for (int u = 0; u < kPlanChunks; ++u) n += __popcll(mask[u][threadIdx.x]);
  const int32_t row0 = plan_scan(p, l, n, wsum);
  if ((int)threadIdx.x <= p.adapters) first[threadIdx.x] = row0;
  __syncthreads();
  if (g >= 0) p.plan[l.rows + first[g] + plan_rank(mask, g)] = (int32_t)threadIdx.x;
}

__global__ __launch_bounds__(kPlanGroup) void k_plan_count(PlanParams p, PlanLayout l) {
  __shared__ uint64_t mask[kPlanChunks][kMaxAdapters + 1];
  plan_masks(p, blockIdx.x, mask);
  const int G = p.adapters + 1;
  if ((int)threadIdx.x >= G) return;
  int32_t n = 0;
  for (int u = 0; u < kPlanChunks; ++u) n += __popcll(mask[u][threadIdx.x]);
  p.plan[l.counts + (int64_t)blockIdx.x * G + threadIdx.x] = n;
}

__global__ __launch_bounds__(kPlanGroup) void k_plan_scan(PlanParams p, PlanLayout l) {
  __shared__ int32_t wsum[2][16];
  const int G = p.adapters + 1, e = threadIdx.x;
  int32_t n = 0;
  if (e < G) {
    constexpr int kB = 16;  // independent loads in flight
    for (int64_t b0 = 0; b0 < l.nblocks; b0 += kB) {
      int32_t v[kB];
#pragma unroll
      for (int u = 0; u < kB; ++u) v[u] = b0 + u < l.nblocks ? p.plan[l.counts + (b0 + u) * G + e] : 0;
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        if (b0 + u < l.nblocks) p.plan[l.counts + (b0 + u) * G + e] = n;
        n += v[u];
      }
    }
  }
  plan_scan(p, l, n, wsum);
}

__global__ __launch_bounds__(kPlanGroup) void k_plan_scatter(PlanParams p, PlanLayout l) {
  __shared__ uint64_t mask[kPlanChunks][kMaxAdapters + 1];
  const int g = plan_masks(p, blockIdx.x, mask);
  if (g < 0) return;
  const int G = p.adapters + 1;
  const int32_t row = p.plan[l.first + g] + p.plan[l.counts + (int64_t)blockIdx.x * G + g] +
                      plan_rank(mask, g);
  p.plan[l.rows + row] = (int32_t)(blockIdx.x * (int64_t)kPlanGroup + threadIdx.x);
}

hipError_t launch_adapter_plan(const PlanParams& p, const PlanLayout& l, hipStream_t st) {
  if (p.tokens <= kPlanGroup) {
    k_plan_small<<<1, kPlanGroup, 0, st>>>(p, l);
    return hipGetLastError();
  }
  k_plan_count<<<(unsigned)l.nblocks, kPlanGroup, 0, st>>>(p, l);
  k_plan_scan<<<1, kPlanGroup, 0, st>>>(p, l);
  k_plan_scatter<<<(unsigned)l.nblocks, kPlanGroup, 0, st>>>(p, l);
  return hipGetLastError();
}

// ---------------------------------------------------------------- operands
// Tile i of the plan; false behind the last one, and for an entry that a plan
// of these sizes cannot hold (a buffer that was never planned).
__device__ __forceinline__ bool plan_tile(const PlanView& v, int64_t i, Tile* t) {
  if (i >= v.max_tiles || i >= v.head[0]) return false;
  *t = v.tiles[i];
  return (uint32_t)t->expert <= (uint32_t)v.adapters && t->nrows >= 1 &&
         t->nrows <= kAdapterTile && t->row0 >= 0 && t->row0 % kAdapterPad == 0 &&
         t->row0 + (t->nrows + kAdapterPad - 1) / kAdapterPad * kAdapterPad <= v.max_rows;
}
// Token of a row, -1 for padding.
__device__ __forceinline__ int64_t plan_token(const PlanView& v, int64_t row) {
  const int64_t t = v.rows[row];
  return t < v.tokens ? t : -1;
}

__device__ __forceinline__ v8bf as_bf16x8(const uint4& u) { return __builtin_bit_cast(v8bf, u); }

// v = hi + lo up to 2^-18 |v|; an infinite hi takes lo = 0.
__device__ __forceinline__ void split_bf16(float v, __bf16* hi, __bf16* lo) {
  const __bf16 h = (__bf16)v;
  const float r = v - (float)h;
  *hi = h;
  *lo = (__bf16)(__builtin_isinf((float)h) ? 0.0f : r);
}
__device__ __forceinline__ void split8(const float4& a, const float4& b, v8bf* hi, v8bf* lo) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __bf16 h, l;
    split_bf16(v[i], &h, &l);
    (*hi)[i] = h;
    (*lo)[i] = l;
  }
}

// 8 rows x 8 columns of bf16 (row i in raw[i]) -> per column its 8 rows.
__device__ __forceinline__ void transpose8(const uint4 (&raw)[8], v8bf (&col)[8]) {
  const auto word = [&](int i, int c) { return c == 0 ? raw[i].x : c == 1 ? raw[i].y : c == 2 ? raw[i].z : raw[i].w; };
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v4u q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = __builtin_amdgcn_perm(word(2 * i + 1, j / 2), word(2 * i, j / 2),
                                   j & 1 ? 0x07060302u : 0x05040100u);
    col[j] = __builtin_bit_cast(v8bf, q);
  }
}

__device__ __forceinline__ v4f mfma_bf16(const v8bf& a, const v8bf& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Sums the accumulators of a block's four waves into wave 0's, in the order
// (0 + 2) + (1 + 3).  red holds 2 N 64 float4.
template <int N>
__device__ __forceinline__ void join_waves(v4f (&acc)[N], v4f* red) {
  const int w = threadIdx.x / kWave, lane = lane_id();
  if (w >= 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[((w - 2) * N + i) * kWave + lane] = acc[i];
  }
  __syncthreads();
  if (w < 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += red[(w * N + i) * kWave + lane];
  }
  __syncthreads();
  if (w == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * kWave + lane] = acc[i];
  }
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += red[i * kWave + lane];
  }
}

// ---------------------------------------------------------------- shrink
// One 64-wide step of K: lane (l16, g) holds elements [8 g, 8 g + 8) of each
// 32-wide half, of W row l16 of a rank block and of X row l16 of a row block.
template <int MT, int RT, bool F32, bool GUARD>
__device__ __forceinline__ void shrink_step(const char* const (&xp)[MT], const uint16_t* const (&wp)[RT],
                                            int k0, int ke, v4f (&acc)[MT * RT]) {
  const int g = lane_id() / 16;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = k0 + 32 * h + 8 * g;
    const bool in = !GUARD || k < ke;
    v8bf a[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
      a[r] = as_bf16x8(in ? *reinterpret_cast<const uint4*>(wp[r] + k) : make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (F32) {
        const float4* s = reinterpret_cast<const float4*>(xp[m] + (int64_t)k * 4);
        v8bf hi, lo;
        split8(in ? s[0] : make_float4(0.f, 0.f, 0.f, 0.f), in ? s[1] : make_float4(0.f, 0.f, 0.f, 0.f), &hi, &lo);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          acc[m * RT + r] = mfma_bf16(a[r], lo, acc[m * RT + r]);
          acc[m * RT + r] = mfma_bf16(a[r], hi, acc[m * RT + r]);
        }
      } else {
        const v8bf b = as_bf16x8(in ? *reinterpret_cast<const uint4*>(xp[m] + (int64_t)k * 2) : make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[m * RT + r] = mfma_bf16(a[r], b, acc[m * RT + r]);
      }
    }
  }
}

template <int MT, int RT, bool F32>
__device__ __forceinline__ void shrink_tile(const ShrinkParams& p, const Tile& tile, int split, v4f* red) {
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int l16 = lane & 15, g = lane >> 4;
  const char* xp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    // rows behind the tile's last repeat it; nothing reads their sums
    const int64_t t = plan_token(p.plan, tile.row0 + min(16 * m + l16, tile.nrows - 1));
    xp[m] = static_cast<const char*>(p.x) + (t < 0 ? 0 : t) * p.x_stride * (F32 ? 4 : 2);
  }
  const uint16_t* wp[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    wp[r] = p.w + ((int64_t)tile.expert * p.rank + min(16 * r + l16, p.rank - 1)) * p.K;
  v4f acc[MT * RT];
#pragma unroll
  for (int i = 0; i < MT * RT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const int kb = split * p.split_k, ke = min(p.K, kb + p.split_k);
  int k = kb + 64 * w;
  for (; k + 64 <= ke; k += 256) shrink_step<MT, RT, F32, false>(xp, wp, k, ke, acc);
  if (k < ke) shrink_step<MT, RT, F32, true>(xp, wp, k, ke, acc);
  join_waves(acc, red);
  if (w != 0) return;
  // lane: row l16 of a row block, ranks [4 g, 4 g + 4) of a rank block
  float* part = p.part + (int64_t)split * p.plan.max_rows * p.rank_pad;
  const int rows = (tile.nrows + kAdapterPad - 1) / kAdapterPad * kAdapterPad;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (16 * m >= rows) break;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      v4f v = acc[m * RT + r];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = 16 * r + 4 * g + i < p.rank ? v[i] : 0.0f;
      if (16 * r < p.rank_pad)
        *reinterpret_cast<v4f*>(part + (int64_t)(tile.row0 + 16 * m + l16) * p.rank_pad + 16 * r + 4 * g) = v;
    }
  }
}

// Block (tile, split): the four waves take the split's 64-wide steps of K in
// turn and join their sums.
template <int RT, bool F32>
__global__ __launch_bounds__(256) void k_adapter_shrink(ShrinkParams p) {
  __shared__ v4f red[2 * 4 * RT * kWave];
  Tile tile;
  if (!plan_tile(p.plan, blockIdx.x, &tile) || tile.expert == p.plan.adapters) return;
  if (tile.nrows <= 16) shrink_tile<1, RT, F32>(p, tile, blockIdx.y, red);
  else shrink_tile<4, RT, F32>(p, tile, blockIdx.y, red);
}

template <bool F32>
static void launch_shrink(const ShrinkParams& p, hipStream_t st) {
  const dim3 grid((unsigned)p.plan.max_tiles, (unsigned)p.splits);
  if (p.rank_pad <= 16) k_adapter_shrink<1, F32><<<grid, 256, 0, st>>>(p);
  else if (p.rank_pad <= 32) k_adapter_shrink<2, F32><<<grid, 256, 0, st>>>(p);
  else if (p.rank_pad <= 64) k_adapter_shrink<4, F32><<<grid, 256, 0, st>>>(p);
  else k_adapter_shrink<8, F32><<<grid, 256, 0, st>>>(p);
}
hipError_t launch_adapter_shrink(const ShrinkParams& p, bool x_f32, hipStream_t st) {
  if (x_f32) launch_shrink<true>(p, st);
  else launch_shrink<false>(p, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------- expand
constexpr int kExpandCols = 128;  // columns of a wave

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  v8bf o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = (__bf16)v[j];
  *reinterpret_cast<v8bf*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Base (or 0) plus add for 8 columns of one token.
template <typename T>
__device__ __forceinline__ void emit8(const ExpandParams& p, int64_t t, int n, const float (&add)[8]) {
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (p.base) load8(static_cast<const T*>(p.base) + t * p.base_stride + n, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += add[j];
  store8(static_cast<T*>(p.out) + t * p.out_stride + n, v);
}

// u of the tile's rows as matrix operands in LDS: per row block and rank block
// a lane's 8 elements, the high halves of ranks [8 g, 8 g + 8) in lane groups
// 0 and 1, the low halves in groups 2 and 3.
template <int MT>
__device__ __forceinline__ void expand_rows(const ExpandParams& p, const Tile& tile, v8bf* frag) {
  const int rb = p.rank_pad / 16;
  const float scale = p.scale[tile.expert];
  const int64_t step = p.plan.max_rows * (int64_t)p.rank_pad;
  for (int i = threadIdx.x; i < MT * rb * 32; i += blockDim.x) {
    const int l = i & 31, m = i / 32 / rb, r = i / 32 % rb;
    const int row = min(16 * m + (l & 15), tile.nrows - 1);
    const float* s = p.part + (int64_t)(tile.row0 + row) * p.rank_pad + 16 * r + 8 * (l >> 4);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int q = 0; q < p.splits; ++q, s += step) {
      const float4 x = reinterpret_cast<const float4*>(s)[0], y = reinterpret_cast<const float4*>(s)[1];
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
    }
    a.x *= scale; a.y *= scale; a.z *= scale; a.w *= scale;
    b.x *= scale; b.y *= scale; b.z *= scale; b.w *= scale;
    v8bf hi, lo;
    split8(a, b, &hi, &lo);
    frag[(m * rb + r) * kWave + l] = hi;
    frag[(m * rb + r) * kWave + l + 32] = lo;
  }
}

// A wave's 128 columns of a tile: lane (l16, g) holds columns 8 l16 + j, which
// are column l16 of matrix j, and rows 4 g + i of a row block, so that it
// reads and writes 8 consecutive elements of a row.
template <int MT, typename T>
__device__ __forceinline__ void expand_tile(const ExpandParams& p, const Tile& tile, int n0, const v8bf* frag) {
  const int lane = lane_id(), l16 = lane & 15, g = lane >> 4;
  const int n = n0 + 8 * l16, rb = p.rank_pad / 16;
  const bool in = n < p.N;
  v4f acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int r = 0; r < rb; ++r) {
    uint4 raw[8];
    v8bf b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = 16 * r + 8 * (g & 1) + i;
      raw[i] = in && q < p.rank
                   ? *reinterpret_cast<const uint4*>(p.w + ((int64_t)tile.expert * p.rank + q) * p.N + n)
                   : make_uint4(0, 0, 0, 0);
    }
    transpose8(raw, b);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const v8bf a = frag[(m * rb + r) * kWave + lane];
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[m][j] = mfma_bf16(a, b[j], acc[m][j]);
    }
  }
  if (!in) return;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * m + 4 * g + i;
      if (row >= tile.nrows) continue;
      const int64_t t = plan_token(p.plan, tile.row0 + row);
      if (t < 0) continue;
      float add[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) add[j] = acc[m][j][i];
      emit8<T>(p, t, n, add);
    }
}

// Block (tile, columns): 128 columns a wave.
template <typename T>
__global__ __launch_bounds__(256) void k_adapter_expand(ExpandParams p) {
  __shared__ v8bf frag[(kAdapterTile / 16) * (kMaxRank / 16) * kWave];
  Tile tile;
  if (!plan_tile(p.plan, blockIdx.x, &tile)) return;
  const int n0 = (blockIdx.y * (blockDim.x / kWave) + threadIdx.x / kWave) * kExpandCols;
  if (tile.expert == p.plan.adapters) {  // no adapter: the base as it is
    if (p.base == p.out && p.base) return;
    const int lane = lane_id(), n = n0 + 8 * (lane & 15);
    const float none[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int row = lane >> 4; row < tile.nrows; row += 4) {
      const int64_t t = plan_token(p.plan, tile.row0 + row);
      if (n < p.N && t >= 0) emit8<T>(p, t, n, none);
    }
    return;
  }
  if (tile.nrows <= 16) expand_rows<1>(p, tile, frag);
  else expand_rows<4>(p, tile, frag);
  __syncthreads();
  if (n0 >= p.N) return;
  if (tile.nrows <= 16) expand_tile<1, T>(p, tile, n0, frag);
  else expand_tile<4, T>(p, tile, n0, frag);
}

hipError_t launch_adapter_expand(const ExpandParams& p, bool out_f32, hipStream_t st) {
  // four waves a block, one where few tiles leave CUs without work
  const int64_t cols = (p.N + kExpandCols - 1) / kExpandCols;
  const int waves = p.plan.max_tiles * cols >= 2048 ? 4 : 1;
  const dim3 grid((unsigned)p.plan.max_tiles, (unsigned)((cols + waves - 1) / waves));
  if (out_f32) k_adapter_expand<float><<<grid, waves * kWave, 0, st>>>(p);
  else k_adapter_expand<uint16_t><<<grid, waves * kWave, 0, st>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------- join
// One block per tile: thread (rank r, 8 rows) writes 16 bytes of each half.
__global__ __launch_bounds__(256) void k_adapter_join(JoinParams p) {
  Tile tile;
  if (!plan_tile(p.plan, blockIdx.x, &tile) || tile.expert == p.plan.adapters) return;
  const int Rp = p.rank_pad;
  const int rows = (tile.nrows + kAdapterPad - 1) / kAdapterPad * kAdapterPad;
  const int64_t step = p.plan.max_rows * (int64_t)Rp;
  const float scale = p.scale[tile.expert];
  for (int i = threadIdx.x; i < rows / 8 * Rp; i += 256) {
    const int r = i % Rp, c = i / Rp * 8;
    v8bf hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = 0.0f;
      if (c + j < tile.nrows) {
        const float* s = p.part + (int64_t)(tile.row0 + c + j) * Rp + r;
        for (int q = 0; q < p.splits; ++q, s += step) v += *s;
        v *= scale;
      }
      __bf16 h, l;
      split_bf16(v, &h, &l);
      hi[j] = h;
      lo[j] = l;
    }
    uint16_t* dst = p.saved + (int64_t)r * p.plan.max_rows + tile.row0 + c;
    *reinterpret_cast<v8bf*>(dst) = hi;
    *reinterpret_cast<v8bf*>(dst + step) = lo;
  }
}

hipError_t launch_adapter_join(const JoinParams& p, hipStream_t st) {
  k_adapter_join<<<(unsigned)p.plan.max_tiles, 256, 0, st>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------- outer
// 32 rows of an adapter a step: lane (l16, g) holds rows [8 g, 8 g + 8) of
// columns [8 l16, 8 l16 + 8) of X, and of rank l16 of a rank block of saved.
template <int RT, bool F32>
__device__ __forceinline__ void outer_sum(const OuterParams& p, const OuterSide& s, int a, int r0, int c0,
                                          v4f (&acc)[RT * 8]) {
  const int lane = lane_id(), w = threadIdx.x / kWave, l16 = lane & 15, g = lane >> 4;
  const int c = c0 + 8 * l16;
  const int64_t M = p.plan.max_rows;
  if (p.plan.tokens == 0) return;
  int64_t b = p.plan.first[a], e = p.plan.first[a + 1];
  b = b < 0 ? 0 : b / kAdapterPad * kAdapterPad;
  e = e > M ? M : e;
  for (int64_t row = b + 32 * w + 8 * g; row - 8 * g < e; row += 128) {
    const bool live = row < e;
    v8bf hi[RT], lo[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint16_t* src = s.saved + (int64_t)(r0 + 16 * r + l16) * M + row;
      const bool in = live && r0 + 16 * r < p.rank_pad;
      hi[r] = as_bf16x8(in ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0));
      lo[r] = as_bf16x8(in ? *reinterpret_cast<const uint4*>(src + M * p.rank_pad) : make_uint4(0, 0, 0, 0));
    }
    uint4 raw[8], low[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = live ? plan_token(p.plan, row + i) : -1;
      raw[i] = low[i] = make_uint4(0, 0, 0, 0);
      if (t >= 0 && c < s.C) {
        if constexpr (F32) {
          const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(s.x) + t * s.x_stride + c);
          v8bf h, l;
          split8(x[0], x[1], &h, &l);
          raw[i] = __builtin_bit_cast(uint4, h);
          low[i] = __builtin_bit_cast(uint4, l);
        } else {
          raw[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(s.x) + t * s.x_stride + c);
        }
      }
    }
    v8bf x[8];
    transpose8(raw, x);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[r * 8 + j] = mfma_bf16(lo[r], x[j], acc[r * 8 + j]);
        acc[r * 8 + j] = mfma_bf16(hi[r], x[j], acc[r * 8 + j]);
      }
    if constexpr (F32) {
      transpose8(low, x);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[r * 8 + j] = mfma_bf16(hi[r], x[j], acc[r * 8 + j]);
    }
  }
}

// Block (128 columns of either side, adapter, 64 ranks): the four waves take
// the adapter's rows in turn.  An adapter without tokens gets zeros.
template <int RT, bool F32>
__global__ __launch_bounds__(256) void k_adapter_outer(OuterParams p) {
  __shared__ v4f red[2 * RT * 8 * kWave];
  const bool second = (int)blockIdx.x >= p.blocks0;
  const OuterSide& s = p.side[second ? 1 : 0];
  const int c0 = ((int)blockIdx.x - (second ? p.blocks0 : 0)) * kExpandCols;
  const int a = blockIdx.y, r0 = blockIdx.z * 16 * RT;
  v4f acc[RT * 8];
#pragma unroll
  for (int i = 0; i < RT * 8; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  if (F32 && second) outer_sum<RT, true>(p, s, a, r0, c0, acc);
  else outer_sum<RT, false>(p, s, a, r0, c0, acc);
  join_waves(acc, red);
  if (threadIdx.x >= kWave) return;
  const int l16 = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int c = c0 + 8 * l16;
  if (c >= s.C) return;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = r0 + 16 * r + 4 * g + i;
      if (q >= p.rank) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[r * 8 + j][i];
      store8(s.grad + ((int64_t)a * p.rank + q) * s.C + c, v);
    }
}

template <bool F32>
static void launch_outer(const OuterParams& p, hipStream_t st) {
  const int64_t cb = p.blocks0 + (p.side[1].C + kExpandCols - 1) / kExpandCols;
  const unsigned z = p.rank_pad > 64 ? 2 : 1;
  const dim3 grid((unsigned)cb, (unsigned)p.plan.adapters, z);
  if (p.rank_pad <= 16) k_adapter_outer<1, F32><<<grid, 256, 0, st>>>(p);
  else if (p.rank_pad <= 32) k_adapter_outer<2, F32><<<grid, 256, 0, st>>>(p);
  else k_adapter_outer<4, F32><<<grid, 256, 0, st>>>(p);
}
hipError_t launch_adapter_outer(const OuterParams& p, bool dout_f32, hipStream_t st) {
  if (dout_f32) launch_outer<true>(p, st);
  else launch_outer<false>(p, st);
  return hipGetLastError();
}

}  // namespace moe
