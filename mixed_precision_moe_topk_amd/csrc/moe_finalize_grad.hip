// Gradient of the router-weighted sum out[t] = sum_j w[t, j] y2[row(t, j)]
// (the finalize step):
//   dweights[t, j]  = sum_h dout[t, h] y2[row(t, j), h]
//   dy2[row(t, j)]  = w[t, j] dout[t]
// Bound by memory: y2 is read once, dy2 (when wanted) written once, dout read
// once per block that needs it.
#include "moe_train.h"

extern "C" __device__ __attribute__((const)) float __ockl_wfred_add_f32(float);

namespace moe {

__device__ __forceinline__ void bf16x4_to_f32(const uint2& u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

// Rounds to bf16 to nearest even; NaN stays NaN (bf16_bits takes finite
// values only).
__device__ __forceinline__ uint32_t bf16_bits_any(float v) {
  return v == v ? bf16_bits(v) : 0x7FC0u | (__float_as_uint(v) >> 16 & 0x8000u);
}

constexpr int kGradThreads = 512;  // at most; see finalize_grad_threads

enum RowGrad : int { kNoRows = 0, kRowsBf16 = 1, kRowsF32 = 2 };

// One block per (token, KC slots from slot blockIdx.y * KC).  Thread i holds
// columns [4 i, 4 i + 4), then those a block's width further, ...; the KC rows
// of a column group are read together, each wave a whole kilobyte of a row.  dy2
// may be y2: a thread writes an element after it has read it.
// Measured (hidden 7168): 16384 tokens x 6 rows, bf16 gradients: 878 us, 5.09
// TB/s, 98 % of the copy's rate; 64 tokens x 8, float32: 6.6 us.  dweights alone
// (the form of a training step with packed experts): 16384 x 6 432 us, 6.5 TB/s,
// 64 x 8 3.4 us.
template <int KC, int ROWS>
__global__ __launch_bounds__(kGradThreads) void k_finalize_grad(const uint16_t* __restrict__ dout,
                                                       const float* __restrict__ weights,
                                                       const float* y2,
                                                       const int32_t* __restrict__ slot_row,
                                                       int32_t k, int32_t H, int64_t rows,
                                                       float* __restrict__ dweights,
                                                       void* dy2) {
  __shared__ float red[kGradThreads / kWave][KC];
  const int64_t t = blockIdx.x;
  const int j0 = blockIdx.y * KC;
  // a slot past the last, or a row outside the batch, reads row 0 and stores
  // nothing (no branch around a read: the reads of a column group go together)
  int64_t row[KC];
  bool ok[KC];
  float w[KC], acc[KC];
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    const int s = j0 + j < k ? j0 + j : k - 1;
    const int64_t r = slot_row[t * k + s];
    ok[j] = j0 + j < k && r >= 0 && r < rows;
    row[j] = ok[j] ? r : 0;
    w[j] = weights[t * k + s];
    acc[j] = 0.0f;
  }
  const int nv = H / 4;
  for (int i = threadIdx.x; i < nv; i += blockDim.x) {
    float d[4];
    bf16x4_to_f32(reinterpret_cast<const uint2*>(dout + t * H)[i], d);
    float4 y[KC];
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const float4* src = reinterpret_cast<const float4*>(y2 + row[j] * H) + i;
      y[j] = KC == 1 ? *src : load_stream(src);
    }
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      acc[j] += d[0] * y[j].x + d[1] * y[j].y + d[2] * y[j].z + d[3] * y[j].w;
      if (ROWS != kNoRows && ok[j]) {
        const v4f g = {w[j] * d[0], w[j] * d[1], w[j] * d[2], w[j] * d[3]};
        if (ROWS == kRowsF32) {
          __builtin_nontemporal_store(g, reinterpret_cast<v4f*>(static_cast<float*>(dy2) + row[j] * H) + i);
        } else {
          typedef uint32_t v2u __attribute__((ext_vector_type(2)));
          const v2u o = {bf16_bits_any(g[0]) | bf16_bits_any(g[1]) << 16, bf16_bits_any(g[2]) | bf16_bits_any(g[3]) << 16};
          __builtin_nontemporal_store(o, reinterpret_cast<v2u*>(static_cast<uint16_t*>(dy2) + row[j] * H) + i);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < KC; ++j) acc[j] = __ockl_wfred_add_f32(acc[j]);
  if (lane_id() == 0) {
#pragma unroll
    for (int j = 0; j < KC; ++j) red[threadIdx.x / kWave][j] = acc[j];
  }
  __syncthreads();
  const int j = threadIdx.x;
  bool mine = false;
#pragma unroll
  for (int q = 0; q < KC; ++q) mine |= q == j && ok[q];
  float sum = 0.0f;
  if (j < KC)
    for (unsigned i = 0; i < blockDim.x / kWave; ++i) sum += red[i][j];
  if (j < KC && j0 + j < k)
    dweights[t * k + j0 + j] = mine ? sum : 0.0f;
}

// Threads of a block: the row's 16-byte pieces in as few rounds as blocks of
// kGradThreads need, all rounds full (H = 7168: four of 448).
unsigned finalize_grad_threads(int32_t H) {
  const int nv = H / 4, rounds = (nv + kGradThreads - 1) / kGradThreads;
  return (unsigned)((nv + rounds * kWave - 1) / (rounds * kWave) * kWave);
}

template <int KC>
static void launch_kc(const uint16_t* dout, const float* weights, const float* y2,
                      const int32_t* slot_row, int64_t T, int32_t k, int32_t H, float* dweights,
                      void* dy2, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)T, (unsigned)((k + KC - 1) / KC));
  const int64_t rows = T * k;
  const unsigned threads = finalize_grad_threads(H);
  if (!dy2) k_finalize_grad<KC, kNoRows><<<grid, threads, 0, st>>>(dout, weights, y2, slot_row, k, H, rows, dweights, dy2);
  else if (f32) k_finalize_grad<KC, kRowsF32><<<grid, threads, 0, st>>>(dout, weights, y2, slot_row, k, H, rows, dweights, dy2);
  else k_finalize_grad<KC, kRowsBf16><<<grid, threads, 0, st>>>(dout, weights, y2, slot_row, k, H, rows, dweights, dy2);
}

hipError_t launch_finalize_grad(const uint16_t* dout, const float* weights, const float* y2,
                                const int32_t* slot_row, int64_t T, int32_t k, int32_t H,
                                float* dweights, void* dy2, bool dy2_f32, hipStream_t st) {
  if (T == 0) return hipSuccess;
  // Few tokens: one slot a block, so that the rows spread over the CUs (us, bf16
  // gradients, hidden 7168, one slot and all: 64 x 8 4.9 and 10.1, 512 x 6 23.8 and
  // 26.0, 1024 x 6 50 and 53, 2048 x 8 145 and 143; dweights alone: 512 x 6 15.7 and
  // 14.9, 1024 x 6 37 and 29).
  // Many: a block reads dout once for all its slots, so the fewest slots that hold
  // top_k (4096 tokens, dweights alone: 4 of 4 79.6, of 6 80.9; 6 of 6 113.6, of 8
  // 114.9; 16384 with bf16 gradients: 6 of 6 832, of 8 840).  Slots behind the last
  // read row 0, from the caches: 5 of 8 102, 7 of 8 131, against 115 and 148 of
  // all used; 9 as 8 and 1: 205, where 16 take 288.
  if (T < 1024) launch_kc<1>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else if (k <= 2) launch_kc<2>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else if (k <= 4) launch_kc<4>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else if (k == 6) launch_kc<6>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else launch_kc<8>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  return hipGetLastError();
}

}  // namespace moe
