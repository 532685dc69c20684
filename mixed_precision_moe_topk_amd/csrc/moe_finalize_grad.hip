// Gradient of the router-weighted sum out[t] = sum_j w[t, j] y2[row(t, j)]
// (the finalize step):
//   dweights[t, j]  = sum_h dout[t, h] y2[row(t, j), h]
//   dy2[row(t, j)]  = w[t, j] dout[t]
// Bound by memory: y2 is read once, dy2 (when wanted) written once, dout read
// once per block that needs it.
#include "moe_train.h"

extern "C" __device__ __attribute__((const)) float __ockl_wfred_add_f32(float);

namespace moe {

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// Rounds to bf16 to nearest even; NaN stays NaN (bf16_bits takes finite
// values only).
__device__ __forceinline__ uint32_t bf16_bits_any(float v) {
  return v == v ? bf16_bits(v) : 0x7FC0u | (__float_as_uint(v) >> 16 & 0x8000u);
}

enum RowGrad : int { kNoRows = 0, kRowsBf16 = 1, kRowsF32 = 2 };

// One block of 256 threads per (token, KC slots from slot blockIdx.y * KC).
// Thread i holds columns [8 i, 8 i + 8), + 2048, ...; the KC rows of a column
// group are read together.  dy2 may be y2: a thread writes an element after it
// has read it.
template <int KC, int ROWS>
__global__ __launch_bounds__(256) void k_finalize_grad(const uint16_t* __restrict__ dout,
                                                       const float* __restrict__ weights,
                                                       const float* y2,
                                                       const int32_t* __restrict__ slot_row,
                                                       int32_t k, int32_t H, int64_t rows,
                                                       float* __restrict__ dweights,
                                                       void* dy2) {
  __shared__ float red[4][KC];
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
  const int nv = H / 8;
  for (int i = threadIdx.x; i < nv; i += 256) {
    float d[8];
    bf16x8_to_f32(reinterpret_cast<const uint4*>(dout + t * H)[i], d);
    float4 y[KC][2];
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const float4* src = reinterpret_cast<const float4*>(y2 + row[j] * H) + 2 * i;
      y[j][0] = load_stream(src);
      y[j][1] = load_stream(src + 1);
    }
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      acc[j] += d[0] * y[j][0].x + d[1] * y[j][0].y + d[2] * y[j][0].z + d[3] * y[j][0].w +
                d[4] * y[j][1].x + d[5] * y[j][1].y + d[6] * y[j][1].z + d[7] * y[j][1].w;
      if (ROWS != kNoRows && ok[j]) {
        float g[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) g[c] = w[j] * d[c];
        if (ROWS == kRowsF32) {
          v4f* dst = reinterpret_cast<v4f*>(static_cast<float*>(dy2) + row[j] * H) + 2 * i;
          __builtin_nontemporal_store(v4f{g[0], g[1], g[2], g[3]}, dst);
          __builtin_nontemporal_store(v4f{g[4], g[5], g[6], g[7]}, dst + 1);
        } else {
          v4u o;
#pragma unroll
          for (int c = 0; c < 4; ++c) o[c] = bf16_bits_any(g[2 * c]) | bf16_bits_any(g[2 * c + 1]) << 16;
          __builtin_nontemporal_store(o, reinterpret_cast<v4u*>(static_cast<uint16_t*>(dy2) + row[j] * H) + i);
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
  if (j < KC && j0 + j < k)
    dweights[t * k + j0 + j] = mine ? (red[0][j] + red[1][j]) + (red[2][j] + red[3][j]) : 0.0f;
}

template <int KC>
static void launch_kc(const uint16_t* dout, const float* weights, const float* y2,
                      const int32_t* slot_row, int64_t T, int32_t k, int32_t H, float* dweights,
                      void* dy2, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)T, (unsigned)((k + KC - 1) / KC));
  const int64_t rows = T * k;
  if (!dy2) k_finalize_grad<KC, kNoRows><<<grid, 256, 0, st>>>(dout, weights, y2, slot_row, k, H, rows, dweights, dy2);
  else if (f32) k_finalize_grad<KC, kRowsF32><<<grid, 256, 0, st>>>(dout, weights, y2, slot_row, k, H, rows, dweights, dy2);
  else k_finalize_grad<KC, kRowsBf16><<<grid, 256, 0, st>>>(dout, weights, y2, slot_row, k, H, rows, dweights, dy2);
}

hipError_t launch_finalize_grad(const uint16_t* dout, const float* weights, const float* y2,
                                const int32_t* slot_row, int64_t T, int32_t k, int32_t H,
                                float* dweights, void* dy2, bool dy2_f32, hipStream_t st) {
  if (T == 0) return hipSuccess;
  // Few tokens: one slot a block, so that the rows spread over the CUs.
  if (T < 1024) launch_kc<1>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else if (k <= 2) launch_kc<2>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else if (k <= 4) launch_kc<4>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else if (k == 6) launch_kc<6>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  else launch_kc<8>(dout, weights, y2, slot_row, T, k, H, dweights, dy2, dy2_f32, st);
  return hipGetLastError();
}

}  // namespace moe
