// Losses of the router and the gradient of its logits.
//
// With p[t] = softmax(z[t]) over all E experts, lse[t] = log sum_e exp z[t, e],
// and for each sequence s its n_s tokens that count, c_s[e] the number of
// their selections of expert e, f_s[e] = E c_s[e] / (k n_s) and P_s[e] the
// mean of p[t, e] over them:
//   balance = mean over the sequences with tokens of sum_e f_s[e] P_s[e]
//   zloss   = mean over all tokens that count of lse[t]^2
// f is constant in the gradient.  The routing weights w[t] are the softmax
// over the selected logits, so with upstream gradients g_b, g_z and dw:
//   dz[t, e] = p[t, e] ((f_s[e] - sum_i p[t, i] f_s[i]) g_b / (S' n_s)
//                       + 2 lse[t] g_z / n)
//              + sum over slots j with ids[t, j] = e of
//                w[t, j] (dw[t, j] - sum_i w[t, i] dw[t, i])
// (S' sequences with tokens, n tokens).  NaN logits rank as -inf, as in the
// router; a token with no logit above -inf has p = 0, lse = 0 and no gradient.
//
// Both passes read the logits once and are bound by that read (and the
// gradient's write).  Everything is summed in float32, in an order that only
// the sizes and the sequences decide.
#include "moe_train.h"

// Wave-wide reductions of the ROCm device library (result in every lane).
extern "C" __device__ __attribute__((const)) float __ockl_wfred_max_f32(float);
extern "C" __device__ __attribute__((const)) float __ockl_wfred_add_f32(float);

namespace moe {

// Logits per lane: the fewest of these that hold all experts.
static int per_lane(int experts) {
  return experts <= 64 ? 1 : experts <= 128 ? 2 : experts <= 256 ? 4 : experts <= 384 ? 6
       : experts <= 512 ? 8 : 16;
}

// Boundary i of the sequences, clamped to the batch.
__device__ __forceinline__ int64_t seq_edge(const int32_t* offs, int64_t tokens, int32_t i) {
  if (!offs) return i ? tokens : 0;
  const int64_t v = offs[i];
  return v < 0 ? 0 : v > tokens ? tokens : v;
}

// The last sequence that starts at or before token t (-1: none), found by the
// whole wave: 64 probes a step.
__device__ __forceinline__ int32_t find_seq(const int32_t* offs, int64_t tokens, int32_t seqs,
                                            int64_t t) {
  int32_t lo = 0, n = seqs;
  bool first = true;
  while (first || n > 1) {
    const int32_t step = (n + kWave - 1) / kWave;
    const int32_t at = lane_id() * step;
    const bool in = at < n && seq_edge(offs, tokens, lo + at) <= t;
    const int hits = __popcll(__ballot(in));
    if (hits == 0) return first ? -1 : lo;
    lo += (hits - 1) * step;
    n = step < n - (hits - 1) * step ? step : n - (hits - 1) * step;
    first = false;
    if (step == 1) break;
  }
  return lo;
}

// Logits lane, lane + 64, ... of one token; NaN as -inf.
template <int PER>
__device__ __forceinline__ void load_logits(const float* row, int E, float (&x)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane_id() + i * kWave;
    const float v = e < E ? row[e] : -INFINITY;
    x[i] = v == v ? v : -INFINITY;
  }
}

// Mask bits of the tokens [t0, t1), at most 64 (bit i: token t0 + i counts).
__device__ __forceinline__ uint64_t mask_bits(const uint8_t* mask, int64_t t0, int64_t t1) {
  const int64_t t = t0 + lane_id();
  return __ballot(t < t1 && (!mask || mask[t] != 0));
}

// Sums over runs of kLossRun tokens, one wave each: probabilities in
// registers, selections in LDS counters.  A wave writes what it has when its
// sequence ends, into slot (run + sequence): along the tokens one of the two
// grows with every slot, so no two share one.  Where a whole block lies in one
// sequence its waves' sums are joined first, and only the first run's slot is
// written.
template <int PER>
__global__ __launch_bounds__(kLossWaves* kWave) void k_loss_part(RouterLossParams p) {
  __shared__ int32_t hist[kLossWaves][PER * kWave];
  __shared__ float join[kLossWaves][PER * kWave];
  __shared__ float join_z[kLossWaves];
  __shared__ int32_t join_n[kLossWaves];
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int E = p.experts, k = p.top_k;
  const int64_t T = p.tokens;
  const int64_t block0 = (int64_t)blockIdx.x * kLossBlock;
  const int64_t block1 = block0 + kLossBlock < T ? block0 + kLossBlock : T;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0;
  const int64_t words = slot_words(E);

  const int32_t bs = find_seq(p.seq_offsets, T, p.seqs, block0);
  const bool whole = bs >= 0 && seq_edge(p.seq_offsets, T, bs + 1) >= block1;

  const int64_t run = (int64_t)blockIdx.x * kLossWaves + w;
  const int64_t t0 = run * kLossRun;
  const int64_t t1 = t0 + kLossRun < block1 ? t0 + kLossRun : block1;
  float acc[PER];
  float z = 0.0f;
  int32_t n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    acc[i] = 0.0f;
    hist[w][lane + i * kWave] = 0;
  }
  const uint64_t on = mask_bits(p.mask, t0, t1);

  auto flush = [&](int32_t s) {
    float* slot = p.slots + (run + s) * words;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + i * kWave;
      if (e < E) {
        slot[e] = acc[i];
        reinterpret_cast<int32_t*>(slot)[E + e] = hist[w][e];
      }
      acc[i] = 0.0f;
      hist[w][e] = 0;
    }
    if (lane == 0) {
      slot[2 * E] = z;
      reinterpret_cast<int32_t*>(slot)[2 * E + 1] = n;
    }
    z = 0.0f;
    n = 0;
  };

  if (t0 < t1) {
    int32_t s = whole ? bs : find_seq(p.seq_offsets, T, p.seqs, t0);
    int64_t end = s >= 0 ? seq_edge(p.seq_offsets, T, s + 1)
                         : seq_edge(p.seq_offsets, T, 0);  // before the first: nothing counts
    float x[PER], nx[PER];
    load_logits<PER>(p.logits + t0 * E, E, nx);
    int32_t nid = lane < k ? p.ids[t0 * k + lane] : -1;
    bool open = false;  // tokens of sequence s seen
    for (int64_t t = t0; t < t1; ++t) {
#pragma unroll
      for (int i = 0; i < PER; ++i) x[i] = nx[i];
      const int32_t id = nid;
      if (t + 1 < t1) {  // the next token's reads run under this one's arithmetic
        load_logits<PER>(p.logits + (t + 1) * E, E, nx);
        nid = lane < k ? p.ids[(t + 1) * k + lane] : -1;
      }
      while (t >= end && s + 1 < p.seqs) {
        if (open) flush(s);
        open = false;
        ++s;
        end = seq_edge(p.seq_offsets, T, s + 1);
      }
      if (t >= end || s < 0) continue;  // behind the last sequence
      open = true;
      if (!((on >> (t - t0)) & 1)) continue;
      ++n;
      if ((uint32_t)id < (uint32_t)E) atomicAdd(&hist[w][id], 1);
      float m = x[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) m = fmaxf(m, x[i]);
      m = __ockl_wfred_max_f32(m);
      if (m == -INFINITY) continue;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        x[i] = __expf(x[i] - m);
        sum += x[i];
      }
      sum = __ockl_wfred_add_f32(sum);
      const float inv = 1.0f / sum;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += x[i] * inv;
      const float lse = m + __logf(sum);
      z += lse * lse;
    }
    if (!whole && open) flush(s);
  }
  if (!whole) return;

#pragma unroll
  for (int i = 0; i < PER; ++i) join[w][lane + i * kWave] = acc[i];
  if (lane == 0) {
    join_z[w] = z;
    join_n[w] = n;
  }
  __syncthreads();
  float* slot = p.slots + ((int64_t)blockIdx.x * kLossWaves + bs) * words;
  for (int e = threadIdx.x; e < E; e += kLossWaves * kWave) {
    float a = 0.0f;
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < kLossWaves; ++i) {
      a += join[i][e];
      c += hist[i][e];
    }
    slot[e] = a;
    reinterpret_cast<int32_t*>(slot)[E + e] = c;
  }
  if (threadIdx.x == 0) {
    float a = 0.0f;
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < kLossWaves; ++i) {
      a += join_z[i];
      c += join_n[i];
    }
    slot[2 * E] = a;
    reinterpret_cast<int32_t*>(slot)[2 * E + 1] = c;
  }
}

// Block (x, s): experts [64 x, 64 x + 64) of sequence s.  Its 16 waves take
// the sequence's slots in turn; then f, P and the block's part of the balance
// loss.  The last block to finish sums the sequences' parts in order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves* kWave) void k_loss_sum(RouterLossParams p) {
  __shared__ float jp[kSumWaves][kWave];
  __shared__ int32_t jc[kSumWaves][kWave];
  __shared__ float jz[kSumWaves];
  __shared__ int32_t jn[kSumWaves];
  __shared__ bool last;
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int E = p.experts;
  const int64_t T = p.tokens, words = slot_words(E);
  const int32_t s = blockIdx.y;
  const int e = blockIdx.x * kWave + lane;
  const int64_t b = seq_edge(p.seq_offsets, T, s), end = seq_edge(p.seq_offsets, T, s + 1);
  float a = 0.0f, z = 0.0f;
  int32_t c = 0, n = 0;
  auto take = [&](int64_t run) {
    const float* slot = p.slots + (run + s) * words;
    if (e < E) {
      a += slot[e];
      c += reinterpret_cast<const int32_t*>(slot)[E + e];
    }
    z += slot[2 * E];
    n += reinterpret_cast<const int32_t*>(slot)[2 * E + 1];
  };
  if (b < end) {
    const int64_t c1 = (end - 1) / kLossBlock;
    for (int64_t blk = b / kLossBlock + w; blk <= c1; blk += kSumWaves) {
      const int64_t t0 = blk * kLossBlock;
      const int64_t t1 = t0 + kLossBlock < T ? t0 + kLossBlock : T;
      if (b <= t0 && t1 <= end) {
        take(blk * kLossWaves);
      } else {
        const int64_t lo = b > t0 ? b : t0, hi = end < t1 ? end : t1;
        for (int64_t run = lo / kLossRun; run <= (hi - 1) / kLossRun; ++run) take(run);
      }
    }
  }
  jp[w][lane] = a;
  jc[w][lane] = c;
  if (lane == 0) {
    jz[w] = z;
    jn[w] = n;
  }
  __syncthreads();
  if (w == 0) {
    a = z = 0.0f;
    c = n = 0;
    for (int i = 0; i < kSumWaves; ++i) {
      a += jp[i][lane];
      c += jc[i][lane];
      z += jz[i];
      n += jn[i];
    }
    const float per = 1.0f / (float)(n > 0 ? n : 1);
    const float mean = a * per;
    float term = 0.0f;
    if (e < E) {
      p.counts[(int64_t)s * E + e] = c;
      p.mean_probs[(int64_t)s * E + e] = mean;
      term = (float)c * ((float)E * per / (float)p.top_k) * mean;
    }
    term = __ockl_wfred_add_f32(term);
    if (lane == 0) {
      p.seq_part[(int64_t)s * gridDim.x + blockIdx.x] = term;
      if (blockIdx.x == 0) {
        p.seq_part[(int64_t)p.seqs * gridDim.x + s] = z;
        p.seq_tokens[s] = n;
      }
      // the parts above are in memory before the count says so
      __threadfence();
      const int32_t done = atomicAdd(p.counter, 1);
      last = done == (int32_t)(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // every block has written its part: sequences in order, one a thread
  float bal = 0.0f, zs = 0.0f;
  int32_t total = 0, live = 0;
  for (int32_t i = threadIdx.x; i < p.seqs; i += kSumWaves * kWave) {
    for (unsigned x = 0; x < gridDim.x; ++x)
      bal += __builtin_nontemporal_load(p.seq_part + (int64_t)i * gridDim.x + x);
    zs += __builtin_nontemporal_load(p.seq_part + (int64_t)p.seqs * gridDim.x + i);
    const int32_t m = __builtin_nontemporal_load(p.seq_tokens + i);
    total += m;
    live += m > 0;
  }
  bal = __ockl_wfred_add_f32(bal);
  zs = __ockl_wfred_add_f32(zs);
  __syncthreads();  // the arrays above are read
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    total += __shfl_xor(total, o);
    live += __shfl_xor(live, o);
  }
  if (lane == 0) {
    jp[w][0] = bal;
    jz[w] = zs;
    jn[w] = total;
    jc[w][0] = live;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bal = zs = 0.0f;
    total = live = 0;
    for (int i = 0; i < kSumWaves; ++i) {
      bal += jp[i][0];
      zs += jz[i];
      total += jn[i];
      live += jc[i][0];
    }
    p.losses[0] = bal / (float)(live > 0 ? live : 1);
    p.losses[1] = zs / (float)(total > 0 ? total : 1);
    p.seq_tokens[p.seqs] = total;
    p.seq_tokens[p.seqs + 1] = live;
  }
}

hipError_t launch_router_loss(const RouterLossParams& p, hipStream_t st) {
  const unsigned blocks = (unsigned)std::max<int64_t>(1, (p.tokens + kLossBlock - 1) / kLossBlock);
  const dim3 block(kLossWaves * kWave);
  switch (per_lane(p.experts)) {
    case 1: k_loss_part<1><<<blocks, block, 0, st>>>(p); break;
    case 2: k_loss_part<2><<<blocks, block, 0, st>>>(p); break;
    case 4: k_loss_part<4><<<blocks, block, 0, st>>>(p); break;
    case 6: k_loss_part<6><<<blocks, block, 0, st>>>(p); break;
    case 8: k_loss_part<8><<<blocks, block, 0, st>>>(p); break;
    default: k_loss_part<16><<<blocks, block, 0, st>>>(p); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((p.experts + kWave - 1) / kWave), (unsigned)p.seqs);
  k_loss_sum<<<grid, kSumWaves * kWave, 0, st>>>(p);
  return hipGetLastError();
}

// One wave per run of kGradRun tokens; the factors f of the sequence stay in
// registers until the next sequence starts.
constexpr int kGradRun = 4;
template <int PER>
__global__ __launch_bounds__(256) void k_router_grad(RouterGradParams p) {
  const int lane = lane_id();
  const int E = p.experts, k = p.top_k;
  const int64_t T = p.tokens;
  const int64_t t0 = ((int64_t)blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave) * kGradRun;
  const int64_t t1 = t0 + kGradRun < T ? t0 + kGradRun : T;
  if (t0 >= T) return;
  const bool losses = p.dlosses != nullptr;
  float gb = 0.0f, gz = 0.0f;
  if (losses) {
    const int32_t total = p.seq_tokens[p.seqs], live = p.seq_tokens[p.seqs + 1];
    gb = p.dlosses[0] / (float)(live > 0 ? live : 1);
    gz = 2.0f * p.dlosses[1] / (float)(total > 0 ? total : 1);
  }
  const uint64_t on = mask_bits(p.mask, t0, t1);
  int32_t s = find_seq(p.seq_offsets, T, p.seqs, t0);
  int64_t end = s >= 0 ? seq_edge(p.seq_offsets, T, s + 1) : seq_edge(p.seq_offsets, T, 0);
  float f[PER];
  auto factors = [&]() {  // g_b f / (S' n) of sequence s
    if (!losses) return;
    const int32_t n = p.seq_tokens[s];
    const float per = 1.0f / (float)(n > 0 ? n : 1);
    const float c = gb * per * ((float)E * per / (float)k);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + i * kWave;
      f[i] = e < E ? (float)p.counts[(int64_t)s * E + e] * c : 0.0f;
    }
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = 0.0f;
  if (s >= 0) factors();
  float nx[PER];
  load_logits<PER>(p.logits + t0 * E, E, nx);
  for (int64_t t = t0; t < t1; ++t) {
    float x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = nx[i];
    if (t + 1 < t1) load_logits<PER>(p.logits + (t + 1) * E, E, nx);
    bool moved = false;
    while (t >= end && s + 1 < p.seqs) {
      ++s;
      end = seq_edge(p.seq_offsets, T, s + 1);
      moved = true;
    }
    if (t >= end || s < 0) continue;  // behind the last sequence: left as it is
    if (moved) factors();
    float m = x[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, x[i]);
    m = __ockl_wfred_max_f32(m);
    float* out = p.dlogits + t * E;
    if (!((on >> (t - t0)) & 1) || m == -INFINITY) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane + i * kWave;
        if (e < E) out[e] = 0.0f;
      }
      continue;
    }
    float g[PER];
    if (losses) {
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        x[i] = __expf(x[i] - m);
        sum += x[i];
        dot += x[i] * f[i];
      }
      sum = __ockl_wfred_add_f32(sum);
      const float inv = 1.0f / sum;
      dot = __ockl_wfred_add_f32(dot) * inv;
      const float lz = (m + __logf(sum)) * gz;
#pragma unroll
      for (int i = 0; i < PER; ++i) g[i] = x[i] * inv * ((f[i] - dot) + lz);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) g[i] = 0.0f;
    }
    if (p.dweights) {
      float wj = 0.0f, dj = 0.0f;
      int32_t id = -1;
      if (lane < k) {
        wj = p.weights[t * k + lane];
        dj = p.dweights[t * k + lane];
        id = p.ids[t * k + lane];
      }
      const float dot = __ockl_wfred_add_f32(wj * dj);
      const float gj = wj * (dj - dot);
      for (int j = 0; j < k; ++j) {
        const int e = __builtin_amdgcn_readlane(id, j);
        const float v = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, gj), j));
#pragma unroll
        for (int i = 0; i < PER; ++i) g[i] += e == lane + i * kWave ? v : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + i * kWave;
      if (e < E) out[e] = g[i];
    }
  }
}

hipError_t launch_router_grad(const RouterGradParams& p, hipStream_t st) {
  if (p.tokens == 0) return hipSuccess;
  const int64_t per_block = kGradRun * 4;
  const unsigned grid = (unsigned)((p.tokens + per_block - 1) / per_block);
  switch (per_lane(p.experts)) {
    case 1: k_router_grad<1><<<grid, 256, 0, st>>>(p); break;
    case 2: k_router_grad<2><<<grid, 256, 0, st>>>(p); break;
    case 4: k_router_grad<4><<<grid, 256, 0, st>>>(p); break;
    case 6: k_router_grad<6><<<grid, 256, 0, st>>>(p); break;
    case 8: k_router_grad<8><<<grid, 256, 0, st>>>(p); break;
    default: k_router_grad<16><<<grid, 256, 0, st>>>(p); break;
  }
  return hipGetLastError();
}

}  // namespace moe
