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
// Both passes read the logits once.  Long batches are bound by that read (and
// the gradient's write), short ones by the chain of a token's reductions and the
// launches.  Everything is summed in float32, in an order that only the sizes and
// the sequences decide.
#include <type_traits>
#include <utility>

#include "moe_train.h"

// Wave-wide reductions of the ROCm device library (result in every lane).
extern "C" __device__ __attribute__((const)) float __ockl_wfred_max_f32(float);
extern "C" __device__ __attribute__((const)) float __ockl_wfred_add_f32(float);

namespace moe {

// Logits per lane: the fewest of these that hold all experts; the reads behind
// the last expert and a smaller batch cost the rest.  4096 tokens, losses and
// gradient: 384 experts 14.2 and 7.9 us, 512: 15.3 and 8.8, 520: 18.1 and 8.9,
// 1024: 18.7 and 10.8.
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

// Walks a wave along the tokens: s, the last sequence that starts at or before
// the token (-1: none), and end, the boundary behind it.  The wave holds 64
// boundaries, one a lane, so that one read finds both where there are at most
// 63 sequences; more are searched 64 at a time.
struct SeqCursor {
  const int32_t* offs;
  int64_t tokens;
  int32_t seqs, s;
  int64_t end;
  int32_t edge;  // lane l: boundary lo + l of the window
  int32_t lo;

  __device__ __forceinline__ SeqCursor(const int32_t* offs_, int64_t tokens_, int32_t seqs_)
      : offs(offs_), tokens(tokens_), seqs(seqs_), s(0), end(tokens_), edge(0), lo(0) {
    // every search starts at the first window: its read needs no token
    if (offs) edge = window(0, 1);
  }
  __device__ __forceinline__ int32_t window(int32_t first, int32_t step) const {
    const int64_t i = first + (int64_t)lane_id() * step;
    return i <= seqs ? (int32_t)seq_edge(offs, tokens, (int32_t)i) : INT32_MAX;
  }
  __device__ __forceinline__ int64_t boundary(int32_t i) const {
    return i - lo < kWave ? __builtin_amdgcn_readlane(edge, i - lo) : seq_edge(offs, tokens, i);
  }
  __device__ __forceinline__ void find(int64_t t) {
    if (!offs) return;  // one sequence of all tokens
    int32_t n = seqs;
    if (n >= kWave) {
      for (int32_t step = 0; n > 1;) {
        step = (n + kWave - 1) / kWave;
        edge = window(lo, step);
        const int hits = __popcll(__ballot(lane_id() * step < n && edge <= t));
        if (hits == 0) break;
        lo += (hits - 1) * step;
        n = min(step, n - (hits - 1) * step);
      }
      edge = window(lo, 1);
    }
    const int hits = __popcll(__ballot(lane_id() < n && edge <= t));
    s = lo + hits - 1;
    end = boundary(s + 1);
  }
  // Moves to the next sequence.
  __device__ __forceinline__ void next() {
    ++s;
    end = boundary(s + 1);
  }
  __device__ __forceinline__ bool inside(int64_t t) const { return t < end && s >= 0; }
};

// Logits lane, lane + 64, ... of a token; NaN as -inf (the larger of the two
// that is a number), like those behind the last expert.
template <int PER>
__device__ __forceinline__ void load_logits(const float* row, int E, float (&x)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {  // no branches: the reads go out together
    const int e = lane_id() + i * kWave;
    const float v = fmaxf(row[e < E ? e : E - 1], -INFINITY);
    x[i] = e < E ? v : -INFINITY;
  }
}
template <int PER>
__device__ __forceinline__ void store_row(float* row, int E, const float (&g)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane_id() + i * kWave;
    if (e < E) row[e] = g[i];
  }
}

// Tokens a wave takes at once: their reductions and reads overlap, and their
// selections fit the wave, slot j of token b in lane 16 b + j.
template <int PER>
constexpr int batch_of() { return PER <= 8 ? 4 : 2; }
static_assert(kMaxTopK <= 16, "a token's selections fit 16 lanes");

// exp(x - m) in place of the logits x of B tokens, their sums and largest
// logits.  A token without a logit above -inf gets zeros and sum 0.  The hardware's
// exp2 of a rounded product: off by at most (3 |x - m| + 4) 2^-24 relative, which
// the largest terms feel least (losses and gradients of 4096 x 256 and 16384 x 384:
// within 1.2e-7 and 2e-7 of their largest, like float32 exp and log).
template <int PER, int B>
__device__ __forceinline__ void exponentials(float (&x)[B][PER], float (&m)[B], float (&sum)[B]) {
#pragma unroll
  for (int b = 0; b < B; ++b) {
    m[b] = x[b][0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m[b] = fmaxf(m[b], x[b][i]);
  }
#pragma unroll
  for (int b = 0; b < B; ++b) m[b] = __ockl_wfred_max_f32(m[b]);
#pragma unroll
  for (int b = 0; b < B; ++b) {
    sum[b] = 0.0f;
    const float base = m[b] == -INFINITY ? 0.0f : m[b];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      x[b][i] = __expf(x[b][i] - base);
      sum[b] += x[b][i];
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) sum[b] = __ockl_wfred_add_f32(sum[b]);
}

// Mask bits of the tokens [t0, t1), at most 64 (bit i: token t0 + i counts).
__device__ __forceinline__ uint64_t mask_bits(const uint8_t* mask, int64_t t0, int64_t t1) {
  const int64_t t = t0 + lane_id();
  return __ballot(t < t1 && (!mask || mask[t] != 0));
}

// Balance and z of a batch from one sequence's sums, for the thread of expert
// e (n tokens, a and c its probability sum and selections).
__device__ __forceinline__ float balance_term(const RouterLossParams& p, int32_t s, int e, int32_t n, float a,
                                              int32_t c) {
  const float per = 1.0f / (float)(n > 0 ? n : 1), mean = a * per;
  p.counts[(int64_t)s * p.experts + e] = c;
  p.mean_probs[(int64_t)s * p.experts + e] = mean;
  return (float)c * ((float)p.experts * per / (float)p.top_k) * mean;
}

// Measured: 16 tokens 4.6 us (SINGLE); 4096 x 256 experts 7.6 us; 16384 x 384 in
// 37 sequences 12 us (25 MB of logits, 2.1 TB/s: half of its time is a wave's
// chain from the first read to the last reduction).
//
// Sums over runs of kLossRun tokens, one wave each, a batch of tokens at a
// time (the chain of a token's reductions is a microsecond long): probabilities
// in registers, selections in LDS counters.  A wave writes what it has when
// its sequence ends, into slot (run + sequence): along the tokens one of the
// two grows with every slot, so no two share one.  Where a whole block lies in
// one sequence its waves' sums are joined first, and only the first run's slot
// is written.  SINGLE: one block holds the batch and one sequence all of it,
// and the block writes the results itself.
template <int PER, bool SINGLE>
__global__ __launch_bounds__(kLossWaves* kWave) void k_loss_part(RouterLossParams p) {
  constexpr int B = batch_of<PER>();
  __shared__ int32_t hist[kLossWaves][PER * kWave];
  __shared__ float join[kLossWaves][PER * kWave];
  __shared__ float join_z[kLossWaves];
  __shared__ int32_t join_n[kLossWaves];
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int E = p.experts, k = p.top_k;
  const int64_t T = p.tokens;
  const int64_t block0 = (int64_t)blockIdx.x * kLossBlock;
  const int64_t block1 = block0 + kLossBlock < T ? block0 + kLossBlock : T;
  if (!SINGLE && blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0;
  const int64_t words = slot_words(E);

  const int64_t run = (int64_t)blockIdx.x * kLossWaves + w;
  const int64_t t0 = run * kLossRun;
  const int64_t t1 = t0 + kLossRun < block1 ? t0 + kLossRun : block1;
  // the first batch's reads run under the search for its sequence
  float nx[B][PER];
  int32_t nid = -1;
  const auto load = [&](int64_t t) {
#pragma unroll
    for (int b = 0; b < B; ++b)  // a batch's last tokens repeat its first, and do not count
      load_logits<PER>(p.logits + (t + b < t1 ? t + b : t) * E, E, nx[b]);
    const int64_t mine = t + lane / 16;
    nid = mine < t1 && lane / 16 < B && lane % 16 < k ? p.ids[mine * k + lane % 16] : -1;
  };
  if (t0 < t1) load(t0);

  SeqCursor seq(p.seq_offsets, T, p.seqs);
  seq.find(block0);
  const int32_t bs = seq.s;
  const bool whole = SINGLE || (bs >= 0 && seq.end >= block1);
  float acc[PER];
  float z = 0.0f;
  int32_t n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    acc[i] = 0.0f;
    hist[w][lane + i * kWave] = 0;
  }
  uint64_t on = mask_bits(p.mask, t0, t1);

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
    if (!whole || SINGLE) {
      seq.lo = 0;
      if (p.seqs >= kWave) seq.edge = seq.window(0, 1);
      seq.find(t0);
    }
    bool open = false;  // tokens of sequence s seen
    for (int64_t t = t0; t < t1; t += B) {
      float x[B][PER], m[B], sum[B];
      const int32_t id = nid;
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < PER; ++i) x[b][i] = nx[b][i];
      if (t + B < t1) load(t + B);  // under this batch's arithmetic
      exponentials<PER, B>(x, m, sum);
      const auto token = [&](int b) {
        ++n;
        if (m[b] == -INFINITY) return;
        const float inv = 1.0f / sum[b];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += x[b][i] * inv;
        const float lse = m[b] + __logf(sum[b]);
        z += lse * lse;
      };
      const uint32_t bits = (uint32_t)(on >> (t - t0));
      if (seq.inside(t) && t + B <= seq.end && t + B <= t1) {  // the batch lies in the sequence
        open = true;
        if ((bits >> lane / 16 & 1) && (uint32_t)id < (uint32_t)E) atomicAdd(&hist[w][id], 1);
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (bits >> b & 1) token(b);
        continue;
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (t + b >= t1) break;
        while (t + b >= seq.end && seq.s + 1 < p.seqs) {
          if (open) flush(seq.s);
          open = false;
          seq.next();
        }
        if (!seq.inside(t + b)) continue;  // before the first sequence or behind the last
        open = true;
        if (!(bits >> b & 1)) continue;
        if (lane / 16 == b && (uint32_t)id < (uint32_t)E) atomicAdd(&hist[w][id], 1);
        token(b);
      }
    }
    if (!whole && open) flush(seq.s);
  }
  if (!whole) return;

#pragma unroll
  for (int i = 0; i < PER; ++i) join[w][lane + i * kWave] = acc[i];
  if (lane == 0) {
    join_z[w] = z;
    join_n[w] = n;
  }
  __syncthreads();
  z = 0.0f;
  n = 0;
#pragma unroll
  for (int i = 0; i < kLossWaves; ++i) {
    z += join_z[i];
    n += join_n[i];
  }
  float* slot = SINGLE ? nullptr : p.slots + ((int64_t)blockIdx.x * kLossWaves + bs) * words;
  float term = 0.0f;
  for (int e = threadIdx.x; e < E; e += kLossWaves * kWave) {
    float a = 0.0f;
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < kLossWaves; ++i) {
      a += join[i][e];
      c += hist[i][e];
    }
    if (SINGLE) {
      term += balance_term(p, 0, e, n, a, c);
    } else {
      slot[e] = a;
      reinterpret_cast<int32_t*>(slot)[E + e] = c;
    }
  }
  if (!SINGLE) {
    if (threadIdx.x == 0) {
      slot[2 * E] = z;
      reinterpret_cast<int32_t*>(slot)[2 * E + 1] = n;
    }
    return;
  }
  term = __ockl_wfred_add_f32(term);
  __syncthreads();  // join_z is read
  if (lane == 0) join_z[w] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    term = 0.0f;
#pragma unroll
    for (int i = 0; i < kLossWaves; ++i) term += join_z[i];
    p.losses[0] = term;
    p.losses[1] = z / (float)(n > 0 ? n : 1);
    p.seq_tokens[0] = p.seq_tokens[1] = n;
    p.seq_tokens[2] = n > 0;
  }
}

// Values that a block of the same launch reads after the counter: stored and
// loaded at the level all XCDs share (their L2s do not see each other's lines),
// which spares the write-back of the whole L2 that a release fence is.
template <typename V>
__device__ __forceinline__ void put_shared(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V get_shared(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// 6.0 us for 4096 tokens and 256 experts, 7.2 for 16384, 384 and 37 sequences:
// latency (boundaries, slots, the joins in LDS, the counter).
//
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
  // slots of the sequence in order: a whole block's, or those of its runs; N at
  // a time, their reads in flight together
  const auto take = [&](auto count, const int64_t (&run)[decltype(count)::value], int have) {
    constexpr int N = decltype(count)::value;
    float va[N], vz[N];
    int32_t vc[N], vn[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float* slot = p.slots + (run[i] + s) * words;
      const bool in = i < have;
      va[i] = in && e < E ? slot[e] : 0.0f;
      vc[i] = in && e < E ? reinterpret_cast<const int32_t*>(slot)[E + e] : 0;
      vz[i] = in ? slot[2 * E] : 0.0f;
      vn[i] = in ? reinterpret_cast<const int32_t*>(slot)[2 * E + 1] : 0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a += va[i];
      c += vc[i];
      z += vz[i];
      n += vn[i];
    }
  };
  if (b < end) {
    const int64_t c0 = b / kLossBlock, c1 = (end - 1) / kLossBlock;
    const auto inside = [&](int64_t blk) {  // the block lies in the sequence
      const int64_t t1 = blk * kLossBlock + kLossBlock;
      return b <= blk * kLossBlock && (t1 < T ? t1 : T) <= end;
    };
    // the blocks at either end, where others share them: the sequence's runs
    for (int side = 0; side < 2; ++side) {
      const int64_t blk = side ? c1 : c0;
      if (inside(blk) || (side && c0 == c1) || w != side) continue;
      const int64_t lo = b > blk * kLossBlock ? b : blk * kLossBlock;
      const int64_t hi = end < (blk + 1) * kLossBlock ? end : (blk + 1) * kLossBlock;
      const int64_t r0 = lo / kLossRun;
      int64_t run[kLossWaves];
#pragma unroll
      for (int i = 0; i < kLossWaves; ++i) run[i] = r0 + i;
      take(std::integral_constant<int, kLossWaves>(), run, (int)((hi - 1) / kLossRun - r0 + 1));
    }
    constexpr int N = 4;
    const int64_t f0 = inside(c0) ? c0 : c0 + 1, f1 = inside(c1) ? c1 : c1 - 1;
    for (int64_t blk = f0 + w; blk <= f1; blk += N * kSumWaves) {
      int64_t run[N];
      int have = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        run[i] = (blk + i * kSumWaves) * kLossWaves;
        have += blk + i * kSumWaves <= f1;
      }
      take(std::integral_constant<int, N>(), run, have);
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
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) {
      a += jp[i][lane];
      c += jc[i][lane];
      z += jz[i];
      n += jn[i];
    }
    const float term = __ockl_wfred_add_f32(e < E ? balance_term(p, s, e, n, a, c) : 0.0f);
    if (lane == 0) {
      put_shared(p.seq_part + (int64_t)s * gridDim.x + blockIdx.x, term);
      if (blockIdx.x == 0) {
        put_shared(p.seq_part + (int64_t)p.seqs * gridDim.x + s, z);
        put_shared(p.seq_tokens + s, n);
      }
      // the parts above have reached memory before the count says so
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
      __builtin_amdgcn_s_waitcnt(0);
      const int32_t done = __hip_atomic_fetch_add(p.counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = done == (int32_t)(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  // every block has written its part: a thread takes every 1024th, in order
  float bal = 0.0f, zs = 0.0f;
  int32_t total = 0, live = 0;
  for (int64_t i = threadIdx.x; i < (int64_t)p.seqs * gridDim.x; i += kSumWaves * kWave) bal += get_shared(p.seq_part + i);
  for (int32_t i = threadIdx.x; i < p.seqs; i += kSumWaves * kWave) {
    zs += get_shared(p.seq_part + (int64_t)p.seqs * gridDim.x + i);
    const int32_t m = get_shared(p.seq_tokens + i);
    total += m;
    live += m > 0;
  }
  bal = __ockl_wfred_add_f32(bal);
  zs = __ockl_wfred_add_f32(zs);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    total += __shfl_xor(total, o);
    live += __shfl_xor(live, o);
  }
  if (lane == 0) {  // the arrays were last read before the barrier above
    jp[w][0] = bal;
    jz[w] = zs;
    jn[w] = total;
    jc[w][0] = live;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bal = zs = 0.0f;
    total = live = 0;
#pragma unroll
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

template <bool SINGLE>
static void launch_part(const RouterLossParams& p, hipStream_t st) {
  const unsigned blocks = (unsigned)std::max<int64_t>(1, (p.tokens + kLossBlock - 1) / kLossBlock);
  const dim3 block(kLossWaves * kWave);
  switch (per_lane(p.experts)) {
    case 1: k_loss_part<1, SINGLE><<<blocks, block, 0, st>>>(p); break;
    case 2: k_loss_part<2, SINGLE><<<blocks, block, 0, st>>>(p); break;
    case 4: k_loss_part<4, SINGLE><<<blocks, block, 0, st>>>(p); break;
    case 6: k_loss_part<6, SINGLE><<<blocks, block, 0, st>>>(p); break;
    case 8: k_loss_part<8, SINGLE><<<blocks, block, 0, st>>>(p); break;
    default: k_loss_part<16, SINGLE><<<blocks, block, 0, st>>>(p); break;
  }
}

hipError_t launch_router_loss(const RouterLossParams& p, hipStream_t st) {
  if (p.tokens <= kLossBlock && p.seqs == 1) {
    launch_part<true>(p, st);
    return hipGetLastError();
  }
  launch_part<false>(p, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((p.experts + kWave - 1) / kWave), (unsigned)p.seqs);
  k_loss_sum<<<grid, kSumWaves * kWave, 0, st>>>(p);
  return hipGetLastError();
}

// Sums over rows of 16 lanes, in every lane of the row.
template <int N>
__device__ __forceinline__ int32_t row_ror(int32_t v) {
  return __builtin_amdgcn_update_dpp(v, v, 0x120 + N, 0xF, 0xF, false);
}
template <int N>
__device__ __forceinline__ float row_ror(float v) {
  return __builtin_bit_cast(float, row_ror<N>(__builtin_bit_cast(int32_t, v)));
}
__device__ __forceinline__ float row_sum(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}
// v of the lane N places before in the row where it holds this lane's key, else
// 0; first: cleared where that lane stands before this one in the row.
template <int N>
__device__ __forceinline__ float row_other(float v, int32_t key, bool& first) {
  // both moves with all lanes on: a lane that is off gives nothing
  const float other = row_ror<N>(v);
  const bool same = row_ror<N>(key) == key;
  if (same && N <= lane_id() % 16) first = false;
  return same ? other : 0.0f;
}
// In the first lane of the row that holds a key (first true): v summed over all
// lanes that hold it, in their order.  The values are added as they are rounded.
template <int... N>
__device__ __forceinline__ float row_same(float v, int32_t key, bool& first, std::integer_sequence<int, N...>) {
#pragma clang fp contract(off)
  float r = v;
  first = true;
  ((r += row_other<15 - N>(v, key, first)), ...);  // the next lane's comes from 15 places before
  return r;
}

// One wave per batch of tokens.  Reads come in two rounds: what the token
// numbers give, then what the sequence and the selections give; with a wave for
// so few tokens their latency is most of its life.  A batch that enters
// another sequence reads that one's factors again.
// Measured: 64 tokens x 256 experts 6.0 us; 16384 x 384 16.2 us (51 MB read and
// written, 3.2 TB/s).
template <int PER>
__global__ __launch_bounds__(256) void k_router_grad(RouterGradParams p) {
  constexpr int B = batch_of<PER>();
  const int lane = lane_id();
  const int E = p.experts, k = p.top_k;
  const int64_t T = p.tokens;
  const int64_t t0 = ((int64_t)blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave) * B;
  const int64_t t1 = t0 + B < T ? t0 + B : T;
  if (t0 >= T) return;
  const bool losses = p.dlosses != nullptr, chosen = p.dweights != nullptr;
  SeqCursor seq(p.seq_offsets, T, p.seqs);
  // lane 16 b + j: selection j of token b (others repeat one of the batch)
  const int64_t slot_t = t0 + min((int64_t)(lane / 16), t1 - t0 - 1);
  const bool slot = slot_t == t0 + lane / 16 && lane % 16 < k;
  const int64_t slot_at = slot_t * k + min(lane % 16, k - 1);
  float wj = 0.0f, dj = 0.0f;
  int32_t id = p.ids[slot_at];
  if (chosen) {
    wj = p.weights[slot_at];
    dj = p.dweights[slot_at];
  }
  float x[B][PER], m[B], sum[B];
#pragma unroll
  for (int b = 0; b < B; ++b) load_logits<PER>(p.logits + (t0 + b < t1 ? t0 + b : t0) * E, E, x[b]);
  float gb = 0.0f, gz = 0.0f;
  if (losses) {
    const int32_t total = p.seq_tokens[p.seqs], live = p.seq_tokens[p.seqs + 1];
    gb = p.dlosses[0] / (float)(live > 0 ? live : 1);
    gz = 2.0f * p.dlosses[1] / (float)(total > 0 ? total : 1);
  }
  const uint64_t on = mask_bits(p.mask, t0, t1);
  id = slot && (uint32_t)id < (uint32_t)E ? id : -1;
  const int32_t at = id < 0 ? 0 : id;
  const float xj = fmaxf(p.logits[slot_t * E + at], -INFINITY);
  seq.find(t0);
  float f[PER], fj = 0.0f;
  auto factors = [&]() {  // g_b f / (S' n) of the cursor's sequence; fj: of the lane's selection
    const int32_t n = p.seq_tokens[seq.s];
    const int32_t* row = p.counts + (int64_t)seq.s * E;
    int32_t c[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = row[min(lane + i * kWave, E - 1)];
    const int32_t cj = row[at];
    const float per = 1.0f / (float)(n > 0 ? n : 1);
    const float scale = gb * per * ((float)E * per / (float)k);
#pragma unroll
    for (int i = 0; i < PER; ++i) f[i] = (float)c[i] * scale;
    fj = (float)cj * scale;
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = 0.0f;
  if (losses && seq.s >= 0) factors();
  // the selections' part: w (dw - sum w dw) of each, summed over a token's
  // selections of one expert (they differ, but for a caller's own ids), which its
  // first one stores
  float sel = 0.0f;
  bool first = true;
  if (chosen) {
    wj = slot ? wj : 0.0f;
    dj = slot ? dj : 0.0f;
    sel = row_same(wj * (dj - row_sum(wj * dj)), id, first, std::make_integer_sequence<int, 15>());
  }
  exponentials<PER, B>(x, m, sum);
  float inv[B], lz[B], dots[B];  // dots: sum of p f with the factors of the token's sequence
#pragma unroll
  for (int b = 0; b < B; ++b) {
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) d += x[b][i] * f[i];
    dots[b] = d;
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    inv[b] = 1.0f / sum[b];
    lz[b] = (m[b] + __logf(sum[b])) * gz;
    dots[b] = losses ? __ockl_wfred_add_f32(dots[b]) * inv[b] : 0.0f;
  }
  bool moved = false;
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int64_t t = t0 + b;
    if (t >= t1) break;
    bool next = false;
    while (t >= seq.end && seq.s + 1 < p.seqs) {
      seq.next();
      next = true;
    }
    if (!seq.inside(t)) continue;  // in no sequence: left as it is
    moved |= next;
    if (next && losses) factors();
    float* out = p.dlogits + t * E;
    const bool live_row = (on >> b & 1) && m[b] != -INFINITY;
    float g[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) g[i] = 0.0f;
    if (live_row && losses) {
      if (moved) {
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) d += x[b][i] * f[i];
        dots[b] = __ockl_wfred_add_f32(d) * inv[b];
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) g[i] = x[b][i] * inv[b] * ((f[i] - dots[b]) + lz[b]);
    }
    store_row<PER>(out, E, g);
    // the selected experts again, with both parts (the wave's stores to an
    // address keep their order)
    if (live_row && chosen && lane / 16 == b && id >= 0 && first)
      out[id] = (losses ? __expf(xj - m[b]) * inv[b] * ((fj - dots[b]) + lz[b]) : 0.0f) + sel;
  }
}

template <int PER>
static void launch_grad(const RouterGradParams& p, hipStream_t st) {
  const int64_t per_block = batch_of<PER>() * 4;
  k_router_grad<PER><<<(unsigned)((p.tokens + per_block - 1) / per_block), 256, 0, st>>>(p);
}
hipError_t launch_router_grad(const RouterGradParams& p, hipStream_t st) {
  if (p.tokens == 0) return hipSuccess;
  switch (per_lane(p.experts)) {
    case 1: launch_grad<1>(p, st); break;
    case 2: launch_grad<2>(p, st); break;
    case 4: launch_grad<4>(p, st); break;
    case 6: launch_grad<6>(p, st); break;
    case 8: launch_grad<8>(p, st); break;
    default: launch_grad<16>(p, st); break;
  }
  return hipGetLastError();
}

}  // namespace moe
