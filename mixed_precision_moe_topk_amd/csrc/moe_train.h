// Launch parameters of the training and adapter operators beside the layer:
// the router's losses and gradients, the gradient of the weighted sum, and
// low-rank adapters.
#pragma once

#include "moe_common.h"

namespace moe {

// ---------------------------------------------------------------- router
constexpr int kLossRun = 8;     // consecutive tokens one wave sums
constexpr int kLossWaves = 8;   // waves (runs) per block of the loss kernel
constexpr int kLossBlock = kLossRun * kLossWaves;

struct RouterLossParams {
  const float* logits;         // [T, E]
  const int32_t* ids;          // [T, k]
  const int32_t* seq_offsets;  // [S + 1], or null: one sequence of all tokens
  const uint8_t* mask;         // [T], or null: every token counts
  int64_t tokens;
  int32_t experts;
  int32_t top_k;
  int32_t seqs;
  // one slot per (run of tokens, sequence): probability sums [E], selections
  // [E], the sum of squared log-sum-exps and the tokens (see slot_words)
  float* slots;
  float* seq_part;   // [S, ceil(E/64)] balance terms, then [S] z sums
  int32_t* counter;  // [1] blocks of the second kernel that have finished
  float* losses;       // [2]
  int32_t* counts;     // [S, E]
  float* mean_probs;   // [S, E]
  int32_t* seq_tokens; // [S + 2]
};
// Words of one slot: E probability sums, E selections, z sum, token count.
__host__ __device__ constexpr int64_t slot_words(int64_t experts) { return 2 * experts + 2; }

struct RouterGradParams {
  const float* logits;
  const int32_t* ids;
  const float* weights;    // [T, k], with dweights
  const float* dweights;   // [T, k] or null
  const int32_t* seq_offsets;
  const uint8_t* mask;
  const int32_t* counts;      // [S, E], with dlosses
  const int32_t* seq_tokens;  // [S + 2], with dlosses
  const float* dlosses;       // [2] or null
  int64_t tokens;
  int32_t experts;
  int32_t top_k;
  int32_t seqs;
  float* dlogits;  // [T, E]
};

hipError_t launch_router_loss(const RouterLossParams& p, hipStream_t st);
hipError_t launch_router_grad(const RouterGradParams& p, hipStream_t st);

// ---------------------------------------------------------------- weighted sum
// dweights [T, k], dy2 [T*k, H] (bf16 bits or float32; null: not wanted).
unsigned finalize_grad_threads(int32_t H);  // threads of a token's block
hipError_t launch_finalize_grad(const uint16_t* dout, const float* weights, const float* y2,
                                const int32_t* slot_row, int64_t T, int32_t k, int32_t H,
                                float* dweights, void* dy2, bool dy2_f32, hipStream_t st);

// ---------------------------------------------------------------- adapters
constexpr int kMaxAdapters = 1023;   // one more group holds the tokens without one
constexpr int kMaxRank = 128;
constexpr int kAdapterTile = 64;     // rows of a tile
constexpr int kAdapterPad = 16;      // an adapter's rows start at a multiple of this
constexpr int kPlanChunk = 64;       // tokens per wave of the plan kernels
constexpr int kPlanGroup = 1024;     // tokens per block of the plan kernels
constexpr int kPlanOne = 8 * kPlanGroup;  // tokens planned in one launch

// Plan of a batch: its tokens grouped by adapter.  Int32 words:
//   head [2]: tiles, and how many of them, the first, hold tokens with an adapter
//   first [L + 2]: first row of each group (multiples of kAdapterPad); group L
//                  holds the tokens without an adapter
//   rows [max_rows]: token of each row, -1 in the padding behind a group
//   tiles [max_tiles][4]: group, first row, rows, unused
//   counts [nblocks, L + 1]: scratch of the plan kernels
struct PlanLayout {
  int64_t first, rows, tiles, counts, total;  // offsets in words
  int64_t max_rows, max_tiles, nblocks;
  PlanLayout(int32_t adapters, int64_t tokens) {
    const int64_t g = adapters + 1, used = tokens < g ? tokens : g;
    max_rows = (tokens + used * (kAdapterPad - 1) + 31) / 32 * 32;
    max_tiles = tokens / kAdapterTile + used;
    nblocks = (tokens + kPlanGroup - 1) / kPlanGroup;
    const auto up = [](int64_t w) { return (w + 63) / 64 * 64; };
    first = 64;
    rows = first + up(g + 1);
    tiles = rows + up(max_rows);
    counts = tiles + up(4 * max_tiles);
    total = counts + up(nblocks * g);
  }
};

// Whether a plan of these sizes can hold the tile: a buffer that was never
// planned, or for another batch, may hold any words.
__host__ __device__ inline bool plan_tile_fits(const Tile& t, int32_t adapters, int64_t max_rows) {
  return t.expert >= 0 && t.expert <= adapters && t.nrows >= 1 && t.nrows <= kAdapterTile &&
         t.row0 >= 0 && t.row0 % kAdapterPad == 0 &&
         (int64_t)t.row0 + (t.nrows + kAdapterPad - 1) / kAdapterPad * kAdapterPad <= max_rows;
}

struct PlanParams {
  const int32_t* adapter_ids;  // [T]
  int64_t tokens;
  int32_t adapters;
  int32_t* plan;
};
hipError_t launch_adapter_plan(const PlanParams& p, const PlanLayout& l, hipStream_t st);

struct PlanView {
  const int32_t* head;
  const int32_t* first;
  const int32_t* rows;
  const Tile* tiles;
  int64_t tokens, max_rows, max_tiles;
  int32_t adapters;
};

// Scaled low-rank rows as operands of expand (frag) and of outer (saved), in
// bf16 parts (layouts in moe_adapter.hip); either may be null.
struct LowRows {
  uint16_t* frag;
  uint16_t* saved;
  int32_t parts;  // of frag: 2, or 3 for float32 results
  int32_t rank_pad, rank_pad32;
  int64_t max_rows;
};
constexpr int kShrinkK = 128;       // elements of K in a unit of shrink's work
constexpr int kShrinkBlocks = 512;  // blocks of shrink
constexpr int kMaxSlots = 8;        // blocks that may share a tile
// How shrink cuts its work: units of a tile, and the fewest units of a block.
struct ShrinkShape {
  int32_t units, min_run;
};
// X[token(row)] . W[adapter]^T in float32, unscaled: part[slot][row][rank_pad],
// a slot for each block that takes part in the row's tile.
struct ShrinkParams {
  PlanView plan;
  ShrinkShape shape;
  const void* x;
  int64_t x_stride;    // elements
  const uint16_t* w;   // [L, R, K] bf16
  int32_t rank, rank_pad, K;
  float* part;
};
// The scaled rows from the slots' sums.
struct JoinParams {
  PlanView plan;
  ShrinkShape shape;
  const float* part;
  const float* scale;
  int32_t rank_pad;
  LowRows low;
};
// out[t] = base[t] + row(t) . W[adapter], the rows from frag or (null) part.
struct ExpandParams {
  PlanView plan;
  ShrinkShape shape;
  const uint16_t* frag;
  const float* part;
  const float* scale;  // [L]
  const uint16_t* w;   // [L, R, N] bf16
  int32_t rank, rank_pad, rank_pad32, N;
  const void* base;    // or null: 0
  int64_t base_stride;
  void* out;
  int64_t out_stride;
  uint16_t* saved;  // with part: where the rows go as operands of outer, or null
  int32_t col_blocks, row_blocks;  // of a tile, set by the launcher
};
// grad[adapter][r][c] = sum over the adapter's rows of saved[r][row] * X[token(row)][c]
struct OuterSide {
  const uint16_t* saved;
  const void* x;
  int64_t x_stride;
  int32_t C;
  float* grad;
  int64_t part_at;  // columns before its own in a slot of the partial sums
};
struct OuterParams {
  PlanView plan;
  OuterSide x, dout;  // dout bf16 or float32
  int32_t rank, rank_pad;
  int64_t chunk;      // most rows of a segment (a multiple of 64)
  int32_t chunks;     // chunks of all rows
  float* part;        // [2 chunks][rank (x.C + dout.C)]
  int32_t cols0, cols;  // column blocks of x and of both, set by the launcher
};
hipError_t launch_adapter_shrink(const ShrinkParams& p, bool x_f32, hipStream_t st);
hipError_t launch_adapter_expand(const ExpandParams& p, bool out_f32, hipStream_t st);
hipError_t launch_adapter_join(const JoinParams& p, hipStream_t st);
hipError_t launch_adapter_outer(const OuterParams& p, bool dout_f32, hipStream_t st);

}  // namespace moe
