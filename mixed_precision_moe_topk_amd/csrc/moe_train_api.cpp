// Host side of the training and adapter entry points of include/moe.h:
// argument checks, size queries and launch sequences.  As in the run calls
// every check comes before any launch, and nothing allocates or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe.h"
#include "moe_host.h"
#include "moe_train.h"

namespace {

using moe::ceil_div;
using moe::is_aligned16;
using moe::set_error;
using moe::set_errorf;

constexpr int64_t kMaxTokens = (int64_t)1 << 26;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

moe_status check_pointers(std::initializer_list<const void*> ps) {
  for (const void* p : ps) {
    if (!p) return set_error(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (!is_aligned16(p)) return set_error(MOE_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  }
  return MOE_OK;
}
// A pointer that may be null.
moe_status check_optional(const void* p) {
  return is_aligned16(p) ? MOE_OK : set_error(MOE_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
}

moe_status check_room(size_t have, size_t need, const char* what) {
  if (have < need)
    return set_errorf(MOE_ERR_WORKSPACE, "%s %zu bytes < %zu required", what, have, need);
  return MOE_OK;
}

// ---------------------------------------------------------------- router
moe_status check_seqs(const int32_t* seq_offsets, int32_t num_seqs) {
  if (num_seqs < 1 || num_seqs > 65535)
    return set_errorf(MOE_ERR_INVALID_ARG, "num_seqs %d outside [1, 65535]", num_seqs);
  if (!seq_offsets && num_seqs != 1)
    return set_error(MOE_ERR_INVALID_ARG, "num_seqs must be 1 without seq_offsets");
  return MOE_OK;
}

struct LossLayout {
  size_t slots, seq_part, counter, total;
  LossLayout(int64_t experts, int64_t tokens, int64_t seqs) {
    const int64_t runs = std::max<int64_t>(1, ceil_div(tokens, moe::kLossBlock)) * moe::kLossWaves;
    slots = 0;
    seq_part = align256((size_t)((runs + seqs) * moe::slot_words(experts) * 4));
    counter = seq_part + align256((size_t)(seqs * (ceil_div(experts, moe::kWave) + 1) * 4));
    total = counter + 256;
  }
};

// ---------------------------------------------------------------- adapters
moe_status check_adapter_tokens(int32_t num_adapters, int64_t num_tokens) {
  if (num_adapters < 1 || num_adapters > moe::kMaxAdapters)
    return set_errorf(MOE_ERR_INVALID_ARG, "num_adapters %d outside [1, %d]", num_adapters,
                      moe::kMaxAdapters);
  if (num_tokens < 0 || num_tokens > kMaxTokens)
    return set_errorf(MOE_ERR_INVALID_ARG, "num_tokens %lld outside [0, 2^26]",
                      (long long)num_tokens);
  return MOE_OK;
}

moe_status check_adapter(const moe_adapter_dims* d, int64_t num_tokens) {
  if (!d) return set_error(MOE_ERR_INVALID_ARG, "dims is null");
  MOE_RETURN_IF(check_adapter_tokens(d->num_adapters, num_tokens));
  if (d->rank < 1 || d->rank > moe::kMaxRank)
    return set_errorf(MOE_ERR_INVALID_ARG, "rank %d outside [1, %d]", d->rank, moe::kMaxRank);
  for (const int32_t n : {d->in_features, d->out_features})
    if (n < 8 || n % 8 != 0 || n > (1 << 18))
      return set_errorf(MOE_ERR_INVALID_ARG, "%d features: a multiple of 8 in [8, 2^18] is needed", n);
  if (d->out_type != MOE_T_BF16 && d->out_type != MOE_T_F32)
    return set_errorf(MOE_ERR_INVALID_ARG, "unknown output type %d", d->out_type);
  return MOE_OK;
}

// Strides in elements; every row starts 16-byte aligned.
moe_status check_stride(int64_t stride, int64_t features) {
  if (stride < features || stride % 8 != 0 || stride > ((int64_t)1 << 32))
    return set_errorf(MOE_ERR_INVALID_ARG,
                      "row stride %lld: a multiple of 8 of at least %lld is needed",
                      (long long)stride, (long long)features);
  return MOE_OK;
}

int32_t rank_pad(const moe_adapter_dims* d) { return (d->rank + 15) / 16 * 16; }

// How shrink cuts a contraction over `features`: a block takes at least a
// seventh of a tile, so that at most 8 blocks share one; from 32768 tokens on a
// whole tile, which keeps the sums' room at two rows a token.
moe::ShrinkShape shrink_shape(int64_t tokens, int64_t features) {
  const int32_t units = (int32_t)ceil_div(features, moe::kShrinkK);
  return {units, tokens >= 32768 ? units : (int32_t)ceil_div(units, 7)};
}
int32_t max_slots(const moe::ShrinkShape& s) { return (s.units - 1) / s.min_run + 2; }

// Up to so many sums (tokens x ranks) expand adds up the parts for itself: every
// wave of 128 columns reads them again, which costs less than the join's launch
// while they are few.  7168 x 7168 features, us a call without and with the join:
// 400 tokens, rank 16: 22.0, 24.3; 800, 16: 27.5, 27.2; 400, 64: 31.3, 30.8; 400,
// 128: 62, 51.  1024 x 2048, 400, 16: 16.8, 20.3.
constexpr int64_t kFewSums = 16384;

// Workspace: the sums of the larger contraction, expand's operands, the backward
// pass's v as outer's operands, and the factors' gradients of the segments.
struct AdapterLayout {
  moe::PlanLayout plan;
  int32_t rp, rp32;
  moe::ShrinkShape shape_x, shape_d;
  size_t part_bytes, frag_bytes, saved_bytes, outer_bytes;
  int64_t chunk;  // rows of a segment of the factors' gradients
  int32_t chunks;
  AdapterLayout(const moe_adapter_dims* d, int64_t tokens)
      : plan(d->num_adapters, tokens), rp(rank_pad(d)), rp32((d->rank + 31) / 32 * 32) {
    shape_x = shrink_shape(tokens, d->in_features);
    shape_d = shrink_shape(tokens, d->out_features);
    part_bytes = align256((size_t)std::max(max_slots(shape_x), max_slots(shape_d)) * plan.max_rows * rp * 4);
    frag_bytes = align256((size_t)plan.max_rows * rp32 * 6);
    saved_bytes = align256((size_t)plan.max_rows * rp * 6);
    // segments of all adapters for as many blocks as run at once (registers
    // allow 3 or 2 a CU by the rank), 256 rows a segment at least: rows are
    // cut into what is left when every adapter has one, or into half as many
    const int64_t wide = rp <= 32 ? 256 : 128;  // columns of a block
    const int64_t cols = ceil_div(d->in_features, wide) +
                         ceil_div(d->out_features, d->out_type == MOE_T_F32 ? 64 : wide);
    const int64_t segments = std::max<int64_t>(1, (rp <= 64 ? 768 : 512) / cols);
    const int64_t cuts = std::max({(int64_t)1, segments / 2, segments - d->num_adapters});
    chunk = std::max<int64_t>(256, ceil_div(ceil_div(plan.max_rows, cuts), 64) * 64);
    // (one where no adapter can have more rows than a segment)
    chunks = tokens <= chunk ? 1 : (int32_t)ceil_div(plan.max_rows, chunk);
    outer_bytes = chunks > 1 ? align256((size_t)chunks * 2 * d->rank *
                                        ((size_t)d->in_features + d->out_features) * 4) : 0;
  }
  size_t outer_at() const { return part_bytes + frag_bytes + saved_bytes; }
  size_t workspace() const { return outer_at() + outer_bytes; }
};

moe::PlanView plan_view(const void* plan, const moe::PlanLayout& l, int32_t adapters,
                        int64_t tokens) {
  const int32_t* p = static_cast<const int32_t*>(plan);
  moe::PlanView v;
  v.head = p;
  v.first = p + l.first;
  v.rows = p + l.rows;
  v.tiles = reinterpret_cast<const moe::Tile*>(p + l.tiles);
  v.tokens = tokens;
  v.max_rows = l.max_rows;
  v.max_tiles = l.max_tiles;
  v.adapters = adapters;
  return v;
}

// One product with a factor on each side: shrink of x with w, then (out not
// null) expand with w2; `saved` (or null) takes the low-rank rows.
struct Product {
  const void* x;
  int64_t x_stride;
  const void* w;
  int32_t features;
  moe::ShrinkShape shape;
  bool x_f32;
  const void* w2;
  int32_t features2;
  const void* base;
  int64_t base_stride;
  void* out;
  int64_t out_stride;
  bool out_f32;
  void* saved;
};

moe_status run_product(const Product& q, const moe::PlanView& v, const AdapterLayout& l,
                       int32_t rank, const float* scale, void* workspace, hipStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part = reinterpret_cast<float*>(ws);
  const bool few = v.tokens * l.rp <= kFewSums;  // expand takes the parts themselves
  moe::LowRows low;
  low.frag = few || !q.out ? nullptr : reinterpret_cast<uint16_t*>(ws + l.part_bytes);
  low.saved = static_cast<uint16_t*>(q.saved);
  low.parts = q.out_f32 ? 3 : 2;
  low.rank_pad = l.rp;
  low.rank_pad32 = l.rp32;
  low.max_rows = l.plan.max_rows;
  const moe::ShrinkParams s = {v, q.shape, q.x, q.x_stride, static_cast<const uint16_t*>(q.w),
                               rank, l.rp, q.features, part};
  MOE_RETURN_IF(moe::check_hip(moe::launch_adapter_shrink(s, q.x_f32, stream), "adapter shrink", stream));
  if (low.frag || (low.saved && !q.out)) {
    const moe::JoinParams j = {v, q.shape, part, scale, l.rp, low};
    MOE_RETURN_IF(moe::check_hip(moe::launch_adapter_join(j, stream), "adapter join", stream));
  }
  if (!q.out) return MOE_OK;
  const moe::ExpandParams e = {v, q.shape, low.frag, part, scale, static_cast<const uint16_t*>(q.w2),
                               rank, l.rp, l.rp32, q.features2, q.base, q.base_stride, q.out,
                               q.out_stride, few ? low.saved : nullptr, 0, 0};
  return moe::check_hip(moe::launch_adapter_expand(e, q.out_f32, stream), "adapter expand", stream);
}

}  // namespace

extern "C" {

moe_status moe_router_loss_query(const moe_dims* dims, int64_t num_tokens, int32_t num_seqs,
                                 size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(moe::check_layer(dims, num_tokens, 1));
  if (num_seqs < 1 || num_seqs > 65535)
    return set_errorf(MOE_ERR_INVALID_ARG, "num_seqs %d outside [1, 65535]", num_seqs);
  *bytes = LossLayout(dims->num_experts, num_tokens, num_seqs).total;
  return moe::set_ok();
}

moe_status moe_router_loss(const moe_dims* dims, const float* router_logits, const int32_t* ids,
                           int64_t num_tokens, int32_t top_k, const int32_t* seq_offsets,
                           int32_t num_seqs, const uint8_t* token_mask, float* losses,
                           int32_t* counts, float* mean_probs, int32_t* seq_tokens,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  MOE_RETURN_IF(moe::check_layer(dims, num_tokens, top_k));
  MOE_RETURN_IF(check_seqs(seq_offsets, num_seqs));
  MOE_RETURN_IF(check_pointers({losses, counts, mean_probs, seq_tokens, workspace}));
  if (num_tokens > 0) MOE_RETURN_IF(check_pointers({router_logits, ids}));
  MOE_RETURN_IF(check_optional(seq_offsets));
  MOE_RETURN_IF(check_optional(token_mask));
  const LossLayout l(dims->num_experts, num_tokens, num_seqs);
  MOE_RETURN_IF(check_room(workspace_bytes, l.total, "workspace"));
  MOE_RETURN_IF(moe::check_gfx950());
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  moe::RouterLossParams p;
  p.logits = router_logits;
  p.ids = ids;
  p.seq_offsets = seq_offsets;
  p.mask = token_mask;
  p.tokens = num_tokens;
  p.experts = dims->num_experts;
  p.top_k = top_k;
  p.seqs = num_seqs;
  p.slots = reinterpret_cast<float*>(ws + l.slots);
  p.seq_part = reinterpret_cast<float*>(ws + l.seq_part);
  p.counter = reinterpret_cast<int32_t*>(ws + l.counter);
  p.losses = losses;
  p.counts = counts;
  p.mean_probs = mean_probs;
  p.seq_tokens = seq_tokens;
  MOE_RETURN_IF(moe::check_hip(moe::launch_router_loss(p, stream), "router loss", stream));
  return moe::set_ok();
}

moe_status moe_router_backward(const moe_dims* dims, const float* router_logits,
                               const int32_t* ids, int64_t num_tokens, int32_t top_k,
                               const int32_t* seq_offsets, int32_t num_seqs,
                               const uint8_t* token_mask, const float* weights,
                               const float* dweights, const float* dlosses, const int32_t* counts,
                               const int32_t* seq_tokens, float* dlogits, hipStream_t stream) {
  MOE_RETURN_IF(moe::check_layer(dims, num_tokens, top_k));
  MOE_RETURN_IF(check_seqs(seq_offsets, num_seqs));
  if (num_tokens == 0) return moe::set_ok();
  if (!dweights && !dlosses)
    return set_error(MOE_ERR_INVALID_ARG, "dweights and dlosses are both null: no gradient");
  MOE_RETURN_IF(check_pointers({router_logits, ids, dlogits}));
  if (dweights) MOE_RETURN_IF(check_pointers({weights, dweights}));
  if (dlosses) MOE_RETURN_IF(check_pointers({dlosses, counts, seq_tokens}));
  MOE_RETURN_IF(check_optional(seq_offsets));
  MOE_RETURN_IF(check_optional(token_mask));
  MOE_RETURN_IF(moe::check_gfx950());
  moe::RouterGradParams p;
  p.logits = router_logits;
  p.ids = ids;
  p.weights = weights;
  p.dweights = dweights;
  p.seq_offsets = seq_offsets;
  p.mask = token_mask;
  p.counts = counts;
  p.seq_tokens = seq_tokens;
  p.dlosses = dlosses;
  p.tokens = num_tokens;
  p.experts = dims->num_experts;
  p.top_k = top_k;
  p.seqs = num_seqs;
  p.dlogits = dlogits;
  MOE_RETURN_IF(moe::check_hip(moe::launch_router_grad(p, stream), "router backward", stream));
  return moe::set_ok();
}

moe_status moe_finalize_backward(const moe_dims* dims, const void* dout, int64_t num_tokens,
                                 int32_t top_k, const float* weights, const float* y2,
                                 const int32_t* slot_row, float* dweights, void* dy2,
                                 int32_t dy2_type, hipStream_t stream) {
  MOE_RETURN_IF(moe::check_layer(dims, num_tokens, top_k));
  if (dy2_type != MOE_T_BF16 && dy2_type != MOE_T_F32)
    return set_errorf(MOE_ERR_INVALID_ARG, "unknown dy2 type %d", dy2_type);
  if (num_tokens == 0) return moe::set_ok();
  if (num_tokens * moe::finalize_grad_threads(dims->hidden) >= (int64_t)1 << 32)
    return set_errorf(MOE_ERR_INVALID_ARG, "num_tokens %lld with hidden %d: more than 2^32 threads",
                      (long long)num_tokens, dims->hidden);
  MOE_RETURN_IF(check_pointers({dout, weights, y2, slot_row, dweights}));
  MOE_RETURN_IF(check_optional(dy2));
  if (dy2 == y2 && dy2_type != MOE_T_F32)
    return set_error(MOE_ERR_INVALID_ARG, "only a float dy2 may be y2");
  MOE_RETURN_IF(moe::check_gfx950());
  MOE_RETURN_IF(moe::check_hip(
      moe::launch_finalize_grad(static_cast<const uint16_t*>(dout), weights, y2, slot_row,
                                num_tokens, top_k, dims->hidden, dweights, dy2,
                                dy2_type == MOE_T_F32, stream),
      "finalize backward", stream));
  return moe::set_ok();
}

moe_status moe_adapter_plan_query(int32_t num_adapters, int64_t num_tokens, size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(check_adapter_tokens(num_adapters, num_tokens));
  *bytes = (size_t)moe::PlanLayout(num_adapters, num_tokens).total * 4;
  return moe::set_ok();
}

moe_status moe_adapter_plan(int32_t num_adapters, const int32_t* adapter_ids, int64_t num_tokens,
                            void* plan, size_t plan_bytes, hipStream_t stream) {
  MOE_RETURN_IF(check_adapter_tokens(num_adapters, num_tokens));
  if (num_tokens == 0) return moe::set_ok();
  MOE_RETURN_IF(check_pointers({adapter_ids, plan}));
  const moe::PlanLayout l(num_adapters, num_tokens);
  MOE_RETURN_IF(check_room(plan_bytes, (size_t)l.total * 4, "plan"));
  MOE_RETURN_IF(moe::check_gfx950());
  moe::PlanParams p;
  p.adapter_ids = adapter_ids;
  p.tokens = num_tokens;
  p.adapters = num_adapters;
  p.plan = static_cast<int32_t*>(plan);
  MOE_RETURN_IF(moe::check_hip(moe::launch_adapter_plan(p, l, stream), "adapter plan", stream));
  return moe::set_ok();
}

moe_status moe_adapter_workspace_query(const moe_adapter_dims* dims, int64_t num_tokens,
                                       size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(check_adapter(dims, num_tokens));
  *bytes = AdapterLayout(dims, num_tokens).workspace();
  return moe::set_ok();
}

moe_status moe_adapter_saved_query(const moe_adapter_dims* dims, int64_t num_tokens,
                                   size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(check_adapter(dims, num_tokens));
  *bytes = AdapterLayout(dims, num_tokens).saved_bytes;
  return moe::set_ok();
}

moe_status moe_adapter_apply(const moe_adapter_dims* dims, const void* x, int64_t x_stride,
                             int64_t num_tokens, const void* plan, size_t plan_bytes,
                             const void* a, const void* b, const float* scale, const void* base,
                             int64_t base_stride, void* out, int64_t out_stride, void* saved,
                             size_t saved_bytes, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  MOE_RETURN_IF(check_adapter(dims, num_tokens));
  if (num_tokens == 0) return moe::set_ok();
  MOE_RETURN_IF(check_pointers({x, plan, a, b, scale, out, workspace}));
  MOE_RETURN_IF(check_optional(base));
  MOE_RETURN_IF(check_optional(saved));
  MOE_RETURN_IF(check_stride(x_stride, dims->in_features));
  MOE_RETURN_IF(check_stride(out_stride, dims->out_features));
  if (base) MOE_RETURN_IF(check_stride(base_stride, dims->out_features));
  if (base == out && base_stride != out_stride)
    return set_error(MOE_ERR_INVALID_ARG, "base is out with another row stride");
  const AdapterLayout l(dims, num_tokens);
  MOE_RETURN_IF(check_room(plan_bytes, (size_t)l.plan.total * 4, "plan"));
  MOE_RETURN_IF(check_room(workspace_bytes, l.workspace(), "workspace"));
  if (saved) MOE_RETURN_IF(check_room(saved_bytes, l.saved_bytes, "saved"));
  MOE_RETURN_IF(moe::check_gfx950());
  const moe::PlanView v = plan_view(plan, l.plan, dims->num_adapters, num_tokens);
  const Product q = {x, x_stride, a, dims->in_features, l.shape_x, false, b, dims->out_features,
                     base, base_stride, out, out_stride, dims->out_type == MOE_T_F32, saved};
  MOE_RETURN_IF(run_product(q, v, l, dims->rank, scale, workspace, stream));
  return moe::set_ok();
}

moe_status moe_adapter_backward(const moe_adapter_dims* dims, const void* dout,
                                int64_t dout_stride, const void* x, int64_t x_stride,
                                int64_t num_tokens, const void* plan, size_t plan_bytes,
                                const void* a, const void* b, const float* scale,
                                const void* saved, size_t saved_bytes, float* da, float* db,
                                const void* dx_base, int64_t dx_base_stride, void* dx,
                                int64_t dx_stride, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  MOE_RETURN_IF(check_adapter(dims, num_tokens));
  if ((da == nullptr) != (db == nullptr))
    return set_error(MOE_ERR_INVALID_ARG, "da and db are wanted together or not at all");
  // (dx of no tokens has no address)
  if (!da && !dx && num_tokens > 0)
    return set_error(MOE_ERR_INVALID_ARG, "neither dx nor da and db: no gradient");
  if (da) MOE_RETURN_IF(check_pointers({da, db}));
  MOE_RETURN_IF(check_optional(dx));
  MOE_RETURN_IF(check_optional(dx_base));
  if (num_tokens > 0) {
    MOE_RETURN_IF(check_pointers({dout, plan, a, b, scale, workspace}));
    if (da) MOE_RETURN_IF(check_pointers({x, saved}));
    MOE_RETURN_IF(check_stride(dout_stride, dims->out_features));
    if (da) MOE_RETURN_IF(check_stride(x_stride, dims->in_features));
    if (dx) MOE_RETURN_IF(check_stride(dx_stride, dims->in_features));
    if (dx && dx_base) MOE_RETURN_IF(check_stride(dx_base_stride, dims->in_features));
    if (dx && dx_base == dx && dx_base_stride != dx_stride)
      return set_error(MOE_ERR_INVALID_ARG, "dx_base is dx with another row stride");
  }
  const AdapterLayout l(dims, num_tokens);
  if (num_tokens > 0) {
    MOE_RETURN_IF(check_room(plan_bytes, (size_t)l.plan.total * 4, "plan"));
    MOE_RETURN_IF(check_room(workspace_bytes, l.workspace(), "workspace"));
    if (da) MOE_RETURN_IF(check_room(saved_bytes, l.saved_bytes, "saved"));
    // dx is written before the factors' gradients read x and dout
    if (da && dx && (dx == x || dx == dout))
      return set_error(MOE_ERR_INVALID_ARG, "dx must not be x or dout");
  }
  if (num_tokens == 0 && !da) return moe::set_ok();
  MOE_RETURN_IF(moe::check_gfx950());
  const moe::PlanView v = plan_view(plan, l.plan, dims->num_adapters, num_tokens);
  const bool f32 = dims->out_type == MOE_T_F32;
  void* vt = num_tokens > 0 ? static_cast<uint8_t*>(workspace) + l.part_bytes + l.frag_bytes : nullptr;
  if (num_tokens > 0) {
    const Product q = {dout, dout_stride, b, dims->out_features, l.shape_d, f32, a,
                       dims->in_features, dx_base, dx_base_stride, dx, dx_stride, false,
                       da ? vt : nullptr};
    MOE_RETURN_IF(run_product(q, v, l, dims->rank, scale, workspace, stream));
  }
  if (!da) return moe::set_ok();
  moe::OuterParams o = {};
  o.plan = v;
  o.x = {static_cast<const uint16_t*>(vt), x, x_stride, dims->in_features, da, 0};
  o.dout = {static_cast<const uint16_t*>(saved), dout, dout_stride, dims->out_features, db,
            dims->in_features};
  o.rank = dims->rank;
  o.rank_pad = l.rp;
  o.chunk = l.chunk;
  o.chunks = l.chunks;
  o.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.outer_at());
  MOE_RETURN_IF(moe::check_hip(moe::launch_adapter_outer(o, f32, stream), "adapter gradients", stream));
  return moe::set_ok();
}

}  // extern "C"
