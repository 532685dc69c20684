// Host side of the dense entry points of include/moe.h: argument checks, size
// queries and launch sequences.  As in the run calls every check comes before
// any launch, and nothing allocates or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe.h"
#include "moe_dense.h"
#include "moe_host.h"

namespace {

using moe::ceil_div;
using moe::DenseGemm;
using moe::is_aligned16;
using moe::set_error;
using moe::set_errorf;

constexpr int64_t kMaxTokens = (int64_t)1 << 26;
constexpr int32_t kMaxFeatures = 1 << 18;
// 2^31 / 128^2 less one piece: int32 sums of int8 products cannot overflow
constexpr int32_t kMaxInt8Features = (1 << 17) - 16;

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
moe_status check_tokens(int64_t num_tokens) {
  if (num_tokens < 0 || num_tokens > kMaxTokens)
    return set_errorf(MOE_ERR_INVALID_ARG, "num_tokens %lld outside [0, 2^26]", (long long)num_tokens);
  return MOE_OK;
}
moe_status check_features(int32_t n, int32_t unit, int32_t limit) {
  if (n < unit || n % unit != 0 || n > limit)
    return set_errorf(MOE_ERR_INVALID_ARG, "%d features: a multiple of %d in [%d, %d] is needed", n, unit,
                      unit, limit);
  return MOE_OK;
}
moe_status check_type(int32_t type, const char* what) {
  if (type != MOE_T_BF16 && type != MOE_T_F32)
    return set_errorf(MOE_ERR_INVALID_ARG, "unknown %s type %d", what, type);
  return MOE_OK;
}
// Strides in elements; a tile's rows lie within 32-bit byte offsets.
moe_status check_stride(int64_t stride, int64_t features) {
  if (stride < features || stride % 8 != 0 || stride > ((int64_t)1 << 22))
    return set_errorf(MOE_ERR_INVALID_ARG,
                      "row stride %lld: a multiple of 8 in [%lld, 2^22] is needed", (long long)stride,
                      (long long)features);
  return MOE_OK;
}
moe_status check_base(const void* base, int64_t base_stride, const void* out, int64_t out_stride,
                      int64_t features, const char* what) {
  MOE_RETURN_IF(check_optional(base));
  if (!base) return MOE_OK;
  MOE_RETURN_IF(check_stride(base_stride, features));
  if (base == out && base_stride != out_stride)
    return set_errorf(MOE_ERR_INVALID_ARG, "%s with another row stride", what);
  return MOE_OK;
}

// Tiles of 64 x 128 by 256 threads, fewer than 2^32 of them in a launch.
moe_status check_grid(int64_t rows, int64_t columns) {
  if (ceil_div(rows, 64) * ceil_div(columns, 128) >= (int64_t)1 << 24)
    return set_errorf(MOE_ERR_INVALID_ARG, "%lld tokens by %lld columns: more results than a launch holds",
                      (long long)rows, (long long)columns);
  return MOE_OK;
}

moe_status check_ffn(const moe_ffn_dims* d, int64_t num_tokens, int32_t unit, int32_t limit) {
  if (!d) return set_error(MOE_ERR_INVALID_ARG, "dims is null");
  MOE_RETURN_IF(check_tokens(num_tokens));
  MOE_RETURN_IF(check_features(d->hidden, unit, limit));
  MOE_RETURN_IF(check_features(d->inter, unit, limit));
  if ((int64_t)d->hidden * d->inter > (int64_t)1 << 30)
    return set_errorf(MOE_ERR_INVALID_ARG, "hidden %d x inter %d: more than 2^30 weights a matrix",
                      d->hidden, d->inter);
  return check_grid(num_tokens, std::max(d->hidden, 2 * d->inter));
}
moe_status check_ffn_bf16(const moe_ffn_dims* d, int64_t num_tokens) {
  return check_ffn(d, num_tokens, 8, kMaxFeatures);
}
moe_status check_ffn_int8(const moe_ffn_dims* d, int64_t num_tokens) {
  return check_ffn(d, num_tokens, 16, kMaxInt8Features);
}
moe_status check_int8(const moe_int8_dims* d, int64_t num_tokens) {
  if (!d) return set_error(MOE_ERR_INVALID_ARG, "dims is null");
  MOE_RETURN_IF(check_tokens(num_tokens));
  MOE_RETURN_IF(check_features(d->in_features, 16, kMaxInt8Features));
  MOE_RETURN_IF(check_features(d->out_features, 8, kMaxFeatures));
  MOE_RETURN_IF(check_grid(num_tokens, d->out_features));
  return check_type(d->out_type, "output");
}

// ---------------------------------------------------------------- tiles and parts
// Which tiles a product takes, and into how many parts K is cut so that the 256 CUs
// have work, goes by an estimate of its time: rounds of blocks that run at once, each
// a number of K steps, and for parts the join that reads them.  Measured on full
// grids of 4 to 64 steps, us a step and besides (launch, first reads, the sums' way
// out), bf16 and int8 alike within a tenth:
//                one block a CU     two
//   256 x 256    1.40 + 15         (256 x 128, the last round's: 0.80 + 10)
//   128 x 128    0.50 + 7.2         0.80 + 9.6
//    64 x 128    0.44 + 4.0         0.60 + 5.5
//    64 x 64     0.24 + 4.2         0.45 + 7.5
// a join 6.5 (with its launch on the host) + 1 for 4 MB.  (The block in bf16, T tokens
// of 7168 x 2048, by 64 x 128, 128 and 256 rows: T = 64: 33, 35, -; 512: 86, 71, 91;
// 2048: 266, 180, 171; with 64 x 64 among them T = 64: 30 -> 26.6, 100: 45 -> 39.)
constexpr int64_t kMinPartSteps = 4;
using moe::kCus;
struct Cost {
  double step, fixed;
};
constexpr Cost kOne[4] = {{1.40, 15.0}, {0.50, 7.2}, {0.44, 4.0}, {0.24, 4.2}};
constexpr Cost kTwo[4] = {{}, {0.80, 9.6}, {0.60, 5.5}, {0.45, 7.5}};
constexpr Cost kHalf = {0.80, 10.0};

int64_t slots(int shape) { return shape == moe::kDenseBig ? kCus : 2 * kCus; }
// `blocks` blocks of `steps` each.
double run_cost(int shape, int64_t blocks, double steps) {
  const Cost one = kOne[shape], all = shape == moe::kDenseBig ? one : kTwo[shape];
  const int64_t rounds = blocks / slots(shape), rest = blocks % slots(shape);
  if (moe::dense_halves(shape, blocks) > 0)
    return (double)rounds * (steps * one.step + one.fixed) + steps * kHalf.step + kHalf.fixed;
  const double full = steps * all.step + all.fixed;
  return (double)rounds * full + (rest > kCus ? full : rest > 0 ? steps * one.step + one.fixed : 0.0);
}
double join_cost(const DenseGemm& g, int64_t parts) {
  return parts > 1 ? 6.5 + (double)parts * (double)g.M * (double)g.N * 1e-6 : 0.0;
}
int64_t steps_of(const DenseGemm& g, bool int8) { return ceil_div(g.K, moe::dense_step(int8, g.terms)); }
void set_parts(DenseGemm& g, int64_t steps, int64_t parts) {
  g.steps = (int32_t)std::max((int64_t)1, ceil_div(steps, std::max((int64_t)1, parts)));
  g.split = (int32_t)std::max((int64_t)1, ceil_div(steps, g.steps));
}

// Whether tiles of 64 x 64 are among the choices.  Their step in the estimate holds for
// one or two tiles of rows; with three and four, long sums take longer than it says.
// The block in bf16 (us, without and with them; the product in question and its steps,
// and hidden x inter):
//   tokens               64          128          160          208          256
//   gate  32 steps   17.7 17.7   20.2 17.8    19.7 17.9    20.4 18.0    21.0 17.9   (2048 x 1024)
//   down  32         33.4 33.4   45.5 39.9    49.1 49.1    48.0 47.9    50.5 50.5   (7168 x 2048)
//   gate  43         21.0 18.7   21.7 19.7    21.3 23.9    22.9 24.7    23.4 24.9   (2744 x 1000)
//   gate  64         27.9 26.8   30.3 30.4    33.0 31.9    37.0 35.7    39.2 36.4   (4096 x 2048)
//   gate  64         21.7 18.0   19.6 19.2    21.5 21.6    23.7 25.1    24.1 25.2   (4096 x 1024)
//   gate  81         31.8 31.5   35.6 35.6    37.5 37.5    41.2 46.2    44.5 59.1   (5128 x 1368)
//   gate 112         33.5 33.5   39.8 39.9    49.1 49.1    47.9 55.4    50.5 58.8   (7168 x 2048)
// and in int8 56 steps (7168 to 2048) 13.5 | 10.6 at 64 tokens, 13.6 | 12.1 at 128, 14.9 |
// 17.4 at 192.
bool few_rows(int64_t M, int64_t steps) { return M <= 128 || (M <= 256 && steps <= 32); }

// One product alone; along: both operands lie along k.
void choose(DenseGemm& g, bool int8, bool along) {
  const int64_t steps = steps_of(g, int8);
  double best = 1e300;
  int shape = 0;
  int64_t parts = 1;
  for (int s = 0; s < (along && few_rows(g.M, steps) ? 4 : 3); ++s) {
    g.shape = s;
    const int64_t tiles = std::max((int64_t)1, moe::dense_tiles(g));
    const int64_t most = std::max((int64_t)1, std::min(slots(s) / tiles, steps / kMinPartSteps));
    for (int64_t n = 1; n <= most; ++n) {
      const double t = run_cost(s, tiles * n, (double)ceil_div(steps, n)) + join_cost(g, n);
      if (t < best) best = t, shape = s, parts = n;
    }
  }
  g.shape = shape;
  set_parts(g, steps, parts);
  g.halves = (int32_t)moe::dense_halves(shape, moe::dense_tiles(g) * g.split);
}

// Products of one launch, of one shape, their K cut into parts of `share` steps at
// most.  Returns the estimate: blocks taken in the order of the launch (longer sums
// first) by whichever slot is free.
double share_out(DenseGemm (&g)[3], int shape, int64_t share) {
  int64_t blocks = 0;
  double total = 0, longest = 0, joins = 0;
  const Cost each = shape == moe::kDenseBig ? kOne[shape] : kTwo[shape];
  for (DenseGemm& q : g) {
    q.shape = shape;
    q.halves = 0;
    const int64_t steps = steps_of(q, false);
    set_parts(q, steps, steps / share);
    const int64_t n = moe::dense_tiles(q) * q.split;
    if (n == 0) continue;
    blocks += n;
    const double cost = (double)q.steps * each.step + each.fixed;
    total += (double)n * cost;
    longest = std::max(longest, cost);
    joins += join_cost(q, q.split);
  }
  int order[3];
  moe::dense_order(g, order);
  // where all blocks are as long, those of the last round may be cut in two
  bool alike = true;
  DenseGemm* last = nullptr;
  for (const int o : order)
    if (moe::dense_tiles(g[o]) > 0) {
      alike = alike && (!last || last->steps == g[o].steps);
      last = &g[o];
    }
  if (!last) return 0.0;
  if (alike) {
    last->halves = (int32_t)std::min(moe::dense_halves(shape, blocks), moe::dense_tiles(*last) * last->split);
    return joins + run_cost(shape, blocks, (double)last->steps);
  }
  // no launch ends before its longest block does
  const double least = std::max(longest, total / (double)slots(shape));
  if (blocks > 64 * slots(shape)) return joins + least;
  struct Free {
    double at;
    int64_t n;
  } free[8] = {{0.0, slots(shape)}};
  int groups = 1;
  double end = 0;
  for (const int o : order) {
    const double cost = (double)g[o].steps * each.step + each.fixed;
    for (int64_t n = moe::dense_tiles(g[o]) * g[o].split; n > 0;) {
      int f = 0;
      for (int k = 1; k < groups; ++k)
        if (free[k].at < free[f].at) f = k;
      const int64_t take = std::min(n, free[f].n);
      const double done = free[f].at + cost;
      n -= take;
      end = std::max(end, done);
      free[f].n -= take;
      if (free[f].n == 0) free[f] = free[--groups];
      int into = -1;
      for (int k = 0; k < groups; ++k)
        if (free[k].at == done) into = k;
      if (into < 0 && groups == 8) return joins + std::max(end, least);
      if (into < 0) free[into = groups++] = {done, 0};
      free[into].n += take;
    }
  }
  return joins + end;
}
void choose(DenseGemm (&g)[3]) {
  double best = 1e300;
  int shape = 0;
  int64_t share = 1;
  for (int s : {(int)moe::kDenseBig, (int)moe::kDenseMid}) {
    int64_t work = 0;
    for (DenseGemm& q : g) {
      q.shape = s;
      work += moe::dense_tiles(q) * steps_of(q, false);
    }
    // a block's fair share of the launch, or a longer one
    const int64_t fair = std::max(kMinPartSteps, ceil_div(work, slots(s)));
    for (int64_t m : {2, 3, 4, 8, 16, 1 << 20}) {
      const double t = share_out(g, s, fair * m / 2);
      if (t < best) best = t, shape = s, share = fair * m / 2;
    }
  }
  share_out(g, shape, share);
}
// Room for the parts of a launch: at most as many tiles as run at once, 64 MB by the
// largest; with at most `rows` x `columns` sums of at most K terms.  Never less for
// fewer rows or terms.
size_t part_bytes(int64_t rows, int64_t columns, int64_t K, bool int8) {
  const int64_t most = ceil_div(K, moe::dense_step(int8, 0)) / kMinPartSteps;
  if (most < 2) return 0;
  const double sums = (double)rows * (double)columns * 4.0 * (double)most;
  const size_t cap = (size_t)kCus * 256 * 256 * 4;
  return align256(sums < (double)cap ? (size_t)sums : cap);
}

moe_status run_product(int mode, DenseGemm g, bool int8, void* parts, const char* what, hipStream_t stream) {
  // (the block of 7168 x 2048 with one token: 19.2 us, by tiles 26.5; two tokens by a
  // kernel of that kind took 27.7)
  if (g.M == 1 && mode != moe::kDenseDgate)
    return moe::check_hip(moe::launch_dense_one(int8, mode, g, stream), what, stream);
  choose(g, int8, mode != moe::kDenseDgate);
  g.part = parts;
  MOE_RETURN_IF(moe::check_hip(mode == moe::kDenseDgate ? moe::launch_dense_dgate(g, stream)
                               : int8 ? moe::launch_dense_gemm_int8(mode, g, stream)
                                      : moe::launch_dense_gemm_bf16(mode, g, stream),
                               what, stream));
  if (g.split > 1) MOE_RETURN_IF(moe::check_hip(moe::launch_dense_join(int8, mode, g, stream), what, stream));
  return MOE_OK;
}

DenseGemm product(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int64_t M, int64_t N,
                  int64_t K, int element) {
  DenseGemm g = {};
  g.a = static_cast<const uint8_t*>(a);
  g.a_stride = a_stride * element;
  g.b = static_cast<const uint8_t*>(b);
  g.b_stride = b_stride * element;
  g.M = M;
  g.N = (int32_t)N;
  g.K = K;
  return g;
}
void store_to(DenseGemm& g, void* out, int64_t stride, bool f32, const void* base, int64_t base_stride) {
  g.e.out = out;
  g.e.out_stride = stride;
  g.e.out_f32 = f32;
  g.e.base = base;
  g.e.base_stride = base_stride;
}

// Workspace of the bf16 block: h or the gradients of gate and up in two terms, then
// the parts.  Saved: gate and up, then h in two terms.
struct FfnLayout {
  size_t gu_bytes, h_bytes, rows, part;
  FfnLayout(const moe_ffn_dims* d, int64_t T) {
    const int64_t H = d->hidden, I = d->inter;
    gu_bytes = align256((size_t)T * 2 * I * 4);
    h_bytes = align256((size_t)T * 2 * I * 2);
    rows = align256((size_t)T * 4 * I * 2);
    const int64_t twice = 2 * ceil_div(T, 64) * 64;
    // (the products of a launch need room together, the weights' for twice the terms)
    part = std::max({part_bytes(T, 2 * I, H, false), part_bytes(T, H, I, false), part_bytes(T, I, H, false),
                     part_bytes(2 * I, H, twice, false) + part_bytes(H, I, twice, false) +
                         part_bytes(T, H, 2 * I, false)});
  }
  size_t workspace() const { return rows + part; }
  size_t saved() const { return gu_bytes + h_bytes; }
};

// Workspace of the int8 block.
struct Int8FfnLayout {
  size_t x_scales, h, h_codes, h_scales, part, total;
  Int8FfnLayout(const moe_ffn_dims* d, int64_t T) {
    const int64_t H = d->hidden, I = d->inter;
    x_scales = align256((size_t)T * H);
    h = x_scales + align256((size_t)T * 4);
    h_codes = h + align256((size_t)T * I * 4);
    h_scales = h_codes + align256((size_t)T * I);
    part = h_scales + align256((size_t)T * 4);
    total = part + std::max(part_bytes(T, 2 * I, H, true), part_bytes(T, H, I, true));
  }
};

size_t int8_parts(const moe_int8_dims* d, int64_t T) {
  return part_bytes(T, d->out_features, d->in_features, true);
}

}  // namespace

extern "C" {

moe_status moe_ffn_workspace_query(const moe_ffn_dims* dims, int64_t num_tokens, size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(check_ffn_bf16(dims, num_tokens));
  *bytes = FfnLayout(dims, num_tokens).workspace();
  return moe::set_ok();
}

moe_status moe_ffn_saved_query(const moe_ffn_dims* dims, int64_t num_tokens, size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(check_ffn_bf16(dims, num_tokens));
  *bytes = FfnLayout(dims, num_tokens).saved();
  return moe::set_ok();
}

moe_status moe_ffn_apply(const moe_ffn_dims* dims, const void* x, int64_t x_stride, int64_t num_tokens,
                         const void* w1, const void* w2, const void* base, int64_t base_stride,
                         void* out, int64_t out_stride, void* saved, size_t saved_bytes,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  MOE_RETURN_IF(check_ffn_bf16(dims, num_tokens));
  if (num_tokens == 0) return moe::set_ok();
  const int64_t T = num_tokens, H = dims->hidden, I = dims->inter;
  MOE_RETURN_IF(check_pointers({x, w1, w2, out, workspace}));
  MOE_RETURN_IF(check_optional(saved));
  MOE_RETURN_IF(check_stride(x_stride, H));
  MOE_RETURN_IF(check_stride(out_stride, H));
  MOE_RETURN_IF(check_base(base, base_stride, out, out_stride, H, "base is out"));
  const FfnLayout l(dims, T);
  MOE_RETURN_IF(check_room(workspace_bytes, l.workspace(), "workspace"));
  if (saved) MOE_RETURN_IF(check_room(saved_bytes, l.saved(), "saved"));
  MOE_RETURN_IF(moe::check_gfx950());
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* h = saved ? static_cast<uint8_t*>(saved) + l.gu_bytes : ws;
  DenseGemm up = product(x, x_stride, w1, H, T, 2 * I, H, 2);
  store_to(up, h, I, false, nullptr, 0);
  up.e.inter = (int32_t)I;
  up.e.gu_out = static_cast<float*>(saved);
  up.e.out_lo = saved ? reinterpret_cast<uint16_t*>(h) + T * I : nullptr;
  MOE_RETURN_IF(run_product(moe::kDenseGate, up, false, ws + l.rows, "block gate and up", stream));
  DenseGemm down = product(h, I, w2, I, T, H, I, 2);
  store_to(down, out, out_stride, false, base, base_stride);
  MOE_RETURN_IF(run_product(moe::kDenseStore, down, false, ws + l.rows, "block down", stream));
  return moe::set_ok();
}

moe_status moe_ffn_backward(const moe_ffn_dims* dims, const void* dout, int64_t dout_stride,
                            const void* x, int64_t x_stride, int64_t num_tokens, const void* w1,
                            const void* w2, const void* saved, size_t saved_bytes, void* dw1,
                            void* dw2, int32_t dw_type, const void* dx_base, int64_t dx_base_stride,
                            void* dx, int64_t dx_stride, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  MOE_RETURN_IF(check_ffn_bf16(dims, num_tokens));
  MOE_RETURN_IF(check_type(dw_type, "gradient"));
  if ((dw1 == nullptr) != (dw2 == nullptr))
    return set_error(MOE_ERR_INVALID_ARG, "dw1 and dw2 are wanted together or not at all");
  // (dx of no tokens has no address)
  if (!dw1 && !dx && num_tokens > 0)
    return set_error(MOE_ERR_INVALID_ARG, "neither dx nor dw1 and dw2: no gradient");
  if (dw1) MOE_RETURN_IF(check_pointers({dw1, dw2}));
  MOE_RETURN_IF(check_optional(dx));
  const int64_t T = num_tokens, H = dims->hidden, I = dims->inter;
  const FfnLayout l(dims, T);
  if (T > 0) {
    // the products of one launch read x and dout while dx is written
    if (dw1 && dx && (dx == x || dx == dout))
      return set_error(MOE_ERR_INVALID_ARG, "dx must not be x or dout");
    MOE_RETURN_IF(check_pointers({dout, w2, saved, workspace}));
    MOE_RETURN_IF(check_stride(dout_stride, H));
    if (dw1) {
      MOE_RETURN_IF(check_pointers({x}));
      MOE_RETURN_IF(check_stride(x_stride, H));
    }
    if (dx) {
      MOE_RETURN_IF(check_pointers({w1}));
      MOE_RETURN_IF(check_stride(dx_stride, H));
      MOE_RETURN_IF(check_base(dx_base, dx_base_stride, dx, dx_stride, H, "dx_base is dx"));
    }
    MOE_RETURN_IF(check_room(workspace_bytes, l.workspace(), "workspace"));
    MOE_RETURN_IF(check_room(saved_bytes, l.saved(), "saved"));
  }
  if (T == 0 && !dw1) return moe::set_ok();
  MOE_RETURN_IF(moe::check_gfx950());
  uint8_t* dgu = static_cast<uint8_t*>(workspace);
  uint8_t* parts = T > 0 ? dgu + l.rows : nullptr;
  const uint8_t* h = T > 0 ? static_cast<const uint8_t*>(saved) + l.gu_bytes : nullptr;
  const bool f32 = dw_type == MOE_T_F32;
  if (T > 0) {
    DenseGemm dh = product(dout, dout_stride, w2, I, T, I, H, 2);
    dh.e.out = dgu;
    dh.e.inter = (int32_t)I;
    dh.e.gu_in = static_cast<const float*>(saved);
    if (dw1 && f32) dh.e.out_lo = reinterpret_cast<uint16_t*>(dgu) + T * 2 * I;
    MOE_RETURN_IF(run_product(moe::kDenseDgate, dh, false, parts, "block gradients of gate and up", stream));
  }
  DenseGemm g[3] = {};  // dw1, dw2, dx
  if (dw1) {
    g[0] = product(dgu, 2 * I, x, T > 0 ? x_stride : H, 2 * I, H, T, 2);
    store_to(g[0], dw1, H, f32, nullptr, 0);
    g[1] = product(dout, T > 0 ? dout_stride : H, h, I, H, I, T, 2);
    store_to(g[1], dw2, I, f32, nullptr, 0);
    g[0].terms = f32 ? 1 : 0;  // of the gradients of gate and up
    g[0].lo = T * 2 * I * 2;
    g[1].terms = f32 ? 2 : 0;  // of h
    g[1].lo = T * I * 2;
  }
  if (dx && T > 0) {
    g[2] = product(dgu, 2 * I, w1, H, T, H, 2 * I, 2);
    store_to(g[2], dx, dx_stride, false, dx_base, dx_base_stride);
  }
  choose(g);
  for (DenseGemm& q : g) {
    q.part = parts;
    if (q.split > 1) parts += align256((size_t)q.split * q.M * q.N * 4);
  }
  MOE_RETURN_IF(moe::check_hip(moe::launch_dense_grads(g, stream), "block gradients", stream));
  for (const DenseGemm& q : g)
    if (q.M > 0 && q.split > 1)
      MOE_RETURN_IF(moe::check_hip(moe::launch_dense_join(false, moe::kDenseStore, q, stream),
                                   "block gradients' join", stream));
  return moe::set_ok();
}

moe_status moe_int8_quantize(const void* x, int32_t x_type, int64_t x_stride, int64_t rows,
                             int32_t features, void* codes, float* scales, hipStream_t stream) {
  MOE_RETURN_IF(check_tokens(rows));
  MOE_RETURN_IF(check_type(x_type, "input"));
  MOE_RETURN_IF(check_features(features, 16, kMaxInt8Features));
  if (rows == 0) return moe::set_ok();
  MOE_RETURN_IF(check_pointers({x, codes, scales}));
  MOE_RETURN_IF(check_stride(x_stride, features));
  MOE_RETURN_IF(moe::check_gfx950());
  MOE_RETURN_IF(moe::check_hip(
      moe::launch_int8_quant(x, x_type == MOE_T_F32, x_stride, rows, features,
                             static_cast<int8_t*>(codes), scales, stream),
      "int8 quantize", stream));
  return moe::set_ok();
}

moe_status moe_int8_workspace_query(const moe_int8_dims* dims, int64_t num_tokens, size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(check_int8(dims, num_tokens));
  *bytes = int8_parts(dims, num_tokens);
  return moe::set_ok();
}

moe_status moe_int8_matmul(const moe_int8_dims* dims, const void* codes, const float* scales,
                           int64_t num_tokens, const void* w, const float* w_scales,
                           const void* base, int64_t base_stride, void* out, int64_t out_stride,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  MOE_RETURN_IF(check_int8(dims, num_tokens));
  if (num_tokens == 0) return moe::set_ok();
  const int64_t T = num_tokens, K = dims->in_features, N = dims->out_features;
  MOE_RETURN_IF(check_pointers({codes, scales, w, w_scales, out}));
  MOE_RETURN_IF(check_optional(workspace));
  MOE_RETURN_IF(check_stride(out_stride, N));
  MOE_RETURN_IF(check_base(base, base_stride, out, out_stride, N, "base is out"));
  const size_t need = int8_parts(dims, T);
  if (need > 0) MOE_RETURN_IF(check_pointers({workspace}));
  MOE_RETURN_IF(check_room(workspace_bytes, need, "workspace"));
  MOE_RETURN_IF(moe::check_gfx950());
  DenseGemm g = product(codes, K, w, K, T, N, K, 1);
  store_to(g, out, out_stride, dims->out_type == MOE_T_F32, base, base_stride);
  g.e.row_scale = scales;
  g.e.col_scale = w_scales;
  MOE_RETURN_IF(run_product(moe::kDenseStore, g, true, workspace, "int8 product", stream));
  return moe::set_ok();
}

moe_status moe_ffn_int8_workspace_query(const moe_ffn_dims* dims, int64_t num_tokens, size_t* bytes) {
  if (!bytes) return set_error(MOE_ERR_INVALID_ARG, "null output pointer");
  MOE_RETURN_IF(check_ffn_int8(dims, num_tokens));
  *bytes = Int8FfnLayout(dims, num_tokens).total;
  return moe::set_ok();
}

moe_status moe_ffn_int8_apply(const moe_ffn_dims* dims, const void* x, int64_t x_stride,
                              int64_t num_tokens, const void* w1, const float* w1_scales,
                              const void* w2, const float* w2_scales, const void* base,
                              int64_t base_stride, void* out, int64_t out_stride, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  MOE_RETURN_IF(check_ffn_int8(dims, num_tokens));
  if (num_tokens == 0) return moe::set_ok();
  const int64_t T = num_tokens, H = dims->hidden, I = dims->inter;
  MOE_RETURN_IF(check_pointers({x, w1, w1_scales, w2, w2_scales, out, workspace}));
  MOE_RETURN_IF(check_stride(x_stride, H));
  MOE_RETURN_IF(check_stride(out_stride, H));
  MOE_RETURN_IF(check_base(base, base_stride, out, out_stride, H, "base is out"));
  const Int8FfnLayout l(dims, T);
  MOE_RETURN_IF(check_room(workspace_bytes, l.total, "workspace"));
  MOE_RETURN_IF(moe::check_gfx950());
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int8_t* codes = reinterpret_cast<int8_t*>(ws);
  float* scales = reinterpret_cast<float*>(ws + l.x_scales);
  float* h = reinterpret_cast<float*>(ws + l.h);
  int8_t* h_codes = reinterpret_cast<int8_t*>(ws + l.h_codes);
  float* h_scales = reinterpret_cast<float*>(ws + l.h_scales);
  MOE_RETURN_IF(moe::check_hip(
      moe::launch_int8_quant(x, false, x_stride, T, (int32_t)H, codes, scales, stream),
      "int8 block quantize", stream));
  DenseGemm up = product(codes, H, w1, H, T, 2 * I, H, 1);
  store_to(up, h, I, true, nullptr, 0);
  up.e.inter = (int32_t)I;
  up.e.row_scale = scales;
  up.e.col_scale = w1_scales;
  choose(up, true, true);
  if (T > 1 && up.split > 1) {
    // the join of the parts quantises h and never stores it
    up.part = ws + l.part;
    MOE_RETURN_IF(moe::check_hip(moe::launch_dense_gemm_int8(moe::kDenseGate, up, stream),
                                 "int8 block gate and up", stream));
    MOE_RETURN_IF(moe::check_hip(moe::launch_dense_join_quant(up, h_codes, h_scales, stream),
                                 "int8 block requantize", stream));
  } else {
    MOE_RETURN_IF(run_product(moe::kDenseGate, up, true, ws + l.part, "int8 block gate and up", stream));
    MOE_RETURN_IF(moe::check_hip(
        moe::launch_int8_quant(h, true, I, T, (int32_t)I, h_codes, h_scales, stream),
        "int8 block requantize", stream));
  }
  DenseGemm down = product(h_codes, I, w2, I, T, H, I, 1);
  store_to(down, out, out_stride, false, base, base_stride);
  down.e.row_scale = h_scales;
  down.e.col_scale = w2_scales;
  MOE_RETURN_IF(run_product(moe::kDenseStore, down, true, ws + l.part, "int8 block down", stream));
  return moe::set_ok();
}

}  // extern "C"
