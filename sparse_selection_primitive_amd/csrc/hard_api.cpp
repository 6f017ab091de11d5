// Host runtime of the hard selections declared in include/lapsum.h: argument
// checks, workspace layout and launches on the caller's stream.  Nothing is
// allocated and no stream is synchronised.
#include <hip/hip_runtime.h>

#include <cmath>
#include <utility>

#include "hard_internal.hpp"

using namespace lapsum;

namespace {

constexpr size_t kAlign = 256;

size_t aligned_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool known_dtype(int32_t d) { return d == LAPSUM_F32 || d == LAPSUM_BF16 || d == LAPSUM_F16; }

lapsum_status check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return LAPSUM_OK;
  if (!ws) return LAPSUM_ERR_NULL;
  return have < need || !aligned(ws, kAlign) ? LAPSUM_ERR_WORKSPACE : LAPSUM_OK;
}

lapsum_status done(hipError_t e) { return e == hipSuccess ? LAPSUM_OK : LAPSUM_ERR_HIP; }

lapsum_status check_route(int32_t dtype, int64_t tokens, int64_t experts, int64_t row_stride,
                          const lapsum_route_options *o) {
  if (!o) return LAPSUM_ERR_NULL;
  if (!known_dtype(dtype)) return LAPSUM_ERR_OPTION;
  if (tokens < 1 || tokens > LAPSUM_MAX_ROWS || experts < 1 || experts > LAPSUM_MAX_EXPERTS) return LAPSUM_ERR_SHAPE;
  if (row_stride < experts) return LAPSUM_ERR_LAYOUT;
  if (o->k < 1 || o->k > experts || o->k > LAPSUM_MAX_CHOICES) return LAPSUM_ERR_OPTION;
  if (o->score != LAPSUM_SCORE_SOFTMAX && o->score != LAPSUM_SCORE_SIGMOID) return LAPSUM_ERR_OPTION;
  if (o->groups < 1 || o->groups > LAPSUM_MAX_GROUPS || experts % o->groups != 0) return LAPSUM_ERR_OPTION;
  if (o->top_groups < 1 || o->top_groups > o->groups) return LAPSUM_ERR_OPTION;
  if (o->renormalise != 0 && o->renormalise != 1) return LAPSUM_ERR_OPTION;
  if (!std::isfinite(o->scale)) return LAPSUM_ERR_OPTION;
  return LAPSUM_OK;
}

RouteArgs route_args(const void *logits, int64_t tokens, int64_t experts, int64_t row_stride,
                     const lapsum_route_options &o) {
  RouteArgs a{};
  a.logits = logits;
  a.tokens = tokens;
  a.stride = row_stride;
  a.experts = (int)experts;
  a.k = o.k;
  a.score = o.score;
  a.groups = o.groups;
  a.top_groups = o.top_groups;
  a.group_size = (int)experts / o.groups;
  a.group_magic = (uint32_t)(((1 << 21) + a.group_size - 1) / a.group_size);
  a.renormalise = o.renormalise;
  a.scale = o.scale;
  return a;
}

lapsum_status check_pairs(int64_t tokens, int64_t k) {
  if (tokens < 1 || k < 1 || k > LAPSUM_MAX_CHOICES || tokens > LAPSUM_MAX_PAIRS / k) return LAPSUM_ERR_SHAPE;
  return LAPSUM_OK;
}

lapsum_status check_rows(int32_t dtype, int64_t tokens, int64_t k, int64_t width, int64_t row_stride) {
  if (!known_dtype(dtype)) return LAPSUM_ERR_OPTION;
  const lapsum_status st = check_pairs(tokens, k);
  if (st != LAPSUM_OK) return st;
  if (width < 1 || width > LAPSUM_MAX_N) return LAPSUM_ERR_SHAPE;
  return row_stride < width ? LAPSUM_ERR_LAYOUT : LAPSUM_OK;
}

RowsArgs rows_args(const void *src, void *dst, int64_t tokens, int64_t k, int64_t width, int64_t stride,
                   const int32_t *slot) {
  RowsArgs a{};
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.k = (int)k;
  a.pairs = tokens * k;
  a.width = width;
  a.stride = stride;
  a.slot = slot;
  return a;
}

size_t plan_bytes(int64_t pairs, int64_t experts) {
  const int64_t tiles = plan_tiles(pairs);
  return tiles > 1 ? aligned_up((size_t)(experts * tiles + experts) * sizeof(uint32_t)) : 0;
}

// Shape and layout of a cache; the pointers are checked by check_cache_pointers.
lapsum_status check_cache(const lapsum_cache *c) {
  if (!c) return LAPSUM_ERR_NULL;
  if (c->dtype != LAPSUM_BF16 && c->dtype != LAPSUM_F16) return LAPSUM_ERR_OPTION;
  if (c->width < 8 || c->width > 256 || c->width % 8 != 0) return LAPSUM_ERR_SHAPE;
  if (c->batch < 1 || c->heads < 1 || c->batch > LAPSUM_MAX_ROWS || c->heads > LAPSUM_MAX_ROWS / c->batch)
    return LAPSUM_ERR_SHAPE;
  if (c->capacity < 1 || c->capacity > LAPSUM_MAX_CACHE) return LAPSUM_ERR_SHAPE;
  const int64_t strides[] = {c->k_stride_batch, c->k_stride_head, c->k_stride_entry,
                             c->v_stride_batch, c->v_stride_head, c->v_stride_entry};
  for (int64_t s : strides)
    if (s < 0 || s % 8 != 0) return LAPSUM_ERR_LAYOUT;
  // 64 entries lie within the 2^31 bytes that a buffer load's offset reaches
  if (c->k_stride_entry > LAPSUM_MAX_ENTRY_STRIDE || c->v_stride_entry > LAPSUM_MAX_ENTRY_STRIDE)
    return LAPSUM_ERR_LAYOUT;
  return LAPSUM_OK;
}
lapsum_status check_cache_pointers(const lapsum_cache *c) {
  if (!c->k || !c->v) return LAPSUM_ERR_NULL;
  return aligned(c->k, 16) && aligned(c->v, 16) ? LAPSUM_OK : LAPSUM_ERR_LAYOUT;
}

// Whether no two entries share memory, by the order of the strides: each has to pass what the
// smaller ones span.  (Layouts whose dimensions are woven into each other without meeting are not told from those that
// meet.)
bool apart(const lapsum_cache &c, int64_t batch, int64_t head, int64_t entry) {
  if (entry < c.width) return false;
  struct {
    int64_t stride, size;
  } d[] = {{entry, c.capacity}, {head, c.heads}, {batch, c.batch}};
  if (d[1].stride < d[0].stride) std::swap(d[0], d[1]);
  if (d[2].stride < d[1].stride) std::swap(d[1], d[2]);
  if (d[1].stride < d[0].stride) std::swap(d[0], d[1]);
  __int128 span = c.width;
  for (const auto &x : d) {
    if (x.size == 1) continue;
    if (x.stride < span) return false;
    span += (__int128)x.stride * (x.size - 1);
  }
  return true;
}

// Whether keys and values lie alike; the stride of a size of one is any.
bool same_strides(const lapsum_cache &c) {
  return (c.batch == 1 || c.k_stride_batch == c.v_stride_batch) && (c.heads == 1 || c.k_stride_head == c.v_stride_head) &&
         (c.capacity == 1 || c.k_stride_entry == c.v_stride_entry);
}

lapsum_status check_attend(const lapsum_cache *c, int64_t news, int64_t q_heads) {
  const lapsum_status st = check_cache(c);
  if (st != LAPSUM_OK) return st;
  if (news < 1 || news > 65536 || q_heads < c->heads || q_heads % c->heads != 0) return LAPSUM_ERR_SHAPE;
  if (q_heads / c->heads > 65536 / news) return LAPSUM_ERR_SHAPE;
  return LAPSUM_OK;
}

lapsum_status check_experts(const lapsum_experts *w, int64_t rows) {
  if (!w) return LAPSUM_ERR_NULL;
  if (!known_dtype(w->dtype)) return LAPSUM_ERR_OPTION;
  if (w->experts < 1 || w->experts > LAPSUM_MAX_EXPERTS || w->inputs < 1 || w->inputs > LAPSUM_MAX_EXPERT_WIDTH ||
      w->outputs < 1 || w->outputs > LAPSUM_MAX_EXPERT_WIDTH || rows < 1 || rows > LAPSUM_MAX_PAIRS)
    return LAPSUM_ERR_SHAPE;
  const bool out_next = w->stride_output == 1 && w->stride_input >= w->outputs;
  const bool in_next = w->stride_input == 1 && w->stride_output >= w->inputs;
  if (!out_next && !in_next) return LAPSUM_ERR_LAYOUT;
  if (w->stride_input > LAPSUM_MAX_EXPERT_STRIDE || w->stride_output > LAPSUM_MAX_EXPERT_STRIDE) return LAPSUM_ERR_LAYOUT;
  return w->stride_expert < 0 ? LAPSUM_ERR_LAYOUT : LAPSUM_OK;
}
lapsum_status check_row_stride(int64_t stride, int64_t width) {
  return stride < width || stride > LAPSUM_MAX_EXPERT_STRIDE ? LAPSUM_ERR_LAYOUT : LAPSUM_OK;
}
// whether a matrix' outputs lie next to each other (of one column or row both hold)
bool outputs_next(const lapsum_experts &w) { return w.stride_output == 1 && w.stride_input >= w.outputs; }

// Whether two stretches of memory meet.
bool meet(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
int64_t type_bytes(int32_t dtype) { return dtype == LAPSUM_F32 ? 4 : 2; }
int64_t rows_bytes(int64_t rows, int64_t width, int64_t stride, int32_t dtype) {
  return ((rows - 1) * stride + width) * type_bytes(dtype);
}
int64_t experts_bytes(const lapsum_experts &w) {  // strides that no memory holds count as the most there is
  const __int128 last = (__int128)(w.experts - 1) * w.stride_expert + (w.inputs - 1) * w.stride_input +
                        (w.outputs - 1) * w.stride_output + 1;
  const __int128 bytes = last * type_bytes(w.dtype), most = (__int128)1 << 62;
  return (int64_t)(bytes < most ? bytes : most);
}

// A layout of memory: `width` bytes next to each other, at every sum of up to three strides (the largest first).
struct Layout {
  struct Dim {
    int64_t stride, size;  // bytes, more than one place each
  };
  const void *at;
  int64_t width;
  int dims;
  Dim dim[3];

  __int128 extent(int from) const {  // of what the dimensions from `from` on span
    __int128 bytes = width;
    for (int i = from; i < dims; ++i) bytes += (__int128)dim[i].stride * (dim[i].size - 1);
    return bytes;
  }
  // Whether a byte of it lies in [lo, hi), from `at` on.  Only places whose extent meets the stretch are looked at, and one that
  // lies in it whole ends the search, so a dimension has a few to look at whatever its size.
  bool meets(__int128 lo, __int128 hi, int from = 0) const {
    if (lo >= extent(from) || hi <= 0) return false;  // as nearly always
    if (from == dims) return true;
    const __int128 stride = dim[from].stride, inner = extent(from + 1);
    __int128 last = (hi - 1) / stride;
    if (last > dim[from].size - 1) last = dim[from].size - 1;
    for (__int128 i = lo < inner ? 0 : (lo - inner) / stride + 1; i <= last; ++i)
      if (meets(lo - i * stride, hi - i * stride, from + 1)) return true;
    return false;
  }
};
struct Block {
  const void *at;  // or NULL: none
  int64_t bytes;
};
bool meet(const Block &a, const Block &b) { return a.at && b.at && meet(a.at, a.bytes, b.at, b.bytes); }
bool meet(const Layout &a, const Block &b) {
  if (!b.at) return false;
  const __int128 lo = (__int128) reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at);
  return a.meets(lo, lo + b.bytes);
}
// Whether a block that is written meets another one that is, or one that is read.
template <int W, int R>
bool any_meet(const Block (&written)[W], const Block (&read)[R]) {
  for (int i = 0; i < W; ++i) {
    for (int j = i + 1; j < W; ++j)
      if (meet(written[i], written[j])) return true;
    for (const Block &b : read)
      if (meet(written[i], b)) return true;
  }
  return false;
}

// The keys or the values of a cache whose entries are apart.
Layout side_of(const lapsum_cache &c, const void *at, int64_t batch, int64_t head, int64_t entry) {
  Layout x{at, (int64_t)c.width * 2, 0, {}};
  for (const Layout::Dim &d : {Layout::Dim{batch, c.batch}, Layout::Dim{head, c.heads}, Layout::Dim{entry, c.capacity}}) {
    if (d.size == 1) continue;
    const __int128 stride = (__int128)d.stride * 2, most = (__int128)1 << 62;
    int i = x.dims++;
    for (; i > 0 && x.dim[i - 1].stride < stride; --i) x.dim[i] = x.dim[i - 1];
    x.dim[i] = {(int64_t)(stride < most ? stride : most), d.size};
  }
  return x;
}
// Whether an entry's keys share memory with an entry's values, for caches that are not one and whose entries are apart: known where
// both lie alike, begin together, or one of them fills what it spans.  (Unlike layouts, both with gaps, that are woven into each
// other are not looked at further.)
bool keys_meet_values(const lapsum_cache &c) {
  if (c.k == c.v) return true;
  const Layout k = side_of(c, c.k, c.k_stride_batch, c.k_stride_head, c.k_stride_entry);
  const Layout v = side_of(c, c.v, c.v_stride_batch, c.v_stride_head, c.v_stride_entry);
  const __int128 all = (__int128)c.batch * c.heads * c.capacity * k.width, most = (__int128)1 << 62;
  if (all < most && k.extent(0) == all) return meet(v, {c.k, (int64_t)all});
  if (all < most && v.extent(0) == all) return meet(k, {c.v, (int64_t)all});
  if (!same_strides(c)) return false;
  const __int128 ahead = (__int128) reinterpret_cast<uintptr_t>(c.v) - reinterpret_cast<uintptr_t>(c.k);
  // An entry's values are at ahead + x from the first keys, another's keys at y.  y - x over all pairs is a layout of twice as
  // many places less one a dimension, which starts at minus its half; they meet where ahead is less than an entry from it.
  Layout apart = k;
  apart.width = 1;
  __int128 half = 0;
  for (int i = 0; i < k.dims; ++i) {
    half += (__int128)k.dim[i].stride * (k.dim[i].size - 1);
    apart.dim[i].size = 2 * k.dim[i].size - 1;
  }
  return apart.meets(half + ahead - k.width + 1, half + ahead + k.width);
}

ProductArgs product_args(const lapsum_experts &w, int64_t rows, const int32_t *offsets) {
  ProductArgs a{};
  a.rows = rows;
  a.experts = (int)w.experts;
  a.offsets = offsets;
  return a;
}

lapsum_status check_beams(int32_t dtype, int64_t batch, int64_t beams, int64_t vocab, int32_t k) {
  if (!known_dtype(dtype)) return LAPSUM_ERR_OPTION;
  if (beams < 1 || beams > LAPSUM_MAX_BEAMS || batch < 1 || batch > LAPSUM_MAX_ROWS / beams || vocab < 1 ||
      vocab > LAPSUM_MAX_VOCAB)
    return LAPSUM_ERR_SHAPE;
  return k < 1 || k > LAPSUM_MAX_BEAMS ? LAPSUM_ERR_OPTION : LAPSUM_OK;
}
// the parts' maxima, then the groups' sums
size_t beam_tops_bytes(int64_t rows, int chunks) { return aligned_up((size_t)rows * (size_t)chunks * sizeof(float)); }
size_t beam_bytes(int64_t batch, int64_t beams, int64_t vocab) {
  int chunk, chunks;
  beam_parts(beams, vocab, chunk, chunks);
  const size_t groups = (size_t)(chunks + kBeamGroup - 1) / kBeamGroup;
  return beam_tops_bytes(batch * beams, chunks) + aligned_up((size_t)(batch * beams) * groups * sizeof(float2));
}

size_t attend_bytes(const AttendPlan &p) {
  return aligned_up(p.part_o) + aligned_up(p.part_ml) + aligned_up(p.dropped) + aligned_up(p.logits);
}

}  // namespace

extern "C" {

lapsum_status lapsum_route_forward(const void *logits, int32_t dtype, int64_t tokens, int64_t experts,
                                   int64_t row_stride, const float *bias, const lapsum_route_options *opt,
                                   float *weights, int32_t *chosen, void *stream) {
  const lapsum_status st = check_route(dtype, tokens, experts, row_stride, opt);
  if (st != LAPSUM_OK) return st;
  if (!logits || !weights || !chosen) return LAPSUM_ERR_NULL;
  RouteArgs a = route_args(logits, tokens, experts, row_stride, *opt);
  a.bias = bias;
  a.weights = weights;
  a.chosen = chosen;
  (void)hipGetLastError();  // drop a non-sticky error that an earlier, unrelated call left pending
  return done(launch_route_forward(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_route_backward(const float *dweights, const void *logits, int32_t dtype, int64_t tokens,
                                    int64_t experts, int64_t row_stride, const int32_t *chosen,
                                    const lapsum_route_options *opt, void *dlogits, void *stream) {
  const lapsum_status st = check_route(dtype, tokens, experts, row_stride, opt);
  if (st != LAPSUM_OK) return st;
  if (!dweights || !logits || !chosen || !dlogits) return LAPSUM_ERR_NULL;
  RouteArgs a = route_args(logits, tokens, experts, row_stride, *opt);
  a.dweights = dweights;
  a.chosen = const_cast<int32_t *>(chosen);  // only read by the backward
  a.dlogits = dlogits;
  (void)hipGetLastError();
  return done(launch_route_backward(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t lapsum_dispatch_plan_workspace_bytes(int64_t tokens, int64_t k, int64_t experts) {
  if (check_pairs(tokens, k) != LAPSUM_OK || experts < 1 || experts > LAPSUM_MAX_EXPERTS) return 0;
  return plan_bytes(tokens * k, experts);
}

lapsum_status lapsum_dispatch_plan(const int32_t *chosen, int64_t tokens, int64_t k, int64_t experts,
                                   int32_t *offsets, int32_t *slot, int32_t *order, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  lapsum_status st = check_pairs(tokens, k);
  if (st != LAPSUM_OK) return st;
  if (experts < 1 || experts > LAPSUM_MAX_EXPERTS) return LAPSUM_ERR_SHAPE;
  if (!chosen || !offsets || !slot || !order) return LAPSUM_ERR_NULL;
  st = check_workspace(workspace, workspace_bytes, plan_bytes(tokens * k, experts));
  if (st != LAPSUM_OK) return st;
  (void)hipGetLastError();
  return done(launch_dispatch_plan(chosen, tokens * k, (int)experts, offsets, slot, order,
                                   static_cast<uint32_t *>(workspace), reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_dispatch_forward(const void *x, int32_t dtype, int64_t tokens, int64_t k, int64_t width,
                                      int64_t row_stride, const int32_t *slot, const int32_t *offsets,
                                      int64_t experts, void *xs, void *stream) {
  const lapsum_status st = check_rows(dtype, tokens, k, width, row_stride);
  if (st != LAPSUM_OK) return st;
  if (experts < 1 || experts > LAPSUM_MAX_EXPERTS) return LAPSUM_ERR_SHAPE;
  if (!x || !slot || !offsets || !xs) return LAPSUM_ERR_NULL;
  RowsArgs a = rows_args(x, xs, tokens, k, width, row_stride, slot);
  a.placed = offsets + experts;
  (void)hipGetLastError();
  return done(launch_dispatch_rows(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_dispatch_backward(const void *dxs, int32_t dtype, int64_t tokens, int64_t k, int64_t width,
                                       const int32_t *slot, void *dx, void *stream) {
  const lapsum_status st = check_rows(dtype, tokens, k, width, width);
  if (st != LAPSUM_OK) return st;
  if (!dxs || !slot || !dx) return LAPSUM_ERR_NULL;
  const RowsArgs a = rows_args(dxs, dx, tokens, k, width, width, slot);
  (void)hipGetLastError();
  return done(launch_sum_rows(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_combine_forward(const void *ys, int32_t dtype, int64_t tokens, int64_t k, int64_t width,
                                     const int32_t *slot, const float *weights, void *y, void *stream) {
  const lapsum_status st = check_rows(dtype, tokens, k, width, width);
  if (st != LAPSUM_OK) return st;
  if (!ys || !slot || !weights || !y) return LAPSUM_ERR_NULL;
  RowsArgs a = rows_args(ys, y, tokens, k, width, width, slot);
  a.weights = weights;
  (void)hipGetLastError();
  return done(launch_sum_rows(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_combine_backward(const void *dy, int64_t row_stride, const void *ys, int32_t dtype,
                                      int64_t tokens, int64_t k, int64_t width, const int32_t *slot,
                                      const float *weights, const int32_t *offsets, int64_t experts, void *dys,
                                      float *dweights, void *stream) {
  const lapsum_status st = check_rows(dtype, tokens, k, width, row_stride);
  if (st != LAPSUM_OK) return st;
  if (experts < 1 || experts > LAPSUM_MAX_EXPERTS) return LAPSUM_ERR_SHAPE;
  if (!dy || !ys || !slot || !weights || !offsets || !dys || !dweights) return LAPSUM_ERR_NULL;
  RowsArgs a = rows_args(ys, dys, tokens, k, width, row_stride, slot);
  a.dy = dy;
  a.weights = weights;
  a.dweights = dweights;
  a.placed = offsets + experts;
  (void)hipGetLastError();
  return done(launch_combine_backward(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t lapsum_cache_attend_workspace_bytes(const lapsum_cache *cache, int64_t news, int64_t q_heads,
                                           int32_t accounts) {
  if (check_attend(cache, news, q_heads) != LAPSUM_OK) return 0;
  return attend_bytes(attend_plan(cache->batch, cache->heads, cache->capacity, news * (q_heads / cache->heads),
                                  news == 1, cache->width, accounts != 0));
}

lapsum_status lapsum_cache_attend(const void *q, const lapsum_cache *cache, const int32_t *lengths, int64_t news,
                                  int64_t q_heads, float scale, const float *account, float *account_out, void *out,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  lapsum_status st = check_attend(cache, news, q_heads);
  if (st != LAPSUM_OK) return st;
  if (!std::isfinite(scale)) return LAPSUM_ERR_OPTION;
  if (!q || !lengths || !out || (account == nullptr) != (account_out == nullptr)) return LAPSUM_ERR_NULL;
  st = check_cache_pointers(cache);
  if (st != LAPSUM_OK) return st;
  if (!aligned(q, 16) || !aligned(out, 16)) return LAPSUM_ERR_LAYOUT;
  const int64_t group = q_heads / cache->heads, rows = news * group;
  const AttendPlan p = attend_plan(cache->batch, cache->heads, cache->capacity, rows, news == 1,
                                   cache->width, account != nullptr);
  st = check_workspace(workspace, workspace_bytes, attend_bytes(p));
  if (st != LAPSUM_OK) return st;
  char *ws = static_cast<char *>(workspace);
  AttendArgs a{};
  a.q = q;
  a.k = cache->k;
  a.v = cache->v;
  a.kb = cache->k_stride_batch;
  a.kh = cache->k_stride_head;
  a.ke = cache->k_stride_entry;
  a.vb = cache->v_stride_batch;
  a.vh = cache->v_stride_head;
  a.ve = cache->v_stride_entry;
  a.batch = (int)cache->batch;
  a.heads = (int)cache->heads;
  a.news = (int)news;
  a.group = (int)group;
  a.rows = (int)rows;
  a.group_magic = (uint32_t)((((uint64_t)1 << 32) + (uint64_t)group - 1) / (uint64_t)group);
  a.width = cache->width;
  a.capacity = cache->capacity;
  a.lengths = lengths;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.splits = p.splits;
  a.account = account;
  a.account_out = account_out;
  a.out = out;
  a.part_o = reinterpret_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float *>(ws + aligned_up(p.part_o));
  ws += aligned_up(p.part_o) + aligned_up(p.part_ml);
  a.dropped = reinterpret_cast<int *>(ws);
  a.logits = p.keep_logits ? reinterpret_cast<float *>(ws + aligned_up(p.dropped)) : nullptr;
  a.blocks = p.blocks;
  (void)hipGetLastError();
  return done(launch_attend(a, cache->dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t lapsum_cache_evict_workspace_bytes(const lapsum_cache *cache, int64_t keep) {
  if (check_cache(cache) != LAPSUM_OK || keep < 1 || keep > cache->capacity) return 0;
  return aligned_up(evict_workspace(cache->batch, cache->heads, cache->capacity, keep));
}

lapsum_status lapsum_cache_evict(const lapsum_cache *cache, const float *account, const int32_t *positions,
                                 const int32_t *lengths, int64_t keep, const int32_t *next_position, int32_t sinks,
                                 int32_t recent, float *account_out, int32_t *positions_out, int32_t *kept,
                                 int32_t *lengths_out, void *workspace, size_t workspace_bytes, void *stream) {
  lapsum_status st = check_cache(cache);
  if (st != LAPSUM_OK) return st;
  if (keep < 1 || keep > cache->capacity) return LAPSUM_ERR_SHAPE;
  if (sinks < 0 || recent < 0) return LAPSUM_ERR_OPTION;
  // entries are written: no two of them may share memory
  if (!apart(*cache, cache->k_stride_batch, cache->k_stride_head, cache->k_stride_entry) ||
      !apart(*cache, cache->v_stride_batch, cache->v_stride_head, cache->v_stride_entry))
    return LAPSUM_ERR_LAYOUT;
  if (!account || !positions || !lengths || !account_out || !positions_out || !kept || !lengths_out ||
      (recent > 0 && !next_position))
    return LAPSUM_ERR_NULL;
  if (lengths_out == lengths) return LAPSUM_ERR_LAYOUT;
  st = check_cache_pointers(cache);
  if (st != LAPSUM_OK) return st;
  st = check_workspace(workspace, workspace_bytes,
                       aligned_up(evict_workspace(cache->batch, cache->heads, cache->capacity, keep)));
  if (st != LAPSUM_OK) return st;
  EvictArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.kb = cache->k_stride_batch;
  a.kh = cache->k_stride_head;
  a.ke = cache->k_stride_entry;
  a.vb = cache->v_stride_batch;
  a.vh = cache->v_stride_head;
  a.ve = cache->v_stride_entry;
  a.batch = cache->batch;
  a.heads = cache->heads;
  a.capacity = cache->capacity;
  a.keep = keep;
  a.entry_bytes = cache->width * 2;
  a.account = account;
  a.positions = positions;
  a.lengths = lengths;
  a.next_position = next_position;
  a.sinks = sinks;
  a.recent = recent;
  a.account_out = account_out;
  a.positions_out = positions_out;
  a.kept = kept;
  a.lengths_out = lengths_out;
  a.workspace = workspace;
  (void)hipGetLastError();
  return done(launch_evict(a, reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_expert_product_forward(const void *xs, int64_t xs_stride, int64_t rows, const lapsum_experts *w,
                                            const int32_t *offsets, void *ys, void *stream) {
  lapsum_status st = check_experts(w, rows);
  if (st != LAPSUM_OK) return st;
  st = check_row_stride(xs_stride, w->inputs);
  if (st != LAPSUM_OK) return st;
  if (!xs || !w->w || !offsets || !ys) return LAPSUM_ERR_NULL;
  const int64_t out = rows_bytes(rows, w->outputs, w->outputs, w->dtype);
  if (meet(ys, out, xs, rows_bytes(rows, w->inputs, xs_stride, w->dtype)) || meet(ys, out, w->w, experts_bytes(*w)))
    return LAPSUM_ERR_LAYOUT;
  ProductArgs a = product_args(*w, rows, offsets);
  a.a = xs;
  a.am = xs_stride;
  a.ak = 1;
  a.b = w->w;
  a.be = w->stride_expert;
  a.bk = w->stride_input;
  a.bn = w->stride_output;
  a.c = ys;
  a.cm = w->outputs;
  a.n = (int)w->outputs;
  a.k = (int)w->inputs;
  (void)hipGetLastError();
  return done(launch_product_rows(a, w->dtype, reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_expert_product_backward_rows(const void *dys, int64_t dys_stride, int64_t rows,
                                                  const lapsum_experts *w, const int32_t *offsets, void *dxs,
                                                  void *stream) {
  // the same product, of the matrices with inputs and outputs changed over
  lapsum_experts t{};
  if (w) {
    t = *w;
    std::swap(t.inputs, t.outputs);
    std::swap(t.stride_input, t.stride_output);
  }
  return lapsum_expert_product_forward(dys, dys_stride, rows, w ? &t : nullptr, offsets, dxs, stream);
}

lapsum_status lapsum_expert_product_backward_weights(const void *xs, int64_t xs_stride, const void *dys,
                                                     int64_t dys_stride, int64_t rows, const int32_t *offsets,
                                                     const lapsum_experts *dw, void *stream) {
  lapsum_status st = check_experts(dw, rows);
  if (st != LAPSUM_OK) return st;
  st = check_row_stride(xs_stride, dw->inputs);
  if (st == LAPSUM_OK) st = check_row_stride(dys_stride, dw->outputs);
  if (st != LAPSUM_OK) return st;
  if (!xs || !dys || !offsets || !dw->w) return LAPSUM_ERR_NULL;
  // matrices are written: no two of them may share memory
  const bool next = outputs_next(*dw);
  const int64_t across = next ? dw->inputs : dw->outputs, along = next ? dw->outputs : dw->inputs;
  const int64_t stride = next ? dw->stride_input : dw->stride_output;
  if (dw->experts > 1 && dw->stride_expert < stride * (across - 1) + along) return LAPSUM_ERR_LAYOUT;
  const int64_t out = experts_bytes(*dw);
  if (meet(dw->w, out, xs, rows_bytes(rows, dw->inputs, xs_stride, dw->dtype)) ||
      meet(dw->w, out, dys, rows_bytes(rows, dw->outputs, dys_stride, dw->dtype)))
    return LAPSUM_ERR_LAYOUT;
  ProductArgs a = product_args(*dw, rows, offsets);
  a.a = next ? xs : dys;
  a.b = next ? dys : xs;
  a.am = 1;
  a.ak = next ? xs_stride : dys_stride;
  a.bk = next ? dys_stride : xs_stride;
  a.bn = 1;
  a.c = dw->w;
  a.ce = dw->stride_expert;
  a.cm = stride;
  a.m = (int)across;
  a.n = (int)along;
  (void)hipGetLastError();
  return done(launch_product_weights(a, dw->dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t lapsum_beam_select_workspace_bytes(int64_t batch, int64_t beams, int64_t vocab, int32_t k) {
  return check_beams(LAPSUM_F32, batch, beams, vocab, k) == LAPSUM_OK ? beam_bytes(batch, beams, vocab) : 0;
}

lapsum_status lapsum_beam_select(const void *logits, int32_t dtype, int64_t batch, int64_t beams, int64_t vocab,
                                 int64_t row_stride, const float *scores, const uint8_t *ended, int32_t end_token,
                                 int32_t k, float *scores_out, int32_t *parents, int32_t *tokens, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  lapsum_status st = check_beams(dtype, batch, beams, vocab, k);
  if (st != LAPSUM_OK) return st;
  if (row_stride < vocab) return LAPSUM_ERR_LAYOUT;
  if (ended && (end_token < 0 || end_token >= vocab)) return LAPSUM_ERR_OPTION;
  if (!logits || !scores || !scores_out || !parents || !tokens) return LAPSUM_ERR_NULL;
  const size_t need = beam_bytes(batch, beams, vocab);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != LAPSUM_OK) return st;
  // one search is read when another is written
  const int64_t rows = batch * beams, places = batch * k * 4;
  const Block written[] = {{scores_out, places}, {parents, places}, {tokens, places}, {workspace, (int64_t)need}};
  const Block read[] = {{scores, rows * 4}, {ended, rows}};
  if (any_meet(written, read)) return LAPSUM_ERR_LAYOUT;
  const __int128 step = (__int128)row_stride * type_bytes(dtype), most = (__int128)1 << 62;
  const Layout x{logits, vocab * type_bytes(dtype), rows > 1, {{(int64_t)(step < most ? step : most), rows}}};
  for (const Block &b : written)
    if (meet(x, b)) return LAPSUM_ERR_LAYOUT;
  BeamArgs a{};
  a.logits = logits;
  a.batch = batch;
  a.stride = row_stride;
  a.beams = (int)beams;
  a.vocab = (int)vocab;
  a.k = k;
  beam_parts(beams, vocab, a.chunk, a.chunks);
  a.scores = scores;
  a.ended = ended;
  a.end_token = end_token;
  a.scores_out = scores_out;
  a.parents = parents;
  a.tokens = tokens;
  a.chunk_magic = (((uint64_t)1 << 32) + (uint64_t)a.chunks - 1) / (uint64_t)a.chunks;
  a.tops = static_cast<float *>(workspace);
  a.sums = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + beam_tops_bytes(batch * beams, a.chunks));
  (void)hipGetLastError();
  return done(launch_beam_select(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

lapsum_status lapsum_cache_reorder(const lapsum_cache *cache, int64_t beams, const int32_t *parents,
                                   const int32_t *lengths, float *account, int32_t *positions, int32_t *lengths_out,
                                   void *stream) {
  lapsum_status st = check_cache(cache);
  if (st != LAPSUM_OK) return st;
  if (beams < 1 || beams > LAPSUM_MAX_BEAMS || cache->batch % beams != 0) return LAPSUM_ERR_SHAPE;
  // entries are written: no two of them may share memory
  if (!apart(*cache, cache->k_stride_batch, cache->k_stride_head, cache->k_stride_entry) ||
      !apart(*cache, cache->v_stride_batch, cache->v_stride_head, cache->v_stride_entry))
    return LAPSUM_ERR_LAYOUT;
  if (!parents || !lengths || !lengths_out) return LAPSUM_ERR_NULL;
  st = check_cache_pointers(cache);
  if (st != LAPSUM_OK) return st;
  ReorderArgs a{};
  // keys that are the values as well move once
  a.one = cache->k == cache->v && same_strides(*cache);
  if (!a.one && keys_meet_values(*cache)) return LAPSUM_ERR_LAYOUT;
  // one workgroup writes when another still reads
  const int64_t per_cache = cache->batch * 4;
  const __int128 entries = (__int128)cache->batch * cache->heads * cache->capacity * 4, most = (__int128)1 << 62;
  const int64_t per_entry = (int64_t)(entries < most ? entries : most);
  const Block written[] = {{lengths_out, per_cache}, {account, per_entry}, {positions, per_entry}};
  const Block read[] = {{lengths, per_cache}, {parents, per_cache}};
  if (any_meet(written, read)) return LAPSUM_ERR_LAYOUT;
  const Layout k = side_of(*cache, cache->k, cache->k_stride_batch, cache->k_stride_head, cache->k_stride_entry);
  const Layout v = side_of(*cache, cache->v, cache->v_stride_batch, cache->v_stride_head, cache->v_stride_entry);
  for (const Block &b : {written[0], written[1], written[2], read[0], read[1]})
    if (meet(k, b) || meet(v, b)) return LAPSUM_ERR_LAYOUT;
  a.k = cache->k;
  a.v = cache->v;
  a.kb = cache->k_stride_batch;
  a.kh = cache->k_stride_head;
  a.ke = cache->k_stride_entry;
  a.vb = cache->v_stride_batch;
  a.vh = cache->v_stride_head;
  a.ve = cache->v_stride_entry;
  a.searches = cache->batch / beams;
  a.heads = cache->heads;
  a.capacity = cache->capacity;
  a.beams = (int)beams;
  a.width = cache->width;
  a.parents = parents;
  a.lengths = lengths;
  a.account = account;
  a.positions = positions;
  a.lengths_out = lengths_out;
  (void)hipGetLastError();
  return done(launch_reorder(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
