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

lapsum_status check_attend(const lapsum_cache *c, int64_t news, int64_t q_heads) {
  const lapsum_status st = check_cache(c);
  if (st != LAPSUM_OK) return st;
  if (news < 1 || news > 65536 || q_heads < c->heads || q_heads % c->heads != 0) return LAPSUM_ERR_SHAPE;
  if (q_heads / c->heads > 65536 / news) return LAPSUM_ERR_SHAPE;
  return LAPSUM_OK;
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

}  // extern "C"
