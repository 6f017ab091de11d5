// Internal interface between the host runtime of the hard selections
// (hard_api.cpp) and their kernel files.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lapsum.h"
#include "lapsum_internal.hpp"

namespace lapsum {

// route.hip
struct RouteArgs {
  const void *logits;
  int64_t tokens, stride;  // row stride of the logits, elements
  int experts;
  const float *bias;       // [experts] or NULL
  int k, score, groups, top_groups, group_size, renormalise;
  float scale;
  uint32_t group_magic;    // ceil(2^21 / group_size): expert / group_size = expert * magic >> 21
  float *weights;          // [tokens][k]
  int32_t *chosen;         // [tokens][k]
  const float *dweights;   // backward: [tokens][k]
  void *dlogits;           // backward: [tokens][experts]
};
hipError_t launch_route_forward(const RouteArgs &a, int dtype, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs &a, int dtype, hipStream_t s);

// dispatch.hip
constexpr int kPlanTile = 1024;  // pairs per workgroup of the plan's count and place launches
int64_t plan_tiles(int64_t pairs);
hipError_t launch_dispatch_plan(const int32_t *chosen, int64_t pairs, int experts, int32_t *offsets, int32_t *slot,
                                int32_t *order, uint32_t *counts, hipStream_t s);

struct RowsArgs {
  const void *src;         // dispatch: x; sums: the expert-ordered rows
  const void *dy;          // combine backward: the tokens' gradient
  void *dst;
  int64_t tokens, stride;  // stride: elements between the token rows that are read
  int64_t pairs;           // tokens * k
  int k;
  int64_t width;
  const int32_t *slot;     // [tokens][k]
  const int32_t *placed;   // device scalar: number of pairs that have a row
  const float *weights;    // [tokens][k] or NULL (all 1)
  float *dweights;         // combine backward: [tokens][k]
};
hipError_t launch_dispatch_rows(const RowsArgs &a, int dtype, hipStream_t s);
hipError_t launch_sum_rows(const RowsArgs &a, int dtype, hipStream_t s);
hipError_t launch_combine_backward(const RowsArgs &a, int dtype, hipStream_t s);

// attend.hip
struct AttendArgs {
  const void *q, *k, *v;
  int64_t kb, kh, ke, vb, vh, ve;  // strides of batch, head, entry (elements)
  int batch, heads, news, group;   // group: query heads per key head
  int rows;                        // news * group
  uint32_t group_magic;            // ceil(2^32 / group) for group > 1: row / group is its product's upper word
  int width;
  int64_t capacity;
  const int32_t *lengths;
  float scale_log2;                // scale * log2(e)
  int splits;                      // workgroups a cache is shared by; 0: one does it all, without a workspace
  const float *account;
  float *account_out;              // NULL: no accounts
  void *out;
  float *part_o;                   // [batch * heads][splits][rows][width]
  float *part_ml;                  // [batch * heads][splits][rows][2]
  float *logits;                   // [batch * heads][blocks][rows][32], or NULL: formed again
  int64_t blocks;                  // of 32 entries
  int *dropped;                    // [batch * heads][splits]: infinities or NaN left out, where that can be
};
struct AttendPlan {
  int splits;
  bool keep_logits;
  int64_t blocks;
  size_t part_o, part_ml, dropped, logits;  // bytes
};
AttendPlan attend_plan(int64_t batch, int64_t heads, int64_t capacity, int64_t rows, bool one, int width,
                       bool accounts);
hipError_t launch_attend(const AttendArgs &a, int dtype, hipStream_t s);

// evict.hip
struct EvictArgs {
  void *k, *v;
  int64_t kb, kh, ke, vb, vh, ve;
  int64_t batch, heads, capacity, keep;
  int entry_bytes;                 // width * element size, a multiple of 16
  const float *account;
  const int32_t *positions, *lengths, *next_position;
  int32_t sinks, recent;
  float *account_out;
  int32_t *positions_out, *kept, *lengths_out;
  void *workspace;
};
size_t evict_workspace(int64_t batch, int64_t heads, int64_t capacity, int64_t keep);
hipError_t launch_evict(const EvictArgs &a, hipStream_t s);


// product.hip: C = A B for every expert, of its own rows.  An element of A is at m * am + k * ak,
// of B at e * be + k * bk + n * bn, of C at m * cm + n, where rows are counted through all experts.
struct ProductArgs {
  const void *a, *b;
  void *c;
  int64_t am, ak, be, bk, bn, ce, cm;
  int64_t rows;             // of all experts and none
  int m, n, k;              // sizes; the one that the rows take the place of is not used
  int experts;
  const int32_t *offsets;   // [experts + 1]
};
hipError_t launch_product_rows(const ProductArgs &a, int dtype, hipStream_t s);     // the rows are m: ys, dxs
hipError_t launch_product_weights(const ProductArgs &a, int dtype, hipStream_t s);  // the rows are k: dw

// beams.hip
struct BeamArgs {
  const void *logits;
  int64_t batch, stride;
  int beams, vocab, k;
  int chunk, chunks;        // tokens of a part, parts of a row
  const float *scores;
  const uint8_t *ended;     // or NULL
  int end_token;
  float *scores_out;
  int32_t *parents, *tokens;
  uint64_t chunk_magic;     // ceil(2^32 / chunks): i / chunks = i * magic >> 32 for all parts of a search
  float *tops;              // [batch * beams][chunks]: maximum of a part
  float2 *sums;             // [batch * beams][groups]: maximum and sum of e^(x - maximum) of kBeamGroup parts
};
constexpr int kBeamGroup = 16;
void beam_parts(int64_t beams, int64_t vocab, int &chunk, int &chunks);
hipError_t launch_beam_select(const BeamArgs &a, int dtype, hipStream_t s);

// reorder.hip
struct ReorderArgs {
  void *k, *v;
  int64_t kb, kh, ke, vb, vh, ve;
  int64_t searches, heads, capacity;
  int beams, width;
  bool one;                 // v is k
  const int32_t *parents, *lengths;
  float *account;           // or NULL
  int32_t *positions;       // or NULL
  int32_t *lengths_out;
};
hipError_t launch_reorder(const ReorderArgs &a, hipStream_t s);

}  // namespace lapsum
