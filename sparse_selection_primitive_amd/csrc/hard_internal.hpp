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

}  // namespace lapsum
