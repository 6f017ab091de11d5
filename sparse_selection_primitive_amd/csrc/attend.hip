// Attention of the newest tokens over a cache, with the account of the weight
// that each entry received.
//
// Mathematics.  Per key head, the `rows` = news * group query rows see the
// entries 0 .. limit(row); z = scale q.k (kept in units of log2), and with the
// running maximum m and sum l of a row one pass over the entries gives
//     out = sum_s 2^(z_s - m) v_s / l,   l = sum_s 2^(z_s - m);
// parts of the cache are joined by m and l.  The account needs the weights
// 2^(z_s - lse), lse = m + log2 l of the whole cache, so it can only be added
// up after the join: for few rows the z of the first pass are kept (4 bytes
// a row and entry, little beside the entry's keys and values), for many rows they
// are formed again from the keys.
//
// Layout.  A wave takes 32 entries at a time, straight from memory into
// registers.  Z' = K Q' by mfma_f32_16x16x32 has the entries as rows, so a
// lane gets 4 entries of one query row and hands them on as the other
// factor of O' = V' P' without moving anything between lanes: the sum over entries
// may take them in any order, so lane group c's eight places of that product are
// its entries 4c..4c+3 and 16+4c..16+4c+3.  For V' a lane needs one element of eight
// entries: it loads the width/16 contiguous elements of each of its entries
// (16 lanes read whole rows) and transposes them in registers.
//
// What bounds it.  A few rows: memory.  Without accounts 200001 entries of 8
// key heads (819 MB) take 137 us with the join, 6.0 TB/s, where a kernel that only reads reaches 6.2; the
// kept logits add 52 MB of writes, which among the reads cost as much as 200 MB of them (a copy of the
// access pattern without arithmetic shows the same), 165 us and 16 us for the
// join.  Many rows: one wave a SIMD, whose vector instructions (46% of its time), matrix
// instructions (33%; 16 cycles for 16 rows, 32 entries and 32 elements) and waits for memory (22%) follow one
// another: 128 rows over 16384 entries of 16 key heads take 50 us (34.4 Gflop with the three parts
// of the weights, 680 Tflop/s) and 27 us for the accounts.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 32;       // entries a wave takes at a time
constexpr int kAttendWaves = 4;  // waves of a workgroup, taking its blocks in turn
constexpr int kStep = kBlock * kAttendWaves;
// Weights are formed against a base kLift powers of two below the maximum that set it, and may
// grow by kSlack more before it moves.  2^15 is an fp16 number, and its smallest weight that is not
// 0 is then 2^-31 of the largest: many entries of little weight beside one of much keep theirs.
constexpr float kLift = 7.0f, kSlack = 8.0f;
// A weight goes into the matrix product as the sum of this many numbers of the cache's type, each the rounding
// of what the ones before leave: three of bf16's 8 bits, or two of fp16's 11, are all 24 bits of an fp32 number.
// With two parts of bf16, 16 bits, outputs that cancel were off by 2^-17.6 of sum p |v| where 24 give 2^-21;
// the third part costs nothing up to 32 rows, where memory is the bound, and of the time of
// 64 rows over two sequences of 16384 entries 9% (43.0 us for 39.6), of 128 rows 1 to 4% (52.6 for 52.2, 54.8 for 52.7).
template <class T>
constexpr int kParts = sizeof(T) == 2 && (float)(T)65536.0f == 65536.0f ? 3 : 2;
constexpr int kMaxSplits = 256;
// A cache goes to one workgroup whole where that is one block a wave, or where
// there are enough caches for every compute unit (times of one call from a graph, 32 query
// heads on 8 of width 128: 200 entries 7.7 us, by splits 9.0; 1000 entries 14.5 and 9.2; 32
// sequences of 500 to 1000 20.7 and 28.5; 64 of 2000 to 4000 137 and 169).  By the capacity, which the host
// knows, not the lengths: 1000 entries in a cache for 131072 take 10.6 us.
constexpr int kWholeShort = 256, kWholeMax = 4096;
constexpr int kWholeCaches = 256;
constexpr int kWholeLogits = 16384;  // fp32 logits that it keeps in LDS, at most
// Up to this many rows the logits are kept for the accounts; beyond they are formed again from the
// keys (4 rows of 64 sequences of 8192 entries: kept 426 us, formed again 507;
// 16 rows of 20000 entries: 27.3 and 35.9; more rows keep more than the keys' bytes).
constexpr int kKeepRows = 16;

LDEV f32x4 mfma(pack_t<bf16> a, pack_t<bf16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
LDEV f32x4 mfma(pack_t<f16> a, pack_t<f16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

LDEV float exp2_of(float z, float m) { return m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(z - m); }

// over the four lane groups of a wave (lanes l, l^16, l^32, l^48)
LDEV float groups_max(float v) {
  v = fmaxf(v, pair_lane<16>(v));
  return fmaxf(v, pair_lane<32>(v));
}
LDEV float groups_sum(float v) {
  v += pair_lane<16>(v);
  return v + pair_lane<32>(v);
}

LDEV int length_of(const AttendArgs &a, int64_t bh) {
  const int64_t n = a.lengths[bh / a.heads];
  return (int)(n < 0 ? 0 : (n > a.capacity ? a.capacity : n));
}
// entries [begin, end) of a split: equal shares of the cache's own length, in whole steps
LDEV void split_range(const AttendArgs &a, int length, int split, int &begin, int &end) {
  const int share = ((length + a.splits - 1) / a.splits + kStep - 1) / kStep * kStep;
  const int64_t b = (int64_t)split * share;
  begin = (int)(b < length ? b : length);
  end = (int)(b + share < length ? b + share : length);
}

template <class T>
LDEV const T *query_row(const AttendArgs &a, int64_t bh, int row) {
  const int64_t b = bh / a.heads, h = bh % a.heads;
  const int i = row / a.group, g = row % a.group;
  return static_cast<const T *>(a.q) + ((b * a.news + i) * ((int64_t)a.heads * a.group) + h * a.group + g) * a.width;
}

// The first row that sees entry e (they are in the order of their tokens).  The accounts leave out
// those before it rather than add their weights of 0: a row of NaN has an lse of NaN, and
// -inf - NaN would reach entries that it does not see.
LDEV int first_row(const AttendArgs &a, int length, int e) {
  const int i = e - (length - a.news);
  return i > 0 ? i * a.group : 0;
}

// this lane's part of 16 query rows (second factor of Z'): row lane % 16, zero past the rows and the width
template <class T, int DP>
LDEV void load_queries(const AttendArgs &a, int64_t bh, int row, pack_t<T> (&q)[DP / 32]) {
  const int c = (threadIdx.x % 64) / 16;
  const T *p = query_row<T>(a, bh, row < a.rows ? row : 0);
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) {
    const int d = i * 32 + c * 8;
    const bool there = row < a.rows && d < a.width;
    const uint4 w = *reinterpret_cast<const uint4 *>(p + (there ? d : 0));
    q[i] = __builtin_bit_cast(pack_t<T>, there ? w : uint4{0, 0, 0, 0});
  }
}

// A window of memory that buffer accesses are held to: what lies past its end
// reads as zero and is not written.  Entries are reached through a window that starts at the
// block's first one, so a load's address is the window (scalar registers) and a 32-bit
// offset of the lane that stays the same from block to block.  All of the
// offset is the lane's: an instruction's scalar offset need not count in the check.
using window_t = __amdgpu_buffer_rsrc_t;
LDEV window_t window_of(const void *first, int64_t bytes) {
  const int64_t most = 0x7FFFFFF0;
  bytes = bytes < 0 ? 0 : (bytes < most ? bytes : most);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(first), 0, (int)bytes, 0x00020000);  // 32-bit format
}
constexpr uint32_t kNowhere = 0x80000000u;  // a lane's offset past every window

// Values are read as streamed (not kept in the cache): 200001 entries in 137
// us instead of 146.  Keys are not: a load touches 16 rows' half lines, and without the
// cache the other halves are fetched again.
constexpr int kCached = 0, kStreamed = 2;
template <int AUX>
LDEV uint4 load_16(window_t w, uint32_t offset) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(w, (int)offset, 0, AUX));
}
template <int AUX>
LDEV uint2 load_8(window_t w, uint32_t offset) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(w, (int)offset, 0, AUX));
}

LDEV void store_16(window_t w, uint32_t offset, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), w, (int)offset, 0, 0);
}

// the entries [first, end) of keys or values; none where first >= end
template <class T>
LDEV window_t entries(const T *base, int64_t stride, int first, int end, int width) {
  const int64_t bytes = ((int64_t)(end - 1 - first) * stride + width) * (int64_t)sizeof(T);
  return window_of(base + (int64_t)first * stride, first < end ? bytes : 0);
}

// This lane's part of 16 keys (first factor of Z'): entry lane % 16 of the
// window's `at`-th entry and on.
template <class T, int DP, bool EXACT>
struct Keys {
  static constexpr int kSteps = DP / 32;
  uint32_t off[EXACT ? 1 : kSteps];
  int stride;  // bytes
  LDEV explicit Keys(const AttendArgs &a) {
    const int lane = threadIdx.x % 64;
    stride = (int)a.ke * 2;
    const uint32_t o = (uint32_t)((lane % 16) * stride + (lane / 16) * 16);
    if constexpr (EXACT) {
      off[0] = o;
    } else {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) off[i] = i * 32 + (lane / 16) * 8 < a.width ? o : kNowhere;
    }
  }
  LDEV void load(window_t w, int at, pack_t<T> (&k)[kSteps]) const {
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      k[i] = __builtin_bit_cast(pack_t<T>, load_16<kCached>(w, off[EXACT ? 0 : i] + (uint32_t)(at * stride) + i * 64));
  }
};

// the place-th entry of this lane's eight in a block
LDEV int entry_of(int place) {
  const int c = (threadIdx.x % 64) / 16;
  return (place / 4) * 16 + c * 4 + place % 4;
}

template <class T, int DP, int AUX>
struct Values {
  static constexpr int W = DP / 16;  // elements per lane and entry
  typedef T vec __attribute__((ext_vector_type(DP / 16)));
  vec v[8];
  // off: this lane's offset in a window (value_offset)
  LDEV void load(window_t w, uint32_t off, int stride) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t at = off + (uint32_t)(((j / 4) * 16 + j % 4) * stride);
      if constexpr (W == 4) {
        v[j] = __builtin_bit_cast(vec, load_8<AUX>(w, at));
      } else if constexpr (W == 8) {
        v[j] = __builtin_bit_cast(vec, load_16<AUX>(w, at));
      } else {
        struct Two {
          uint4 x, y;
        } two = {load_16<AUX>(w, at), load_16<AUX>(w, at + 16)};
        v[j] = __builtin_bit_cast(vec, two);
      }
    }
  }
  // sets infinities and NaN to zero (by their exponents, on the packed words); whether there were any
  LDEV bool drop() {
    constexpr uint32_t kExponent = (float)(T)65536.0f == 65536.0f ? 0x7F80u : 0x7C00u;  // bf16, fp16
    typedef uint32_t words __attribute__((ext_vector_type(W / 2)));
    bool any = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      words x = __builtin_bit_cast(words, v[j]);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const bool low = (x[i] & kExponent) == kExponent, high = ((x[i] >> 16) & kExponent) == kExponent;
        any |= low || high;
        x[i] &= (low ? 0xFFFF0000u : 0xFFFFFFFFu) & (high ? 0x0000FFFFu : 0xFFFFFFFFu);
      }
      v[j] = __builtin_bit_cast(vec, x);
    }
    return any;
  }
  static LDEV uint32_t value_offset(const AttendArgs &a) {
    const int lane = threadIdx.x % 64, d = (lane % 16) * W;
    return d < a.width ? (uint32_t)((lane / 16) * 4 * (int)a.ve * 2 + d * 2) : kNowhere;
  }
  LDEV pack_t<T> column(int n) const {
    pack_t<T> w;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = v[j][n];
    return w;
  }
};

// What becomes of a block's logits: kept in the workspace for the accounts, kept in
// LDS, or dropped.
struct KeepNone {
  LDEV void operator()(int, int, f32x4, f32x4) const {}
};
struct KeepFar {  // [blocks][rows][32]
  float *logits;
  int rows, row;  // row: this lane's of the first tile
  // rows past the last one go nowhere; no branch, so the waits for the loads stay exact
  LDEV void operator()(int e0, int t, f32x4 z0, f32x4 z1) const {
    const window_t to = window_of(logits + (int64_t)(e0 / kBlock) * rows * kBlock,
                                  (int64_t)rows * kBlock * (int64_t)sizeof(float));
    const int c = (threadIdx.x % 64) / 16, at = ((row + 16 * t) * kBlock + 4 * c) * (int)sizeof(float);
    store_16(to, (uint32_t)at, z0);
    store_16(to, (uint32_t)at + 64, z1);
  }
};
struct KeepNear {  // [rows][stride], one tile of rows
  float *logits;
  int rows, stride;
  LDEV void operator()(int e0, int, f32x4 z0, f32x4 z1) const {
    const int lane = threadIdx.x % 64, c = lane / 16, r = lane % 16;
    if (r >= rows) return;
    float *to = logits + r * stride + e0 + 4 * c;
    *reinterpret_cast<f32x4 *>(to) = z0;
    *reinterpret_cast<f32x4 *>(to + 16) = z1;
  }
};

// One wave's pass over the blocks first, first + stride, .. of the entries up to
// `end`, for 16 * NT rows from row0: the rows' bases (see kLift), their sums (this lane's
// share) and outputs.  Returns whether values were left out (see drop()).
template <class T, int DP, int NT, bool EXACT, bool ONE, int AUX, class Keep>
LDEV bool attend_entries(const AttendArgs &a, int64_t bh, int row0, int length, int first, int end, int stride,
                         const Keep keep, float (&m)[NT], float (&l)[NT], f32x4 (&o)[NT][DP / 16]) {
  constexpr int W = DP / 16;
  const int lane = threadIdx.x % 64, c = lane / 16, r = lane % 16;
  const int64_t b = bh / a.heads, h = bh % a.heads;
  const T *keys = static_cast<const T *>(a.k) + b * a.kb + h * a.kh;
  const T *values = static_cast<const T *>(a.v) + b * a.vb + h * a.vh;

  // a block's keys are asked for as soon as the last block's are used up, its
  // values likewise, so each is on its way while the other is worked on (past the
  // last block from an empty window: a branch here would make the compiler
  // wait for the keys where only the values are needed)
  const Keys<T, DP, EXACT> key(a);
  Values<T, DP, AUX> v;
  const uint32_t value_off = decltype(v)::value_offset(a);
  pack_t<T> k[2][DP / 32];
  pack_t<T> q[NT][DP / 32];
  int limit[NT];  // the last entry this lane's row sees
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + 16 * t + r;
    load_queries<T, DP>(a, bh, row, q[t]);
    limit[t] = length - a.news + row / a.group;
  }
  // the order of the loads is the loop's: keys before values
  __builtin_amdgcn_sched_barrier(0);
  {
    const window_t w = entries(keys, a.ke, first, end, a.width);
    key.load(w, 0, k[0]);
    key.load(w, 16, k[1]);
  }
  __builtin_amdgcn_sched_barrier(0);
  v.load(entries(values, a.ve, first, end, a.width), value_off, (int)a.ve * 2);
  __builtin_amdgcn_sched_barrier(0);

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.0f;
#pragma unroll
    for (int n = 0; n < W; ++n) o[t][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  bool dropped = false;
  for (int e0 = first; e0 < end; e0 += stride) {
    f32x4 z[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      z[t][0] = z[t][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        z[t][0] = mfma(k[0][i], q[t][i], z[t][0]);
        z[t][1] = mfma(k[1][i], q[t][i], z[t][1]);
      }
    }
    const window_t next_keys = entries(keys, a.ke, e0 + stride, end, a.width);
    key.load(next_keys, 0, k[0]);
    key.load(next_keys, 16, k[1]);
    // some row does not see some entry of the block
    const bool edge = e0 + kBlock > end || e0 + kBlock - 1 > length - a.news;
    pack_t<T> part[NT][kParts<T>];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[t][u][i] *= a.scale_log2;
        }
      }
      if (edge) {
        const int most = min(limit[t], end - 1) - e0 - 4 * c;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * u + i > most) z[t][u][i] = -INFINITY;
        }
      }
      keep(e0, t, z[t][0], z[t][1]);
      float top = fmaxf(fmaxf(fmaxf(z[t][0][0], z[t][0][1]), fmaxf(z[t][0][2], z[t][0][3])),
                        fmaxf(fmaxf(z[t][1][0], z[t][1][1]), fmaxf(z[t][1][2], z[t][1][3])));
      // A maximum that grows a little moves nothing: the first blocks would otherwise
      // rescale the outputs nearly every time.
      if (__any(top > m[t] + (kLift + kSlack))) {
        const float next = fmaxf(m[t], groups_max(top) - kLift);
        const float f = exp2_of(m[t], next);
        l[t] *= f;
#pragma unroll
        for (int n = 0; n < W; ++n) o[t][n] *= f;
        m[t] = next;
      }
      const float base = m[t] == -INFINITY ? 0.0f : m[t];
      f32x8 p;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(z[t][i / 4][i % 4] - base);
      }
      // the block's weights among themselves first: many small ones would each round away in a large sum
      l[t] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
      for (int i = 0; i < kParts<T>; ++i) {
        part[t][i] = __builtin_convertvector(p, pack_t<T>);
        p -= __builtin_convertvector(part[t][i], f32x8);
      }
    }
    // NaN or infinity among values that some row does not see must not meet
    // that row's zero weights: they are left out here and added by the join
    if (!ONE && edge) dropped |= v.drop();
#pragma unroll
    for (int n = 0; n < W; ++n) {
      const pack_t<T> col = v.column(n);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < kParts<T>; ++i) o[t][n] = mfma(col, part[t][i], o[t][n]);
      }
    }
    v.load(entries(values, a.ve, e0 + stride, end, a.width), value_off, (int)a.ve * 2);
  }
  return dropped;
}

// The waves of a workgroup share its entries (BY_ROWS false: few rows, so the
// entries' bytes are what counts; a wave takes every fourth block and the
// waves are joined at the end) or its rows (BY_ROWS: every wave goes through
// all the entries for rows of its own, and what one wave loads the others find in
// the cache of their compute unit).
template <class T, int DP, int NT, bool EXACT, bool BY_ROWS, bool ONE, bool KEEP>
__global__ __launch_bounds__(64 * kAttendWaves, DP <= 128 ? 2 : 1) void attend_kernel(const AttendArgs a) {
  constexpr int W = DP / 16;
  constexpr int kRows = 16 * NT;
  constexpr int kPad = DP + 4;  // floats per row in LDS: 16 rows' 16-byte accesses fall on all banks
  struct Shared {
    float m[kAttendWaves][kRows], l[kAttendWaves][kRows];
    int dropped[kAttendWaves];
    float o[BY_ROWS ? 1 : kAttendWaves][BY_ROWS ? 1 : kRows][BY_ROWS ? 4 : kPad];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64, c = lane / 16, r = lane % 16;
  const int split = blockIdx.x % a.splits;
  const int row0 = (int)(blockIdx.x / a.splits) * kRows * (BY_ROWS ? kAttendWaves : 1) + (BY_ROWS ? wave * kRows : 0);
  if (BY_ROWS && row0 >= a.rows) return;  // no barrier follows on that path
  const int length = length_of(a, bh);
  int begin, end;
  split_range(a, length, split, begin, end);
  float *ml = a.part_ml + ((bh * a.splits + split) * a.rows + row0) * 2;
  const int rows_here = min(a.rows - row0, kRows);
  if (begin >= end) {  // the same for the whole workgroup
    for (int i = BY_ROWS ? lane : threadIdx.x; i < rows_here; i += BY_ROWS ? 64 : blockDim.x) {
      ml[2 * i] = -INFINITY;
      ml[2 * i + 1] = 0.0f;
    }
    if (!ONE && threadIdx.x == 0) a.dropped[bh * a.splits + split] = 0;
    return;
  }
  constexpr int kStride = BY_ROWS ? kBlock : kStep;
  const int first = begin + (BY_ROWS ? 0 : wave * kBlock);
  // values that no other wave reads are streamed
  constexpr int AUX = BY_ROWS ? kCached : kStreamed;
  float m[NT], l[NT];
  f32x4 o[NT][W];
  bool dropped;
  if constexpr (KEEP) {
    const KeepFar keep{a.logits + bh * a.blocks * a.rows * kBlock, a.rows, row0 + r};
    dropped = attend_entries<T, DP, NT, EXACT, ONE, AUX>(a, bh, row0, length, first, end, kStride, keep, m, l, o);
  } else {
    dropped = attend_entries<T, DP, NT, EXACT, ONE, AUX>(a, bh, row0, length, first, end, kStride, KeepNone(), m, l, o);
  }

  int *const flag = a.dropped + bh * a.splits + split;
  if constexpr (!ONE && BY_ROWS) {  // every wave has seen the same values
    const bool any = __any(dropped);
    if (lane == 0) *flag = any ? 1 : 0;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) l[t] = groups_sum(l[t]);
  float *part = a.part_o + ((bh * a.splits + split) * a.rows + row0) * a.width;
  if constexpr (BY_ROWS) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = 16 * t + r;
      if (row >= rows_here) continue;
      if (c == 0) {
        ml[2 * row] = m[t];
        ml[2 * row + 1] = l[t];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int n = 0; n < W; n += 4) {
          const int d = (4 * c + i) * W + n;
          if (EXACT || d < a.width)
            *reinterpret_cast<f32x4 *>(part + (int64_t)row * a.width + d) =
                f32x4{o[t][n][i], o[t][n + 1][i], o[t][n + 2][i], o[t][n + 3][i]};
        }
      }
    }
    return;
  }
  // join the waves: a common maximum, then their sums in the waves' order
  if constexpr (!ONE) sh.dropped[wave] = __any(dropped) ? 1 : 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (c == 0) {
      sh.m[wave][16 * t + r] = m[t];
      sh.l[wave][16 * t + r] = l[t];
    }
  }
  __syncthreads();
  if (!ONE && threadIdx.x == 0) *flag = sh.dropped[0] | sh.dropped[1] | sh.dropped[2] | sh.dropped[3];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float all = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttendWaves; ++w) all = fmaxf(all, sh.m[w][16 * t + r]);
    const float f = exp2_of(m[t], all);
    if (wave == 0 && c == 0 && 16 * t + r < rows_here) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttendWaves; ++w) sum += exp2_of(sh.m[w][16 * t + r], all) * sh.l[w][16 * t + r];
      ml[2 * (16 * t + r)] = all;
      ml[2 * (16 * t + r) + 1] = sum;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int n = 0; n < W; n += 4)
        *reinterpret_cast<f32x4 *>(&sh.o[wave][16 * t + r][(4 * c + i) * W + n]) =
            f32x4{o[t][n][i] * f, o[t][n + 1][i] * f, o[t][n + 2][i] * f, o[t][n + 3][i] * f};
    }
  }
  __syncthreads();
  const int packs = a.width / 4;  // the width is a multiple of 8
  for (int i = threadIdx.x; i < rows_here * packs; i += blockDim.x) {
    const int row = i / packs, d = (i % packs) * 4;
    f32x4 sum = *reinterpret_cast<const f32x4 *>(&sh.o[0][row][d]);
#pragma unroll
    for (int w = 1; w < kAttendWaves; ++w) sum += *reinterpret_cast<const f32x4 *>(&sh.o[w][row][d]);
    *reinterpret_cast<f32x4 *>(part + (int64_t)row * a.width + d) = sum;
  }
}

// Infinities and NaN among the values of the newest entries that the products
// left out, added to four elements of a row's output (one that they did not leave out is in
// the sum already, and stays).
template <class T>
LDEV void add_dropped(const AttendArgs &a, int64_t bh, int row, int length, int d, f32x4 &o) {
  const int64_t b = bh / a.heads, h = bh % a.heads;
  const T *v = static_cast<const T *>(a.v) + b * a.vb + h * a.vh + d;
  const int last = length - a.news + row / a.group;
  for (int e = max(0, length - a.news - kBlock); e <= last; ++e) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float x = (float)v[(int64_t)e * a.ve + n];
      if (!(fabsf(x) < INFINITY)) o[n] += x;
    }
  }
}

template <class T>
LDEV void store_out(const AttendArgs &a, int64_t bh, int row, int d, f32x4 o) {
  typedef T vec4 __attribute__((ext_vector_type(4)));
  T *out = const_cast<T *>(query_row<T>(a, bh, row) - static_cast<const T *>(a.q) + static_cast<T *>(a.out));
  *reinterpret_cast<vec4 *>(out + d) = vec4{(T)o[0], (T)o[1], (T)o[2], (T)o[3]};
}

// A short cache by one workgroup: its logits stay in LDS, so output and
// accounts are finished here, without a workspace and a second launch.
constexpr int whole_waves(int dp) { return dp <= 128 ? 8 : 4; }  // 8 waves have 256 registers each
template <class T, int DP, bool EXACT, bool ONE>
__global__ __launch_bounds__(64 * whole_waves(DP)) void attend_whole_kernel(const AttendArgs a, const int logit_stride) {
  constexpr int W = DP / 16, WAVES = whole_waves(DP), kPad = DP + 4;
  struct Shared {
    float m[WAVES][16], l[WAVES][16];
    float lse[16], inv[16];
    int dropped[WAVES];
    float o[4][16][kPad];
  };
  __shared__ Shared sh;
  extern __shared__ float logits[];  // [rows][logit_stride], where there are accounts
  lds_poison(sh);
  if (a.account_out != nullptr) lds_poison(logits, a.rows * logit_stride * (int)sizeof(float));
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64, c = lane / 16, r = lane % 16;
  const int length = length_of(a, bh);

  float m[1], l[1];
  f32x4 o[1][W];
  bool dropped;
  if (a.account_out != nullptr) {
    dropped = attend_entries<T, DP, 1, EXACT, ONE, kStreamed>(a, bh, 0, length, wave * kBlock, length, WAVES * kBlock,
                                                              KeepNear{logits, a.rows, logit_stride}, m, l, o);
  } else {
    dropped = attend_entries<T, DP, 1, EXACT, ONE, kStreamed>(a, bh, 0, length, wave * kBlock, length, WAVES * kBlock,
                                                              KeepNone(), m, l, o);
  }
  l[0] = groups_sum(l[0]);
  if (c == 0) {
    sh.m[wave][r] = m[0];
    sh.l[wave][r] = l[0];
  }
  if constexpr (!ONE) sh.dropped[wave] = __any(dropped) ? 1 : 0;
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sh.m[w][r]);
#pragma unroll
  for (int w = 0; w < WAVES; ++w) sum += exp2_of(sh.m[w][r], top) * sh.l[w][r];
  if (wave == 0 && c == 0) {
    sh.lse[r] = sum > 0.0f ? top + log2f(sum) : (sum == 0.0f ? INFINITY : sum);
    sh.inv[r] = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  const float f = exp2_of(m[0], top);
#pragma unroll
  for (int n = 0; n < W; ++n) o[0][n] *= f;
  // the waves' outputs in four buffers, the upper half's handed to the lower half's waves first
  const auto each = [&](auto use) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int n = 0; n < W; n += 4)
        use(*reinterpret_cast<f32x4 *>(&sh.o[wave & 3][r][(4 * c + i) * W + n]), n, i);
    }
  };
  const auto put = [&](f32x4 &at, int n, int i) {
    at = f32x4{o[0][n][i], o[0][n + 1][i], o[0][n + 2][i], o[0][n + 3][i]};
  };
  if constexpr (WAVES > 4) {
    if (wave >= 4) each(put);
    __syncthreads();
    if (wave < 4) {
      each([&](f32x4 &at, int n, int i) {
#pragma unroll
        for (int x = 0; x < 4; ++x) o[0][n + x][i] += at[x];
      });
    }
    // a wave reads and writes the same places, so no barrier in between
  }
  if (wave < 4) each(put);
  __syncthreads();
  bool again = false;
  if constexpr (!ONE) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) again |= sh.dropped[w] != 0;
  }
  const int packs = a.width / 4;
  for (int i = threadIdx.x; i < a.rows * packs; i += blockDim.x) {
    const int row = i / packs, d = (i % packs) * 4;
    f32x4 x = *reinterpret_cast<const f32x4 *>(&sh.o[0][row][d]);
#pragma unroll
    for (int w = 1; w < 4; ++w) x += *reinterpret_cast<const f32x4 *>(&sh.o[w][row][d]);
    x *= sh.inv[row];
    if (again) add_dropped<T>(a, bh, row, length, d, x);
    store_out<T>(a, bh, row, d, x);
  }
  if (a.account_out == nullptr) return;
  for (int e = threadIdx.x; e < length; e += blockDim.x) {
    float w = 0.0f;
    const int from = ONE ? 0 : first_row(a, length, e);
    for (int i = 0; i < a.rows; ++i) {
      const float off = sh.lse[i];
      w += __builtin_amdgcn_exp2f(logits[i * logit_stride + e] - (i < from ? 0.0f : off));
    }
    a.account_out[bh * a.capacity + e] = a.account[bh * a.capacity + e] + w;
  }
}

// The splits' maxima and sums of a row as one, by a team of 16 lanes: its
// lse in units of log2 (+inf for a row that sees nothing, so its weights are 0).
LDEV float row_lse(const AttendArgs &a, int64_t bh, int row) {
  const int j = threadIdx.x % 16;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + bh * a.splits * a.rows + row;
  float top = -INFINITY, sum = 0.0f;
  for (int s = j; s < a.splits; s += 16) {
    const float2 x = ml[(int64_t)s * a.rows];
    const float next = fmaxf(top, x.x);
    sum = sum * exp2_of(top, next) + exp2_of(x.x, next) * x.y;
    top = next;
  }
  const float all = team_max<16>(top);
  sum = team_sum<16>(sum * exp2_of(top, all));
  return sum > 0.0f ? all + log2f(sum) : (sum == 0.0f ? INFINITY : sum);
}

// out of one row: its parts, each weighed by its maximum, summed over the splits
template <class T, int TH, bool ONE>
LDEV void join_row(const AttendArgs &a, int64_t bh, int row, float *lse) {
  struct Shared {
    float weight[TH];
    float top[TH / 64], sum[TH / 64];
    f32x4 o[TH];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int tid = threadIdx.x, wave = tid / 64;
  static_assert(kMaxSplits <= TH, "one split per thread");
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + bh * a.splits * a.rows + row;
  float2 x = {-INFINITY, 0.0f};
  if (tid < a.splits) x = ml[(int64_t)tid * a.rows];
  const bool again = !ONE && __syncthreads_or(tid < a.splits && a.dropped[bh * a.splits + tid] != 0) != 0;
  float top = team_max<64>(x.x);
  if (tid % 64 == 0) sh.top[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < TH / 64; ++w) top = fmaxf(top, sh.top[w]);
  const float f = exp2_of(x.x, top);
  sh.weight[tid] = f;
  const float part = team_sum<64>(f * x.y);
  if (tid % 64 == 0) sh.sum[wave] = part;
  __syncthreads();
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < TH / 64; ++w) sum += sh.sum[w];
  if (lse != nullptr && tid == 0)
    lse[bh * a.rows + row] = sum > 0.0f ? top + log2f(sum) : (sum == 0.0f ? INFINITY : sum);
  // a thread takes 4 elements of every n-th split
  const int packs = a.width / 4, teams = TH / packs, team = tid / packs, d = (tid % packs) * 4;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (team < teams) {
    const float *po = a.part_o + (bh * a.splits * a.rows + row) * a.width + d;
    const int64_t step = (int64_t)a.rows * a.width;
#pragma unroll 8
    for (int s = team; s < a.splits; s += teams) {
      const float w = sh.weight[s];
      if (w != 0.0f) o += w * *reinterpret_cast<const f32x4 *>(po + s * step);  // an empty split has no part
    }
  }
  sh.o[tid] = o;
  __syncthreads();
  if (team != 0) return;
  for (int t = 1; t < teams; ++t) o += sh.o[t * packs + tid];
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  o *= inv;
  if (again) add_dropped<T>(a, bh, row, length_of(a, bh), d, o);
  store_out<T>(a, bh, row, d, o);
}

template <int TH, bool ONE>
LDEV void add_kept(const AttendArgs &a, int64_t bh) {
  const int length = length_of(a, bh);
  const int base = ((int)blockIdx.x - a.rows) * (4 * TH);
  if (base >= length) return;
  struct Shared {
    float lse[kKeepRows];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int row = threadIdx.x / 16;  // a team of 16 lanes each
  if (row < a.rows) {
    const float x = row_lse(a, bh, row);
    if (threadIdx.x % 16 == 0) sh.lse[row] = x;
  }
  __syncthreads();
  const int e = base + 4 * (int)threadIdx.x;
  if (e >= length) return;
  f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
  const float *z = a.logits + (bh * a.blocks + e / kBlock) * a.rows * kBlock + e % kBlock;
  // Whether some row does not see some entry is asked for the wave as a whole, so it goes through the rows once
  // (2 sequences of 16384 entries, 4 new tokens: 35.4 us; by lane, so twice in one wave, 42.0).
  if (ONE || !__any(e + 3 > length - a.news)) {
#pragma unroll 4
    for (int i = 0; i < a.rows; ++i) {
      const f32x4 y = *reinterpret_cast<const f32x4 *>(z + i * kBlock);
#pragma unroll
      for (int n = 0; n < 4; ++n) w[n] += __builtin_amdgcn_exp2f(y[n] - sh.lse[i]);
    }
  } else {
    int from[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) from[n] = first_row(a, length, e + n);
#pragma unroll 4
    for (int i = 0; i < a.rows; ++i) {
      const f32x4 y = *reinterpret_cast<const f32x4 *>(z + i * kBlock);
      const float off = sh.lse[i];
#pragma unroll
      for (int n = 0; n < 4; ++n) w[n] += __builtin_amdgcn_exp2f(y[n] - (i < from[n] ? 0.0f : off));  // y is -inf before
    }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n)
    if (e + n < length) a.account_out[bh * a.capacity + e + n] = a.account[bh * a.capacity + e + n] + w[n];
}

// The first a.rows workgroups of a cache join its rows; the others (KEEP) add up the
// accounts of 4 entries a thread from the kept logits:
// account_out = account + sum over rows of 2^(z - lse).  ONE (nothing was left out, and every row
// sees every entry) and KEEP as in the attend_kernel before it, so that no case carries the
// other's code: with it the join of 64 rows took 8.8 us for 6.7.
template <class T, int TH, bool ONE, bool KEEP>
__global__ __launch_bounds__(TH) void attend_join_kernel(const AttendArgs a, float *lse) {
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  if ((int)blockIdx.x < a.rows) {
    join_row<T, TH, ONE>(a, bh, (int)blockIdx.x, lse);
    return;
  }
  if constexpr (KEEP) add_kept<TH, ONE>(a, bh);
}

// the same, z formed again: a wave takes 64 entries and goes through all rows
template <class T, int DP, bool EXACT>
__global__ __launch_bounds__(256) void account_formed_kernel(const AttendArgs a, const float *lse) {
  constexpr int KT = 4;
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  const int lane = threadIdx.x % 64, c = lane / 16, r = lane % 16;
  const int length = length_of(a, bh);
  const int e0 = (int)(blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64)) * 16 * KT;
  if (e0 >= length) return;
  const int64_t b = bh / a.heads, h = bh % a.heads;
  const T *keys = static_cast<const T *>(a.k) + b * a.kb + h * a.kh;
  const Keys<T, DP, EXACT> key(a);
  const window_t win = entries(keys, a.ke, e0, length, a.width);
  pack_t<T> k[KT][DP / 32];
  f32x4 w[KT];
#pragma unroll
  for (int u = 0; u < KT; ++u) {
    key.load(win, 16 * u, k[u]);
    w[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  static_assert(KT == 4, "16 entries a lane group, one a lane in the end");
  const int mine = e0 + 16 * (r / 4) + 4 * c + r % 4;
  const float before = mine < length ? a.account[bh * a.capacity + mine] : 0.0f;
  // some row does not see some entry
  const bool edge = e0 + 16 * KT - 1 > length - a.news;
  // this lane's row of 16 from `row0` (one past the last is read as the first, and left out below)
  const T *queries = query_row<T>(a, bh, 0);
  const int64_t news_stride = (int64_t)a.heads * a.group * a.width;
  struct Rows {
    pack_t<T> q[DP / 32];
    float off;
    int most;  // the last of the lane group's entries that the row sees
  };
  const auto load = [&](int row0, Rows &x) {
    const int row = row0 + r < a.rows ? row0 + r : 0;
    const int i = a.group == 1 ? row : (int)__umulhi((uint32_t)row, a.group_magic);
    const T *p = queries + i * news_stride + (row - i * a.group) * a.width;
#pragma unroll
    for (int n = 0; n < DP / 32; ++n) {
      const int d = n * 32 + c * 8;
      const bool there = EXACT || d < a.width;
      const uint4 w = *reinterpret_cast<const uint4 *>(p + (there ? d : 0));
      // zero past the width, as the keys are: an infinity of the row itself would meet their zeros
      x.q[n] = __builtin_bit_cast(pack_t<T>, there ? w : uint4{0, 0, 0, 0});
    }
    x.off = lse[bh * a.rows + row];
    x.most = row0 + r < a.rows ? length - a.news + i - e0 - 4 * c : -1;
  };
  const auto add = [&](int row0, const Rows &x) {
    const bool some = edge || row0 + 16 > a.rows;
#pragma unroll
    for (int u = 0; u < KT; ++u) {
      f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < DP / 32; ++n) z = mfma(k[u][n], x.q[n], z);
      if (some) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[u][i] += 16 * u + i > x.most ? 0.0f : __builtin_amdgcn_exp2f(z[i] * a.scale_log2 - x.off);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[u][i] += __builtin_amdgcn_exp2f(z[i] * a.scale_log2 - x.off);
      }
    }
  };
  // two sets of rows in turn, one on its way while the other is worked on
  Rows x, y;
  load(0, x);
  for (int row0 = 0; row0 < a.rows; row0 += 32) {
    load(row0 + 16, y);
    add(row0, x);
    load(row0 + 32, x);
    if (row0 + 16 < a.rows) add(row0 + 16, y);
  }
  // lane r of a group takes the sum of its r-th entry
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < KT; ++u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = team_sum<16>(w[u][i]);
      sum = r == 4 * u + i ? x : sum;
    }
  }
  if (mine < length) a.account_out[bh * a.capacity + mine] = before + sum;
}

template <class T, int TH, bool ONE, bool KEEP>
hipError_t join(const AttendArgs &a, float *lse, hipStream_t s) {
  const int64_t sums = KEEP ? (a.capacity + 4 * TH - 1) / (4 * TH) : 0;
  attend_join_kernel<T, TH, ONE, KEEP>
      <<<rows_grid((unsigned)(a.rows + sums), (int64_t)a.batch * a.heads), dim3(TH), 0, s>>>(a, lse);
  return hipGetLastError();
}

template <class T, int DP, int NT, bool EXACT, bool BY_ROWS, bool ONE, bool KEEP>
hipError_t attend(const AttendArgs &a, hipStream_t s) {
  const int64_t caches = (int64_t)a.batch * a.heads;
  const int per = 16 * NT * (BY_ROWS ? kAttendWaves : 1), row_blocks = (a.rows + per - 1) / per;
  attend_kernel<T, DP, NT, EXACT, BY_ROWS, ONE, KEEP>
      <<<rows_grid((unsigned)(a.splits * row_blocks), caches), dim3(64 * kAttendWaves), 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool formed = a.account_out != nullptr && !KEEP;
  // the rows' lse, where the logits are formed again, follow the parts' maxima and sums
  float *lse = formed ? a.part_ml + caches * a.splits * a.rows * 2 : nullptr;
  // 512 threads where there are many parts (one sequence of 8192 entries, 64 splits: 14.0 us, 15.5 with
  // 256), 256 where there are few (128 rows, 16 splits: 52.6 us, 61.5 with 512)
  e = a.splits > 16 ? join<T, 512, ONE, KEEP>(a, lse, s) : join<T, 256, ONE, KEEP>(a, lse, s);
  if (e != hipSuccess || !formed) return e;
  account_formed_kernel<T, DP, EXACT>
      <<<rows_grid((unsigned)((a.capacity + 255) / 256), caches), dim3(256), 0, s>>>(a, lse);
  return hipGetLastError();
}
// LDS floats per row of a whole cache's logits: whole blocks, and four more so that the rows' 16-byte
// accesses fall on all banks
int whole_stride(int64_t capacity) { return (int)((capacity + kBlock - 1) / kBlock * kBlock + 4); }

// 16 rows are one tile of the matrix instruction, 32 two that share the entries
// (ONE: up to 16 rows of a single new token, which see every entry; more rows of one token run as those of
// several do, their values checked and joined in the same way); beyond, each wave takes 32
// rows of its own and all entries, which leaves waves idle at up to 96 rows but is better than
// 16 rows each, since every wave reads the keys and values (64 rows over two
// sequences of 16384 entries: 43.0 us, with 16 rows each 50.0).  32 rows of 256
// elements would not fit a wave's registers.
template <class T, int DP, bool EXACT>
hipError_t attend_rows(const AttendArgs &a, hipStream_t s) {
  if (a.splits == 0) {  // whole caches
    const int stride = whole_stride(a.capacity);
    const size_t lds = a.account_out != nullptr ? (size_t)a.rows * stride * sizeof(float) : 0;
    const dim3 grid = rows_grid(1, (int64_t)a.batch * a.heads), threads(64 * whole_waves(DP));
    if (a.news == 1) attend_whole_kernel<T, DP, EXACT, true><<<grid, threads, lds, s>>>(a, stride);
    else attend_whole_kernel<T, DP, EXACT, false><<<grid, threads, lds, s>>>(a, stride);
    return hipGetLastError();
  }
  const bool keep = a.logits != nullptr;  // at most 16 rows
  if (a.rows <= 16) {
    if (a.news == 1)
      return keep ? attend<T, DP, 1, EXACT, false, true, true>(a, s)
                  : attend<T, DP, 1, EXACT, false, true, false>(a, s);
    return keep ? attend<T, DP, 1, EXACT, false, false, true>(a, s)
                : attend<T, DP, 1, EXACT, false, false, false>(a, s);
  }
  if constexpr (DP <= 128) {
    if (a.rows <= 32) return attend<T, DP, 2, EXACT, false, false, false>(a, s);
    return attend<T, DP, 2, EXACT, true, false, false>(a, s);
  } else {
    return attend<T, DP, 1, EXACT, true, false, false>(a, s);
  }
}
template <class T, int DP>
hipError_t attend_width(const AttendArgs &a, hipStream_t s) {
  return a.width == DP ? attend_rows<T, DP, true>(a, s) : attend_rows<T, DP, false>(a, s);
}
template <class T>
hipError_t attend_type(const AttendArgs &a, hipStream_t s) {
  if (a.width <= 64) return attend_width<T, 64>(a, s);
  if (a.width <= 128) return attend_width<T, 128>(a, s);
  return attend_width<T, 256>(a, s);
}

}  // namespace

AttendPlan attend_plan(int64_t batch, int64_t heads, int64_t capacity, int64_t rows, bool one, int width,
                       bool accounts) {
  AttendPlan p{};
  const int64_t caches = batch * heads;
  if (rows <= 16 && capacity <= (caches >= kWholeCaches ? kWholeMax : kWholeShort) &&
      rows * whole_stride(capacity) <= kWholeLogits)
    return p;  // whole caches
  // rows per workgroup, as attend_rows() chooses them
  const int64_t rows_per = rows <= 16 ? 16 : (width <= 128 ? (rows <= 32 ? 32 : 128) : 64);
  const int64_t groups = caches * ((rows + rows_per - 1) / rows_per);
  // Workgroups over all.  768 fit the chip at once (three a compute unit), and one
  // round of them is best where their shares are equal: one sequence of 200001 entries takes 137 us,
  // in three rounds 146.  Sequences of several lengths need a finer grain: 64 of 512 to 8192
  // entries, at random, take 1 to 8% less in three rounds, 8 of 100 to 32768 up to 17%; evenly spread lengths 2% more,
  // 3 of 50000 to 100000 4%.  With more rows, or wider ones, a
  // split's part of the outputs weighs more: 32 new tokens over 16384 entries take 53 us with
  // one workgroup a compute unit, 65 with two and 85 with half of them idle.
  // At up to 64 rows half of a workgroup's waves are idle, so two share a compute unit where the
  // entries are many: 64 rows over 100000 entries take 109 us with 512 workgroups, 133 with 256, over
  // 8192 entries 24.8 and 21.9.
  const bool halves = rows > 32 && rows <= 64 && width <= 128 && caches * capacity >= 1 << 17;
  const int64_t wanted = halves ? 512 : (rows > 16 || width > 128 ? 256 : (batch > 1 && one ? 2304 : 768));
  int64_t splits = (wanted + groups - 1) / groups;
  const int64_t most = (capacity + kStep - 1) / kStep;
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits < 1) splits = 1;
  p.splits = (int)splits;
  p.keep_logits = accounts && rows <= kKeepRows;
  p.blocks = (capacity + kBlock - 1) / kBlock;
  p.part_o = (size_t)(caches * splits * rows) * width * sizeof(float);
  p.part_ml = (size_t)(caches * splits * rows) * 2 * sizeof(float) + (size_t)(caches * rows) * sizeof(float);
  p.dropped = (size_t)(caches * splits) * sizeof(int);
  p.logits = p.keep_logits ? (size_t)(caches * rows) * p.blocks * kBlock * sizeof(float) : 0;
  return p;
}

hipError_t launch_attend(const AttendArgs &a, int dtype, hipStream_t s) {
  return dtype == LAPSUM_BF16 ? attend_type<bf16>(a, s) : attend_type<f16>(a, s);
}

}  // namespace lapsum
