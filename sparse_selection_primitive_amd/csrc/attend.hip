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
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 32;       // entries a wave takes at a time
constexpr int kAttendWaves = 4;  // waves of a workgroup, taking its blocks in turn
constexpr int kStep = kBlock * kAttendWaves;
constexpr int kKeepRows = 16;    // up to this many rows the logits are kept for the accounts

LDEV f32x4 mfma(pack_t<bf16> a, pack_t<bf16> b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
LDEV f32x4 mfma(pack_t<f16> a, pack_t<f16> b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

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

// this lane's part of 16 keys (first factor of Z'): entry first + lane % 16, held to the last one
template <class T, int DP, bool EXACT>
LDEV void load_keys(const AttendArgs &a, const T *keys, int first, int last, pack_t<T> (&k)[DP / 32]) {
  const int lane = threadIdx.x % 64, c = lane / 16;
  const int e = first + lane % 16;
  const T *p = keys + (int64_t)(e < last ? e : last) * a.ke;
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) {
    const int d = i * 32 + c * 8;
    const bool there = EXACT || d < a.width;
    const uint4 w = *reinterpret_cast<const uint4 *>(p + (there ? d : 0));
    k[i] = __builtin_bit_cast(pack_t<T>, there ? w : uint4{0, 0, 0, 0});
  }
}

// the place-th entry of this lane's eight in a block
LDEV int entry_of(int place) {
  const int c = (threadIdx.x % 64) / 16;
  return (place / 4) * 16 + c * 4 + place % 4;
}

template <class T, int DP>
struct Values {
  static constexpr int W = DP / 16;  // elements per lane and entry
  typedef T vec __attribute__((ext_vector_type(DP / 16)));
  vec v[8];
  template <bool EXACT>
  LDEV void load(const AttendArgs &a, const T *values, int first, int last) {
    const int d = (threadIdx.x % 16) * W;
    const bool there = EXACT || d < a.width;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = first + entry_of(j);
      const T *p = values + (int64_t)(e < last ? e : last) * a.ve + (there ? d : 0);
      v[j] = *reinterpret_cast<const vec *>(p);
      if (!there) v[j] = (T)0.0f;
    }
  }
  LDEV pack_t<T> column(int n) const {
    pack_t<T> w;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = v[j][n];
    return w;
  }
};

template <class T, int DP, int NT, bool EXACT>
__global__ __launch_bounds__(64 * kAttendWaves) void attend_kernel(const AttendArgs a) {
  constexpr int W = DP / 16;
  constexpr int kRows = 16 * NT;
  struct Shared {
    float m[kAttendWaves][kRows], l[kAttendWaves][kRows];
    float o[kRows][DP];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  const int split = blockIdx.x % a.splits, row0 = (blockIdx.x / a.splits) * kRows;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, c = lane / 16, r = lane % 16;
  const int length = length_of(a, bh);
  int begin, end;
  split_range(a, length, split, begin, end);
  float *ml = a.part_ml + ((bh * a.splits + split) * a.rows + row0) * 2;
  const int rows_here = min(a.rows - row0, kRows);
  if (begin >= end) {  // the same for the whole workgroup
    for (int i = threadIdx.x; i < rows_here; i += blockDim.x) {
      ml[2 * i] = -INFINITY;
      ml[2 * i + 1] = 0.0f;
    }
    return;
  }
  const int64_t b = bh / a.heads, h = bh % a.heads;
  const T *keys = static_cast<const T *>(a.k) + b * a.kb + h * a.kh;
  const T *values = static_cast<const T *>(a.v) + b * a.vb + h * a.vh;

  pack_t<T> q[NT][DP / 32];
  int limit[NT];  // the last entry this lane's row sees
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + 16 * t + r;
    load_queries<T, DP>(a, bh, row, q[t]);
    limit[t] = length - a.news + row / a.group;
  }

  float m[NT], l[NT];
  f32x4 o[NT][W];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.0f;
#pragma unroll
    for (int n = 0; n < W; ++n) o[t][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  for (int e0 = begin + wave * kBlock; e0 < end; e0 += kStep) {
    pack_t<T> k[2][DP / 32];
    Values<T, DP> v;
    load_keys<T, DP, EXACT>(a, keys, e0, end - 1, k[0]);
    load_keys<T, DP, EXACT>(a, keys, e0 + 16, end - 1, k[1]);
    v.template load<EXACT>(a, values, e0, end - 1);
    // some row does not see some entry of the block
    const bool edge = e0 + kBlock > end || e0 + kBlock - 1 > length - a.news;
    bool broken = false;
    if (edge) {
      bool odd = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (e0 + entry_of(j) >= end) v.v[j] = (T)0.0f;
#pragma unroll
        for (int n = 0; n < W; ++n) odd |= !(fabsf((float)v.v[j][n]) < INFINITY);
      }
      broken = a.news > 1 && __any(odd);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 z[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        z[0] = mfma(k[0][i], q[t][i], z[0]);
        z[1] = mfma(k[1][i], q[t][i], z[1]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[u][i] *= a.scale_log2;
          if (edge) {
            const int e = e0 + 16 * u + 4 * c + i;
            if (e > limit[t] || e >= end) z[u][i] = -INFINITY;
          }
        }
      }
      if (a.logits != nullptr && row0 + 16 * t + r < a.rows) {
        float *to = a.logits + (bh * a.rows + row0 + 16 * t + r) * a.logit_stride + e0 + 4 * c;
        *reinterpret_cast<f32x4 *>(to) = z[0];
        *reinterpret_cast<f32x4 *>(to + 16) = z[1];
      }
      float top = fmaxf(fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[0][2], z[0][3])),
                        fmaxf(fmaxf(z[1][0], z[1][1]), fmaxf(z[1][2], z[1][3])));
      top = groups_max(top);
      const float next = fmaxf(m[t], top);
      if (__any(next > m[t])) {
        const float f = exp2_of(m[t], next);
        l[t] *= f;
#pragma unroll
        for (int n = 0; n < W; ++n) o[t][n] *= f;
        m[t] = next;
      }
      // the weights go into the product in two parts, so they keep 16 bits or more of their mantissa there
      pack_t<T> hi, lo;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = exp2_of(z[u][i], m[t]);
          l[t] += p;
          hi[4 * u + i] = (T)p;
          lo[4 * u + i] = (T)(p - (float)hi[4 * u + i]);
        }
      }
      if (!broken) {
#pragma unroll
        for (int n = 0; n < W; ++n) {
          const pack_t<T> col = v.column(n);
          o[t][n] = mfma(col, hi, o[t][n]);
          o[t][n] = mfma(col, lo, o[t][n]);
        }
      } else {
        // NaN or infinity among values that some row does not see: one new
        // token at a time, what it does not see set to zero
        for (int i = 0; i < a.news; ++i) {
          const int sees = length - a.news + i;
          const bool mine = (row0 + 16 * t + r) / a.group == i;
#pragma unroll
          for (int n = 0; n < W; ++n) {
            pack_t<T> col = v.column(n);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (e0 + entry_of(j) > sees) col[j] = (T)0.0f;
            f32x4 part = mfma(col, hi, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
            part = mfma(col, lo, part);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (mine) o[t][n][x] += part[x];
          }
        }
      }
    }
  }

  // join the waves: a common maximum, then their sums in the waves' order
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] = groups_sum(l[t]);
    if (c == 0) {
      sh.m[wave][16 * t + r] = m[t];
      sh.l[wave][16 * t + r] = l[t];
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float all = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttendWaves; ++w) all = fmaxf(all, sh.m[w][16 * t + r]);
    const float f = exp2_of(m[t], all);
#pragma unroll
    for (int n = 0; n < W; ++n) o[t][n] *= f;
    if (wave == 0 && c == 0 && 16 * t + r < rows_here) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttendWaves; ++w) sum += exp2_of(sh.m[w][16 * t + r], all) * sh.l[w][16 * t + r];
      ml[2 * (16 * t + r)] = all;
      ml[2 * (16 * t + r) + 1] = sum;
    }
  }
  for (int w = 0; w < kAttendWaves; ++w) {
    if (wave == w) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int n = 0; n < W; ++n) {
            float *at = &sh.o[16 * t + r][(4 * c + i) * W + n];
            *at = w == 0 ? o[t][n][i] : *at + o[t][n][i];
          }
        }
      }
    }
    __syncthreads();
  }
  float *part = a.part_o + ((bh * a.splits + split) * a.rows + row0) * a.width;
  for (int i = threadIdx.x; i < rows_here * a.width; i += blockDim.x) part[i] = sh.o[i / a.width][i % a.width];
}

// lse of a row over the splits (in units of log2), and its inverse sum at maximum `top`
LDEV void join_row(const AttendArgs &a, int64_t bh, int row, float &top, float &sum) {
  top = -INFINITY;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.part_ml[((bh * a.splits + s) * a.rows + row) * 2]);
  sum = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float *ml = a.part_ml + ((bh * a.splits + s) * a.rows + row) * 2;
    sum += exp2_of(ml[0], top) * ml[1];
  }
}

// out: one workgroup per 16 rows and cache; lse into the logits' place when they are formed again
template <class T>
__global__ __launch_bounds__(256) void attend_join_kernel(const AttendArgs a, float *lse) {
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  const int row = blockIdx.x;
  float top, sum;
  join_row(a, bh, row, top, sum);
  if (lse != nullptr && threadIdx.x == 0) lse[bh * a.rows + row] = sum > 0.0f ? top + log2f(sum) : (sum == 0.0f ? INFINITY : sum);
  T *out = const_cast<T *>(query_row<T>(a, bh, row) - static_cast<const T *>(a.q) + static_cast<T *>(a.out));
  for (int d = threadIdx.x; d < a.width; d += blockDim.x) {
    float o = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
      const int64_t at = (bh * a.splits + s) * a.rows + row;
      const float m = a.part_ml[at * 2];
      if (m != -INFINITY) o += exp2_of(m, top) * a.part_o[at * a.width + d];
    }
    out[d] = (T)(sum == 0.0f ? 0.0f : o / sum);
  }
}

// account_out = account + sum over rows of 2^(z - lse), z kept
__global__ __launch_bounds__(256) void account_kept_kernel(const AttendArgs a, const float *lse) {
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= length_of(a, bh)) return;
  float w = 0.0f;
  for (int row = 0; row < a.rows; ++row)
    w += __builtin_amdgcn_exp2f(a.logits[(bh * a.rows + row) * a.logit_stride + e] - lse[bh * a.rows + row]);
  a.account_out[bh * a.capacity + e] = a.account[bh * a.capacity + e] + w;
}

// the same, z formed again: a wave takes 64 entries and goes through all rows
template <class T, int DP, bool EXACT>
__global__ __launch_bounds__(256) void account_formed_kernel(const AttendArgs a, const float *lse) {
  constexpr int KT = 4;
  const int64_t bh = grid_row();
  if (bh >= (int64_t)a.batch * a.heads) return;
  const int lane = threadIdx.x % 64, c = lane / 16, r = lane % 16;
  const int length = length_of(a, bh);
  const int e0 = (blockIdx.x * 4 + threadIdx.x / 64) * 16 * KT;
  if (e0 >= length) return;
  const int64_t b = bh / a.heads, h = bh % a.heads;
  const T *keys = static_cast<const T *>(a.k) + b * a.kb + h * a.kh;
  pack_t<T> k[KT][DP / 32];
  f32x4 w[KT];
#pragma unroll
  for (int u = 0; u < KT; ++u) {
    load_keys<T, DP, EXACT>(a, keys, e0 + 16 * u, length - 1, k[u]);
    w[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  for (int row0 = 0; row0 < a.rows; row0 += 16) {
    const int row = row0 + r;
    pack_t<T> q[DP / 32];
    load_queries<T, DP>(a, bh, row, q);
    const float off = row < a.rows ? lse[bh * a.rows + row] : INFINITY;
    const int limit = length - a.news + row / a.group;
#pragma unroll
    for (int u = 0; u < KT; ++u) {
      f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) z = mfma(k[u][i], q[i], z);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f(z[i] * a.scale_log2 - off);
        if (e0 + 16 * u + 4 * c + i <= limit && row < a.rows) w[u][i] += p;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < KT; ++u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sum = team_sum<16>(w[u][i]);
      const int e = e0 + 16 * u + 4 * c + i;
      if (r == 0 && e < length) a.account_out[bh * a.capacity + e] = a.account[bh * a.capacity + e] + sum;
    }
  }
}

template <class T, int DP, int NT, bool EXACT>
hipError_t attend(const AttendArgs &a, hipStream_t s) {
  const int64_t caches = (int64_t)a.batch * a.heads;
  const int row_blocks = (a.rows + 16 * NT - 1) / (16 * NT);
  attend_kernel<T, DP, NT, EXACT>
      <<<rows_grid((unsigned)(a.splits * row_blocks), caches), dim3(64 * kAttendWaves), 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // the rows' lse follows the parts' maxima and sums
  float *lse = a.account_out == nullptr ? nullptr : a.part_ml + caches * a.splits * a.rows * 2;
  attend_join_kernel<T><<<rows_grid((unsigned)a.rows, caches), dim3(256), 0, s>>>(a, lse);
  e = hipGetLastError();
  if (e != hipSuccess || lse == nullptr) return e;
  if (a.logits != nullptr) {
    account_kept_kernel<<<rows_grid((unsigned)((a.capacity + 255) / 256), caches), dim3(256), 0, s>>>(a, lse);
  } else {
    account_formed_kernel<T, DP, EXACT>
        <<<rows_grid((unsigned)((a.capacity + 255) / 256), caches), dim3(256), 0, s>>>(a, lse);
  }
  return hipGetLastError();
}
template <class T, int DP>
hipError_t attend_width(const AttendArgs &a, hipStream_t s) {
  const bool exact = a.width == DP;
  if constexpr (DP <= 128) {  // 32 rows of 256 elements would not fit the registers
    if (a.rows > 16) return exact ? attend<T, DP, 2, true>(a, s) : attend<T, DP, 2, false>(a, s);
  }
  return exact ? attend<T, DP, 1, true>(a, s) : attend<T, DP, 1, false>(a, s);
}
template <class T>
hipError_t attend_type(const AttendArgs &a, hipStream_t s) {
  if (a.width <= 64) return attend_width<T, 64>(a, s);
  if (a.width <= 128) return attend_width<T, 128>(a, s);
  return attend_width<T, 256>(a, s);
}

}  // namespace

AttendPlan attend_plan(int64_t batch, int64_t heads, int64_t capacity, int64_t rows, int width, bool accounts) {
  AttendPlan p{};
  const int64_t caches = batch * heads, rows_per = rows <= 16 || width > 128 ? 16 : 32;
  const int64_t row_blocks = (rows + rows_per - 1) / rows_per;
  int64_t splits = (1024 + caches * row_blocks - 1) / (caches * row_blocks);
  const int64_t most = (capacity + kStep - 1) / kStep;
  if (splits > most) splits = most;
  if (splits > 128) splits = 128;
  if (splits < 1) splits = 1;
  p.splits = (int)splits;
  p.keep_logits = accounts && rows <= kKeepRows;
  p.logit_stride = (capacity + kBlock - 1) / kBlock * kBlock;
  p.part_o = (size_t)(caches * splits * rows) * width * sizeof(float);
  p.part_ml = (size_t)(caches * splits * rows) * 2 * sizeof(float) + (size_t)(caches * rows) * sizeof(float);
  p.logits = p.keep_logits ? (size_t)(caches * rows) * p.logit_stride * sizeof(float) : 0;
  return p;
}

hipError_t launch_attend(const AttendArgs &a, int dtype, hipStream_t s) {
  return dtype == LAPSUM_BF16 ? attend_type<bf16>(a, s) : attend_type<f16>(a, s);
}

}  // namespace lapsum
