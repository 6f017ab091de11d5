// Dispatch of tokens to experts and back: the expert order of the chosen
// (token, choice) pairs, the token rows laid out in it, and the weighted sum
// of the experts' outputs, each with its gradient.
//
// The plan is a stable counting sort by expert.  A wave ranks its 64 pairs by
// matching experts bit by bit with ballots, so a pair's place depends on its
// index alone and the result is the same on every run.
//
// The row kernels only move data: k rows of `width` elements per token.  A
// thread owns 16 bytes of a token's row and goes through the token's
// k slots, so the token's side is read or written once and the experts' side
// is touched in whole rows.
//
// What bounds them: memory.  8192 tokens of 2048 bf16 elements, 8 choices (268 MB
// on the experts' side): dispatch 54 us (302 MB, 5.6 TB/s), combine and the sums of the dispatch's
// gradient 54 us each (5.6 TB/s), combine's gradient 109 us (570 MB, 5.2 TB/s).  The plan of the 65536 pairs is
// three launches of 5 us (10.5 from a graph), of up to 1024 pairs one of 3 us: launches and chains of
// latencies, its bytes are few.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

constexpr int kPlanWaves = kPlanTile / 64;

// Lanes of the wave that hold the same value below 2^bits (dead lanes: none).
LDEV unsigned long long same_lanes(uint32_t v, bool live, int bits) {
  unsigned long long m = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const bool one = ((v >> b) & 1u) != 0;
    const unsigned long long set = __ballot(one);
    m &= one ? set : ~set;
  }
  return m;
}
LDEV int lanes_below(unsigned long long m) {
  return __popcll(m & ((1ull << (threadIdx.x % 64)) - 1ull));
}

// Counts of a tile: count[wave][expert] pairs per wave (LDS, cleared by the
// caller); returns the pair's rank among its expert's pairs of its wave.
LDEV int rank_in_wave(uint16_t *count, int experts, int e, bool live, int bits) {
  const unsigned long long same = same_lanes((uint32_t)e, live, bits);
  const int rank = lanes_below(same);
  if (live && rank == 0) count[(threadIdx.x / 64) * experts + e] = (uint16_t)__popcll(same);
  return rank;
}

// Pairs per expert of each tile: counts[expert][tile].
__global__ __launch_bounds__(kPlanTile) void plan_count_kernel(const int32_t *chosen, int64_t pairs, int experts,
                                                               int bits, int tiles, uint32_t *counts) {
  extern __shared__ uint16_t count[];  // [kPlanWaves][experts]
  lds_poison(count, kPlanWaves * experts * (int)sizeof(uint16_t));
  for (int i = threadIdx.x; i < kPlanWaves * experts; i += kPlanTile) count[i] = 0;
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * kPlanTile + threadIdx.x;
  const int e = i < pairs ? chosen[i] : -1;
  rank_in_wave(count, experts, e, (uint32_t)e < (uint32_t)experts, bits);
  __syncthreads();
  for (int x = threadIdx.x; x < experts; x += kPlanTile) {
    uint32_t n = 0;
    for (int w = 0; w < kPlanWaves; ++w) n += count[w * experts + x];
    counts[(int64_t)x * tiles + blockIdx.x] = n;
  }
}

// One workgroup per expert: its tile counts become the pairs in earlier
// tiles; its total goes behind them (totals[expert]).
__global__ __launch_bounds__(256) void plan_scan_kernel(uint32_t *counts, int experts, int tiles, uint32_t *totals) {
  struct Shared {
    uint32_t wave[4];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  uint32_t *c = counts + (int64_t)blockIdx.x * tiles;
  uint32_t carry = 0;
  for (int base = 0; base < tiles; base += 256) {
    const int i = base + (int)threadIdx.x;
    const uint32_t v = i < tiles ? c[i] : 0;
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const uint32_t u = __shfl_up(inc, o, 64);
      if ((int)(threadIdx.x % 64) >= o) inc += u;
    }
    if (threadIdx.x % 64 == 63) sh.wave[threadIdx.x / 64] = inc;
    __syncthreads();
    uint32_t before = carry, all = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < (int)(threadIdx.x / 64)) before += sh.wave[w];
      all += sh.wave[w];
    }
    if (i < tiles) c[i] = before + inc - v;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Exclusive sums of n <= kPlanTile values, one per thread, by the whole
// workgroup; `all` gets the total.
LDEV uint32_t exclusive_sum(uint32_t v, uint32_t *wave_sums, uint32_t &all) {
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint32_t u = __shfl_up(inc, o, 64);
    if ((int)(threadIdx.x % 64) >= o) inc += u;
  }
  if (threadIdx.x % 64 == 63) wave_sums[threadIdx.x / 64] = inc;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w < (int)(threadIdx.x / 64)) before += wave_sums[w];
    all += wave_sums[w];
  }
  __syncthreads();
  return before + inc - v;
}

// The places of a tile's pairs.  counts == NULL: the only tile, whose own
// counts are the totals.
__global__ __launch_bounds__(kPlanTile) void plan_place_kernel(const int32_t *chosen, int64_t pairs, int experts,
                                                               int bits, int tiles, const uint32_t *counts,
                                                               const uint32_t *totals, int32_t *offsets,
                                                               int32_t *slot, int32_t *order) {
  extern __shared__ uint16_t count[];  // [kPlanWaves][experts], then the experts' starts [experts]
  __shared__ uint32_t wave_sums[kPlanWaves];
  lds_poison(wave_sums);
  lds_poison(count, experts * (kPlanWaves * (int)sizeof(uint16_t) + (int)sizeof(uint32_t)));
  uint32_t *start = reinterpret_cast<uint32_t *>(count + kPlanWaves * experts);
  for (int i = threadIdx.x; i < kPlanWaves * experts; i += kPlanTile) count[i] = 0;
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * kPlanTile + threadIdx.x;
  const int e = i < pairs ? chosen[i] : -1;
  const bool live = (uint32_t)e < (uint32_t)experts;
  const int rank = rank_in_wave(count, experts, e, live, bits);
  __syncthreads();
  // one thread per expert (experts <= kPlanTile): waves' counts to the pairs before them
  const int x = threadIdx.x;
  uint32_t here = 0;
  if (x < experts) {
    for (int w = 0; w < kPlanWaves; ++w) {
      const uint32_t n = count[w * experts + x];
      count[w * experts + x] = (uint16_t)here;
      here += n;
    }
  }
  uint32_t all = 0;
  const uint32_t total = x < experts ? (counts != nullptr ? totals[x] : here) : 0;
  const uint32_t first = exclusive_sum(total, wave_sums, all);
  if (x < experts) {
    start[x] = first + (counts != nullptr ? counts[(int64_t)x * tiles + blockIdx.x] : 0);
    if (blockIdx.x == 0) offsets[x] = (int32_t)first;
  }
  if (blockIdx.x == 0 && x == 0) offsets[experts] = (int32_t)all;
  __syncthreads();
  if (i < pairs) {
    int at = -1;
    if (live) {
      at = (int)(start[e] + count[(threadIdx.x / 64) * experts + e]) + rank;
      order[at] = (int32_t)i;
    }
    slot[i] = at;
    if (i >= (int64_t)all) order[i] = -1;  // behind the last pair: no place there
  }
}

int bits_for(int experts) {
  int b = 0;
  while ((1 << b) < experts) ++b;
  return b;
}

// ----------------------------------------------------------------- rows
// Threads per token by the row's length in 16-byte packs; a workgroup of 256
// threads takes 256 / G tokens.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
LDEV uint4 stream_load(const uint4 *p);
LDEV void stream_store(uint4 *p, uint4 v);

// What a thread moves at a time: a pack of 16 bytes, or one element where
// rows are not 16-byte aligned.  Kept as it is in memory.
template <class T, bool PACKS>
struct Unit {
  static constexpr int N = Pack<T>::N;
  pack_t<T> v;
  LDEV float at(int n) const { return (float)v[n]; }
  static LDEV Unit load(const T *p) { return Unit{load_pack(p)}; }
  static LDEV Unit stream(const T *p) {
    return Unit{__builtin_bit_cast(pack_t<T>, stream_load(reinterpret_cast<const uint4 *>(p)))};
  }
  LDEV void store(T *p) const { stream_store(reinterpret_cast<uint4 *>(p), __builtin_bit_cast(uint4, v)); }
  LDEV void cached(T *p) const { store_pack(p, v); }
  static LDEV Unit zero() { return Unit{__builtin_bit_cast(pack_t<T>, uint4{0, 0, 0, 0})}; }
  static LDEV Unit of(const float (&f)[N]) {
    Unit u;
#pragma unroll
    for (int n = 0; n < N; ++n) u.v[n] = (T)f[n];
    return u;
  }
};
template <class T>
struct Unit<T, false> {
  static constexpr int N = 1;
  T v;
  LDEV float at(int) const { return (float)v; }
  static LDEV Unit load(const T *p) { return Unit{*p}; }
  static LDEV Unit stream(const T *p) { return Unit{*p}; }
  LDEV void store(T *p) const { *p = v; }
  LDEV void cached(T *p) const { *p = v; }
  static LDEV Unit zero() { return Unit{(T)0.0f}; }
  static LDEV Unit of(const float (&f)[1]) { return Unit{(T)f[0]}; }
};

LDEV int slot_at(const RowsArgs &a, int64_t pair) {
  const int s = a.slot[pair];
  return (uint64_t)(int64_t)s < (uint64_t)a.pairs ? s : -1;
}

// Rows of the experts' side are read or written once and are far more than the
// caches hold: streamed past them.
LDEV uint4 stream_load(const uint4 *p) {
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
  return __builtin_bit_cast(uint4, v);
}
LDEV void stream_store(uint4 *p, uint4 v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4 *>(p));
}

constexpr int kAhead = 8;  // rows of a token whose loads are under way together

// The token of this thread: the same for its whole wave, so slots and weights
// are scalar loads.
template <int G>
LDEV int64_t token_of() {
  return (int64_t)blockIdx.x * (256 / G) + __builtin_amdgcn_readfirstlane(threadIdx.x / G);
}

// The slots (and weights) of up to kAhead pairs from `pair`; absent ones -1 (and 0).
LDEV void slots_of(const RowsArgs &a, int64_t pair, int left, int (&s)[kAhead], float (&w)[kAhead]) {
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    s[i] = i < left ? slot_at(a, pair + i) : -1;
    w[i] = i < left && a.weights != nullptr ? a.weights[pair + i] : 1.0f;
  }
}

// xs[slot[t][j]] = x[t]; the rows behind the last pair are zeroed by the
// tokens whose pairs have those indices.
template <class T, bool PACKS, int G>
__global__ __launch_bounds__(256) void dispatch_rows_kernel(const RowsArgs a) {
  using U = Unit<T, PACKS>;
  const int64_t token = token_of<G>();
  if (token >= a.tokens) return;
  const int64_t placed = *a.placed;
  const T *src = static_cast<const T *>(a.src) + token * a.stride;
  T *dst = static_cast<T *>(a.dst);
  for (int64_t c = (int64_t)(threadIdx.x % G) * U::N; c < a.width; c += (int64_t)G * U::N) {
    const U u = U::load(src + c);
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
      const int64_t pair = token * a.k + j0;
      int s[kAhead];
      float w[kAhead];
      slots_of(a, pair, a.k - j0, s, w);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s[i] >= 0) u.store(dst + (int64_t)s[i] * a.width + c);
        if (i < a.k - j0 && pair + i >= placed) U::zero().store(dst + (pair + i) * a.width + c);
      }
    }
  }
}

// y[t] = sum_j w[t][j] ys[slot[t][j]], in the order of j, in fp32
template <class T, bool PACKS, int G>
__global__ __launch_bounds__(256) void sum_rows_kernel(const RowsArgs a) {
  using U = Unit<T, PACKS>;
  const int64_t token = token_of<G>();
  if (token >= a.tokens) return;
  const T *src = static_cast<const T *>(a.src);
  T *dst = static_cast<T *>(a.dst) + token * a.width;
  for (int64_t c = (int64_t)(threadIdx.x % G) * U::N; c < a.width; c += (int64_t)G * U::N) {
    float sum[U::N];
#pragma unroll
    for (int i = 0; i < U::N; ++i) sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
      int s[kAhead];
      float w[kAhead];
      slots_of(a, token * a.k + j0, a.k - j0, s, w);
      U u[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (s[i] >= 0) u[i] = U::stream(src + (int64_t)s[i] * a.width + c);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s[i] < 0) continue;
#pragma unroll
        for (int n = 0; n < U::N; ++n) sum[n] = __builtin_fmaf(w[i], u[i].at(n), sum[n]);
      }
    }
    U::of(sum).cached(dst + c);
  }
}

// dys[slot] = w dy[t], dweights = <dy[t], ys[slot]>: one pass over both.  The
// products' sum goes over a wave's lanes, then over the waves, in a fixed order.
template <class T, bool PACKS, int G>
__global__ __launch_bounds__(256) void combine_backward_kernel(const RowsArgs a) {
  using U = Unit<T, PACKS>;
  struct Shared {
    float part[LAPSUM_MAX_CHOICES][4];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int64_t token = token_of<G>();
  const bool live = token < a.tokens;
  const int64_t placed = *a.placed;
  const T *dy = static_cast<const T *>(a.dy) + (live ? token : 0) * a.stride;
  const T *ys = static_cast<const T *>(a.src);
  T *dys = static_cast<T *>(a.dst);
  const int lane = threadIdx.x % G;
  for (int j0 = 0; j0 < a.k && live; j0 += kAhead) {
    const int64_t pair = token * a.k + j0;
    int s[kAhead];
    float w[kAhead], dot[kAhead];
    slots_of(a, pair, a.k - j0, s, w);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) dot[i] = 0.0f;
    for (int64_t c = (int64_t)lane * U::N; c < a.width; c += (int64_t)G * U::N) {
      const U g = U::load(dy + c);
      U u[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (s[i] >= 0) u[i] = U::stream(ys + (int64_t)s[i] * a.width + c);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s[i] >= 0) {
          float d[U::N];
#pragma unroll
          for (int n = 0; n < U::N; ++n) {
            dot[i] = __builtin_fmaf(g.at(n), u[i].at(n), dot[i]);
            d[n] = w[i] * g.at(n);
          }
          U::of(d).store(dys + (int64_t)s[i] * a.width + c);
        }
        if (i < a.k - j0 && pair + i >= placed) U::zero().store(dys + (pair + i) * a.width + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i >= a.k - j0) continue;
      dot[i] = wave_reduce(dot[i], [](float x, float y) { return x + y; });
      if (threadIdx.x % 64 == 0) {
        if constexpr (G == 64) a.dweights[pair + i] = dot[i];
        else sh.part[j0 + i][threadIdx.x / 64] = dot[i];
      }
    }
  }
  if constexpr (G > 64) {
    __syncthreads();
    if (live && lane < a.k)
      a.dweights[token * a.k + lane] =
          (sh.part[lane][0] + sh.part[lane][1]) + (sh.part[lane][2] + sh.part[lane][3]);
  }
}

enum Kind { kDispatch, kSum, kBackward };

template <class T, bool PACKS, int G>
hipError_t rows(const RowsArgs &a, Kind kind, hipStream_t s) {
  constexpr int per = 256 / G;
  const dim3 grid((unsigned)((a.tokens + per - 1) / per));
  if (kind == kDispatch) dispatch_rows_kernel<T, PACKS, G><<<grid, dim3(256), 0, s>>>(a);
  else if (kind == kSum) sum_rows_kernel<T, PACKS, G><<<grid, dim3(256), 0, s>>>(a);
  else combine_backward_kernel<T, PACKS, G><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
template <class T>
hipError_t rows_of(const RowsArgs &a, Kind kind, hipStream_t s) {
  const auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool packs = a.width % Pack<T>::N == 0 && a.stride % Pack<T>::N == 0 && aligned(a.src) && aligned(a.dst) &&
                     aligned(a.dy);
  // A wave per token for up to 64 units, a workgroup beyond: 8192 rows of 512 bf16 elements, 8 choices,
  // take 14.5, 14.3 and 30.7 us (dispatch, sums, combine's gradient) with a wave each, 15.0, 16.4 and
  // 49.2 with a workgroup; of 2048 elements 78, 72 and 128 with a wave, 55, 55 and 109 with a
  // workgroup.  Packs where widths and addresses allow them (2048 elements one by one: 106, 78 and 137).
  const int64_t units = packs ? a.width / Pack<T>::N : a.width;
  if (packs) return units <= 64 ? rows<T, true, 64>(a, kind, s) : rows<T, true, 256>(a, kind, s);
  return units <= 64 ? rows<T, false, 64>(a, kind, s) : rows<T, false, 256>(a, kind, s);
}
hipError_t rows_any(const RowsArgs &a, Kind kind, int dtype, hipStream_t s) {
  if (dtype == LAPSUM_F32) return rows_of<f32>(a, kind, s);
  if (dtype == LAPSUM_BF16) return rows_of<bf16>(a, kind, s);
  return rows_of<f16>(a, kind, s);
}

}  // namespace

int64_t plan_tiles(int64_t pairs) { return (pairs + kPlanTile - 1) / kPlanTile; }

hipError_t launch_dispatch_plan(const int32_t *chosen, int64_t pairs, int experts, int32_t *offsets, int32_t *slot,
                                int32_t *order, uint32_t *counts, hipStream_t s) {
  const int tiles = (int)plan_tiles(pairs), bits = bits_for(experts);
  const size_t lds = (size_t)kPlanWaves * experts * sizeof(uint16_t), start = (size_t)experts * sizeof(uint32_t);
  uint32_t *totals = nullptr;
  if (tiles > 1) {
    totals = counts + (size_t)experts * tiles;
    plan_count_kernel<<<dim3(tiles), dim3(kPlanTile), lds, s>>>(chosen, pairs, experts, bits, tiles, counts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    plan_scan_kernel<<<dim3(experts), dim3(256), 0, s>>>(counts, experts, tiles, totals);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else {
    counts = nullptr;
  }
  plan_place_kernel<<<dim3(tiles), dim3(kPlanTile), lds + start, s>>>(chosen, pairs, experts, bits, tiles, counts,
                                                                      totals, offsets, slot, order);
  return hipGetLastError();
}

hipError_t launch_dispatch_rows(const RowsArgs &a, int dtype, hipStream_t s) { return rows_any(a, kDispatch, dtype, s); }
hipError_t launch_sum_rows(const RowsArgs &a, int dtype, hipStream_t s) { return rows_any(a, kSum, dtype, s); }
hipError_t launch_combine_backward(const RowsArgs &a, int dtype, hipStream_t s) {
  return rows_any(a, kBackward, dtype, s);
}

}  // namespace lapsum
