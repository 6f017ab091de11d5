// The experts' products: rows in expert order times the matrix of their expert, and the gradients.
//
// With R_e the rows of expert e, X their inputs, Y their outputs and W_e its matrix,
//     Y = X W_e,   dX = dY W_e',   dW_e = X' dY     (R_e x inputs x outputs each).
// All three are C = A B for every expert: in the first two the rows are a size of C (ragged), in the third they are
// what is summed over.  How many rows an expert has is known on the device only, so a workgroup finds its
// expert and rows from the offsets: tiles are counted through the experts in order, one wave's lanes a
// few experts each.
//
// Few rows are bounded by reading the matrices: 192 rows of 135 experts of 2048 x 1024 take 70 us (566 MB, 8.1 TB/s
// with what the last call left in the memory-side cache), 8 rows of 8 experts 7.8 to 8.0 us (34 MB).  Many rows are
// bounded by the matrix instructions and the power that they and LDS draw: 16384 rows of 8 experts of 4096 x 14336 take 1.69 ms
// (1.14 PFLOP/s, the clock at 1.6 to 2.0 of 2.4 GHz; the library's product of one expert after another 1.84 ms).  In
// between the matrices' way from memory and the ragged ends count as well: 65536 rows of 256 experts of 2048 x 1024
// 0.38 to 0.43 ms, the same for the rows' gradient, 0.43 to 0.49 for the matrices' (of which 0.17 ms are writing 1.1 GB).
#include <cmath>
#include <type_traits>

#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

LDEV f32x4 mfma(pack_t<bf16> a, pack_t<bf16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
LDEV f32x4 mfma(pack_t<f16> a, pack_t<f16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

LDEV int in_rows(const ProductArgs &p, int64_t o) { return (int)(o < 0 ? 0 : (o > p.rows ? p.rows : o)); }
// An offset that the whole wave asks for: a scalar load, since a vector one would wait for all loads that are under way.
LDEV int offset_of(const ProductArgs &p, int i) {
  using scalars = const __attribute__((address_space(4))) int32_t *;
  return in_rows(p, ((scalars)(uintptr_t)p.offsets)[__builtin_amdgcn_readfirstlane(i)]);
}

// The rows in order are those before the first expert's, every expert's, and those behind the
// last one's: experts + 2 ranges, of which the first and the last are no expert's.  `offset`: of g - 1, or any other
// where there is none.
LDEV int range_begin(const ProductArgs &p, int g, int offset) {
  return g == 0 ? 0 : (g <= p.experts + 1 ? offset : (int)p.rows);
}
LDEV int offset_before(const ProductArgs &p, int g) { return g < 1 ? 0 : (g <= p.experts + 1 ? g - 1 : p.experts); }
// a lane's own range
LDEV int range_begin(const ProductArgs &p, int g) {
  return range_begin(p, g, in_rows(p, p.offsets[offset_before(p, g)]));
}
// the whole wave's
LDEV int range_begin_all(const ProductArgs &p, int g) {
  g = __builtin_amdgcn_readfirstlane(g);
  return range_begin(p, g, offset_of(p, offset_before(p, g)));
}

struct RowTile {
  int expert;      // -1: no expert's
  int first, end;  // rows of the tile
};
// The tiles of `size` rows, counted through the ranges in order: lanes take `per` neighbouring ranges each.  Every wave counts
// by itself.  The bounds of up to kBounds ranges a lane are asked for at once and stay in its registers; of
// more (from 511 experts on) they are read again.
struct RowTiles {
  static constexpr int kBounds = 8;
  int bound[kBounds + 1];
  int per, mine, upto;  // ranges of a lane; tiles of this lane's and up to them

  static LDEV int tiles_of(int a, int b, int size) { return b > a ? (b - a + size - 1) / size : 0; }
  LDEV void count(const ProductArgs &p, int size) {
    const int ranges = p.experts + 2, first = lane_id() * (per = (ranges + 63) / 64);
#pragma unroll
    for (int i = 0; i <= kBounds; ++i) {
      const int g = first + (i < per ? i : per);
      bound[i] = range_begin(p, g < ranges ? g : ranges);
    }
    mine = 0;
#pragma unroll
    for (int i = 0; i < kBounds; ++i) mine += tiles_of(bound[i], bound[i + 1], size);
    for (int i = kBounds; i < per; ++i) {
      const int g = first + i;
      if (g < ranges) mine += tiles_of(range_begin(p, g), range_begin(p, g + 1), size);
    }
    upto = (int)wave_incl_scan((uint32_t)mine);
  }
  LDEV int total() const { return read_lane(upto, 63); }
  // the index-th of them; false: there are no more
  LDEV bool find(const ProductArgs &p, int size, int index, RowTile &t) const {
    if (index >= total()) return false;
    const int at = __builtin_ctzll(__ballot(upto > index)), first = at * per;
    int left = index - read_lane(upto - mine, at);
    const auto here = [&](int g, int a, int b) {
      const int n = tiles_of(a, b, size);
      if (left >= n) {
        left -= n;
        return false;
      }
      t.expert = g >= 1 && g <= p.experts ? g - 1 : -1;
      t.first = a + left * size;
      t.end = t.first + size < b ? t.first + size : b;
      return true;
    };
#pragma unroll
    for (int i = 0; i < kBounds; ++i)
      if (i < per && here(first + i, read_lane(bound[i], at), read_lane(bound[i + 1], at))) return true;
    for (int i = kBounds; i < per; ++i)
      if (here(first + i, range_begin_all(p, first + i), range_begin_all(p, first + i + 1))) return true;
    return false;
  }
};
// as many tiles as there can be: a range that has rows adds one to those that are full
int64_t most_row_tiles(const ProductArgs &p, int size) {
  return p.rows / size + (p.rows < p.experts + 2 ? p.rows : p.experts + 2);
}

// ------------------------------------------------------------------ any layout
// A tile of 64 x 64, its factors brought to LDS an element at a time: for fp32, and for sizes, strides and pointers that are
// no multiples of 16 bytes.  Bound by the addresses and bounds of single elements.  fp32: 75 to 86 TFLOP/s (8192 tokens of 256
// experts of 2048 x 1024 with both gradients 11.1 ms, elementary products 18.7); bf16, 64 experts of 2047 x 1023 with 1024
// rows: 200.
constexpr int kAny = 64, kAnyK = 32;

template <class T, bool SUM_ROWS>
__global__ __launch_bounds__(256) void product_any_kernel(ProductArgs p) {
  constexpr int kRow = kAnyK + 16 / (int)sizeof(T);  // 16 rows of one column in different banks
  __shared__ struct {
    T a[kAny][kRow], b[kAny][kRow];
  } sh;
  lds_poison(sh);
  const int n0 = blockIdx.x * kAny;
  int m0, m1, k0, k1, e;
  if (SUM_ROWS) {
    const int tiles = (p.m + kAny - 1) / kAny;
    if (grid_row() >= (int64_t)tiles * p.experts) return;
    e = (int)(grid_row() / tiles);
    m0 = (int)(grid_row() % tiles) * kAny;
    m1 = m0 + kAny < p.m ? m0 + kAny : p.m;
    k0 = offset_of(p, e);
    k1 = offset_of(p, e + 1);
  } else {
    RowTile t;
    RowTiles all;
    all.count(p, kAny);
    if (!all.find(p, kAny, (int)grid_row(), t)) return;
    e = t.expert;
    m0 = t.first;
    m1 = t.end;
    k0 = 0;
    k1 = e < 0 ? 0 : p.k;
  }
  const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);
  if (!SUM_ROWS && e >= 0) b += e * p.be;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, i = threadIdx.x;
  f32x4 c[4] = {};
  T xa[8], xb[8];  // of the next step
  // neighbouring lanes take neighbouring elements where there are any
  const auto at = [&](int64_t next, int j) { return next == 1 ? (j * 256 + i) / kAnyK : (j * 256 + i) % kAny; };
  const auto in = [&](int64_t next, int j) { return next == 1 ? (j * 256 + i) % kAnyK : (j * 256 + i) / kAny; };
  const auto ask = [&](int k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ma = at(p.ak, j), ka = k + in(p.ak, j), nb = at(p.bk, j), kb = k + in(p.bk, j);
      xa[j] = m0 + ma < m1 && ka < k1 ? a[(m0 + ma) * p.am + ka * p.ak] : (T)0.0f;
      xb[j] = n0 + nb < p.n && kb < k1 ? b[(n0 + nb) * p.bn + kb * p.bk] : (T)0.0f;
    }
  };
  if (k0 < k1) ask(k0);
  for (int k = k0; k < k1; k += kAnyK) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sh.a[at(p.ak, j)][in(p.ak, j)] = xa[j];
      sh.b[at(p.bk, j)][in(p.bk, j)] = xb[j];
    }
    __syncthreads();
    if (k + kAnyK < k1) ask(k + kAnyK);
    const int row = wave * 16 + lane % 16;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int s = 0; s < kAnyK; s += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(sh.a[row][s + lane / 16], sh.b[j * 16 + lane % 16][s + lane / 16], c[j],
                                                      0, 0, 0);
    } else {
      const pack_t<T> f = load_pack(&sh.a[row][lane / 16 * 8]);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = mfma(f, load_pack(&sh.b[j * 16 + lane % 16][lane / 16 * 8]), c[j]);
    }
    __syncthreads();
  }
  T *out = static_cast<T *>(p.c) + (SUM_ROWS ? e * p.ce : 0);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int m = m0 + wave * 16 + lane / 16 * 4 + r;
    if (m >= m1) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + j * 16 + lane % 16;
      if (n < p.n) out[m * p.cm + n] = (T)c[j][r];
    }
  }
}

template <class T, bool SUM_ROWS>
hipError_t any(const ProductArgs &p, hipStream_t s) {
  const unsigned nt = (unsigned)((p.n + kAny - 1) / kAny);
  const int64_t mt = SUM_ROWS ? (int64_t)((p.m + kAny - 1) / kAny) * p.experts : most_row_tiles(p, kAny);
  product_any_kernel<T, SUM_ROWS><<<rows_grid(nt, mt), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

// ------------------------------------------------------------- 16 bytes at a time
// A window of memory that loads are held to: what lies past its end reads as zero.  Steps of a tile lie within 2^31 bytes.
using window_t = __amdgpu_buffer_rsrc_t;
constexpr int kStreamed = 2;  // not kept in the caches: the products are another's to read (3% of a training batch)
constexpr uint32_t kNowhere = 0x80000000u;  // a lane's offset past every window

// 64 x 16 bytes from the lanes' offsets to consecutive places of LDS from `to` on (bytes).  Written out, since the compiler
// would have every later read of LDS wait for it; whoever reads waits by arrived().  The compiler does not look into it
// either, so it keeps the distances itself: one wait state from a write of m0 to a load to LDS, five from a vector
// instruction's write of a scalar register (the window's) to a load that reads it.
LDEV void load_to_lds(window_t w, uint32_t to, uint32_t offset) {
  uint32_t m0;  // the compiler's; the place goes there
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 2\n\t"
      "buffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(to), "v"(offset), "s"(w)
      : "memory");
}
LDEV uint32_t lds_at(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

constexpr int kDepth = 32;  // of a step: elements of the sum

// One factor's side of a tile: SIZE places along C by kDepth of the sum, in LDS, brought there by WAVES waves.
//
// NEXT: the sum's elements lie next to each other in memory.  LDS holds rows of one place, 64 bytes, whose 16-byte
// chunks change places by the row, so that eight lanes that read one chunk of neighbouring rows meet all
// banks.  SPREAD: rows 16 i + j hold places 8 j + i of each 128, so that what a lane reads from rows 16 apart are
// neighbouring places.
// Otherwise places lie next to each other: LDS holds kDepth rows of SIZE.
template <class T, int SIZE, bool NEXT, bool SPREAD, int WAVES>
struct Side {
  static constexpr int kLoads = SIZE * kDepth * 2 / 1024 / WAVES;
  const char *at;     // of the step
  int64_t advance;    // bytes from step to step
  int step;           // elements between rows of memory
  int whole, rest;    // bytes of the window of a whole step and of the last one, where that is not whole
  uint32_t to;        // LDS of this wave's first load, of the first stage
  uint32_t offset;    // of this lane's part of the wave's first load
  int chunk;          // NEXT: the lane's chunk of the step's sum

  // rows of memory between the wave's first load and load `i`
  static constexpr int rows_to(int i) {
    if (!NEXT) return i * (WAVES * 64 / (SIZE / 8));
    if (!SPREAD) return i * WAVES * 16;
    return i * WAVES / 8 * 128 + i * WAVES % 8;  // 16 rows a wave, 8 such to 128 places
  }
  LDEV void start(int64_t stride, uint32_t lds) {
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    to = lds + wave * 1024;
    step = (int)stride;
    at = nullptr;
    whole = rest = 0;
    if (NEXT) {
      advance = kDepth * 2;
      chunk = lane % 4 ^ (lane / 8 & 3);  // the same for all loads: their rows are 16 apart
      static_assert(!NEXT || !SPREAD || 8 % WAVES == 0, "the places of a wave's loads");
      const int place = SPREAD ? lane / 4 * 8 + wave : wave * 16 + lane / 4;
      offset = (uint32_t)(place * step * 2) + (uint32_t)(chunk * 16);
    } else {
      constexpr int kPer = SIZE / 8;  // chunks of a row
      static_assert(NEXT || WAVES * 64 % kPer == 0, "a wave's loads are whole rows apart");
      const int x = wave * 64 + lane;
      advance = kDepth * stride * 2;
      offset = (uint32_t)(x / kPer * step * 2) + (uint32_t)(x % kPer * 16);
    }
  }
  // To a tile: the element at its first place and the sum's first element; places and elements of the sum that are there.
  LDEV void aim(const T *first, int places, int sum) {
    at = reinterpret_cast<const char *>(first);
    places = places < SIZE ? places : SIZE;
    const int left = sum % kDepth;
    whole = NEXT ? ((places - 1) * step + kDepth) * 2 : ((kDepth - 1) * step + places) * 2;
    rest = NEXT ? ((places - 1) * step + left) * 2 : ((left - 1) * step + places) * 2;
  }
  // The step's part, of which `left` elements of the sum are there (none or fewer: zeros), to LDS: load `i` of this wave.
  window_t window;
  uint32_t from;
  LDEV void begin(int left) {
    const int bytes = left >= kDepth ? whole : (left > 0 ? rest : 0);
    window = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(at), 0, bytes, 0x00020000);
    from = NEXT && chunk * 8 >= left ? kNowhere : offset;
    at += advance;
  }
  LDEV void load(int i, uint32_t stage) const {
    load_to_lds(window, to + stage + i * (WAVES * 1024), from + (uint32_t)(rows_to(i) * step * 2));
  }
};

// two 16-bit elements, the low or the high ones of two words
LDEV uint32_t pair_low(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
LDEV uint32_t pair_high(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// What a lane holds of one side's step for N matrix instructions: with NEXT the operands themselves (SPREAD or not, by
// what LDS holds); otherwise eight rows of the sum by N neighbouring places (first + N * lane % 16 + i for
// operand i), which operand() turns over.
template <class T, int SIZE, bool NEXT, int N>
struct Held {
  static constexpr int kReads = NEXT ? N : 8;
  uint32_t w[kReads][NEXT ? 4 : N / 2];
  // where this lane reads from, in elements from the side's part of a stage
  LDEV static int place(int first) {
    const int lane = lane_id();
    return NEXT ? (first + lane % 16) * kDepth + ((lane / 16) ^ (lane / 2 & 3)) * 8
                : lane / 16 * 8 * SIZE + first + lane % 16 * N;
  }
  LDEV void read(int i, const T *from) {
    const T *p = from + i * (NEXT ? 16 * kDepth : SIZE);
    if constexpr (NEXT || N == 8)
      *reinterpret_cast<uint4 *>(w[i]) = *reinterpret_cast<const uint4 *>(p);
    else
      *reinterpret_cast<uint2 *>(w[i]) = *reinterpret_cast<const uint2 *>(p);
  }
  LDEV pack_t<T> operand(int i) const {
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (NEXT)
        d[j] = w[i][j];
      else
        d[j] = i % 2 == 0 ? pair_low(w[2 * j][i / 2], w[2 * j + 1][i / 2]) : pair_high(w[2 * j][i / 2], w[2 * j + 1][i / 2]);
    }
    return __builtin_bit_cast(pack_t<T>, uint4{d[0], d[1], d[2], d[3]});
  }
};

template <class T, int WM, int WAVES_M, int WAVES_N, bool A_NEXT, bool B_NEXT>
struct Tile {
  static constexpr int kWaves = WAVES_M * WAVES_N, kM = WM * WAVES_M, kN = 128 * WAVES_N, kFrags = WM / 16;
  using A = Side<T, kM, A_NEXT, false, kWaves>;
  using B = Side<T, kN, B_NEXT, true, kWaves>;
  static constexpr int kLoads = A::kLoads + B::kLoads;  // of a wave and step
  struct Operands {
    Held<T, kM, A_NEXT, kFrags> a;
    Held<T, kN, B_NEXT, 8> b;
  };
  static constexpr int kReadsA = decltype(Operands::a)::kReads;
  f32x4 c[kFrags][8];

  // The products of a step, column by column, and between them what `between(j)` does: the columns stay in order, so
  // that neither loads nor reads of LDS hold up the matrix instructions.
  template <class F>
  LDEV void step(const Operands &x, const F &between) {
    pack_t<T> fa[kFrags];
#pragma unroll
    for (int i = 0; i < kFrags; ++i) fa[i] = x.a.operand(i);
    pack_t<T> fb = x.b.operand(0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      between(j);
      pack_t<T> next = fb;
      if (j < 7) next = x.b.operand(j + 1);
#pragma unroll
      for (int i = 0; i < kFrags; ++i) c[i][j] = mfma(fa[i], fb, c[i][j]);
      fb = next;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // Places [0, m) x [0, n) of the tile.  Always kStores stores of a wave, so that they can be counted.
  static constexpr int kStores = kFrags * 4;
  LDEV void store(T *out, int64_t stride, int m, int n) const {
    int lane = lane_id();
    asm volatile("" : "+v"(lane));  // places are formed again for each tile, not held (and spilled) through the steps
    const int wave = threadIdx.x / 64, wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int col = wn * 128 + lane % 16 * 8, step = (int)stride;
    m = m < kM ? m : kM;
    n = n < kN ? n : kN;
    const window_t window = __builtin_amdgcn_make_buffer_rsrc(out, 0, ((m - 1) * step + n) * 2, 0x00020000);
    const uint32_t none = col < n ? 0u : kNowhere;
#pragma unroll
    for (int i = 0; i < kFrags; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int in = lane / 16 * 4 + r, row = wm * WM + (A_NEXT ? i * 16 + in : in * kFrags + i);
        pack_t<T> v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (T)c[i][j][r];
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), window,
                                               (int)((uint32_t)(row * step * 2 + col * 2) | none), 0, kStreamed);
      }
  }
  LDEV void clear() {
#pragma unroll
    for (int i = 0; i < kFrags; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) c[i][j] = f32x4{};
  }
};

// All but the last LOADS loads to LDS of every wave are there, and what every wave has read from LDS is in its registers.
template <int LOADS>
LDEV void arrived() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS) : "memory");
}

// Tiles of rows counted through the ranges, in LDS: before[g] of them come before range g.
struct RowTable {
  int before[LAPSUM_MAX_EXPERTS + 3];
  LDEV int total(const ProductArgs &p) const { return __builtin_amdgcn_readfirstlane(before[p.experts + 2]); }
  LDEV void fill(const ProductArgs &p, int size) {
    if (threadIdx.x < 64) {
      RowTiles all;
      all.count(p, size);
      const int ranges = p.experts + 2, first = lane_id() * all.per;
      int at = all.upto - all.mine;
#pragma unroll
      for (int i = 0; i < RowTiles::kBounds; ++i)
        if (i < all.per && first + i < ranges) {
          before[first + i] = at;
          at += RowTiles::tiles_of(all.bound[i], all.bound[i + 1], size);
        }
      for (int i = RowTiles::kBounds; i < all.per && first + i < ranges; ++i) {
        before[first + i] = at;
        at += RowTiles::tiles_of(range_begin(p, first + i), range_begin(p, first + i + 1), size);
      }
      if (lane_id() == 63) before[ranges] = all.upto;
    }
    __syncthreads();
  }
  // the range of the index-th tile; index below total().  Every lane of the wave asks.
  LDEV int range_of(const ProductArgs &p, int index) const {
    const int ranges = p.experts + 2, per = (ranges + 63) / 64, lane = lane_id();
    const auto end = [&](int g) { return before[g + 1 < ranges ? g + 1 : ranges]; };
    const int part = __builtin_ctzll(__ballot(end(lane * per + per - 1) > index)) * per;
    return part + __builtin_ctzll(__ballot(lane >= per || end(part + lane) > index));  // per is at most 17
  }
};

template <class T>
struct TilePlace {
  const T *a, *b;
  T *out;
  int m, n, sum;  // places that are there (or more than the tile holds), elements of the sum
};

// Workgroups stay, as many as there is room for, and take tile after tile, so that a tile's first loads are under way
// while the last one is still multiplied and stored.  They go round the eight dies; each die takes a run of tiles,
// which share factors.
//
// What loads is ahead of what multiplies by kStages steps, in whatever tile that is; tiles have an even number of steps
// (the last may be zeros), so that the two sets of operands change places evenly.
template <class T, int WM, int WAVES_M, int WAVES_N, int kStages, bool A_NEXT, bool B_NEXT, bool SUM_ROWS>
__global__ __launch_bounds__(64 * WAVES_M *WAVES_N, 2) void product_tile_kernel(ProductArgs p) {
  using Work = Tile<T, WM, WAVES_M, WAVES_N, A_NEXT, B_NEXT>;
  constexpr int kA = Work::kM * kDepth, kStage = kA + Work::kN * kDepth;
  __shared__ T lds[kStages * kStage];
  lds_poison(lds);
  const int tiles_n = (p.n + Work::kN - 1) / Work::kN, tiles_m = SUM_ROWS ? (p.m + Work::kM - 1) / Work::kM : 0;
  int total;
  __shared__ std::conditional_t<SUM_ROWS, int, RowTable> table;
  lds_poison(table);
  if constexpr (SUM_ROWS) {
    total = tiles_m * tiles_n * p.experts;
  } else {
    table.fill(p, Work::kM);
    // of offsets that do not ascend no more than ascending ones would have
    const int rows = table.total(p), most = (int)(p.rows / Work::kM) + p.experts + 2;
    total = (rows < most ? rows : most) * tiles_n;
  }
  const int each = (total + 7) / 8, round = gridDim.x / 8;
  // this workgroup's index-th tile
  const auto place = [&](int index, TilePlace<T> &x) {
    const int i = index * round + (int)blockIdx.x / 8, t = (int)blockIdx.x % 8 * each + i;
    if (i >= each || t >= total) return false;
    x.a = static_cast<const T *>(p.a);
    x.b = static_cast<const T *>(p.b);
    x.out = static_cast<T *>(p.c);
    int n0;
    if constexpr (SUM_ROWS) {
      const int e = t / (tiles_m * tiles_n), in = t % (tiles_m * tiles_n), m0 = in % tiles_m * Work::kM;
      n0 = in / tiles_m * Work::kN;
      const int k0 = offset_of(p, e), k1 = offset_of(p, e + 1);
      x.sum = k1 - k0;
      x.m = p.m - m0;
      x.a += k0 * p.ak + m0;
      x.b += k0 * p.bk + n0;
      x.out += e * p.ce + m0 * p.cm + n0;
    } else {
      // A range's tiles come after one another, up to kGroup tiles of rows through all columns: their columns of a matrix
      // are read once.  30018 rows to 64 experts of 1416 x 2056 draw 0.80 GB from memory, in groups across ranges 1.27
      // (0.46 are there), in 292 us for 320; 65536 rows to 256 of 2048 x 1024 1.86 GB for 2.09 (1.34), in the same 455 us.
      constexpr int kGroup = 8;
      const int g = table.range_of(p, t / tiles_n), before = __builtin_amdgcn_readfirstlane(table.before[g]);
      const int rows = __builtin_amdgcn_readfirstlane(table.before[g + 1]) - before, in_range = t - before * tiles_n;
      const int first = in_range / (kGroup * tiles_n) * kGroup, group = rows - first < kGroup ? rows - first : kGroup;
      const int in = in_range - first * tiles_n;
      const int begin = range_begin_all(p, g), end = range_begin_all(p, g + 1);
      RowTile r;
      r.expert = g >= 1 && g <= p.experts ? g - 1 : -1;
      r.first = begin + (first + in % group) * Work::kM;
      r.end = r.first + Work::kM < end ? r.first + Work::kM : end;
      n0 = in / group * Work::kN;
      x.m = r.end - r.first;
      x.sum = r.expert < 0 ? 0 : p.k;
      x.a += r.first * p.am;
      x.b += (r.expert < 0 ? 0 : r.expert) * p.be + n0 * p.bn;
      x.out += r.first * p.cm + n0;
    }
    x.n = p.n - n0;
    return true;
  };

  TilePlace<T> now;
  if (!place(0, now)) return;
  typename Work::A sa;
  typename Work::B sb;
  sa.start(A_NEXT ? p.am : p.ak, lds_at(lds));
  sb.start(B_NEXT ? p.bn : p.bk, lds_at(lds + kA));
  int ahead = 0, asked = 0;  // the next tile to load; what is left of the sum of the one that is loaded
  int to = 0, from = 0, fresh = 0;
  const int wave = threadIdx.x / 64;
  const int place_a = decltype(Work::Operands::a)::place(wave / WAVES_N * WM);
  const int place_b = kA + decltype(Work::Operands::b)::place(wave % WAVES_N * 128);
  bool more = true, half = false;  // half: a tile's second step of two is next
  TilePlace<T> x = now;            // the tile that is loaded, the (ahead - 1)-th
  const auto begin = [&] {
    if (asked <= 0 && !half && more) {
      do {
        more = place(ahead++, x);
      } while (more && x.sum <= 0);
      if (more) {
        sa.aim(x.a, x.m, x.sum);
        sb.aim(x.b, x.n, x.sum);
        asked = x.sum;
      }
    }
    sa.begin(asked);
    sb.begin(asked);
    asked -= kDepth;
    half = !half;
  };
  const auto load = [&](int i) {
    if (i < Work::A::kLoads)
      sa.load(i, to * 2);
    else
      sb.load(i - Work::A::kLoads, to * 2);
  };
  const auto after = [&](int stage) { return stage == (kStages - 1) * kStage ? 0 : stage + kStage; };
  Work w;
  // Step t computes on what the step before has read from LDS, reads what the next one computes on, and asks for
  // what is kStages steps away, whose place step t's own part has left.  Past the end zeros are asked for, so that
  // as many loads are under way in every step.
  const auto step = [&](const typename Work::Operands &now, typename Work::Operands &next) {
    // stores count as loads do, for as long as loads from before them are waited for
    if (fresh > 0) {
      --fresh;
      arrived<(kStages - 2) * Work::kLoads + Work::kStores>();
    } else {
      arrived<(kStages - 2) * Work::kLoads>();
    }
    from = after(from);
    const T *pa = lds + from + place_a, *pb = lds + from + place_b;
    w.step(now, [&](int j) {
#pragma unroll
      for (int i = j * Work::kReadsA / 8; i < (j + 1) * Work::kReadsA / 8; ++i) next.a.read(i, pa);
      next.b.read(j, pb);
#pragma unroll
      for (int i = (j * Work::kLoads + 7) / 8; i < ((j + 1) * Work::kLoads + 7) / 8; ++i) load(i);
      if (j == 7) {
        begin();  // the next step's
        to = after(to);
      }
    });
  };
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) {
    begin();
#pragma unroll
    for (int i = 0; i < Work::kLoads; ++i) load(i);
    to = after(to);
  }
  begin();
  typename Work::Operands u, v;
  arrived<(kStages - 1) * Work::kLoads>();
#pragma unroll
  for (int i = 0; i < Work::kReadsA; ++i) u.a.read(i, lds + place_a);
#pragma unroll
  for (int i = 0; i < 8; ++i) u.b.read(i, lds + place_b);
#pragma unroll 1
  for (int index = 1;; ++index) {
    w.clear();
#pragma unroll 1
    for (int sum = now.sum; sum > 0; sum -= 2 * kDepth) {
      step(u, v);
      step(v, u);
    }
    w.store(now.out, p.cm, now.m, now.n);
    fresh = kStages - 1;
    if (more && ahead == index + 1)
      now = x;  // mostly
    else if (!place(index, now))
      break;
  }
  // no load may reach LDS that is another workgroup's
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <class T, int WM, int WAVES_M, int WAVES_N, int STAGES, bool A_NEXT, bool B_NEXT, bool SUM_ROWS>
hipError_t tiles(const ProductArgs &p, hipStream_t s) {
  using Work = Tile<T, WM, WAVES_M, WAVES_N, A_NEXT, B_NEXT>;
  const int64_t nt = (p.n + Work::kN - 1) / Work::kN;
  const int64_t mt = SUM_ROWS ? (int64_t)((p.m + Work::kM - 1) / Work::kM) * p.experts : most_row_tiles(p, Work::kM);
  if (mt > 0x7FFFFFFF / nt) return hipErrorInvalidValue;  // more than memory holds
  const int64_t room = 256 * 8 / (WAVES_M * WAVES_N);  // eight waves a compute unit
  const int64_t groups = nt * mt < room ? (nt * mt + 7) / 8 * 8 : room;
  product_tile_kernel<T, WM, WAVES_M, WAVES_N, STAGES, A_NEXT, B_NEXT, SUM_ROWS>
      <<<dim3((unsigned)groups), dim3(64 * WAVES_M * WAVES_N), 0, s>>>(p);
  return hipGetLastError();
}

// ------------------------------------------------------------------ few rows
// 16 MT rows by 16 NT columns a workgroup, whose waves share the sum: a matrix goes from memory to the operands'
// registers, without LDS, as much of it under way as the registers hold, and the waves' sums are added at the end.
constexpr int kFewDepth = 4;  // steps of 32 that are asked for at once

template <class T, int MT, int NT, int WAVES, bool B_NEXT>
__global__ __launch_bounds__(64 * WAVES) void product_few_kernel(ProductArgs p) {
  constexpr int M = 16 * MT, N = 16 * NT, kWords = B_NEXT ? 4 : NT / 2;
  __shared__ float sums[WAVES][M][N];
  lds_poison(sums);
  RowTile r;
  RowTiles all;
  all.count(p, M);
  if (!all.find(p, M, (int)grid_row(), r)) return;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int n0 = blockIdx.x * N, m = r.end - r.first, n = p.n - n0 < N ? p.n - n0 : N;
  f32x4 c[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) c[i][j] = f32x4{};
  if (r.expert >= 0) {
    const T *a = static_cast<const T *>(p.a) + r.first * p.am;
    const T *b = static_cast<const T *>(p.b) + r.expert * p.be + n0 * p.bn;
    const int sa = (int)p.am, sb = (int)(B_NEXT ? p.bn : p.bk);
    // this lane's place in a step: of A the row lane % 16 and eight elements, of B as in Held
    const uint32_t oa = (uint32_t)(lane % 16 * sa * 2 + lane / 16 * 16);
    const uint32_t ob = (uint32_t)(B_NEXT ? lane % 16 * NT * sb * 2 + lane / 16 * 16
                                          : lane / 16 * 8 * sb * 2 + lane % 16 * NT * 2);
    // steps go round the waves, kFewDepth neighbouring ones each
#pragma unroll 1
    for (int k0 = wave * kFewDepth * 32; k0 < p.k; k0 += WAVES * kFewDepth * 32) {
      uint4 fa[kFewDepth][MT];
      uint32_t fb[kFewDepth][B_NEXT ? NT : 8][kWords];
#pragma unroll
      for (int d = 0; d < kFewDepth; ++d) {
        const int k = k0 + d * 32, left = p.k - k < 32 ? p.k - k : 32;  // may be none
        const uint32_t none = lane / 16 * 8 >= left ? kNowhere : 0u;
        const window_t wb = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T *>(b + (int64_t)k * (B_NEXT ? 1 : sb)), 0,
            left <= 0 ? 0 : (B_NEXT ? ((n - 1) * sb + left) * 2 : ((left - 1) * sb + n) * 2), 0x00020000);
#pragma unroll
        for (int i = 0; i < (B_NEXT ? NT : 8); ++i) {
          const uint32_t o = ob + (uint32_t)(i * sb * 2);
          if constexpr (B_NEXT)
            *reinterpret_cast<uint4 *>(fb[d][i]) =
                __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(wb, (int)(o | none), 0, 0));
          else if constexpr (NT == 8)
            *reinterpret_cast<uint4 *>(fb[d][i]) =
                __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(wb, (int)o, 0, 0));
          else
            *reinterpret_cast<uint2 *>(fb[d][i]) =
                __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(wb, (int)o, 0, 0));
        }
        const window_t wa = __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(a + k), 0,
                                                              left <= 0 ? 0 : ((m - 1) * sa + left) * 2, 0x00020000);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          fa[d][i] = __builtin_bit_cast(
              uint4, __builtin_amdgcn_raw_buffer_load_b128(wa, (int)((oa + (uint32_t)(i * 16 * sa * 2)) | none), 0, 0));
      }
#pragma unroll
      for (int d = 0; d < kFewDepth; ++d)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (B_NEXT)
              w[q] = fb[d][j][q];
            else
              w[q] = j % 2 == 0 ? pair_low(fb[d][2 * q][j / 2], fb[d][2 * q + 1][j / 2])
                                : pair_high(fb[d][2 * q][j / 2], fb[d][2 * q + 1][j / 2]);
          }
          const pack_t<T> f = __builtin_bit_cast(pack_t<T>, uint4{w[0], w[1], w[2], w[3]});
#pragma unroll
          for (int i = 0; i < MT; ++i) c[i][j] = mfma(__builtin_bit_cast(pack_t<T>, fa[d][i]), f, c[i][j]);
        }
    }
  }
  // lane l has the rows l / 16 * 4 + 0 .. 3 and the columns l % 16 * NT + 0 .. NT - 1 of each 16 rows
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < NT; ++j) sums[wave][i * 16 + lane / 16 * 4 + q][lane % 16 * NT + j] = c[i][j][q];
  __syncthreads();
  T *out = static_cast<T *>(p.c) + r.first * p.cm + n0;
  for (int x = threadIdx.x; x < M * N / 2; x += 64 * WAVES) {
    const int row = x / (N / 2), col = x % (N / 2) * 2;
    if (row >= m || col >= n) continue;
    float2 s = {0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float2 y = *reinterpret_cast<const float2 *>(&sums[w][row][col]);
      s.x += y.x;
      s.y += y.y;
    }
    typedef T pair_t __attribute__((ext_vector_type(2)));
    *reinterpret_cast<pair_t *>(out + row * p.cm + col) = pair_t{(T)s.x, (T)s.y};
  }
}

template <class T, int MT, int NT, int WAVES, bool B_NEXT>
hipError_t few(const ProductArgs &p, hipStream_t s) {
  const unsigned nt = (unsigned)((p.n + 16 * NT - 1) / (16 * NT));
  product_few_kernel<T, MT, NT, WAVES, B_NEXT>
      <<<rows_grid(nt, most_row_tiles(p, 16 * MT)), dim3(64 * WAVES), 0, s>>>(p);
  return hipGetLastError();
}

bool whole(const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; }
bool whole(int64_t n) { return n % 8 == 0; }

// Which kernel takes the rows: by how long each would take, as far as the host knows sizes (not how the rows are
// spread: experts that rows meet by chance have x rows each, x / size + 1/2 tiles).  Figures of bf16, in us.  On a grid
// of 4, 32 and 256 experts of 512 x 512, 2048 x 1024 and 1024 x 4096 with 1 to 400 rows each, both ways of storing, what the
// rule takes is within 1.2 us or 11% of the fastest of the four.  All rows are taken for rows of the call's experts: with a slice
// of the offsets, whose rows are fewer, it can take a kernel for more rows than there are: 32 of 256 experts of 2048 x 1024 with 4
// rows each 33.5 us for 23.0, with 24 47.9 for 34.2.
//  - 16 rows a workgroup: a start, then what its tiles draw, from the caches faster than from memory.  4 experts of 2048 x 1024
//    with 12 rows each: 8.8 (32 rows a workgroup 9.5, tiles of 128 x 256 31.8), with 400 44 (34, 33.5); 32 experts of 1024 x
//    4096 with a row each 26.6 (24.8, 32.8), with 48 80 (84, 45).
//  - 32 rows: the caches' draw halved, a start that grows with the sum, which four waves share.  4 experts of 1024 x 4096,
//    48 rows each: 12.0 (16 rows 16.7, tiles 19.4); 256 experts of 2048 x 1024 with 24 rows 257 (241, 205).
//  - 128 x 256: 0.42 a step where every workgroup has a compute unit to itself, else a round of 512; or the matrices' way
//    from memory.
//  - 256 x 256 takes as long as 1.85 of those; where the sum lies next to each other in a matrix, so that its lines come in halves,
//    1.6; few rounds are whole ones.  8 experts of 4096 x 14336 with 2048 rows 1710 for 1830, 256 experts of 2048 x 1024 with
//    256 510 for 430, of 1024 x 2048, lines in halves, 437 for 470, 64 experts of 2056 x 1416 with 469 rows 306 for 366, 32 of
//    2048 x 1024 with 400, two rounds for one, 91 for 69; their matrices' gradients 430 for 490 (256) and 320 for 345 (64).
enum Kind { kFew16, kFew32, kTile128, kTile256 };
Kind tile_kind(double tiles128, double tiles256, bool halves) {
  if (tiles128 <= 256) return kTile128;
  const auto rounds = [](double tiles, double each) { return tiles > 3 * each ? tiles / each : std::ceil(tiles / each); };
  const double as_long = halves ? 1.6 : 1.85;
  return tiles256 * as_long < tiles128 && rounds(tiles256, 256) * as_long < 2 * rounds(tiles128, 512) ? kTile256 : kTile128;
}
Kind rows_kind(const ProductArgs &p) {
  const bool halves = p.bk == 1;
  const double rows = (double)p.rows, met = p.experts * (1.0 - std::exp(-rows / p.experts)), x = rows / met;
  const auto tiles = [&](int size) { return met * std::fmax(1.0, x / size + 0.5); };
  const double matrix = (double)p.k * p.n * 2e-6, all = met * matrix;  // MB
  const double rate16 = all > 200 ? 5.5 : halves ? 5.2 : 9.0, rate32 = halves ? 7.0 : 8.5;
  const double few16 = 4.5 + std::fmax(tiles(16) * matrix / rate16, all / 5.8);
  const double few32 = 4 + p.k / (halves ? 256.0 : 512.0) + std::fmax(tiles(32) * matrix / rate32, all / 4.5);
  const double columns = std::ceil(p.n / 256.0), tiles128 = tiles(128) * columns;
  const double steps = (tiles128 <= 256 ? 0.42 : 0.95 * std::ceil(tiles128 / 512)) * p.k / 32, memory = all / 6.2;
  const double tile = 4 + std::fmax(steps, memory) + 0.1 * std::fmin(steps, memory);
  if (few16 <= few32 && few16 < tile) return kFew16;
  if (few32 < tile) return kFew32;
  return tile_kind(tiles128, tiles(256) * columns, halves);
}

template <class T, bool B_NEXT>
hipError_t rows_in(const ProductArgs &p, hipStream_t s) {
  switch (rows_kind(p)) {
    case kFew16:
      if constexpr (B_NEXT)
        return few<T, 1, 2, 8, true>(p, s);
      else  // wide rows of a matrix where there are workgroups enough (192 rows to 256 experts of 2048 x 1024: 72, else 80)
        return most_row_tiles(p, 16) * p.n >= 1024 * 128 ? few<T, 1, 8, 4, false>(p, s) : few<T, 1, 4, 8, false>(p, s);
    case kFew32: return few<T, 2, 4, 4, B_NEXT>(p, s);
    case kTile128: return tiles<T, 64, 2, 2, 3, true, B_NEXT, false>(p, s);
    case kTile256: return tiles<T, 64, 4, 2, 4, true, B_NEXT, false>(p, s);
  }
  return hipErrorInvalidValue;
}
template <class T>
hipError_t rows_of(const ProductArgs &p, hipStream_t s) {
  if (whole(p.a) && whole(p.b) && whole(p.c) && whole(p.am) && whole(p.be) && whole(p.bk == 1 ? p.bn : p.bk) &&
      whole(p.cm) && whole(p.n) && whole(p.k))
    return p.bk == 1 ? rows_in<T, true>(p, s) : rows_in<T, false>(p, s);
  return any<T, false>(p, s);
}
template <class T>
hipError_t weights_of(const ProductArgs &p, hipStream_t s) {
  if (whole(p.a) && whole(p.b) && whole(p.c) && whole(p.ak) && whole(p.bk) && whole(p.ce) && whole(p.cm) &&
      whole(p.m) && whole(p.n))
    return tile_kind(std::ceil(p.m / 128.0) * std::ceil(p.n / 256.0) * p.experts,
                     std::ceil(p.m / 256.0) * std::ceil(p.n / 256.0) * p.experts, false) == kTile256
               ? tiles<T, 64, 4, 2, 4, false, false, true>(p, s)
               : tiles<T, 64, 2, 2, 3, false, false, true>(p, s);
  return any<T, true>(p, s);
}

}  // namespace

hipError_t launch_product_rows(const ProductArgs &p, int dtype, hipStream_t s) {
  if (dtype == LAPSUM_F32) return any<f32, false>(p, s);
  return dtype == LAPSUM_BF16 ? rows_of<bf16>(p, s) : rows_of<f16>(p, s);
}
hipError_t launch_product_weights(const ProductArgs &p, int dtype, hipStream_t s) {
  if (dtype == LAPSUM_F32) return any<f32, true>(p, s);
  return dtype == LAPSUM_BF16 ? weights_of<bf16>(p, s) : weights_of<f16>(p, s);
}

}  // namespace lapsum
