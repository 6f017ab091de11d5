// The caches of a beam search follow its beams: beam j's cache becomes its parent's, in place.
//
// Parents are any map of the beams: some caches are taken over by several, some by none, and some change
// places.  One thread holds the same 16 bytes of every beam's cache: it reads those that another beam takes over, then
// writes, so no order among the beams matters and no second cache is needed.  A beam that is its own parent is
// not written, a cache that nobody else takes is not read.
//
// Bound by memory: every cache that is taken over read once, every changed one written once.  16 searches of 4 beams, 8
// heads of up to 8192 entries of 128, with accounts and positions, by the parents: 1.55 to 2.23 GB in 311 to 460 us (4.8 to
// 5.4 TB/s; a copy reaches 5.2); 12 of 5 beams, 2 heads of up to 3001 of 96: 110 to 141 MB in 19 to 26 us; one search of 4 beams of 1000
// entries 5.0 to 7.5 us for 8 to 33 MB.  From
// 17 beams on a thread holds 8 bytes of each beam's, and few threads fit: 40 beams of 4000 entries 3.0 TB/s.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

// (structs of as many would go through memory)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

LDEV int clamped(int64_t n, int64_t capacity) { return (int)(n < 0 ? 0 : (n > capacity ? capacity : n)); }

// The beams of a search, one a lane: whose cache each takes over, and how many entries it has.  Asked with all lanes.
struct Family {
  int parent, length;  // parent -1: none, or itself
  // the beams that take p's cache over
  LDEV uint64_t takers(int p) const { return __ballot(parent == p); }
  // its entries, none where nobody takes it
  LDEV int reach(int p) const { return takers(p) != 0 ? read_lane(length, p) : 0; }
};

// One column: what the beams hold at `at`, `stride` bytes from beam to beam, of entry `entry`.
template <int NB, class V>
struct Column {
  V held[NB];
  LDEV void take(const Family &f, const char *at, int64_t stride, int entry) {
#pragma unroll
    for (int p = 0; p < NB; ++p) {
      const int reach = f.reach(p);
      if (entry < reach) held[p] = *reinterpret_cast<const V *>(at + p * stride);
    }
  }
  LDEV void give(const Family &f, char *at, int64_t stride, int entry) const {
#pragma unroll
    for (int p = 0; p < NB; ++p) {
      const int reach = f.reach(p);
      for (uint64_t left = f.takers(p); left != 0; left &= left - 1) {
        const int j = __builtin_ctzll(left);
        if (entry < reach) *reinterpret_cast<V *>(at + j * stride) = held[p];
      }
    }
  }
};

constexpr int kNoEntry = 0x7FFFFFFF;
constexpr int64_t kMostGroups = 1 << 20;  // of a search and head; beyond, workgroups take several parts

// Workgroups of twice `tile` entries' keys or values (in turn; 256 columns of V are a tile), then, blockIdx.x from `parts`
// on, of 256 entries' accounts and positions.  Keys and values of one tile by one workgroup: 16 searches of 4 beams with up to
// 8192 entries 430 us, by two of two tiles 370 (short caches the same, 7.0), of 8 tiles 377 (12.5), with streamed accesses 366 to 372.
template <int NB, class V>
__global__ __launch_bounds__(256) void reorder_kernel(ReorderArgs a, int tile, int64_t parts) {
  const uint32_t row = (uint32_t)grid_row(), heads = (uint32_t)a.heads;  // at most 2^24
  const int64_t b = row / heads, h = row % heads;
  if (b >= a.searches) return;
  const int lane = lane_id(), beams = a.beams;
  Family f{-1, 0};
  if (lane < beams) {
    f.parent = a.parents[b * beams + lane];
    f.length = clamped(a.lengths[b * beams + lane], a.capacity);
  }
  const bool there = f.parent >= 0 && f.parent < beams;
  const int theirs = __shfl(f.length, there ? f.parent : 0, 64);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x < beams) a.lengths_out[b * beams + lane] = there ? theirs : 0;
  if (!there || f.parent == lane) f.parent = -1;
  int most = 0;  // entries of the longest cache that is taken over
#pragma unroll
  for (int p = 0; p < NB; ++p) {
    const int reach = f.reach(p);
    most = reach > most ? reach : most;
  }
  for (int64_t part = blockIdx.x; part < parts; part += gridDim.x) {
    const int64_t e0 = part / 2 * (2 * tile);
    if (e0 >= most) break;
    const bool values = part % 2 != 0;
    if (values && a.one) continue;
    const int64_t beam = (values ? a.vb : a.kb) * 2, head = (values ? a.vh : a.kh) * 2, step = (values ? a.ve : a.ke) * 2;
    const int per = a.width * 2 / (int)sizeof(V);  // columns of an entry
    const int e = threadIdx.x / per, c = (threadIdx.x - e * per) * (int)sizeof(V);
    char *at = static_cast<char *>(values ? a.v : a.k) + b * beams * beam + h * head + (e0 + e) * step + c;
    char *then = at + tile * step;
    const int entry = e < tile ? (int)e0 + e : kNoEntry, second = e < tile ? (int)e0 + tile + e : kNoEntry;
    Column<NB, V> x, y;
    x.take(f, at, beam, entry);
    constexpr bool kBoth = NB * sizeof(V) <= 128;  // where the registers hold both tiles' columns
    if (kBoth) y.take(f, then, beam, second);
    x.give(f, at, beam, entry);
    if (!kBoth) y.take(f, then, beam, second);
    y.give(f, then, beam, second);
  }
  if (a.account == nullptr && a.positions == nullptr) return;
  // the workgroups behind those of the keys and values, or where there are none (very long caches), all
  const int64_t before = (int64_t)gridDim.x > parts ? parts : 0;
  for (int64_t part = (int64_t)blockIdx.x - before; part >= 0; part += gridDim.x - before) {
    const int64_t e0 = part * 256 + threadIdx.x;
    if (part * 256 >= most) break;
    const int entry = e0 < most ? (int)e0 : kNoEntry;
    const int64_t first = ((b * beams * a.heads + h) * a.capacity + e0) * 4, beam = a.heads * a.capacity * 4;
    char *account = reinterpret_cast<char *>(a.account) + first, *positions = reinterpret_cast<char *>(a.positions) + first;
    Column<NB, uint32_t> x, y;
    if (a.account != nullptr) x.take(f, account, beam, entry);
    if (a.positions != nullptr) y.take(f, positions, beam, entry);
    if (a.account != nullptr) x.give(f, account, beam, entry);
    if (a.positions != nullptr) y.give(f, positions, beam, entry);
  }
}

template <int NB, class V>
hipError_t reorder(const ReorderArgs &a, hipStream_t s) {
  const int per = a.width * 2 / (int)sizeof(V), tile = 256 / per;
  const int64_t parts = (a.capacity + 2 * tile - 1) / (2 * tile) * 2;
  const int64_t extra = a.account != nullptr || a.positions != nullptr ? (a.capacity + 255) / 256 : 0;
  const int64_t groups = parts + extra <= kMostGroups ? parts + extra : kMostGroups;
  reorder_kernel<NB, V><<<rows_grid((unsigned)groups, a.searches * a.heads), dim3(256), 0, s>>>(a, tile, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_reorder(const ReorderArgs &a, hipStream_t s) {
  // a thread's registers hold the column: 16 bytes of up to 16 beams, 8 of up to 64
  if (a.beams <= 4) return reorder<4, u32x4>(a, s);
  if (a.beams <= 8) return reorder<8, u32x4>(a, s);
  if (a.beams <= 16) return reorder<16, u32x4>(a, s);
  if (a.beams <= 32) return reorder<32, u32x2>(a, s);
  return reorder<64, u32x2>(a, s);
}

}  // namespace lapsum
