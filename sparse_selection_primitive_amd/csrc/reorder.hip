// The caches of a beam search follow its beams: beam j's cache becomes its parent's, in place.
//
// Parents are any map of the beams: some caches are taken over by several, some by none, and some change
// places.  One thread holds the same 16 bytes of every beam's cache: it reads those that another beam takes over, then
// writes, so no order among the beams matters and no second cache is needed.  A beam that is its own parent is
// not written, a cache that nobody else takes is not read.
//
// Bound by memory: every cache that is taken over read once, every changed one written once.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

LDEV int clamped(int64_t n, int64_t capacity) { return (int)(n < 0 ? 0 : (n > capacity ? capacity : n)); }

// One column: what the beams hold at `at` elements of a V, `stride` (bytes) between beams.
template <int NB, class V>
struct Column {
  V held[NB];
  template <class S>
  LDEV void take(const S &sh, const char *at, int64_t stride, int entry) {
#pragma unroll
    for (int p = 0; p < NB; ++p)
      if (entry < sh.reach(p)) held[p] = *reinterpret_cast<const V *>(at + p * stride);
  }
  template <class S>
  LDEV void give(const S &sh, char *at, int64_t stride, int entry) const {
#pragma unroll
    for (int p = 0; p < NB; ++p) {
      if (entry >= sh.reach(p)) continue;
      for (uint64_t left = sh.takers(p); left != 0; left &= left - 1)
        *reinterpret_cast<V *>(at + __builtin_ctzll(left) * stride) = held[p];
    }
  }
};

// which beams take each beam's cache over, and how many entries (0 where none does)
template <int NB>
struct Family {
  uint64_t mask[NB];
  int length[NB];
  LDEV int reach(int p) const { return __builtin_amdgcn_readfirstlane(length[p]); }
  LDEV uint64_t takers(int p) const {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)mask[p]);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(mask[p] >> 32));
    return (uint64_t)hi << 32 | lo;
  }
};

template <int NB, class V>
__global__ __launch_bounds__(256) void reorder_kernel(ReorderArgs a, int tile) {
  __shared__ Family<NB> sh;
  lds_poison(sh);
  const int64_t b = grid_row() / a.heads, h = grid_row() % a.heads;
  if (b >= a.searches) return;
  const int lane = lane_id(), beams = a.beams;
  int parent = -1, length = 0;
  if (lane < beams) {
    parent = a.parents[b * beams + lane];
    length = clamped(a.lengths[b * beams + lane], a.capacity);
  }
  if (parent < 0 || parent >= beams) parent = -1;
  const int theirs = __shfl(length, parent < 0 ? 0 : parent, 64);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x < beams) a.lengths_out[b * beams + lane] = parent < 0 ? 0 : theirs;
  if (threadIdx.x < 64) {
#pragma unroll 1
    for (int p = 0; p < NB; ++p) {
      const uint64_t m = __ballot(lane < beams && parent == p && lane != p);
      if (lane == 0) {
        sh.mask[p] = m;
        sh.length[p] = m != 0 ? read_lane(length, p) : 0;
      }
    }
  }
  __syncthreads();
  int most = 0;
#pragma unroll
  for (int p = 0; p < NB; ++p) most = sh.reach(p) > most ? sh.reach(p) : most;
  const int64_t e0 = (int64_t)blockIdx.x * tile;
  if (e0 >= most) return;
  const int entries = most - (int)e0 < tile ? most - (int)e0 : tile;
  const int per = a.width * 2 / (int)sizeof(V);  // columns of an entry
  char *k = static_cast<char *>(a.k) + (b * beams * a.kb + h * a.kh + e0 * a.ke) * 2;
  char *v = static_cast<char *>(a.v) + (b * beams * a.vb + h * a.vh + e0 * a.ve) * 2;
  for (int u = threadIdx.x; u < entries * per; u += 256) {
    const int e = u / per, c = (u - e * per) * (int)sizeof(V);
    Column<NB, V> x;
    char *at = k + e * a.ke * 2 + c;
    x.take(sh, at, a.kb * 2, (int)e0 + e);
    x.give(sh, at, a.kb * 2, (int)e0 + e);
    at = v + e * a.ve * 2 + c;
    x.take(sh, at, a.vb * 2, (int)e0 + e);
    x.give(sh, at, a.vb * 2, (int)e0 + e);
  }
  const int64_t first = (b * beams * a.heads + h) * a.capacity + e0, beam = a.heads * a.capacity * 4;
  for (int e = threadIdx.x; e < entries; e += 256) {
    Column<NB, uint32_t> x;
    if (a.account != nullptr) {
      char *at = reinterpret_cast<char *>(a.account + first + e);
      x.take(sh, at, beam, (int)e0 + e);
      x.give(sh, at, beam, (int)e0 + e);
    }
    if (a.positions != nullptr) {
      char *at = reinterpret_cast<char *>(a.positions + first + e);
      x.take(sh, at, beam, (int)e0 + e);
      x.give(sh, at, beam, (int)e0 + e);
    }
  }
}

template <int NB, class V>
hipError_t reorder(const ReorderArgs &a, hipStream_t s) {
  const int64_t rows = a.searches * a.heads;
  const int tile = 32;
  reorder_kernel<NB, V><<<rows_grid((unsigned)((a.capacity + tile - 1) / tile), rows), dim3(256), 0, s>>>(a, tile);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_reorder(const ReorderArgs &a, hipStream_t s) {
  // a thread's registers hold the column: 16 bytes of up to 16 beams, 4 of up to 64
  if (a.beams <= 4) return reorder<4, uint4>(a, s);
  if (a.beams <= 8) return reorder<8, uint4>(a, s);
  if (a.beams <= 16) return reorder<16, uint4>(a, s);
  return reorder<64, uint32_t>(a, s);
}

}  // namespace lapsum
