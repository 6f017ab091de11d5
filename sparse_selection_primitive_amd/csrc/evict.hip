// Eviction from a cache by the account of the attention its entries received.
//
// Which entries stay is an exact selection: the accounts become unsigned keys
// whose order is the order of staying (protected entries highest, NaN
// lowest), the keep-th largest key is found digit by digit, and of the
// entries that hold exactly that key the lowest slots stay.  Nothing is
// sorted.  The survivors in front of slot `keep` stay where they are and those
// behind it fill the holes in front, so the bytes moved are those of the
// entries behind the budget that survive, not those of the budget.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;
constexpr int kMoveSlots = 256;  // slots per workgroup of the move

LDEV int64_t evict_length(const EvictArgs &a, int64_t row) {
  const int64_t n = a.lengths[row / a.heads];
  return n < 0 ? 0 : (n > a.capacity ? a.capacity : n);
}

struct RowKeys {
  const float *account;
  const int32_t *positions;
  int32_t sinks, from;  // protected: position < sinks or position >= from
  LDEV uint32_t key(int64_t i) const {
    const int32_t p = positions[i];
    const float x = account[i];
    if (p < sinks || p >= from) return 0xFFFFFFFFu;
    return x != x ? 0u : key_of(x + 0.0f);  // -0 counts as 0
  }
};
LDEV RowKeys row_keys(const EvictArgs &a, int64_t row) {
  RowKeys k;
  k.account = a.account + row * a.capacity;
  k.positions = a.positions + row * a.capacity;
  k.sinks = a.sinks;
  k.from = INT32_MAX;
  if (a.recent > 0) {
    const int64_t f = (int64_t)a.next_position[row / a.heads] - a.recent;
    k.from = (int32_t)(f < INT32_MIN ? INT32_MIN : f);
  }
  return k;
}

// exclusive count of `flag` over the workgroup's threads; `all` the total
LDEV int count_before(bool flag, int *waves, int &all) {
  const unsigned long long m = __ballot(flag);
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  if (lane == 0) waves[wave] = __popcll(m);
  __syncthreads();
  int before = __popcll(m & ((1ull << lane) - 1ull));
  all = 0;
  for (int w = 0; w < kSelectWaves; ++w) {
    if (w < wave) before += waves[w];
    all += waves[w];
  }
  __syncthreads();
  return before;
}

// kept[0 .. keep): one workgroup per cache row.  holes: scratch [rows][keep].
__global__ __launch_bounds__(kSelectThreads) void evict_select_kernel(const EvictArgs a, int32_t *holes) {
  struct Shared {
    uint32_t hist[256];
    int waves[kSelectWaves];
    uint32_t prefix;
    uint32_t want;  // how many entries of the keys that begin with `prefix` stay
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int64_t row = grid_row();
  if (row >= a.batch * a.heads) return;
  const int tid = threadIdx.x;
  const int64_t n = evict_length(a, row), keep = a.keep;
  int32_t *kept = a.kept + row * keep;
  for (int64_t i = tid; i < keep; i += kSelectThreads) kept[i] = i < n ? (int32_t)i : -1;
  if (n <= keep) return;
  holes += row * keep;
  const RowKeys keys = row_keys(a, row);

  uint32_t prefix = 0, want = (uint32_t)keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) sh.hist[tid] = 0;
    __syncthreads();
    const uint32_t high = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int64_t i = tid; i < n; i += kSelectThreads) {
      const uint32_t k = keys.key(i);
      if ((k & high) == prefix) atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 64) {  // bins from the top: lane l holds bins 255 - 4l .. 252 - 4l
      uint32_t v[4], sum = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) sum += v[x] = sh.hist[255 - 4 * tid - x];
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 64; o *= 2) {
        const uint32_t u = __shfl_up(inc, o, 64);
        if (tid >= o) inc += u;
      }
      uint32_t above = inc - sum;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (above < want && want <= above + v[x]) {
          sh.prefix = prefix | ((uint32_t)(255 - 4 * tid - x) << shift);
          sh.want = want - above;
        }
        above += v[x];
      }
    }
    __syncthreads();
    prefix = sh.prefix;
    want = sh.want;
    __syncthreads();
  }

  // slots in ascending order: of the entries with exactly the key `prefix` the first `want` stay
  int64_t same = 0, moved = 0;
  for (int64_t base = 0; base < n; base += kSelectThreads) {
    const int64_t i = base + tid;
    const uint32_t k = i < n ? keys.key(i) : 0u;
    int all;
    const bool equal = i < n && k == prefix;
    const int64_t rank = same + count_before(equal, sh.waves, all);
    same += all;
    const bool stays = i < n && (k > prefix || (equal && rank < (int64_t)want));
    const bool hole = i < keep && !stays, mover = i >= keep && stays;
    // a tile can hold both: the holes lie in front, and their number is not needed with the movers'
    const int h = count_before(hole, sh.waves, all);
    const int holes_here = all;
    if (hole) holes[moved + h] = (int32_t)i;
    if (base < keep) moved += holes_here;
    if (base + kSelectThreads >= keep) {
      if (base < keep) {  // the last tile with holes: from here on `moved` counts movers
        __syncthreads();
        moved = 0;
      }
      const int m = count_before(mover, sh.waves, all);
      if (mover) kept[holes[moved + m]] = (int32_t)i;
      moved += all;
    }
  }
}

// The survivors' accounts and positions, and the keys and values of those that move.
__global__ __launch_bounds__(256) void evict_move_kernel(const EvictArgs a) {
  const int64_t row = grid_row();
  if (row >= a.batch * a.heads) return;
  const int64_t n = evict_length(a, row);
  const int64_t after = n < a.keep ? n : a.keep;
  const int64_t base = (int64_t)blockIdx.x * kMoveSlots;
  const int64_t i = base + threadIdx.x;
  const int64_t b = row / a.heads, h = row % a.heads;
  if (base == 0 && h == 0 && threadIdx.x == 0) a.lengths_out[b] = (int32_t)after;
  if (base >= after) return;
  int from = -1;
  if (i < after) {
    from = a.kept[row * a.keep + i];
    a.account_out[row * a.capacity + i] = a.account[row * a.capacity + from];
    a.positions_out[row * a.capacity + i] = a.positions[row * a.capacity + from];
    if (from == (int)i) from = -1;
  }
  // each wave moves its own 64 slots' entries: 16 bytes a lane and entry
  const int lane = threadIdx.x % 64;
  const int packs = a.entry_bytes / 16, team = lane / packs, teams = 64 / packs;
  char *k = static_cast<char *>(a.k) + (b * a.kb + h * a.kh) * 2;
  char *v = static_cast<char *>(a.v) + (b * a.vb + h * a.vh) * 2;
  const int64_t first = base + (threadIdx.x / 64) * 64;
  unsigned long long todo = __ballot(from >= 0);
  while (todo != 0) {
    // the next `teams` entries, one per team
    int mine = -1;
    for (int t = 0; t < teams && todo != 0; ++t) {
      const int bit = __ffsll(todo) - 1;
      todo &= todo - 1;
      if (t == team) mine = bit;
    }
    const int src = __shfl(from, mine < 0 ? 0 : mine, 64);
    if (mine >= 0) {
      const int64_t at = (int64_t)(lane % packs) * 16, to = first + mine;
      const uint4 x = *reinterpret_cast<const uint4 *>(k + (int64_t)src * a.ke * 2 + at);
      const uint4 y = *reinterpret_cast<const uint4 *>(v + (int64_t)src * a.ve * 2 + at);
      *reinterpret_cast<uint4 *>(k + to * a.ke * 2 + at) = x;
      *reinterpret_cast<uint4 *>(v + to * a.ve * 2 + at) = y;
    }
  }
}

}  // namespace

size_t evict_workspace(int64_t batch, int64_t heads, int64_t capacity, int64_t keep) {
  return (size_t)(batch * heads) * (size_t)keep * sizeof(int32_t);
}

hipError_t launch_evict(const EvictArgs &a, hipStream_t s) {
  const int64_t rows = a.batch * a.heads;
  evict_select_kernel<<<rows_grid(1, rows), dim3(kSelectThreads), 0, s>>>(a, static_cast<int32_t *>(a.workspace));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  evict_move_kernel<<<rows_grid((unsigned)((a.keep + kMoveSlots - 1) / kMoveSlots), rows), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace lapsum
