// Eviction from a cache by the account of the attention its entries received.
//
// Which entries stay is an exact selection: the accounts become unsigned keys
// whose order is the order of staying (protected entries highest, NaN
// lowest), the keep-th largest key is found digit by digit, and of the
// entries that hold exactly that key the lowest slots stay.  Nothing is
// sorted.  The survivors in front of slot `keep` stay where they are and those
// behind it fill the holes in front, so the bytes moved are those of the
// entries behind the budget that survive, not those of the budget.
//
// Slots in order, let before(i) be the number of survivors before slot i and F the
// number of those in front of slot keep.  A hole at slot i is the
// (i - before(i))-th, a survivor behind the budget the (before(i) - F)-th, so
// one scan of the survivors ranks both.
//
// Rows of up to 16384 entries: one workgroup holds the row's keys in its
// registers, so the accounts are read once.  Longer rows: tiles of 4096
// entries on as many workgroups, one launch a digit; the last leaves the tiles' counts.
//
// What bounds it.  One entry over the budget: a chain of latencies, 7.5 us for 256 rows of 4097
// (the accounts and positions, 8.4 MB, read; a minimum over the row; then, read again from the cache, written with
// the slots, 12.6 MB).  130001 entries of 8 rows to a quarter: the moves, 39 us for 201 MB
// (5.2 TB/s), and five launches of 5 to 12 us before them that find the key and the places, the longest of
// them for its barriers, two in each of four rounds.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;
// Entries of a row that one workgroup holds: 16 a thread, what its registers allow.
// 8 rows of 8192 to a half take 23 us, by tiles 33; 256 rows of 16384 275 and 327, and 26 and 99 where one entry
// leaves; only few rows of 16384 that lose many are better by tiles (8 to a half: 41 and 36).  By the
// capacity, which the host knows, not the lengths: of 20000 slots one entry leaves 8 rows in 29 us, of 16384 in 12.
constexpr int kRowMax = 16384;
// Up to this many entries the selecting workgroup moves itself, beyond a second launch
// does (256 rows, 64 of 4160 entries leave: 15.7 us, with the second launch 21.1).
constexpr int kFewMoves = 64;
constexpr int kMoveSlots = 256;

LDEV int evict_length(const EvictArgs &a, int64_t row) {
  const int64_t n = a.lengths[row / a.heads];
  return (int)(n < 0 ? 0 : (n > a.capacity ? a.capacity : n));
}

struct RowKeys {
  const float *account;
  const int32_t *positions;
  int32_t sinks, past;  // protected: position < sinks or position > past
  LDEV uint32_t key(int64_t i) const { return key(positions[i], account[i]); }
  LDEV uint32_t key(int32_t p, float x) const {
    if (p < sinks || p > past) return 0xFFFFFFFFu;
    return x != x ? 0u : key_of(x + 0.0f);  // -0 counts as 0
  }
};
LDEV RowKeys row_keys(const EvictArgs &a, int64_t row) {
  RowKeys k;
  k.account = a.account + row * a.capacity;
  k.positions = a.positions + row * a.capacity;
  k.sinks = a.sinks;
  k.past = INT32_MAX;  // none
  if (a.recent > 0) {
    const int64_t past = (int64_t)a.next_position[row / a.heads] - a.recent - 1;
    k.past = (int32_t)(past < INT32_MIN ? INT32_MIN : past);  // the lowest position is below the sinks, so all are protected
  }
  return k;
}

// One entry's keys and values from slot `src` to slot `to`, 16 bytes a lane
// (`lane` of a.entry_bytes / 16).
struct Mover {
  char *k, *v;
  int64_t ke, ve;  // bytes
  LDEV Mover(const EvictArgs &a, int64_t row) {
    const int64_t b = row / a.heads, h = row % a.heads;
    k = static_cast<char *>(a.k) + (b * a.kb + h * a.kh) * 2;
    v = static_cast<char *>(a.v) + (b * a.vb + h * a.vh) * 2;
    ke = a.ke * 2;
    ve = a.ve * 2;
  }
  LDEV void move(int64_t src, int64_t to, int lane) const {
    const int64_t at = (int64_t)lane * 16;
    const uint4 x = *reinterpret_cast<const uint4 *>(k + src * ke + at);
    const uint4 y = *reinterpret_cast<const uint4 *>(v + src * ve + at);
    *reinterpret_cast<uint4 *>(k + to * ke + at) = x;
    *reinterpret_cast<uint4 *>(v + to * ve + at) = y;
  }
};

// From a histogram of 2^BITS bins (LDS), the bin in which the want-th entry
// from the top lies, by one wave: bin and the number wanted inside it.
template <int BITS>
LDEV void find_bin(const uint32_t *hist, uint32_t want, uint32_t *bin, uint32_t *inside) {
  constexpr int PER = (1 << BITS) / 64;
  const int lane = threadIdx.x % 64;
  uint32_t sum = 0;
#pragma unroll
  for (int x = 0; x < PER; ++x) sum += hist[(1 << BITS) - 1 - (lane * PER + x)];
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint32_t u = __shfl_up(inc, o, 64);
    if (lane >= o) inc += u;
  }
  uint32_t above = inc - sum;
  if (above < want && want <= inc) {
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const uint32_t b = (1 << BITS) - 1 - (lane * PER + x), n = hist[b];
      if (above < want && want <= above + n) {
        *bin = b;
        *inside = want - above;
      }
      above += n;
    }
  }
}

// ----------------------------------------------------- rows in registers
// V entries a thread: entry v * 1024 + thread.
template <int V>
__global__ __launch_bounds__(kSelectThreads) void evict_row_kernel(const EvictArgs a, const bool move_here) {
  struct Shared {
    uint32_t hist[256];
    int count[V * kSelectWaves];    // per round and wave, then the counts before
    unsigned long long worst[kSelectWaves];
    uint32_t prefix, want;
    int total;
    int32_t movers[V * kSelectThreads / 2];
    int32_t holes[kFewMoves];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int64_t row = grid_row();
  if (row >= a.batch * a.heads) return;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int n = evict_length(a, row), keep = (int)a.keep, after = n < keep ? n : keep;
  int32_t *kept = a.kept + row * a.keep;
  const RowKeys keys = row_keys(a, row);
  const int64_t base = row * a.capacity;
  const bool apart = a.account_out != a.account || a.positions_out != a.positions;
  if (tid == 0 && row % a.heads == 0) a.lengths_out[row / a.heads] = after;

  if (n <= keep) {
    for (int i = tid; i < keep; i += kSelectThreads) {
      kept[i] = i < n ? i : -1;
      if (i < n && apart) {
        a.account_out[base + i] = a.account[base + i];
        a.positions_out[base + i] = a.positions[base + i];
      }
    }
    return;
  }
  uint32_t k[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * kSelectThreads + tid;
    k[v] = i < n ? keys.key(i) : 0u;
  }

  if (n == keep + 1) {
    // one entry leaves: the smallest key, of equal ones the highest slot
    unsigned long long worst = ~0ull;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t i = (uint32_t)(v * kSelectThreads + tid);
      if ((int)i < n) {
        const unsigned long long x = ((unsigned long long)k[v] << 32) | (0xFFFFFFFFu - i);
        worst = x < worst ? x : worst;
      }
    }
    worst = wave_reduce(worst, [](unsigned long long x, unsigned long long y) { return x < y ? x : y; });
    if (lane == 0) sh.worst[wave] = worst;
    __syncthreads();
    worst = sh.worst[0];
#pragma unroll
    for (int w = 1; w < kSelectWaves; ++w) worst = sh.worst[w] < worst ? sh.worst[w] : worst;
    const int hole = (int)(0xFFFFFFFFu - (uint32_t)worst);  // == keep: the last entry itself leaves
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * kSelectThreads + tid;
      if (i >= keep) continue;
      const int from = i == hole ? keep : i;
      kept[i] = from;
      if (apart || from != i) {
        a.account_out[base + i] = a.account[base + from];
        a.positions_out[base + i] = a.positions[base + from];
      }
    }
    if (hole < keep && tid < a.entry_bytes / 16) Mover(a, row).move(keep, hole, tid);
    return;
  }

  uint32_t prefix = 0, want = (uint32_t)keep, equal = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) sh.hist[tid] = 0;
    __syncthreads();
    const uint32_t high = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v * kSelectThreads + tid < n && (k[v] & high) == prefix) atomicAdd(&sh.hist[(k[v] >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (wave == 0) find_bin<8>(sh.hist, want, &sh.prefix, &sh.want);
    __syncthreads();
    equal = sh.hist[sh.prefix];
    prefix |= sh.prefix << shift;
    want = sh.want;
    __syncthreads();
  }

  // counts before each round and wave; the scan's total in sh.total
  const auto scan = [&]() {
    __syncthreads();
    if (wave == 0) {
      constexpr int PER = (V * kSelectWaves + 63) / 64;
      int own[PER], sum = 0;
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int at = lane * PER + x;
        own[x] = at < V * kSelectWaves ? sh.count[at] : 0;
        sum += own[x];
      }
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 64; o *= 2) {
        const int u = __shfl_up(inc, o, 64);
        if (lane >= o) inc += u;
      }
      int before = inc - sum;
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int at = lane * PER + x;
        if (at < V * kSelectWaves) sh.count[at] = before;
        before += own[x];
      }
    }
    __syncthreads();
  };
  const unsigned long long below = (1ull << lane) - 1ull;

  // stays: bit v of a mask
  uint32_t stays = 0;
  if (equal != want) {  // some of the entries with exactly the last key leave: rank them by slot
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const unsigned long long m = __ballot(v * kSelectThreads + tid < n && k[v] == prefix);
      if (lane == 0) sh.count[v * kSelectWaves + wave] = __popcll(m);
    }
    scan();
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * kSelectThreads + tid;
    bool s = i < n && k[v] >= prefix;
    if (equal != want) {
      const bool same = i < n && k[v] == prefix;
      const unsigned long long m = __ballot(same);
      const uint32_t rank = (uint32_t)(sh.count[v * kSelectWaves + wave] + __popcll(m & below));
      if (same && rank >= want) s = false;
    }
    stays |= s ? 1u << v : 0u;
  }
  __syncthreads();
  if (tid == 0) sh.total = 0;
  int behind = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool s = ((stays >> v) & 1u) != 0;
    const unsigned long long m = __ballot(s);
    if (lane == 0) sh.count[v * kSelectWaves + wave] = __popcll(m);
    behind += __popcll(__ballot(s && v * kSelectThreads + tid >= keep));
  }
  __syncthreads();
  if (lane == 0 && behind != 0) atomicAdd(&sh.total, behind);
  scan();
  const int front = keep - sh.total;  // survivors in front of slot keep
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * kSelectThreads + tid;
    const bool s = ((stays >> v) & 1u) != 0;
    const int before = sh.count[v * kSelectWaves + wave] + __popcll(__ballot(s) & below);
    if (s && i >= keep) sh.movers[before - front] = i;  // fewer than n - keep and keep, so at most half of the row
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * kSelectThreads + tid;
    const bool s = ((stays >> v) & 1u) != 0;
    const int before = sh.count[v * kSelectWaves + wave] + __popcll(__ballot(s) & below);
    if (i >= keep) continue;
    const int from = s ? i : sh.movers[i - before];
    kept[i] = from;
    if (apart || from != i) {
      a.account_out[base + i] = a.account[base + from];
      a.positions_out[base + i] = a.positions[base + from];
    }
    if (!s && move_here) sh.holes[i - before] = i;
  }
  if (!move_here) return;  // the same for the whole launch
  __syncthreads();
  const Mover mover(a, row);
  const int packs = a.entry_bytes / 16, teams = 64 / packs, team = lane / packs;
  if (team < teams) {
    for (int m = wave * teams + team; m < sh.total; m += kSelectWaves * teams)
      mover.move(sh.movers[m], sh.holes[m], lane % packs);
  }
}

// The keys and values of the entries that move, from `kept`: a wave takes 64 slots.
__global__ __launch_bounds__(256) void evict_move_kernel(const EvictArgs a) {
  const int64_t row = grid_row();
  if (row >= a.batch * a.heads) return;
  const int n = evict_length(a, row), after = n < a.keep ? n : (int)a.keep;
  const int64_t i = (int64_t)blockIdx.x * kMoveSlots + threadIdx.x;
  if (n <= a.keep) return;
  const int from = i < after ? a.kept[row * a.keep + i] : -1;
  const int lane = threadIdx.x % 64;
  const int packs = a.entry_bytes / 16, team = lane / packs, teams = 64 / packs;
  const Mover mover(a, row);
  const int64_t first = i - lane;
  unsigned long long todo = __ballot(from >= 0 && from != (int)i);
  while (todo != 0) {
    // the next `teams` entries, one per team
    int mine = -1;
    for (int t = 0; t < teams && todo != 0; ++t) {
      const int bit = __ffsll(todo) - 1;
      todo &= todo - 1;
      if (t == team) mine = bit;
    }
    const int src = __shfl(from, mine < 0 ? 0 : mine, 64);
    if (mine >= 0) mover.move(src, first + mine, lane % packs);
  }
}

// ------------------------------------------------------------ long rows
// Tiles of a row: those of the slots in front of `keep`, then those behind.
constexpr int kTileThreads = 1024;
constexpr int kTileRounds = 4;
constexpr int kTileMin = kTileThreads * kTileRounds;
constexpr int kMaxTiles = 256;  // of either part; one thread each where they are summed up

struct Tiles {
  int size, front, count;  // entries per tile; tiles in front of keep; tiles
};
Tiles tiles_of(int64_t capacity, int64_t keep) {
  const int64_t longest = keep > capacity - keep ? keep : capacity - keep;
  int64_t size = (longest + kMaxTiles / 2 - 1) / (kMaxTiles / 2);
  size = (size + kTileMin - 1) / kTileMin * kTileMin;
  Tiles t;
  t.size = (int)size;
  t.front = (int)((keep + size - 1) / size);
  t.count = t.front + (int)((capacity - keep + size - 1) / size);
  return t;
}

struct LongRow {  // a row's state in the workspace
  uint32_t prefix[2], want[2];  // after a digit: the key's digits so far, and how many of those stay
  int32_t moves;
  int32_t pad;
};
struct LongArgs {
  EvictArgs e;
  Tiles t;
  LongRow *state;      // [rows]
  uint32_t *hist;      // [rows][3][2048]
  uint32_t *tails;     // [rows][tiles][kTail]: entries of a tile whose key is at least that of the first two
                       // digits found and last digit b (b = 1024: those above the first two digits)
  int32_t *holes, *movers;  // [rows][limit]
  int64_t limit;       // most entries that can move
};
constexpr int kDigits = 3;
constexpr int kBins = 2048;
LDEV int digit_shift(int d) { return d == 0 ? 21 : (d == 1 ? 10 : 0); }
LDEV uint32_t digit_mask(int d) { return d == 2 ? 1023u : 2047u; }
constexpr int kTail = 1025;

LDEV void tile_range(const LongArgs &a, int n, int tile, int &begin, int &end) {
  const int keep = (int)a.e.keep;
  const int64_t first = tile < a.t.front ? (int64_t)tile * a.t.size : keep + (int64_t)(tile - a.t.front) * a.t.size;
  const int64_t stop = tile < a.t.front ? keep : n;
  begin = (int)first;
  end = (int)(first + a.t.size < stop ? first + a.t.size : stop);
}

LDEV int block_sum(int v, int *waves) {
  v = wave_reduce(v, [](int x, int y) { return x + y; });
  __syncthreads();
  if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = v;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kTileThreads / 64; ++w) sum += waves[w];
  return sum;
}
// exclusive sum of v over the threads; `all` the total
LDEV int block_before(int v, int *waves, int &all) {
  int inc = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int u = __shfl_up(inc, o, 64);
    if ((int)(threadIdx.x % 64) >= o) inc += u;
  }
  __syncthreads();
  if (threadIdx.x % 64 == 63) waves[threadIdx.x / 64] = inc;
  __syncthreads();
  int before = inc - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < kTileThreads / 64; ++w) {
    if (w < (int)(threadIdx.x / 64)) before += waves[w];
    all += waves[w];
  }
  return before;
}

// The digits found so far, and how many of the entries that begin with them stay: digit d - 1 is
// the bin of its histogram in which the last survivor lies, two bins a thread.
LDEV void settle_digit(const LongArgs &a, int64_t row, int d, int *waves, uint32_t *found, uint32_t &prefix,
                       uint32_t &want) {
  prefix = 0;
  want = (uint32_t)a.e.keep;
  if (d == 0) return;
  static_assert(kBins == 2 * kTileThreads, "two bins a thread");
  const int pair = kTileThreads - 1 - (int)threadIdx.x;  // from the top
  const uint2 n = reinterpret_cast<const uint2 *>(a.hist + (row * kDigits + d - 1) * kBins)[pair];
  if (d > 1) {
    prefix = a.state[row].prefix[d - 2];
    want = a.state[row].want[d - 2];
  }
  int all;
  const uint32_t before = (uint32_t)block_before((int)(n.x + n.y), waves, all);
  if (before < want && want <= before + n.x + n.y) {
    const bool upper = want <= before + n.y;
    found[0] = 2 * (uint32_t)pair + (upper ? 1u : 0u);
    found[1] = want - before - (upper ? 0u : n.y);
  }
  __syncthreads();
  prefix |= found[0] << digit_shift(d - 1);
  want = found[1];
  if (d < kDigits && blockIdx.x == 0 && threadIdx.x == 0) {
    a.state[row].prefix[d - 1] = prefix;
    a.state[row].want[d - 1] = want;
  }
  __syncthreads();
}

// A tile's first kTileRounds rounds, one entry a thread and round: asked for before the digits are
// settled, so that one latency covers the other (with that, and the digits found by the whole workgroup,
// 8 rows of 131072 take 70 us instead of 81).  All of a tile in rows of up to 2^19 entries.
struct Ahead {
  int32_t position[kTileRounds];
  float account[kTileRounds];
  LDEV Ahead(const RowKeys &keys, int begin, int n) {
#pragma unroll
    for (int x = 0; x < kTileRounds; ++x) {
      const int i = min(begin + x * kTileThreads + (int)threadIdx.x, n - 1);
      position[x] = keys.positions[i];
      account[x] = keys.account[i];
    }
  }
};

__global__ __launch_bounds__(256) void evict_clear_kernel(uint32_t *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// Digit d of the keys that begin with the digits found so far.  With the last one a tile also
// leaves its counts from every digit on, so that the next launch, which finds the
// digit, has the tiles' survivors at once (8 rows of 131072: 83 us with a launch of its own for that, 81 without).
__global__ __launch_bounds__(kTileThreads) void evict_digit_kernel(const LongArgs a, const int d) {
  struct Shared {
    uint32_t hist[kBins];
    uint32_t found[2];
    int waves[kTileThreads / 64];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int64_t row = grid_row();
  if (row >= a.e.batch * a.e.heads) return;
  const int n = evict_length(a.e, row);
  if (n <= a.e.keep) return;
  const RowKeys keys = row_keys(a.e, row);
  int begin, end;
  tile_range(a, n, blockIdx.x, begin, end);
  const Ahead ahead(keys, begin, n);
  for (int i = threadIdx.x; i < kBins; i += kTileThreads) sh.hist[i] = 0;
  uint32_t prefix, want;
  settle_digit(a, row, d, sh.waves, sh.found, prefix, want);
  __syncthreads();
  const int shift = digit_shift(d);
  const uint32_t mask = digit_mask(d), high = d == 0 ? 0u : ~((mask << shift) | ((1u << shift) - 1u));
  int above = 0;
  const auto count = [&](uint32_t k) {
    if ((k & high) == prefix) atomicAdd(&sh.hist[(k >> shift) & mask], 1u);
    above += (k & high) > prefix ? 1 : 0;
  };
#pragma unroll
  for (int x = 0; x < kTileRounds; ++x)
    if (begin + x * kTileThreads + (int)threadIdx.x < end) count(keys.key(ahead.position[x], ahead.account[x]));
#pragma unroll 4
  for (int i = begin + kTileMin + (int)threadIdx.x; i < end; i += kTileThreads) count(keys.key(i));
  __syncthreads();
  uint32_t *to = a.hist + (row * kDigits + d) * kBins;
  for (int i = threadIdx.x; i < kBins; i += kTileThreads)
    if (sh.hist[i] != 0) atomicAdd(&to[i], sh.hist[i]);
  if (d != kDigits - 1) return;
  static_assert(kTileThreads == kTail - 1, "one thread for each last digit");
  above = block_sum(above, sh.waves);
  const int digit = kTileThreads - 1 - (int)threadIdx.x, here = (int)sh.hist[digit];
  int all;
  const int more = block_before(here, sh.waves, all);
  uint32_t *tail = a.tails + (row * a.t.count + blockIdx.x) * kTail;
  tail[digit] = (uint32_t)(above + more + here);
  if (threadIdx.x == 0) tail[kTail - 1] = (uint32_t)above;
}

// Ranks of the holes and of the survivors that fill them; the accounts and
// positions of the entries that stay where they are.
__global__ __launch_bounds__(kTileThreads) void evict_place_kernel(const LongArgs a) {
  struct Shared {
    uint32_t found[2];
    int waves[kTileThreads / 64];
    int pre[2];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int64_t row = grid_row();
  if (row >= a.e.batch * a.e.heads) return;
  const int tid = threadIdx.x, tile = blockIdx.x;
  const int n = evict_length(a.e, row), keep = (int)a.e.keep, after = n < keep ? n : keep;
  int32_t *kept = a.e.kept + row * a.e.keep;
  const int64_t base = row * a.e.capacity;
  const bool apart = a.e.account_out != a.e.account || a.e.positions_out != a.e.positions;
  if (tile == 0 && tid == 0) {
    if (row % a.e.heads == 0) a.e.lengths_out[row / a.e.heads] = after;
    if (n <= keep) a.state[row].moves = 0;
  }
  if (n <= keep) {
    if (tile >= a.t.front) return;
    const int64_t first = (int64_t)tile * a.t.size, stop = first + a.t.size < keep ? first + a.t.size : keep;
    for (int64_t i = first + tid; i < stop; i += kTileThreads) {
      kept[i] = i < n ? (int32_t)i : -1;
      if (i < n && apart) {
        a.e.account_out[base + i] = a.e.account[base + i];
        a.e.positions_out[base + i] = a.e.positions[base + i];
      }
    }
    return;
  }
  const RowKeys keys = row_keys(a.e, row);
  int begin, end;
  tile_range(a, n, tile, begin, end);
  const Ahead ahead(keys, begin, n);
  uint32_t key, of_key;
  settle_digit(a, row, kDigits, sh.waves, sh.found, key, of_key);
  const int want = (int)of_key;
  // tiles' survivors: entries above the key, and of those that hold it the first `want` of the row
  int all;
  int2 mine = {0, 0};  // entries above the key, entries that hold it
  if (tid < a.t.count) {
    const uint32_t *tail = a.tails + (row * a.t.count + tid) * kTail + (key & digit_mask(kDigits - 1));
    mine.x = (int)tail[1];
    mine.y = (int)(tail[0] - tail[1]);
  }
  const int same_before = block_before(mine.y, sh.waves, all);
  int left = want - same_before;
  left = left < 0 ? 0 : (left < mine.y ? left : mine.y);
  const int stay = mine.x + left;
  const int stay_before = block_before(stay, sh.waves, all);
  const int front = block_sum(tid < a.t.front ? stay : 0, sh.waves);
  __syncthreads();
  if (tid == tile) {
    sh.pre[0] = same_before;
    sh.pre[1] = stay_before;
  }
  __syncthreads();
  int same_at = sh.pre[0], stay_at = sh.pre[1];
  if (tile == 0 && tid == 0) a.state[row].moves = keep - front;

  const int lane = tid % 64, wave = tid / 64;
  const unsigned long long below = (1ull << lane) - 1ull;
  const auto round = [&](int at, uint32_t k) {
    const int i = at + tid;
    const bool same = i < end && k == key;
    // both counts of a wave in one word
    const unsigned long long ms = __ballot(same), mg = __ballot(i < end && k > key);
    __syncthreads();
    if (lane == 0) sh.waves[wave] = __popcll(ms) | (__popcll(mg) << 16);
    __syncthreads();
    int same_b = same_at + __popcll(ms & below), above_b = __popcll(mg & below), same_all = 0, above_all = 0;
#pragma unroll
    for (int w = 0; w < kTileThreads / 64; ++w) {
      const int x = sh.waves[w];
      if (w < wave) {
        same_b += x & 0xFFFF;
        above_b += x >> 16;
      }
      same_all += x & 0xFFFF;
      above_all += x >> 16;
    }
    // survivors before this slot: those above the key, and the holders of the key among the first `want`
    const int holders = (same_b < want ? same_b : want) - (same_at < want ? same_at : want);
    const int before = stay_at + above_b + holders;
    const bool s = i < end && (k > key || (same && same_b < want));
    if (i < end) {
      if (tile < a.t.front) {
        if (s) {
          kept[i] = i;
          if (apart) {
            a.e.account_out[base + i] = a.e.account[base + i];
            a.e.positions_out[base + i] = a.e.positions[base + i];
          }
        } else {
          a.holes[row * a.limit + i - before] = i;
        }
      } else if (s) {
        a.movers[row * a.limit + before - front] = i;
      }
    }
    const int same_next = same_at + same_all;
    stay_at += above_all + (same_next < want ? same_next : want) - (same_at < want ? same_at : want);
    same_at = same_next;
  };
#pragma unroll
  for (int x = 0; x < kTileRounds; ++x)
    if (begin + x * kTileThreads < end)  // the same for the whole workgroup
      round(begin + x * kTileThreads, keys.key(ahead.position[x], ahead.account[x]));
  for (int at = begin + kTileMin; at < end; at += kTileThreads) round(at, keys.key(min(at + tid, n - 1)));
}

// The entries that move, a team of lanes each.
__global__ __launch_bounds__(256) void evict_fill_kernel(const LongArgs a) {
  const int64_t row = grid_row();
  if (row >= a.e.batch * a.e.heads) return;
  const int moves = a.state[row].moves;
  const int lane = threadIdx.x % 64;
  const int packs = a.e.entry_bytes / 16, teams = 64 / packs, team = lane / packs;
  if (team >= teams) return;
  const Mover mover(a.e, row);
  const int64_t base = row * a.e.capacity;
  const int step = (int)gridDim.x * 4 * teams;
  for (int m = ((int)blockIdx.x * 4 + (int)threadIdx.x / 64) * teams + team; m < moves; m += step) {
    const int to = a.holes[row * a.limit + m], src = a.movers[row * a.limit + m];
    mover.move(src, to, lane % packs);
    if (lane % packs == 0) {
      a.e.kept[row * a.e.keep + to] = src;
      a.e.account_out[base + to] = a.e.account[base + src];
      a.e.positions_out[base + to] = a.e.positions[base + src];
    }
  }
}

struct LongLayout {
  size_t state, hist, tails, holes, movers, bytes;
  int64_t limit;
};
LongLayout long_layout(int64_t rows, int64_t capacity, int64_t keep) {
  const Tiles t = tiles_of(capacity, keep);
  LongLayout l;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  l.limit = keep < capacity - keep ? keep : capacity - keep;
  if (l.limit < 1) l.limit = 1;
  l.state = take((size_t)rows * sizeof(LongRow));
  l.hist = take((size_t)rows * kDigits * kBins * sizeof(uint32_t));
  l.tails = take((size_t)rows * t.count * kTail * sizeof(uint32_t));
  l.holes = take((size_t)(rows * l.limit) * sizeof(int32_t));
  l.movers = take((size_t)(rows * l.limit) * sizeof(int32_t));
  l.bytes = at;
  return l;
}

hipError_t evict_long(const EvictArgs &e, hipStream_t s) {
  const int64_t rows = e.batch * e.heads;
  const LongLayout l = long_layout(rows, e.capacity, e.keep);
  char *ws = static_cast<char *>(e.workspace);
  LongArgs a;
  a.e = e;
  a.t = tiles_of(e.capacity, e.keep);
  a.state = reinterpret_cast<LongRow *>(ws + l.state);
  a.hist = reinterpret_cast<uint32_t *>(ws + l.hist);
  a.tails = reinterpret_cast<uint32_t *>(ws + l.tails);
  a.holes = reinterpret_cast<int32_t *>(ws + l.holes);
  a.movers = reinterpret_cast<int32_t *>(ws + l.movers);
  a.limit = l.limit;
  const int64_t words = rows * kDigits * kBins, blocks = (words + 1023) / 1024;
  evict_clear_kernel<<<dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s>>>(a.hist, words);
  hipError_t err = hipGetLastError();
  const dim3 grid = rows_grid((unsigned)a.t.count, rows), threads(kTileThreads);
  for (int d = 0; d < kDigits && err == hipSuccess; ++d) {
    evict_digit_kernel<<<grid, threads, 0, s>>>(a, d);
    err = hipGetLastError();
  }
  if (err != hipSuccess) return err;
  evict_place_kernel<<<grid, threads, 0, s>>>(a);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  // about 8 entries a team, on 4096 workgroups at most over all rows
  const int64_t per = 4 * (64 / (e.entry_bytes / 16)) * 8;
  int64_t fill = (a.limit + per - 1) / per, most = 4096 / rows;
  if (most < 1) most = 1;
  if (fill > most) fill = most;
  evict_fill_kernel<<<rows_grid((unsigned)fill, rows), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <int V>
hipError_t evict_rows(const EvictArgs &a, hipStream_t s) {
  const int64_t rows = a.batch * a.heads, limit = a.keep < a.capacity - a.keep ? a.keep : a.capacity - a.keep;
  const bool here = limit <= kFewMoves;
  evict_row_kernel<V><<<rows_grid(1, rows), dim3(kSelectThreads), 0, s>>>(a, here);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || here) return e;
  evict_move_kernel<<<rows_grid((unsigned)((a.keep + kMoveSlots - 1) / kMoveSlots), rows), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t evict_workspace(int64_t batch, int64_t heads, int64_t capacity, int64_t keep) {
  return capacity > kRowMax ? long_layout(batch * heads, capacity, keep).bytes : 0;
}

hipError_t launch_evict(const EvictArgs &a, hipStream_t s) {
  if (a.capacity > kRowMax) return evict_long(a, s);
  // Entries a thread by the row's slots.  5, so that a budget of 4096 and the entry over it do not take 8 (256 rows
  // of 4097 slots: 7.2 us, with 8 a thread 7.9; of 3000 6.5 and 7.2; 8 rows of 4097 to 2048 17.0 and 18.5).
  // 3, 9 and 12 as well would save 0.1 us of 2049 slots, 1.0 of 8193 and 0.8 of 12000, and are not built.
  if (a.capacity <= 2 * kSelectThreads) return evict_rows<2>(a, s);
  if (a.capacity <= 5 * kSelectThreads) return evict_rows<5>(a, s);
  if (a.capacity <= 8 * kSelectThreads) return evict_rows<8>(a, s);
  return evict_rows<16>(a, s);
}

}  // namespace lapsum
