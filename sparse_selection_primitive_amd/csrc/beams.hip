// One step of a beam search: the k best continuations of a search's beams over beams and vocabulary.
//
// score(i, v) = scores[i] + (x - M) - log S with M = max_u x[i, u] and S = sum_u e^(x[i, u] - M).
//
// First launch: rows are cut into parts of 512 tokens (16 lanes a part); each leaves its maximum, and each
// workgroup its sum of e^(x - maximum).  That is the one pass over the logits, and no selection takes part in it.
// Second launch, a workgroup a search: the sums give every beam's log S, so the parts' maxima become scores.  All of
// the k best continuations lie in the k best parts (by score, then by place): a part
// that is not among them has k parts before it, each with a continuation before all of its own.  So only
// these k parts are read again, and of their tokens only those at or above the k-th best part's score can be among the
// k best.
//
// Bound by the logits' one pass where they are many (64 searches of 8 beams over 131072 tokens, bf16, a tenth of the beams ended:
// 121 MB in 22.8 us, 5.3 TB/s; the exponentials' vector instructions would take 15), else by latencies: the second launch, 6.2 to
// 8.3 us, is a chain of two rounds of memory and eight barriers (sums 2.0, scores and their k-th 1.2, parts 0.9, tokens
// 1.6).  Workgroups of 256 threads take 7.8 to 13 there: the same steps with more a thread.
//
// Equal scores go by their place, and places are unique, so results do not depend on the order in which candidates are
// gathered (an atomic count in LDS).
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

constexpr int kPart = 512;        // tokens, or a power of two times as many
constexpr int kMostParts = 8192;  // of a search: the second launch's share stays small
constexpr int kThreads = 1024, kRows = kThreads / 16;
constexpr int kList = 1024;
constexpr float kLog2e = 1.44269504f;

// 16 bytes of a row, which may start at any element
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Loose {
  pack_t<T> v;
};
// the tokens [t, t + N) of a row, -inf past its end
template <class T>
LDEV void load_tokens(const T *row, int t, int vocab, float (&x)[Pack<T>::N]) {
  constexpr int N = Pack<T>::N;
  if (t + N <= vocab) {
    const pack_t<T> w = reinterpret_cast<const Loose<T> *>(row + t)->v;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)w[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = t + i < vocab ? (float)row[t + i] : -INFINITY;
  }
}

// An exponential, a product and an addition to a join: up to 4 2^-24 of the sum.  With the rounded arguments, which weigh as much as
// the row's entropy, a row of V tokens errs by (33 + 2.3 ln V + 4 joins) 2^-24 at most, 106 for 50000; ascending maxima 5.
//
// joins (m, s) with (m2, s2): sums of e^(x - maximum), of -inf alone (-inf, 0); where the maximum is
// +inf, s counts what is +inf
LDEV void join(float &m, float &s, float m2, float s2) {
  const float to = fmaxf(m, m2);
  // at equal maxima the difference would be NaN for infinities
  s = (m == to ? s : s * __builtin_amdgcn_exp2f((m - to) * kLog2e)) +
      (m2 == to ? s2 : s2 * __builtin_amdgcn_exp2f((m2 - to) * kLog2e));
  m = to;
}
template <int M>
LDEV void join_lanes(float &m, float &s) {
  const float m2 = pair_lane<M>(m), s2 = pair_lane<M>(s);
  join(m, s, m2, s2);
}

template <class T>
__global__ __launch_bounds__(256) void beam_parts_kernel(BeamArgs a) {
  constexpr int N = Pack<T>::N, L = kPart / (16 * N);
  const int64_t row = grid_row();
  if (row >= a.batch * a.beams || (a.ended != nullptr && a.ended[row] != 0)) return;
  const int part = blockIdx.x * kBeamGroup + threadIdx.x / 16, lane = threadIdx.x % 16;
  __shared__ float2 sums[256 / 64];
  lds_poison(sums);
  const T *x = static_cast<const T *>(a.logits) + row * a.stride;
  float m = -INFINITY, s = 0.0f;
  const int64_t begin = (int64_t)part * a.chunk;
  for (int64_t t0 = begin; t0 < begin + a.chunk && t0 < a.vocab; t0 += kPart) {  // none behind the last part
    float v[L][N];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int64_t t = t0 + (i * 16 + lane) * N;
      load_tokens(x, (int)(t < a.vocab ? t : a.vocab), a.vocab, v[i]);
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) top = fmaxf(top, v[i][j]);
    float sum = 0.0f;
    // e^(x - top) = 2^(x c - h) 2^-l with h + l the product top c in two parts, without a subtraction a token.  l is up to half
    // a step of h and both powers hold it: below 2^24 it is at most 1, at 10^10 it is 440, and 2^l 2^-l is no number.
    if (top > -16777216.0f && top < 16777216.0f) {
      const float h = top * kLog2e, l = __builtin_fmaf(top, kLog2e, -h);
#pragma unroll
      for (int i = 0; i < L; ++i) {
        float part_sum = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) part_sum += __builtin_amdgcn_exp2f(__builtin_fmaf(v[i][j], kLog2e, -h));
        sum += part_sum;
      }
      sum *= __builtin_amdgcn_exp2f(-l);
    } else {  // nothing, masked tokens alone (by any finite value, too), large logits, or infinities
#pragma unroll
      for (int i = 0; i < L; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float d = v[i][j] == top ? 0.0f : v[i][j] - top;  // NaN stays, -inf below -inf is not counted
          sum += top == -INFINITY && d == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(d * kLog2e);
        }
    }
    join(m, s, top, sum);
  }
  join_lanes<1>(m, s);
  join_lanes<2>(m, s);
  join_lanes<4>(m, s);
  join_lanes<8>(m, s);
  if (lane == 0 && part < a.chunks) a.tops[row * a.chunks + part] = m;
  join_lanes<16>(m, s);
  join_lanes<32>(m, s);
  if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = float2{m, s};
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 256 / 64; ++w) join(m, s, sums[w].x, sums[w].y);
    a.sums[row * ((a.chunks + kBeamGroup - 1) / kBeamGroup) + blockIdx.x] = float2{m, s};
  }
}

// --------------------------------------------------------------- selection
// A candidate: its score and its place.  Before another: a higher score, or an equal one and a lower place.
struct Best {
  double score;
  int place;
  LDEV bool before(const Best &o) const { return score > o.score || (score == o.score && place < o.place); }
};
constexpr double kNone = -INFINITY;

struct alignas(16) Beam {
  double base;  // scores - log S; -inf: no continuation
  float top;    // M
  int done;     // ended
  LDEV double score(float x) const {
    const double s = base + (x == top ? 0.0 : (double)x - (double)top);
    return s > kNone ? s : kNone;  // NaN is none
  }
};
struct Shared {
  Beam beam[LAPSUM_MAX_BEAMS];
  double row_best[kRows];
  double least;                   // no candidate below it is among the k best
  int listed;
  double score[kList];
  int place[kList];
  double best_score[LAPSUM_MAX_BEAMS];  // of the selected ones, in order
  int best_place[LAPSUM_MAX_BEAMS];
  double wave_score[kThreads / 64];
  int wave_place[kThreads / 64];
};

LDEV int row_sum(int v) {  // over 16 lanes
  v += (int)xor_lanes<1>((uint32_t)v);
  v += (int)xor_lanes<2>((uint32_t)v);
  v += (int)xor_lanes<7>((uint32_t)v);
  return v + (int)xor_lanes<15>((uint32_t)v);
}

// The k first of the listed candidates in their order, each ranked by how many come before it.
LDEV void rank_listed(Shared &sh, int n, int k) {
  for (int i = threadIdx.x; i < k; i += kThreads) {
    sh.best_score[i] = kNone;
    sh.best_place[i] = -1;
  }
  __syncthreads();
  for (int e = threadIdx.x / 16; e < n; e += kRows) {  // 16 lanes each
    const Best me{sh.score[e], sh.place[e]};
    int rank = 0;
    for (int i = threadIdx.x % 16; i < n; i += 16) rank += Best{sh.score[i], sh.place[i]}.before(me) ? 1 : 0;
    rank = row_sum(rank);
    if (rank < k && threadIdx.x % 16 == 0) {
      sh.best_score[rank] = me.score;
      sh.best_place[rank] = me.place;
    }
  }
  __syncthreads();
}

// The same when they do not fit the list: one after the other, each the first behind the last one.  each(f) calls
// f(candidate) for all candidates of this thread.
template <class Each>
LDEV void select_in_turn(Shared &sh, int k, const Each &each) {
  Best last{INFINITY, -1};
  for (int j = 0; j < k; ++j) {
    Best b{kNone, 0x7FFFFFFF};
    each([&](const Best &c) {
      if (c.score > kNone && last.before(c) && c.before(b)) b = c;
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const Best o{__shfl_xor(b.score, d, 64), __shfl_xor(b.place, d, 64)};
      if (o.before(b)) b = o;
    }
    if (threadIdx.x % 64 == 0) {
      sh.wave_score[threadIdx.x / 64] = b.score;
      sh.wave_place[threadIdx.x / 64] = b.place;
    }
    __syncthreads();
    for (int w = 0; w < kThreads / 64; ++w) {
      const Best o{sh.wave_score[w], sh.wave_place[w]};
      if (o.before(b)) b = o;
    }
    if (threadIdx.x == 0) {
      sh.best_score[j] = b.score;
      sh.best_place[j] = b.score > kNone ? b.place : -1;
    }
    last = b;
    __syncthreads();
  }
}

// The k first of all candidates at or above sh.least.
template <class Each>
LDEV void select(Shared &sh, int k, const Each &each) {
  const double least = sh.least;
  each([&](const Best &c) {
    if (c.score > kNone && c.score >= least) {
      const int at = atomicAdd(&sh.listed, 1);
      if (at < kList) {
        sh.score[at] = c.score;
        sh.place[at] = c.place;
      }
    }
  });
  __syncthreads();
  const int n = sh.listed;
  if (n <= kList)
    rank_listed(sh, n, k);
  else
    select_in_turn(sh, k, each);
}

template <class T>
__global__ __launch_bounds__(kThreads) void beam_select_kernel(BeamArgs a) {
  constexpr int N = Pack<T>::N;
  __shared__ Shared sh;
  __shared__ int chosen[LAPSUM_MAX_BEAMS];
  lds_poison(sh);
  lds_poison(chosen);
  const int64_t search = grid_row();
  if (search >= a.batch) return;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int all = a.beams * a.chunks, groups = (a.chunks + kBeamGroup - 1) / kBeamGroup;
  const float *tops = a.tops + search * a.beams * a.chunks;
  const float2 *sums = a.sums + search * a.beams * groups;

  // this thread's parts, asked for before the sums are joined
  constexpr int kMine = kMostParts / kThreads;
  float mine_top[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = j * kThreads + threadIdx.x;
    if (i < all) mine_top[j] = tops[i];  // of an ended beam whatever is there: not looked at
  }
  for (int i = wave; i < a.beams; i += kThreads / 64) {
    // all asked for at once; what an ended beam's sums hold is not looked at
    const float score = a.scores[search * a.beams + i];
    const bool ended = a.ended != nullptr && a.ended[search * a.beams + i] != 0;
    float m = -INFINITY, s = 0.0f;
    for (int c = lane; c < groups; c += 64) {
      const float2 x = sums[i * groups + c];
      join(m, s, x.x, x.y);
    }
    join_lanes<1>(m, s);
    join_lanes<2>(m, s);
    join_lanes<4>(m, s);
    join_lanes<8>(m, s);
    join_lanes<16>(m, s);
    join_lanes<32>(m, s);
    if (lane == 0) {
      const bool finite = score > -INFINITY && score < INFINITY;
      const bool none = !finite || (!ended && !(s > 0.0f));  // a NaN sum, or nothing above -inf
      sh.beam[i] = Beam{none ? kNone : (ended ? (double)score : (double)score - log_pos((double)s)),
                        ended || none ? 0.0f : m, ended};
    }
  }
  if (threadIdx.x == 0) sh.listed = 0;
  __syncthreads();

  // the best parts
  double mine_score[kMine];
  const int end_part = a.ended != nullptr ? a.end_token / a.chunk : 0;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = j * kThreads + threadIdx.x;
    mine_score[j] = kNone;
    if (i < all) {
      const int beam = (int)((uint64_t)i * a.chunk_magic >> 32);
      const Beam x = sh.beam[beam];
      mine_score[j] = !x.done ? x.score(mine_top[j]) : (i - beam * a.chunks == end_part ? x.base : kNone);
    }
  }
  const auto each_part = [&](const auto &f) {
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (mine_score[j] > kNone) f(Best{mine_score[j], j * kThreads + (int)threadIdx.x});
  };
  // the k-th best of the rows of 16 lanes' best: k candidates are at least that
  double mine = kNone;
  each_part([&](const Best &c) { mine = fmax(mine, c.score); });
  mine = team_max<16>(mine);
  if (threadIdx.x % 16 == 0) sh.row_best[threadIdx.x / 16] = mine;
  __syncthreads();
  {
    const int row = threadIdx.x / 16, first = threadIdx.x % 16 * (kRows / 16);
    int before = 0;
#pragma unroll
    for (int i = 0; i < kRows / 16; ++i) {
      const Best o{sh.row_best[first + i], first + i};
      before += o.before(Best{mine, row}) ? 1 : 0;
    }
    before = row_sum(before);
    if (before == a.k - 1 && threadIdx.x % 16 == 0) sh.least = mine;
  }
  __syncthreads();
  select(sh, a.k, each_part);

  // the best tokens of these parts
  if ((int)threadIdx.x < a.k) chosen[threadIdx.x] = sh.best_place[threadIdx.x];
  if (threadIdx.x == 0) {
    sh.least = sh.best_score[a.k - 1];
    sh.listed = 0;
  }
  __syncthreads();
  const int shift = __builtin_ctz(a.chunk / N);
  const auto each_token = [&](const auto &f) {
    for (int u = threadIdx.x; u < a.k << shift; u += kThreads) {
      const int part = chosen[u >> shift];
      if (part < 0) continue;
      const int beam = (int)((uint64_t)part * a.chunk_magic >> 32);
      const int t = (part - beam * a.chunks) * a.chunk + (u & ((1 << shift) - 1)) * N;
      if (t >= a.vocab) continue;
      const Beam y = sh.beam[beam];
      if (y.done) {
        if (a.end_token >= t && a.end_token < t + N) f(Best{y.base, beam * a.vocab + a.end_token});
        continue;
      }
      float x[N];
      load_tokens(static_cast<const T *>(a.logits) + (search * a.beams + beam) * a.stride, t, a.vocab, x);
#pragma unroll
      for (int j = 0; j < N; ++j) f(Best{y.score(x[j]), beam * a.vocab + t + j});
    }
  };
  select(sh, a.k, each_token);
  if ((int)threadIdx.x < a.k) {
    const int place = sh.best_place[threadIdx.x];
    const int64_t at = search * a.k + threadIdx.x;
    a.scores_out[at] = (float)sh.best_score[threadIdx.x];
    a.parents[at] = place < 0 ? -1 : place / a.vocab;
    a.tokens[at] = place < 0 ? -1 : place % a.vocab;
  }
}

template <class T>
hipError_t beams(const BeamArgs &a, hipStream_t s) {
  beam_parts_kernel<T><<<rows_grid((unsigned)((a.chunks + kBeamGroup - 1) / kBeamGroup), a.batch * a.beams), dim3(256), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  beam_select_kernel<T><<<rows_grid(1, a.batch), dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

void beam_parts(int64_t beams, int64_t vocab, int &chunk, int &chunks) {
  int64_t size = kPart;
  while (beams * ((vocab + size - 1) / size) > kMostParts) size *= 2;
  chunk = (int)size;
  chunks = (int)((vocab + size - 1) / size);
}

hipError_t launch_beam_select(const BeamArgs &a, int dtype, hipStream_t s) {
  if (dtype == LAPSUM_F32) return beams<f32>(a, s);
  if (dtype == LAPSUM_BF16) return beams<bf16>(a, s);
  return beams<f16>(a, s);
}

}  // namespace lapsum
