// Routing of tokens to experts: the hard top-k of a router's scores, its
// weights, and the gradient of the weights with respect to the logits.
//
// Mathematics.  s = softmax(x) or 1/(1 + e^-x), c = s + bias; a group scores
// the sum of its two largest c, the best groups stay open, the k largest c of
// the open groups are chosen (equal values: the lowest index), and
// w_j = scale s_j / S with S the sum of the chosen s, or 1.
//
// A team of L lanes holds a row, V scores a lane, all in registers: the row
// is read once and nothing goes back to memory but the k choices.  A score
// and its expert travel as one fp64 number, c exact in the upper bits (an
// fp32 value leaves the 29 lowest bits of the fp64 mantissa free) and the
// expert in the lowest ten, set so that of equal c the lower expert is the
// larger number.  Then one max gives score and place at once, all numbers of a row
// differ, and compare-exchange is a max and a min.  Each lane orders the
// largest of its own numbers once; a round takes the maximum of the lanes' heads by a
// DPP butterfly, and the lane that held it moves up.
//
// What bounds it: vector instructions, about 225 a row of 256 experts (scores 60, the fp64
// numbers 25, ordering 55, eight rounds 50).  16384 rows of 256 fp32 logits
// take 9.3 us (17.8 MB, 1.9 TB/s), 32768 bf16 rows with bias and groups 18.0 us, the
// gradient of those 10.2 us (34 MB with the gathered logits' 64-byte
// sectors, 3.3 TB/s); 16 rows 4.9 us, the length of one row's chain.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

constexpr int kWaves = 4;
constexpr float kLargest = 3.40282347e38f;

// The fp64 number of (c, expert).  Minus infinity becomes the lowest fp32
// value, which no available expert has.
LDEV double number_of(float c, int expert) {
  c = __builtin_amdgcn_fmed3f(c + 0.0f, -kLargest, kLargest);  // -0 counts as 0
  unsigned long long u = (unsigned long long)__double_as_longlong((double)c);
  u |= (unsigned long long)(c < 0.0f ? expert : LAPSUM_MAX_EXPERTS - 1 - expert);
  return __longlong_as_double((long long)u);
}
LDEV bool available(double d) { return d > -(double)kLargest; }
LDEV int expert_of(double d) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(d);
  const int low = (int)(u & (LAPSUM_MAX_EXPERTS - 1));
  return (u >> 63) != 0 ? low : LAPSUM_MAX_EXPERTS - 1 - low;
}

LDEV void exchange(double &x, double &y) {
  const double a = fmax(x, y), b = fmin(x, y);
  x = a;
  y = b;
}
// Descending merge-exchange network (Batcher 1968) on N registers from a[at].
template <int N, int V>
LDEV void sort_descending(double (&a)[V], int at) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) exchange(a[at + i + j], a[at + i + j + q]);
        }
      }
    }
  }
}
// The K largest of V numbers, descending, to the front (K = V, or V / 2).
template <int K, int V>
LDEV void sort_largest(double (&a)[V]) {
  if constexpr (K == V) {
    sort_descending<V>(a, 0);
  } else {
    static_assert(2 * K == V, "two halves");
    sort_descending<K>(a, 0);
    sort_descending<K>(a, K);
    // of two descending halves, the larger of a[i] and a[V - 1 - i] are the K largest, in bitonic order
#pragma unroll
    for (int i = 0; i < K; ++i) a[i] = fmax(a[i], a[V - 1 - i]);
#pragma unroll
    for (int q = K / 2; q >= 1; q /= 2) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if ((i & q) == 0) exchange(a[i], a[i + q]);
    }
  }
}

// Place of an expert's score in LDS: a pad every 32 keeps lanes that walk
// groups of a power of two on different banks.
LDEV int place(int e) { return e + (e >> 5); }
constexpr int places(int e) { return e + e / 32 + 1; }

// Lane j of a team holds the experts of its packs: pack i is L * P experts
// wide, so the team's 16-byte loads are contiguous.
template <class T, int L, int V>
LDEV int expert_at(int j, int v) {
  constexpr int P = Pack<T>::N < V ? Pack<T>::N : V;
  return (v / P) * (L * P) + j * P + v % P;
}

template <class T, int L, int V>
LDEV void load_row(const T *row, int experts, bool packs, int j, float (&x)[V]) {
  constexpr int P = Pack<T>::N < V ? Pack<T>::N : V;
  if (P == Pack<T>::N && packs) {
#pragma unroll
    for (int i = 0; i < V / P; ++i) {
      const int e = expert_at<T, L, V>(j, i * P);
      if (e < experts) {
        const pack_t<T> w = load_pack(row + e);
#pragma unroll
        for (int v = 0; v < P; ++v) x[i * P + v] = (float)w[v];
      } else {
#pragma unroll
        for (int v = 0; v < P; ++v) x[i * P + v] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_at<T, L, V>(j, v);
      x[v] = e < experts ? (float)row[e] : -INFINITY;
    }
  }
}

// e^(x - m), m the row's maximum; 1 where both are the same infinity.
LDEV float share_of(float x, float m) { return exp_full(x == m ? 0.0f : x - m); }

LDEV float sigmoid(float x) {
  const float e = exp_full(-fabsf(x));
  return (x > 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e);
}

// The two largest of what has been seen, b1 >= b2.
LDEV void best_two(float &b1, float &b2, float y) {
  b2 = __builtin_amdgcn_fmed3f(b1, b2, y);
  b1 = fmaxf(b1, y);
}
// Their sum; a group with one available expert is as one with none, also where that one's c is +inf.
// Two that are available never score as none: a sum below the range is the lowest number.
LDEV float group_score(float b1, float b2, int size) {
  return size == 1 ? b1 : (b2 == -INFINITY ? -INFINITY : fmaxf(b1 + b2, -kLargest));
}
template <int M>
LDEV void best_two_across(float &b1, float &b2) {
  const float x1 = pair_lane<M>(b1), x2 = pair_lane<M>(b2);
  b2 = fmaxf(fminf(b1, x1), fmaxf(b2, x2));
  b1 = fmaxf(b1, x1);
}

// Numbers A + 1 .. B of a lane one place up if it won the round.  Written out
// by recursion: a loop would have its selects turned into indexed reads before it is unrolled.
template <int A, int B, int V>
LDEV void move_up(double (&num)[V], bool won) {
  if constexpr (A < B) {
    const double next = num[A + 1], own = num[A];
    num[A] = won ? next : own;
    move_up<A + 1, B>(num, won);
  }
}
// Up to eight rounds; choice i goes to lane i of the team.  After round I a lane has
// at most K - 1 - I numbers left that can still be chosen.
template <int L, int K, int I, int V>
LDEV void choose(double (&num)[V], int k, int j, double &mine) {
  if constexpr (I < 8) {
    if (I >= k) return;  // k is the same for the whole launch
    const double best = team_max<L>(num[0]);
    if (I == j) mine = best;
    constexpr int last = K - 1 - I > 0 ? K - 1 - I : 0;
    const bool won = num[0] == best;
    move_up<0, last>(num, won);
    if constexpr (I >= K - 1) num[0] = won ? -INFINITY : num[0];  // a lane of fewer than eight numbers
    choose<L, K, I + 1>(num, k, j, mine);
  }
}

// packs: the rows can be read in 16-byte packs (host-checked alignment, and
// a whole number of packs per row).  spread: the lanes that share a group, a
// power of two, where groups are whole packs of neighbouring lanes; else 0.
// KM: most choices (8 or 32).
template <class T, int L, int V, int KM>
__global__ __launch_bounds__(64 * kWaves) void route_forward_kernel(const RouteArgs a, const bool packs,
                                                                    const int spread) {
  constexpr int R = 64 / L;              // rows per wave
  constexpr int C = (KM + L - 1) / L;    // choices a lane records, at most
  constexpr int K = KM < V ? KM : V;     // numbers of a lane that can be chosen
  constexpr int P = Pack<T>::N < V ? Pack<T>::N : V;
  constexpr int kN = places(L * V);
  struct Shared {
    float s[kWaves][R][kN];
    float group[kWaves][R][LAPSUM_MAX_GROUPS];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int wave = threadIdx.x / 64, team = (threadIdx.x % 64) / L, j = threadIdx.x % L;
  const int64_t token = ((int64_t)blockIdx.x * kWaves + wave) * R + team;
  const bool live = token < a.tokens;
  const T *row = static_cast<const T *>(a.logits) + (live ? token : 0) * a.stride;

  float x[V];
  load_row<T, L, V>(row, live ? a.experts : 0, packs, j, x);
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    nan |= x[v] != x[v];
    x[v] = x[v] != x[v] ? -INFINITY : x[v];
  }
  nan = team_max<L>(nan ? 1.0f : 0.0f) > 0.0f;

  // c: the scores the choice goes by
  float c[V];
  float m = 0.0f, r = 0.0f;  // softmax: maximum and the inverse sum
  if (a.score == LAPSUM_SCORE_SOFTMAX) {
    m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = team_max<L>(m);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = share_of(x[v], m);
      sum += c[v];
    }
    sum = team_sum<L>(sum);
    r = m > -INFINITY ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] *= r;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = sigmoid(x[v]);
  }
  if (a.bias != nullptr && packs) {  // whole packs inside the row
#pragma unroll
    for (int i = 0; i < V / P; ++i) {
      const int e = expert_at<T, L, V>(j, i * P);
      const float *bias = a.bias + (e < a.experts ? e : 0);
#pragma unroll
      for (int v = 0; v < P; ++v) c[i * P + v] += bias[v];
    }
  } else if (a.bias != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_at<T, L, V>(j, v);
      c[v] += a.bias[e < a.experts ? e : 0];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (x[v] == -INFINITY || !(c[v] > -kLargest)) c[v] = -INFINITY;  // not available: NaN and the lowest number too

  if (a.groups > 1) {
    float *group = sh.group[wave][team];
    if (spread > 0) {
      // a pack lies in one group, and the group's packs in neighbouring lanes
#pragma unroll
      for (int i = 0; i < V / P; ++i) {
        float b1 = c[i * P], b2 = -INFINITY;
#pragma unroll
        for (int v = 1; v < P; ++v) best_two(b1, b2, c[i * P + v]);
        if constexpr (L > 1) { if (spread > 1) best_two_across<1>(b1, b2); }
        if constexpr (L > 2) { if (spread > 2) best_two_across<2>(b1, b2); }
        if constexpr (L > 4) { if (spread > 4) best_two_across<4>(b1, b2); }
        if constexpr (L > 8) { if (spread > 8) best_two_across<8>(b1, b2); }
        if constexpr (L > 16) { if (spread > 16) best_two_across<16>(b1, b2); }
        if constexpr (L > 32) { if (spread > 32) best_two_across<32>(b1, b2); }
        const int e = expert_at<T, L, V>(j, i * P);
        if (e < a.experts && (j & (spread - 1)) == 0)
          group[(uint32_t)e * a.group_magic >> 21] = group_score(b1, b2, a.group_size);
      }
    } else {
      float *sc = sh.s[wave][team];
#pragma unroll
      for (int v = 0; v < V; ++v) sc[place(expert_at<T, L, V>(j, v))] = c[v];
      wave_sync();
      for (int g = j; g < a.groups; g += L) {
        float b1 = -INFINITY, b2 = -INFINITY;
        for (int i = 0; i < a.group_size; ++i) best_two(b1, b2, sc[place(g * a.group_size + i)]);
        group[g] = group_score(b1, b2, a.group_size);
      }
    }
    wave_sync();
    // the groups in the order of their scores: a group's place is the number of groups before it
    unsigned long long open = 0;
    for (int g = 0; g < a.groups; g += L) {
      const int mine = g + j;
      const float y = mine < a.groups ? group[mine] : 0.0f;
      int before = 0;
      for (int h = 0; h < a.groups; ++h) {
        const float z = group[h];
        before += (z > y || (z == y && h < mine)) ? 1 : 0;
      }
      const unsigned long long in = __ballot(mine < a.groups && before < a.top_groups);
      constexpr unsigned long long kTeam = L == 64 ? ~0ull : (1ull << (L % 64)) - 1ull;
      open |= ((in >> (team * L)) & kTeam) << g;
    }
    // lanes past the last expert may name a group past the 64th; whatever bit they read, their c stays -inf
    const auto shut_at = [&](int e) { return ((open >> (((uint32_t)e * a.group_magic >> 21) & 63u)) & 1ull) == 0; };
    if (spread > 0) {
#pragma unroll
      for (int i = 0; i < V / P; ++i) {
        const bool shut = shut_at(expert_at<T, L, V>(j, i * P));
#pragma unroll
        for (int v = 0; v < P; ++v)
          if (shut) c[i * P + v] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (shut_at(expert_at<T, L, V>(j, v))) c[v] = -INFINITY;
      }
    }
  }

  double num[V];
#pragma unroll
  for (int v = 0; v < V; ++v) num[v] = number_of(c[v], expert_at<T, L, V>(j, v));
  sort_largest<K>(num);

  double mine[C];  // choice i * L + j of this row
#pragma unroll
  for (int i = 0; i < C; ++i) mine[i] = -INFINITY;
  if constexpr (KM == 8) {
    choose<L, K, 0>(num, a.k, j, mine[0]);
  } else {
#pragma unroll
    for (int r2 = 0; r2 < C; ++r2) {
      const int n = min(a.k - r2 * L, L);
      for (int i = 0; i < n; ++i) {
        const double best = team_max<L>(num[0]);
        if (i == j) mine[r2] = best;
        if (num[0] == best) {
#pragma unroll
          for (int v = 0; v + 1 < V; ++v) num[v] = num[v + 1];
          num[V - 1] = -INFINITY;
        }
      }
    }
  }

  // The chosen scores: the c themselves, or formed again from the logits where a bias is in them, or where a
  // renormalised softmax may have left out the row's maximum (by the bias, or by the groups): its weights
  // are the softmax of the chosen logits alone, so they are formed against the maximum of those,
  // as the gradient's are, and keep their size however far the choice lies below the row's maximum.
  float w[C], sum = 0.0f;
  const bool soft = a.score == LAPSUM_SCORE_SOFTMAX, alone = soft && a.renormalise != 0;
  if (a.bias == nullptr && !(alone && a.groups > 1)) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const unsigned long long u = (unsigned long long)__double_as_longlong(mine[i]) & ~1023ull;
      w[i] = available(mine[i]) ? (float)__longlong_as_double((long long)u) : 0.0f;
      sum += w[i];
    }
  } else {
    float y[C];
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] = available(mine[i]) ? (float)row[expert_of(mine[i])] : -INFINITY;
    if (alone) {
      m = y[0];
#pragma unroll
      for (int i = 1; i < C; ++i) m = fmaxf(m, y[i]);
      m = team_max<L>(m);
      r = 1.0f;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      w[i] = !available(mine[i]) ? 0.0f : (soft ? share_of(y[i], m) * r : sigmoid(y[i]));
      sum += w[i];
    }
  }
  sum = a.renormalise != 0 ? team_sum<L>(sum) : 1.0f;
  // divided first: scale / sum overflows where all of the chosen scores are small
  if (sum == 0.0f) sum = INFINITY;
  if (!live) return;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int at = i * L + j;
    if (at < a.k) {
      a.weights[token * a.k + at] = nan ? NAN : w[i] / sum * a.scale;
      a.chosen[token * a.k + at] = available(mine[i]) ? expert_of(mine[i]) : -1;
    }
  }
}

// Gradient.  A row's logits are read whole only where a softmax is not
// renormalised; otherwise the k chosen ones are enough, because a
// renormalised softmax is the softmax of the chosen logits alone.  The k
// gradients are laid into a row of zeros in LDS, and the row goes out in
// packs.
template <class T, int L, int V>
__global__ __launch_bounds__(64 * kWaves) void route_backward_kernel(const RouteArgs a, const bool packs,
                                                                     const bool out_packs) {
  constexpr int R = 64 / L;
  constexpr int C = (LAPSUM_MAX_CHOICES + L - 1) / L;
  constexpr int P = Pack<T>::N < V ? Pack<T>::N : V;
  struct Shared {
    float d[kWaves][R][L * V];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int wave = threadIdx.x / 64, team = (threadIdx.x % 64) / L, j = threadIdx.x % L;
  const int64_t token = ((int64_t)blockIdx.x * kWaves + wave) * R + team;
  if (token >= a.tokens) return;  // whole teams leave; nothing below crosses teams but wave_sync
  const T *row = static_cast<const T *>(a.logits) + token * a.stride;
  float *d = sh.d[wave][team];
#pragma unroll
  for (int v = 0; v < V; ++v) d[expert_at<T, L, V>(j, v)] = 0.0f;
  wave_sync();

  int e[C];
  float x[C], g[C];
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const int i = r * L + j;
    e[r] = i < a.k ? a.chosen[token * a.k + i] : -1;
    if ((uint32_t)e[r] >= (uint32_t)a.experts) e[r] = -1;
    x[r] = e[r] >= 0 ? (float)row[e[r]] : -INFINITY;
    g[r] = e[r] >= 0 ? a.dweights[token * a.k + i] : 0.0f;
  }

  const bool soft = a.score == LAPSUM_SCORE_SOFTMAX;
  float s[C];
  if (soft && a.renormalise == 0) {
    float z[V];
    load_row<T, L, V>(row, a.experts, packs, j, z);
    float m = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, z[v]);
    m = team_max<L>(m);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[v] = share_of(z[v], m);
      sum += z[v];
    }
    sum = team_sum<L>(sum);
    const float inv = m == -INFINITY ? 0.0f : 1.0f / sum;
    float dot = 0.0f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      s[r] = share_of(x[r], m) * inv;
      g[r] *= a.scale;
      dot += g[r] * s[r];
      if (e[r] >= 0) d[e[r]] = g[r];
    }
    dot = team_sum<L>(dot);
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = expert_at<T, L, V>(j, v);
      d[i] = z[v] * inv * (d[i] - dot);
    }
    wave_sync();
  } else {
    float m = -INFINITY;
    if (soft) {
#pragma unroll
      for (int r = 0; r < C; ++r) m = fmaxf(m, x[r]);
      m = team_max<L>(m);
    }
    float sum = 0.0f, mean = 0.0f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      s[r] = soft ? share_of(x[r], m) : sigmoid(x[r]);
      if (x[r] == -INFINITY) s[r] = 0.0f;
      sum += s[r];
    }
    // from here s is the share of the sum: the terms keep their size where all of the scores are small
    if (a.renormalise != 0) {
      sum = team_sum<L>(sum);
      if (sum == 0.0f) sum = INFINITY;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        s[r] /= sum;
        mean += g[r] * s[r];
      }
      mean = team_sum<L>(mean);
    }
#pragma unroll
    for (int r = 0; r < C; ++r) {
      if (e[r] < 0) continue;
      float dx = a.scale * (g[r] - mean) * s[r];
      if (!soft) dx *= sigmoid(-x[r]);  // 1 - sigmoid(x), without the difference's rounding
      d[e[r]] = dx;
    }
    wave_sync();
  }

  T *out = static_cast<T *>(a.dlogits) + token * a.experts;
  if (P == Pack<T>::N && out_packs) {
#pragma unroll
    for (int i = 0; i < V / P; ++i) {
      const int at = expert_at<T, L, V>(j, i * P);
      if (at < a.experts) {
        pack_t<T> w;
#pragma unroll
        for (int v = 0; v < P; ++v) w[v % Pack<T>::N] = (T)d[at + v];
        store_pack(out + at, w);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = expert_at<T, L, V>(j, v);
      if (at < a.experts) out[at] = (T)d[at];
    }
  }
}

template <class T, int L, int V>
hipError_t forward(const RouteArgs &a, hipStream_t s) {
  constexpr int N = Pack<T>::N, P = N < V ? N : V;
  const bool packs = a.experts % N == 0 && a.stride % N == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  int spread = a.group_size % P == 0 ? a.group_size / P : 0;
  if (spread > L || (spread & (spread - 1)) != 0) spread = 0;
  // 16384 bf16 rows of 256 in 8 groups: 10.2 us by butterflies, 12.6 through LDS
  constexpr int rows = kWaves * (64 / L);
  const dim3 grid((unsigned)((a.tokens + rows - 1) / rows)), threads(64 * kWaves);
  // a lane orders its 8 or 32 largest: for 8 choices of 256 experts 9.1 us, with the longer order 14.7
  if (a.k <= 8) route_forward_kernel<T, L, V, 8><<<grid, threads, 0, s>>>(a, packs, spread);
  else route_forward_kernel<T, L, V, 32><<<grid, threads, 0, s>>>(a, packs, spread);
  return hipGetLastError();
}
template <class T, int L, int V>
hipError_t backward(const RouteArgs &a, hipStream_t s) {
  constexpr int P = Pack<T>::N;
  const bool whole = a.experts % P == 0;
  const bool packs = whole && a.stride % P == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  const bool out_packs = whole && reinterpret_cast<uintptr_t>(a.dlogits) % 16 == 0;
  constexpr int rows = kWaves * (64 / L);
  route_backward_kernel<T, L, V>
      <<<dim3((unsigned)((a.tokens + rows - 1) / rows)), dim3(64 * kWaves), 0, s>>>(a, packs, out_packs);
  return hipGetLastError();
}

// Lanes and scores per lane by the number of experts: 16 scores a lane keep
// a wave's share of the butterflies small (several rows share each step).
// 16384 rows of 256 take 9.1 us on 16 lanes, 15.1 on 32; of 128 5.6 on 8, 8.6 on 16; of 64
// 4.1 with 8 scores a lane, 5.2 with 16.
template <class T>
hipError_t forward_of(const RouteArgs &a, hipStream_t s) {
  if (a.experts <= 64) return forward<T, 8, 8>(a, s);
  if (a.experts <= 128) return forward<T, 8, 16>(a, s);
  if (a.experts <= 256) return forward<T, 16, 16>(a, s);
  if (a.experts <= 512) return forward<T, 32, 16>(a, s);
  return forward<T, 64, 16>(a, s);
}
template <class T>
hipError_t backward_of(const RouteArgs &a, hipStream_t s) {
  if (a.experts <= 64) return backward<T, 8, 8>(a, s);
  if (a.experts <= 128) return backward<T, 8, 16>(a, s);
  if (a.experts <= 256) return backward<T, 16, 16>(a, s);
  if (a.experts <= 512) return backward<T, 32, 16>(a, s);
  return backward<T, 64, 16>(a, s);
}

}  // namespace

hipError_t launch_route_forward(const RouteArgs &a, int dtype, hipStream_t s) {
  if (dtype == LAPSUM_F32) return forward_of<f32>(a, s);
  if (dtype == LAPSUM_BF16) return forward_of<bf16>(a, s);
  return forward_of<f16>(a, s);
}
hipError_t launch_route_backward(const RouteArgs &a, int dtype, hipStream_t s) {
  if (dtype == LAPSUM_F32) return backward_of<f32>(a, s);
  if (dtype == LAPSUM_BF16) return backward_of<bf16>(a, s);
  return backward_of<f16>(a, s);
}

}  // namespace lapsum
