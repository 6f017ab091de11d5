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
// differ, and compare-exchange is a max and a min.  Each lane sorts its
// own V numbers once; a round takes the maximum of the lanes' heads by a DPP
// butterfly, and the lane that held it moves up.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

constexpr int kWaves = 4;

// the fp64 number of (c, expert); experts that are not available are -inf
LDEV double number_of(float c, int expert) {
  if (!(c > -INFINITY)) return -INFINITY;
  c = fminf(c + 0.0f, 3.40282347e38f);  // -0 counts as 0; an infinite c as the largest finite one
  unsigned long long u = (unsigned long long)__double_as_longlong((double)c);
  u |= (unsigned long long)(c < 0.0f ? expert : LAPSUM_MAX_EXPERTS - 1 - expert);
  return __longlong_as_double((long long)u);
}
LDEV int expert_of(double d) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(d);
  const int low = (int)(u & (LAPSUM_MAX_EXPERTS - 1));
  return (u >> 63) != 0 ? low : LAPSUM_MAX_EXPERTS - 1 - low;
}

// Descending merge-exchange network (Batcher 1968) on V registers.
template <int V>
LDEV void sort_descending(double (&a)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double x = a[i + j], y = a[i + j + q];
            a[i + j] = fmax(x, y);
            a[i + j + q] = fmin(x, y);
          }
        }
      }
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

LDEV float sigmoid(float x) {
  const float e = exp_full(-fabsf(x));
  return (x > 0.0f ? 1.0f : e) / (1.0f + e);
}

// packs: the rows can be read in 16-byte packs (host-checked alignment, and
// a whole number of packs per row)
template <class T, int L, int V>
__global__ __launch_bounds__(64 * kWaves) void route_forward_kernel(const RouteArgs a, const bool packs) {
  constexpr int R = 64 / L;              // rows per wave
  constexpr int C = (LAPSUM_MAX_CHOICES + L - 1) / L;  // choices a lane records, at most
  constexpr int kN = places(L * V);
  struct Shared {
    float s[kWaves][R][kN];
    float group[kWaves][R][LAPSUM_MAX_GROUPS];
    int open[kWaves][R][LAPSUM_MAX_GROUPS];
  };
  __shared__ Shared sh;
  lds_poison(sh);
  const int wave = threadIdx.x / 64, team = (threadIdx.x % 64) / L, j = threadIdx.x % L;
  const int64_t token = ((int64_t)blockIdx.x * kWaves + wave) * R + team;
  const bool live = token < a.tokens;
  float *sc = sh.s[wave][team];

  float x[V];
  if (live) {
    load_row<T, L, V>(static_cast<const T *>(a.logits) + token * a.stride, a.experts, packs, j, x);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = -INFINITY;
  }
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (x[v] != x[v]) {
      nan = true;
      x[v] = -INFINITY;
    }
  }
  nan = team_max<L>(nan ? 1.0f : 0.0f) > 0.0f;

  float s[V];
  if (a.score == LAPSUM_SCORE_SOFTMAX) {
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = team_max<L>(m);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = x[v] == -INFINITY ? 0.0f : (x[v] == m ? 1.0f : exp_full(x[v] - m));
      sum += s[v];
    }
    sum = team_sum<L>(sum);
    const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] *= r;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = x[v] == -INFINITY ? 0.0f : sigmoid(x[v]);
  }

  // c: the scores the choice goes by
  float c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_at<T, L, V>(j, v);
    c[v] = s[v];
    if (a.bias != nullptr && e < a.experts) c[v] += a.bias[e];
    if (x[v] == -INFINITY || c[v] != c[v]) c[v] = -INFINITY;
  }
  if (a.groups > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) sc[place(expert_at<T, L, V>(j, v))] = c[v];
    wave_sync();
    for (int g = j; g < a.groups; g += L) {
      float b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < a.group_size; ++i) {
        const float y = sc[place(g * a.group_size + i)];
        b2 = fmaxf(b2, fminf(b1, y));
        b1 = fmaxf(b1, y);
      }
      sh.group[wave][team][g] = a.group_size > 1 ? b1 + b2 : b1;
    }
    wave_sync();
    for (int g = j; g < a.groups; g += L) {
      const float mine = sh.group[wave][team][g];
      int before = 0;
      for (int h = 0; h < a.groups; ++h) {
        const float y = sh.group[wave][team][h];
        before += (y > mine || (y == mine && h < g)) ? 1 : 0;
      }
      sh.open[wave][team][g] = before < a.top_groups ? 1 : 0;
    }
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_at<T, L, V>(j, v);
      if (e < a.experts) {
        if (sh.open[wave][team][(uint32_t)e * a.group_magic >> 21] == 0) c[v] = -INFINITY;
      }
    }
    wave_sync();
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sc[place(expert_at<T, L, V>(j, v))] = s[v];
  wave_sync();

  double num[V];
#pragma unroll
  for (int v = 0; v < V; ++v) num[v] = number_of(c[v], expert_at<T, L, V>(j, v));
  sort_descending<V>(num);

  double mine[C];  // choice r * L + j of this row
#pragma unroll
  for (int r = 0; r < C; ++r) mine[r] = -INFINITY;
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const int n = min(a.k - r * L, L);
    for (int i = 0; i < n; ++i) {
      const double best = team_max<L>(num[0]);
      if (i == j) mine[r] = best;
      if (num[0] == best) {  // one lane of the team (several only when nothing is left)
#pragma unroll
        for (int v = 0; v + 1 < V; ++v) num[v] = num[v + 1];
        num[V - 1] = -INFINITY;
      }
    }
  }

  float w[C], sum = 0.0f;
#pragma unroll
  for (int r = 0; r < C; ++r) {
    w[r] = mine[r] > -INFINITY ? sc[place(expert_of(mine[r]))] : 0.0f;
    sum += w[r];
  }
  sum = a.renormalise != 0 ? team_sum<L>(sum) : 1.0f;
  const float f = sum > 0.0f ? a.scale / sum : 0.0f;
  if (!live) return;
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const int i = r * L + j;
    if (i < a.k) {
      a.weights[token * a.k + i] = nan ? NAN : w[r] * f;
      a.chosen[token * a.k + i] = mine[r] > -INFINITY ? expert_of(mine[r]) : -1;
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
      z[v] = z[v] == -INFINITY ? 0.0f : (z[v] == m ? 1.0f : exp_full(z[v] - m));
      sum += z[v];
    }
    sum = team_sum<L>(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      s[r] = x[r] == -INFINITY ? 0.0f : (x[r] == m ? inv : exp_full(x[r] - m) * inv);
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
      if (x[r] == -INFINITY) s[r] = 0.0f;
      else if (soft) s[r] = x[r] == m ? 1.0f : exp_full(x[r] - m);
      else s[r] = sigmoid(x[r]);
      sum += s[r];
      mean += g[r] * s[r];
    }
    if (a.renormalise != 0) {
      sum = team_sum<L>(sum);
      mean = team_sum<L>(mean);
    } else {
      sum = 1.0f;
      mean = 0.0f;
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      if (e[r] < 0) continue;
      float dx = a.scale * (g[r] - mean * inv) * inv * s[r];
      if (!soft) dx *= 1.0f - s[r];
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
  constexpr int P = Pack<T>::N;
  const bool packs = a.experts % P == 0 && a.stride % P == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  constexpr int rows = kWaves * (64 / L);
  route_forward_kernel<T, L, V>
      <<<dim3((unsigned)((a.tokens + rows - 1) / rows)), dim3(64 * kWaves), 0, s>>>(a, packs);
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
