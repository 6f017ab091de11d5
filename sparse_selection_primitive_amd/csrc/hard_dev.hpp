// Device building blocks of the hard selections: element types, 16-byte
// accesses and reductions over teams of lanes.
#pragma once

#include "lapsum_device.hpp"

namespace lapsum {

using f32 = float;
using bf16 = __bf16;
using f16 = _Float16;

// 16 bytes of elements
template <class T>
struct Pack {
  static constexpr int N = 16 / (int)sizeof(T);
  typedef T type __attribute__((ext_vector_type(16 / sizeof(T))));
};
template <class T>
using pack_t = typename Pack<T>::type;

template <class T>
LDEV pack_t<T> load_pack(const T *p) {
  return __builtin_bit_cast(pack_t<T>, *reinterpret_cast<const uint4 *>(p));
}
template <class T>
LDEV void store_pack(T *p, pack_t<T> v) {
  *reinterpret_cast<uint4 *>(p) = __builtin_bit_cast(uint4, v);
}

// Reductions over aligned teams of L lanes (a power of two up to 64), the
// result on every lane of the team.
template <int M>
LDEV float pair_lane(float v) {
  return __uint_as_float(xor_lanes<M == 4 ? 7 : (M == 8 ? 15 : M)>(__float_as_uint(v)));
}
template <int M>
LDEV double pair_lane(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(v);
  constexpr int P = M == 4 ? 7 : (M == 8 ? 15 : M);
  return __longlong_as_double(
      (long long)(((unsigned long long)xor_lanes<P>((uint32_t)(u >> 32)) << 32) | xor_lanes<P>((uint32_t)u)));
}
template <int L, class T, class Op>
LDEV T team_reduce(T v, Op op) {
  if constexpr (L > 1) v = op(v, pair_lane<1>(v));
  if constexpr (L > 2) v = op(v, pair_lane<2>(v));
  if constexpr (L > 4) v = op(v, pair_lane<4>(v));
  if constexpr (L > 8) v = op(v, pair_lane<8>(v));
  if constexpr (L > 16) v = op(v, pair_lane<16>(v));
  if constexpr (L > 32) v = op(v, pair_lane<32>(v));
  return v;
}
template <int L>
LDEV float team_max(float v) {
  return team_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
LDEV float team_sum(float v) {
  return team_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
LDEV double team_max(double v) {
  return team_reduce<L>(v, [](double a, double b) { return fmax(a, b); });
}

// Orders this wave's LDS accesses on both sides (LDS serves one wave's
// accesses in order, so only the compiler has to be held).
LDEV void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// e^d, d <= 0, to about 1 ulp: the product d log2(e) is carried in two parts,
// so its rounding does not grow with |d|; d = -inf gives 0.
LDEV float exp_full(float d) {
  const float h = d * 1.44269502f;
  float l = __builtin_fmaf(d, 1.44269502f, -h);
  l = __builtin_fmaf(d, 1.92596303e-8f, l);
  const float e = __builtin_amdgcn_exp2f(h);
  // at d = -inf the parts are inf - inf; below -150 the power is 0 anyway
  return d < -150.0f ? 0.0f : __builtin_fmaf(e * l, 0.693147182f, e);
}

}  // namespace lapsum
