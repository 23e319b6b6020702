// Device helpers of the layer operators: vectors of elements with one rounding to bf16,
// and sums over the lanes of a row.
#pragma once

#include "gdn_device.h"

namespace gdn {

typedef __bf16 bhalf4 __attribute__((ext_vector_type(4)));
typedef __bf16 bhalf2 __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));

// Element types of the layer operators: float, or __bf16 (conversions from float round
// to nearest even, v_cvt_pk_bf16_f32).
template <typename E, int N> using vec = E __attribute__((ext_vector_type(N)));

template <typename E>
__device__ __forceinline__ void load4(const E* p, float* x) {
  const vec<E, 4> r = *reinterpret_cast<const vec<E, 4>*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = float(r[i]);
}
template <typename E>
__device__ __forceinline__ void store4(E* p, const float* x) {
  vec<E, 4> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = E(x[i]);
  *reinterpret_cast<vec<E, 4>*>(p) = r;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// Sum over aligned groups of L lanes (2, 4, 8 or 16), in every lane: quads by
// permutation, then the mirror images of eight and sixteen lanes.
template <int L>
__device__ __forceinline__ float row_sum(float x) {
  x += dpp<0xB1>(x);                           // lane ^ 1
  if constexpr (L >= 4) x += dpp<0x4E>(x);     // lane ^ 2
  if constexpr (L >= 8) x += dpp<0x141>(x);    // the other quad of eight lanes
  if constexpr (L >= 16) x += dpp<0x140>(x);   // the other eight of a row
  return x;
}

}  // namespace gdn
