// ortho_device.hpp -- how the orthogonalisation's kernels read x.
#pragma once
#include "sl_device.hpp"
#include "sl_ops.hpp"

namespace sl {

template <int T>
__device__ __forceinline__ float ortho_widen(typename OrthoElem<T>::type v) {
  if constexpr (T == OT_F32)
    return __builtin_bit_cast(float, v);
  else
    return to_f32<T == OT_F16 ? DT_F16 : DT_BF16>(v);
}

// eight values of matrix b of x at rows i .. (along_rows) or columns j ..,
// zero from row p.m and from column j_end on
template <int T>
__device__ __forceinline__ void ortho_load8(const OrthoParams& p, int64_t b, int64_t i, int64_t j, int64_t j_end, bool along_rows,
                                            float (&v)[8]) {
  typedef typename OrthoElem<T>::type E;
  typedef E vec8 __attribute__((ext_vector_type(8), aligned(sizeof(E))));
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  if (i >= p.m || j >= j_end) return;
  const E* x = (const E*)p.x + b * p.x_bs + i * p.x_rs + j * p.x_cs;
  const int64_t step = along_rows ? p.x_rs : p.x_cs, left = along_rows ? p.m - i : j_end - j;
  if (step == 1 && left >= 8) {
    const vec8 w = *(const vec8*)x;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ortho_widen<T>(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) v[e] = ortho_widen<T>(x[e * step]);
  }
}

}  // namespace sl
