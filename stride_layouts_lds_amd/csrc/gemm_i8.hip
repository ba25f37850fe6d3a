// gemm_i8.hip -- the product of int8 codes with one fp32 scale per row of
// either operand (a token's, an output channel's):
//   D[m,n] = C[m,n] + sa[m] sb[n] sum_k A[m,k] B[n,k]
// on v_mfma_i32_16x16x64_i8 (dense.hpp).  The sum is exact in int32 for K below
// 131072 (128 x 128 x K < 2^31), so that the order of its parts does not matter; it
// is rounded to fp32 once, multiplied by sa and by sb, and C added, in fp32.
#include <type_traits>

#include "dense.hpp"

namespace sl {
namespace {

struct ScaledSum {
  const float *sa, *sb;
  __device__ __forceinline__ ScaledSum(const DenseParams& p, int64_t batch) : sa(p.sa + batch * p.sa_bs), sb(p.sb[0] + batch * p.sb_bs[0]) {}
  __device__ __forceinline__ void finish(const DenseParams& p, int64_t batch, int64_t m, int64_t n, floatx4 v) const {
    const float a = sa[m * p.sa_rs];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = v[r] * a * sb[(n + r < p.N ? n + r : p.N - 1) * p.sb_rs[0]];
    const int64_t valid = p.N - n;
    if (p.c) {
      const floatx4 c = dense_load(p.c, p.type, batch * p.c_bs + m * p.c_rs + n * p.c_cs, p.c_cs, p.flags & DF_C_VEC, valid);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += c[r];
    }
    dense_store(p.d, p.type, batch * p.d_bs + m * p.d_rs + n * p.d_cs, p.d_cs, p.flags & DF_D_VEC, valid, v);
  }
};

}  // namespace

hipError_t launch_gemm_i8(const DenseParams& p, const DensePlan& plan, hipStream_t s) { return dense_launch<EK_I8, false, ScaledSum>(p, plan, s); }

}  // namespace sl
