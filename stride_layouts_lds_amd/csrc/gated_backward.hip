// gated_backward.hip -- the matrix products of the gated feed-forward block's
// backward pass, on operands that gated_prepare.hip has laid along the axis
// they contract over:
//   dx = [dg | du] [Wg ; Wu],   dWg = dg^T x,   dWu = du^T x
// the weights' gradients as one product of a batch of pairs.
#include <type_traits>

#include "dense.hpp"

namespace sl {
namespace {

template <int OT>
struct Gradient {
  int32_t s;
  __device__ __forceinline__ Gradient(const DenseParams& p, int64_t batch) : s((int32_t)batch & p.b_shift) {}
  __device__ __forceinline__ void finish(const DenseParams& p, int64_t batch, int64_t m, int64_t n, floatx4 v) const {
    const int64_t off = (batch >> p.b_shift) * p.kept_bs[s] + m * p.kept_rs[s] + n * p.kept_cs[s];
    dense_store(p.kept[s], OT, off, p.kept_cs[s], s ? p.flags & (2 * DF_KEPT_VEC) : p.flags & DF_KEPT_VEC, p.N - n, v);
  }
  template <int RPI, class GET>
  __device__ __forceinline__ void rows(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    uint16_t* d = (uint16_t*)p.kept[s] + (batch >> p.b_shift) * p.kept_bs[s] + m * p.kept_rs[s] + n;
#pragma unroll 4
    for (int it = 0; it < count; ++it) {
      float v[8];
      get(it, 0, v);
      dense_store8<OT>(d, v);
      d += RPI * p.kept_rs[s];
    }
  }
};

}  // namespace

hipError_t launch_gated_products(const DenseParams& p, int32_t kind, const DensePlan& plan, hipStream_t s) {
  if (kind == EK_F16) return dense_launch<EK_F16, false, Gradient<OT_F16>>(p, plan, s);
  return dense_launch<EK_BF16, false, Gradient<OT_BF16>>(p, plan, s);
}

}  // namespace sl
