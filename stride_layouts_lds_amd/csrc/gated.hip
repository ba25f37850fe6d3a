// gated.hip -- the gated feed-forward block in one kernel:
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u
// on fp16, bf16 or int8 operands (dense.hpp's pair of products), g and u
// stored where they are wanted for the backward pass.  g and u stay in fp32
// until h is formed; each output is rounded once.
#include <type_traits>

#include "activation.hpp"
#include "dense.hpp"

namespace sl {
namespace {

template <bool SCALED>
struct Gate {
  const float *sa, *sg, *su;
  __device__ __forceinline__ Gate(const DenseParams& p, int64_t batch) : sa(nullptr), sg(nullptr), su(nullptr) {
    if constexpr (SCALED) sa = p.sa + batch * p.sa_bs, sg = p.sb[0] + batch * p.sb_bs[0], su = p.sb[1] + batch * p.sb_bs[1];
  }
  __device__ __forceinline__ void finish(const DenseParams& p, int64_t batch, int64_t m, int64_t n, floatx4 g, floatx4 u) const {
    if constexpr (SCALED) {
      const float a = sa[m * p.sa_rs];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t at = n + r < p.N ? n + r : p.N - 1;
        g[r] = g[r] * a * sg[at * p.sb_rs[0]];
        u[r] = u[r] * a * su[at * p.sb_rs[1]];
      }
    }
    const int64_t valid = p.N - n;
    if (p.kept[0]) {
      dense_store(p.kept[0], p.type, batch * p.kept_bs[0] + m * p.kept_rs[0] + n * p.kept_cs[0], p.kept_cs[0], p.flags & DF_KEPT_VEC, valid, g);
      dense_store(p.kept[1], p.type, batch * p.kept_bs[1] + m * p.kept_rs[1] + n * p.kept_cs[1], p.kept_cs[1], p.flags & (2 * DF_KEPT_VEC),
                  valid, u);
    }
    floatx4 h;
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = activate(p.act, g[r]) * u[r];
    dense_store(p.d, p.type, batch * p.d_bs + m * p.d_rs + n * p.d_cs, p.d_cs, p.flags & DF_D_VEC, valid, h);
  }
};

}  // namespace

hipError_t launch_gated(const DenseParams& p, int32_t kind, const DensePlan& plan, hipStream_t s) {
  switch (kind) {
    case EK_F16: return dense_launch<EK_F16, true, Gate<false>>(p, plan, s);
    case EK_BF16: return dense_launch<EK_BF16, true, Gate<false>>(p, plan, s);
    case EK_I8: return dense_launch<EK_I8, true, Gate<true>>(p, plan, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sl
