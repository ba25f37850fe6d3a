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

template <int EK>
struct Gate {
  static constexpr bool SCALED = EK == EK_I8;
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
  template <int OT, int ACT, int RPI, int V, class GET>
  __device__ __forceinline__ void rows_of(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    typedef typename OrthoElem<OT>::type E;
    float bg[V], bu[V];
    const float* a = nullptr;
    if constexpr (SCALED) {
      a = sa + m * p.sa_rs;
#pragma unroll
      for (int e = 0; e < V; ++e) bg[e] = sg[(n + e) * p.sb_rs[0]], bu[e] = su[(n + e) * p.sb_rs[1]];
    }
    E* d = (E*)p.d + batch * p.d_bs + m * p.d_rs + n;
    const bool keep = p.kept[0];
    E* kg = (E*)p.kept[0] + batch * p.kept_bs[0] + m * p.kept_rs[0] + n;
    E* ku = (E*)p.kept[1] + batch * p.kept_bs[1] + m * p.kept_rs[1] + n;
#pragma unroll 2
    for (int it = 0; it < count; ++it) {
      float g[V], u[V], h[V];
      get(it, 0, g);
      get(it, 1, u);
      if constexpr (SCALED) {
        const float as = *a;
        a += RPI * p.sa_rs;
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = g[e] * as * bg[e], u[e] = u[e] * as * bu[e];
      }
      if (keep) {
        dense_store_cols<OT, V>(kg, g);
        dense_store_cols<OT, V>(ku, u);
        kg += RPI * p.kept_rs[0], ku += RPI * p.kept_rs[1];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = activate(ACT, g[e]) * u[e];
      dense_store_cols<OT, V>(d, h);
      d += RPI * p.d_rs;
    }
  }
  template <int OT, int RPI, int V, class GET>
  __device__ __forceinline__ void rows_by_act(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    switch (p.act) {
      case ACT_SILU: rows_of<OT, ACT_SILU, RPI, V>(p, batch, m, n, count, get); break;
      case ACT_GELU: rows_of<OT, ACT_GELU, RPI, V>(p, batch, m, n, count, get); break;
      case ACT_GELU_TANH: rows_of<OT, ACT_GELU_TANH, RPI, V>(p, batch, m, n, count, get); break;
      default: rows_of<OT, ACT_RELU, RPI, V>(p, batch, m, n, count, get);
    }
  }
  template <int RPI, int V, class GET>
  __device__ __forceinline__ void rows(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    if constexpr (EK == EK_F16) rows_by_act<OT_F16, RPI, V>(p, batch, m, n, count, get);
    else if constexpr (EK == EK_BF16) rows_by_act<OT_BF16, RPI, V>(p, batch, m, n, count, get);
    else if (p.type == OT_F16) rows_by_act<OT_F16, RPI, V>(p, batch, m, n, count, get);
    else if (p.type == OT_BF16) rows_by_act<OT_BF16, RPI, V>(p, batch, m, n, count, get);
    else if constexpr (V < 8) rows_by_act<OT_F32, RPI, V>(p, batch, m, n, count, get);  // (DF_ROWS8 is of 16-bit types)
  }
};

}  // namespace

hipError_t launch_gated(const DenseParams& p, int32_t kind, const DensePlan& plan, hipStream_t s) {
  switch (kind) {
    case EK_F16: return dense_launch<EK_F16, true, Gate<EK_F16>>(p, plan, s);
    case EK_BF16: return dense_launch<EK_BF16, true, Gate<EK_BF16>>(p, plan, s);
    case EK_I8: return dense_launch<EK_I8, true, Gate<EK_I8>>(p, plan, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sl
