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
  // V values of a row as they are stored.  (Where V is eight fp16 and bf16 each have their copy of
  // the code; otherwise ANY16 is either: with copies of all of it the kernel's
  // registers went to memory, and told apart row by row eights take 2 of 33 us more, 4000 x
  // 3000 x 2064 + C.)
  static constexpr int ANY16 = -1;
  template <int OT, int V>
  struct Stored {
    static constexpr bool F32 = OT == OT_F32;
    typedef typename std::conditional<F32, float, uint16_t>::type E;
    typedef E vec __attribute__((ext_vector_type(V == 1 ? 2 : V)));
    vec w;
    __device__ __forceinline__ void load(const E* at) {
      if constexpr (V == 1) w[0] = *at;
      else w = *(const vec*)at;
    }
    __device__ __forceinline__ void store(E* at) const {
      if constexpr (V == 1) *at = w[0];
      else *(vec*)at = w;
    }
    template <int DT>
    __device__ __forceinline__ void add_as(float (&v)[V]) const {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (F32) v[e] += w[e];
        else v[e] += to_f32<DT>((uint16_t)w[e]);
      }
    }
    template <int DT>
    __device__ __forceinline__ void set_as(const float (&v)[V]) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (F32) w[e] = v[e];
        else w[e] = from_f32<DT>(v[e]);
      }
    }
    __device__ __forceinline__ void add_to(float (&v)[V], bool bf16) const {
      if (OT == OT_BF16 || (OT == ANY16 && bf16)) add_as<DT_BF16>(v);
      else add_as<DT_F16>(v);
    }
    __device__ __forceinline__ void set(const float (&v)[V], bool bf16) {
      if (OT == OT_BF16 || (OT == ANY16 && bf16)) set_as<DT_BF16>(v);
      else set_as<DT_F16>(v);
    }
  };
  template <int OT, bool HAS_C, int RPI, int V, class GET>
  __device__ __forceinline__ void rows_of(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    typedef Stored<OT, V> S;
    typedef typename S::E E;
    const bool bf16 = p.type == OT_BF16;
    float b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) b[e] = sb[(n + e) * p.sb_rs[0]];
    E* d = (E*)p.d + batch * p.d_bs + m * p.d_rs + n;
    const E* c = HAS_C ? (const E*)p.c + batch * p.c_bs + m * p.c_rs + n : nullptr;
    const float* a = sa + m * p.sa_rs;
    // N rows at a time, their scales and C requested together: one after the
    // other each waited for memory (4000 x 3000 x 2064 + C: 12 of 48 us)
    auto some = [&](int32_t it0, auto many) {
      constexpr int N = decltype(many)::value;
      float as[N];
      S w[HAS_C ? N : 1];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        as[i] = a[(it0 + i) * RPI * p.sa_rs];
        if constexpr (HAS_C) w[i].load(c + (it0 + i) * RPI * p.c_rs);
      }
      if constexpr (HAS_C) __builtin_amdgcn_sched_barrier(0);  // (or each load moves next to its use)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v[V];
        S out;
        get(it0 + i, 0, v);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = v[e] * as[i] * b[e];
        if constexpr (HAS_C) w[i].add_to(v, bf16);
        out.set(v, bf16);
        out.store(d);
        d += RPI * p.d_rs;
      }
    };
    int32_t it = 0;
#pragma unroll 1
    for (; it + 8 <= count; it += 8) some(it, std::integral_constant<int, 8>{});
#pragma unroll 1
    for (; it < count; ++it) some(it, std::integral_constant<int, 1>{});
  }
  template <int OT, int RPI, int V, class GET>
  __device__ __forceinline__ void rows_to(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    if (p.c) rows_of<OT, true, RPI, V>(p, batch, m, n, count, get);
    else rows_of<OT, false, RPI, V>(p, batch, m, n, count, get);
  }
  template <int RPI, int V, class GET>
  __device__ __forceinline__ void rows(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    if constexpr (V == 8) {  // (DF_ROWS8 is of 16-bit types)
      if (p.type == OT_F16) rows_to<OT_F16, RPI, V>(p, batch, m, n, count, get);
      else rows_to<OT_BF16, RPI, V>(p, batch, m, n, count, get);
    } else {
      if (p.type == OT_F32) rows_to<OT_F32, RPI, V>(p, batch, m, n, count, get);
      else rows_to<ANY16, RPI, V>(p, batch, m, n, count, get);
    }
  }
};

}  // namespace

hipError_t launch_gemm_i8(const DenseParams& p, const DensePlan& plan, hipStream_t s) { return dense_launch<EK_I8, false, ScaledSum>(p, plan, s); }

}  // namespace sl
