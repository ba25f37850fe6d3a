// quantize_rows.hip -- row quantisation to int8: per row of x
//   top = max(max |x|, 2^-100),  s = top / 127,  q = the integer nearest to 127 x / top,
// s correctly rounded to fp32, ties of the code to even; a row with a NaN or an
// infinity has scale NaN and codes 0, so whatever is computed from it shows it.
//
// The codes are those of the exact quotient.  16-bit x: 127 x and top have at
// most 18 and 11 bits, so the quotient is a tie or at least 2^-12 off one; a
// product with 1 / top and one residual step give an exact quotient exactly and
// any other within 2^-17.  fp32 x: the quotient can lie within 2^-25 of a tie,
// which fp32 cannot tell; the same two steps in 64 bits.
#include <type_traits>

#include "sl_device.hpp"
#include "sl_ops.hpp"

namespace sl {
namespace {

constexpr uint32_t kAbs = 0x7FFFFFFFu, kInfBits = 0x7F800000u;

template <int T>
using RowElem = typename std::conditional<T == OT_F32, uint32_t, uint16_t>::type;

template <int T>
__device__ __forceinline__ float widen(RowElem<T> v) {
  if constexpr (T == OT_F32) return __builtin_bit_cast(float, v);
  else return to_f32<T == OT_F16 ? DT_F16 : DT_BF16>(v);
}

template <int T>
struct RowScale {
  typedef typename std::conditional<T == OT_F32, double, float>::type R;
  R d, r;   // 2^-7 top and its reciprocal (no overflow at the largest top)
  float s;
  bool bad; // the row holds a NaN or an infinity: its codes are 0, and code() is not asked (a NaN has no integer)
  __device__ __forceinline__ explicit RowScale(uint32_t top_bits) : bad(top_bits >= kInfBits) {
    const float top = fmaxf(__builtin_bit_cast(float, bad ? 0x3F800000u : top_bits), 0x1p-100f);
    constexpr float k = 1.f / 127.f;
    const float s0 = top * k;
    s = bad ? __builtin_nanf("") : __builtin_fmaf(__builtin_fmaf(-127.f, s0, top), k, s0);
    d = (R)top * (R)0x1p-7f;
    if constexpr (T == OT_F32) {
      r = 1.0 / d;
    } else {
      const float r0 = __builtin_amdgcn_rcpf(d);
      r = __builtin_fmaf(__builtin_fmaf(-d, r0, 1.f), r0, r0);
    }
  }
  __device__ __forceinline__ int32_t code(float x) const {
    const R v = (R)x * (R)0.9921875f;  // 127 / 128
    if constexpr (T == OT_F32) {
      const double q = v * r;
      return (int32_t)__builtin_rint(__builtin_fma(__builtin_fma(-d, q, v), r, q));
    } else {
      const float q = v * r;
      return (int32_t)__builtin_rintf(__builtin_fmaf(__builtin_fmaf(-d, q, v), r, q));
    }
  }
};

__device__ __forceinline__ uint32_t bigger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// the largest over a workgroup's `threads` (those of a row: whole waves)
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = bigger(m, (uint32_t)__shfl_xor((int)m, d));
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) m = bigger(m, lds[w]);
  }
  return m;
}

__device__ __forceinline__ void store8(int8_t* q, int64_t c, int64_t q_cols, const int32_t (&w)[8]) {
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) lo |= ((uint32_t)w[e] & 255u) << (8 * e), hi |= ((uint32_t)w[4 + e] & 255u) << (8 * e);
  if (c + 8 <= q_cols) {
    *(u32x2*)(q + c) = u32x2{lo, hi};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < q_cols) q[c + e] = (int8_t)w[e];
  }
}

// the codes of a row without numbers, a thread's: columns c0 .. + 7 of every `step`
__device__ __forceinline__ void store_zeros(int8_t* q, int64_t c0, int64_t step, int64_t q_cols) {
  const int32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t c = c0; c < q_cols; c += step) store8(q, c, q_cols, w);
}

// Rows contiguous: TPR threads to a row, which holds it in registers (VPT
// pieces of 8 values each), so x is read once.  VPT 0: any length, read twice.
// Bound by memory: 8192 x 4096 bf16 in 18 us, 5.6 TB/s; one row of 4096 in 2.1 us.
template <int T, int TPR, int VPT>
__global__ __launch_bounds__(256) void quantize_whole_rows_kernel(const QuantizeRowsParams p) {
  typedef RowElem<T> E;
  typedef E vec8 __attribute__((ext_vector_type(8)));
  typedef E vec8u __attribute__((ext_vector_type(8), aligned(sizeof(E))));
  __shared__ uint32_t lds[4];
  constexpr int RPW = 256 / TPR;
  const int64_t id = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  if (id >= p.batch * p.rows) return;  // whole waves; with more to a row none
  const int64_t b = id / p.rows, row = id % p.rows;
  const int32_t t = threadIdx.x % TPR;
  const E* X = (const E*)p.x + b * p.x_bs + row * p.x_rs;
  int8_t* Q = p.q + b * p.q_bs + row * p.q_rs;
  auto load = [&](int64_t c) {
    vec8 v;
    if (c + 8 <= p.cols) {
      v = *(const vec8u*)(X + c);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < p.cols ? X[c + e] : (E)0;
    }
    return v;
  };
  auto top = [&](const vec8& v, uint32_t m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = bigger(m, __builtin_bit_cast(uint32_t, widen<T>(v[e])) & kAbs);
    return m;
  };
  auto write = [&](const RowScale<T>& s, const vec8& v, int64_t c) {
    int32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = s.code(widen<T>(v[e]));
    store8(Q, c, p.q_cols, w);
  };
  uint32_t m = 0;
  if constexpr (VPT > 0) {
    vec8 v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = load(8 * (t + (int64_t)TPR * i));
#pragma unroll
    for (int i = 0; i < VPT; ++i) m = top(v[i], m);
    const RowScale<T> s((uint32_t)__builtin_amdgcn_readfirstlane((int)row_max<TPR>(m, lds)));  // one for the wave
    if (t == 0) p.s[b * p.s_bs + row * p.s_rs] = s.s;
    if (s.bad) return store_zeros(Q, 8 * t, 8 * TPR, p.q_cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t c = 8 * (t + (int64_t)TPR * i);
      if (c < p.q_cols) write(s, v[i], c);
    }
  } else {
    for (int64_t c = 8 * t; c < p.cols; c += 8 * TPR) m = top(load(c), m);
    const RowScale<T> s((uint32_t)__builtin_amdgcn_readfirstlane((int)row_max<TPR>(m, lds)));  // one for the wave
    if (t == 0) p.s[b * p.s_bs + row * p.s_rs] = s.s;
    if (s.bad) return store_zeros(Q, 8 * t, 8 * TPR, p.q_cols);
    for (int64_t c = 8 * t; c < p.q_cols; c += 8 * TPR) write(s, load(c), c);
  }
}

// Any strides: a lane to a row, 64 rows to a workgroup (of a matrix stored
// column after column neighbouring lanes read neighbouring values), its waves
// taking 16 columns in turn; x is read twice.
constexpr int kStridedWaves = 16;
template <int T>
__global__ __launch_bounds__(64 * kStridedWaves) void quantize_strided_rows_kernel(const QuantizeRowsParams p, uint32_t tiles_r) {
  typedef RowElem<T> E;
  __shared__ uint32_t tops[kStridedWaves][64];
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t b = blockIdx.x / tiles_r, row = (int64_t)(blockIdx.x % tiles_r) * 64 + lane;
  const bool in = row < p.rows;
  const E* X = (const E*)p.x + b * p.x_bs + (in ? row : 0) * p.x_rs;
  uint32_t m = 0;
  for (int64_t c = 16 * wave; c < p.cols; c += 16 * kStridedWaves) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (c + e < p.cols) m = bigger(m, __builtin_bit_cast(uint32_t, widen<T>(X[(c + e) * p.x_cs])) & kAbs);
  }
  tops[wave][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kStridedWaves; ++w) m = bigger(m, tops[w][lane]);
  if (!in) return;
  const RowScale<T> s(m);
  if (wave == 0) p.s[b * p.s_bs + row * p.s_rs] = s.s;
  int8_t* Q = p.q + b * p.q_bs + row * p.q_rs;
  if (s.bad) {
    for (int32_t h = 0; h < 16; h += 8) store_zeros(Q, 16 * wave + h, 16 * kStridedWaves, p.q_cols);
    return;
  }
  for (int64_t c = 16 * wave; c < p.q_cols; c += 16 * kStridedWaves) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t at = c + 8 * h + e;
        w[e] = at < p.cols ? s.code(widen<T>(X[at * p.x_cs])) : 0;
      }
      if (c + 8 * h < p.q_cols) store8(Q, c + 8 * h, p.q_cols, w);
    }
  }
}

bool strided(const QuantizeRowsParams& p) { return p.x_cs != 1 && p.cols > 1; }

// threads to a row and pieces a thread: a wave to a row while there are rows
// enough to fill the chip, else four; 0 pieces: the row is read twice
struct Shape {
  int tpr, vpt;
};
Shape shape_of(const QuantizeRowsParams& p) {
  const bool many = p.batch * p.rows >= 1024;
  if (p.q_cols <= 1024) return {64, 2};
  if (p.q_cols <= 4096) return many ? Shape{64, 8} : Shape{256, 2};
  if (p.q_cols <= 16384) return {256, 8};
  return {256, 0};
}

template <int T>
hipError_t go(const QuantizeRowsParams& p, hipStream_t s) {
  const dim3 grid((uint32_t)quantize_rows_groups(p)), block(256);
  if (strided(p)) {
    hipLaunchKernelGGL(quantize_strided_rows_kernel<T>, grid, dim3(64 * kStridedWaves), 0, s, p, (uint32_t)((p.rows + 63) / 64));
    return hipGetLastError();
  }
  const Shape h = shape_of(p);
  if (h.tpr == 64 && h.vpt == 2) hipLaunchKernelGGL((quantize_whole_rows_kernel<T, 64, 2>), grid, block, 0, s, p);
  else if (h.tpr == 64) hipLaunchKernelGGL((quantize_whole_rows_kernel<T, 64, 8>), grid, block, 0, s, p);
  else if (h.vpt == 2) hipLaunchKernelGGL((quantize_whole_rows_kernel<T, 256, 2>), grid, block, 0, s, p);
  else if (h.vpt == 8) hipLaunchKernelGGL((quantize_whole_rows_kernel<T, 256, 8>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((quantize_whole_rows_kernel<T, 256, 0>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace

int32_t quantize_rows_threads(const QuantizeRowsParams& p) { return strided(p) ? 64 * kStridedWaves : 256; }

int64_t quantize_rows_groups(const QuantizeRowsParams& p) {
  if (strided(p)) return p.batch * ((p.rows + 63) / 64);
  const int64_t rpw = 256 / shape_of(p).tpr;
  return (p.batch * p.rows + rpw - 1) / rpw;
}

hipError_t launch_quantize_rows(const QuantizeRowsParams& p, hipStream_t s) {
  switch (p.type) {
    case OT_F16: return go<OT_F16>(p, s);
    case OT_BF16: return go<OT_BF16>(p, s);
    case OT_F32: return go<OT_F32>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sl
