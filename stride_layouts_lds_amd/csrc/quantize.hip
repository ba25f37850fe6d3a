// quantize.hip -- block quantisation to E4M3: each block of 128 consecutive
// values of a row (or of 128 x 128 values) gets one fp32 scale,
//   top = max(max |x|, 2^-100),  s = top / 448,  q = E4M3(448 x / top),
// both quotients correctly rounded to fp32 and the code to the nearest E4M3
// value, ties to even; a block with a NaN or an infinity has scale NaN and
// NaN codes, so whatever is computed from it shows it.  "Transposed" is the
// same of x's transpose, blocked along x's rows: a product that contracts
// over the rows reads its operands with that axis contiguous.
//
// Bound by memory: x is read once and every code written once.  Measured:
// 8192 x 4096 bf16 both ways 27 to 31 us (134 MB, 4.4 to 4.9 TB/s), along the
// rows alone 21 (101 MB, 4.7), 4000 x 3000 fp32 in square blocks both ways 17.
// Two kernels.
//
// Along the columns alone, blocks of 1 x 128: 16 lanes hold a block (8 values
// each), four rows per group of lanes in flight; nothing crosses a wave.
//
// With the transpose, or blocks of 128 x 128: one workgroup per 128 x 128
// tile, every value in registers (a thread holds 8 rows x 8 columns), so x
// is read once for both outputs.  The largest magnitudes along a row meet
// over 16 lanes, along a column over the thread's rows, the wave's four row
// groups and then, through LDS, the four waves.  The transposed codes go
// through LDS so that each instruction stores whole 128-byte rows.
#include "sl_ops.hpp"

#include "sl_device.hpp"

namespace sl {
namespace {

constexpr uint32_t kAbs = 0x7FFFFFFFu, kInfBits = 0x7F800000u;

// The code's quotient 448 x / top as one correctly rounded fp32 division at
// three multiply-adds a value: with v = 7/16 x, d = top / 2^10 (both exact
// but for fp32 x, whose product rounds as 448 x does) and r = 1 / d rounded,
// one residual step takes v r to the nearest fp32 of v / d.  A multiplication
// by 448 / top would round twice and miss the ties that 8-bit significands
// hit often.
struct BlockScale {
  float d, r, s;
  __device__ __forceinline__ explicit BlockScale(uint32_t top_bits) {
    const float top = fmaxf(__builtin_bit_cast(float, top_bits), 0x1p-100f);
    d = top * 0x1p-10f;
    // 1 / d: the hardware's reciprocal and one Newton step; top / 448: a
    // product with the rounded 1 / 448 and one residual step (top is at least
    // 2^-100, so nothing here is subnormal)
    const float r0 = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(__builtin_fmaf(-d, r0, 1.f), r0, r0);
    constexpr float k = 1.f / 448.f;
    const float s0 = top * k;
    s = __builtin_fmaf(__builtin_fmaf(-448.f, s0, top), k, s0);
    if (top_bits >= kInfBits) d = r = s = __builtin_nanf("");
  }
  __device__ __forceinline__ float quotient(float x) const {
    const float v = x * 0.4375f;
    const float q = v * r;
    return __builtin_fmaf(__builtin_fmaf(-d, q, v), r, q);
  }
};

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

template <int T>
struct Elem {
  typedef uint16_t type;
};
template <>
struct Elem<OT_F32> {
  typedef uint32_t type;
};
template <int T>
__device__ __forceinline__ float widen(typename Elem<T>::type v) {
  if constexpr (T == OT_F32)
    return __builtin_bit_cast(float, v);
  else
    return to_f32<T == OT_F16 ? DT_F16 : DT_BF16>(v);
}

// eight consecutive columns of a row from column c0 (zero at and past
// `cols`); CONTIG: unit column stride, one wide load that needs no more
// than the element's own alignment
template <int T, bool CONTIG, bool WHOLE = false>
__device__ __forceinline__ void load8(const typename Elem<T>::type* row, int64_t cs, int64_t c0, int64_t cols,
                                      bool row_ok, float (&v)[8]) {
  typedef typename Elem<T>::type E;
  typedef E vec8 __attribute__((ext_vector_type(8), aligned(sizeof(E))));
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  if (!WHOLE && !row_ok) return;
  if (CONTIG && (WHOLE || c0 + 8 <= cols)) {
    const vec8 x = *(const vec8*)(row + c0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = widen<T>(x[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (WHOLE || c0 + e < cols) v[e] = widen<T>(row[(c0 + e) * cs]);
  }
}

// the largest over the 16 lanes that share lane / 16
__device__ __forceinline__ uint32_t max16(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
    m = m > o ? m : o;
  }
  return m;
}

__device__ __forceinline__ uint32_t max8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[e]) & kAbs;
    m = m > b ? m : b;
  }
  return m;
}

constexpr int kRowsPerGroup = 4;                       // rows of one block column per 16 lanes
constexpr int kRowTile = 16 * kRowsPerGroup;           // rows per workgroup of the row kernel

template <int T, bool CONTIG>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantizeParams p, uint32_t blocks_c, uint32_t tiles_r) {
  typedef typename Elem<T>::type E;
  const uint32_t id = blockIdx.x;
  const int64_t bc = id % blocks_c, tr = id / blocks_c % tiles_r, b = id / blocks_c / tiles_r;
  const int32_t g = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t c0 = bc * kScaleBlock + 8 * l;
  const E* X = (const E*)p.x + b * p.x_bs;
  float v[kRowsPerGroup][8];
#pragma unroll
  for (int i = 0; i < kRowsPerGroup; ++i) {
    const int64_t r = tr * kRowTile + 16 * i + g;
    load8<T, CONTIG>(X + r * p.x_rs, p.x_cs, c0, p.cols, r < p.rows, v[i]);
  }
#pragma unroll
  for (int i = 0; i < kRowsPerGroup; ++i) {
    const int64_t r = tr * kRowTile + 16 * i + g;
    const BlockScale bs(max16(max8(v[i])));
    if (r >= p.rows) continue;
    if (l == 0) p.s[b * p.s_bs + r * p.s_rs + bc * p.s_cs] = bs.s;
    uint8_t* Q = p.q + b * p.q_bs + r * p.q_rs + c0;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = c0 + e < p.cols ? bs.quotient(v[i][e]) : 0.f;
    const u32x2 w = u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
    if (c0 + 8 <= p.q_cols) {
      *(u32x2*)Q = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e < p.q_cols) Q[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
  }
}

// The values as new ones: the compiler would otherwise keep what one stage
// computed of each (its magnitude, 7/16 of it) for the next, another 64
// registers.
__device__ __forceinline__ void renew(float (&v)[8][8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(v[i][e]));
}

// thread t of a tile: columns 8 (t % 16) .. + 7 of rows 8 (t / 16) .. + 7.
// WHOLE: 128 x 128 values in x and codes in every output, so nothing is
// checked.
template <int T, bool CONTIG, bool SQUARE, bool WHOLE>
__device__ __forceinline__ void quantize_tile(const QuantizeParams& p, int64_t bc, int64_t br, int64_t b, char* codes,
                                              uint32_t (*tops)[128]) {
  typedef typename Elem<T>::type E;
  const int32_t g = threadIdx.x >> 4, l = threadIdx.x & 15, wave = threadIdx.x >> 6;
  const int64_t r0 = br * 128 + 8 * g, c0 = bc * 128 + 8 * l;
  const E* X = (const E*)p.x + b * p.x_bs;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<T, CONTIG, WHOLE>(X + (r0 + i) * p.x_rs, p.x_cs, c0, p.cols, WHOLE || r0 + i < p.rows, v[i]);

  uint32_t row_top[8], col_top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) row_top[i] = max8(v[i]);
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = m > row_top[i] ? m : row_top[i];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
      m = m > o ? m : o;
    }
    if ((threadIdx.x & 63) == 0) tops[wave][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = m > tops[w][0] ? m : tops[w][0];
#pragma unroll
    for (int i = 0; i < 8; ++i) row_top[i] = col_top[i] = m;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) row_top[i] = max16(row_top[i]);
    if (p.qt) {
      renew(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = __builtin_bit_cast(uint32_t, v[i][e]) & kAbs;
          m = m > x ? m : x;
        }
#pragma unroll
        for (int d = 16; d < 64; d <<= 1) {
          const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
          m = m > o ? m : o;
        }
        if ((threadIdx.x & 63) < 16) tops[wave][8 * l + e] = m;
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t m = tops[0][8 * l + e];
#pragma unroll
        for (int w = 1; w < 4; ++w) m = m > tops[w][8 * l + e] ? m : tops[w][8 * l + e];
        col_top[e] = m;
      }
    }
  }

  renew(v);
  const BlockScale whole(row_top[0]);  // SQUARE: the block's
  if (p.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + i;
      __builtin_amdgcn_sched_barrier(0);  // one row's scale and codes at a time: registers for four waves a SIMD
      const BlockScale bs = SQUARE ? whole : BlockScale(row_top[i]);
      if (!WHOLE && r >= p.rows) continue;
      if (SQUARE ? threadIdx.x == 0 && i == 0 : l == 0)
        p.s[b * p.s_bs + (SQUARE ? br : r) * p.s_rs + bc * p.s_cs] = bs.s;
      uint8_t* Q = p.q + b * p.q_bs + r * p.q_rs + c0;
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = WHOLE || c0 + e < p.cols ? bs.quotient(v[i][e]) : 0.f;
      const u32x2 w = u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
      if (WHOLE || c0 + 8 <= p.q_cols) {
        *(u32x2*)Q = w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c0 + e < p.q_cols) Q[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
  if (p.qt) {
    renew(v);
    // column c's 128 codes as 16 pieces of 8 bytes, piece g at g ^ (c / 8):
    // a wave's 64 stores of one register then spread over the pieces
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      __builtin_amdgcn_sched_barrier(0);
      const BlockScale bs = SQUARE ? whole : BlockScale(col_top[e]);
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = WHOLE || r0 + i < p.rows ? bs.quotient(v[i][e]) : 0.f;
      *(u32x2*)(codes + (8 * l + e) * 128 + 8 * (g ^ l)) =
          u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
      if (SQUARE ? threadIdx.x == 0 && e == 0 : g == 0 && (WHOLE || c0 + e < p.cols))
        p.st[b * p.st_bs + (SQUARE ? bc : c0 + e) * p.st_rs + br * p.st_cs] = bs.s;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // 16 lanes store one column's 128 codes
      const int32_t cl = 16 * e + g;
      const int64_t c = bc * 128 + cl, r = br * 128 + 8 * l;
      const u32x2 w = *(const u32x2*)(codes + cl * 128 + 8 * (l ^ (cl >> 3)));
      if (!WHOLE && c >= p.cols) continue;
      uint8_t* Q = p.qt + b * p.qt_bs + c * p.qt_rs + r;
      if (WHOLE || r + 8 <= p.qt_cols) {
        *(u32x2*)Q = w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (r + i < p.qt_cols) Q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
    }
  }
}

template <int T, bool CONTIG, bool SQUARE>
__global__ __launch_bounds__(256, 4) void quantize_tile_kernel(const QuantizeParams p, uint32_t blocks_c, uint32_t blocks_r) {
  __shared__ __attribute__((aligned(16))) char codes[128 * 128];
  __shared__ uint32_t tops[4][128];
  const uint32_t id = blockIdx.x;
  const int64_t bc = id % blocks_c, br = id / blocks_c % blocks_r, b = id / blocks_c / blocks_r;
  if ((bc + 1) * 128 <= p.cols && (br + 1) * 128 <= p.rows)
    quantize_tile<T, CONTIG, SQUARE, true>(p, bc, br, b, codes, tops);
  else
    quantize_tile<T, CONTIG, SQUARE, false>(p, bc, br, b, codes, tops);
}

bool rows_only(const QuantizeParams& p) { return !p.qt && !p.square; }

template <int T, bool CONTIG>
void go(const QuantizeParams& p, hipStream_t s) {
  const uint32_t bc = (uint32_t)((p.cols + 127) / 128), br = (uint32_t)((p.rows + 127) / 128);
  const int64_t rows = quantize_rows(p);
  const dim3 grid((uint32_t)(p.batch * ((p.rows + rows - 1) / rows) * bc)), block(kQuantizeThreads);
  if (rows_only(p))
    hipLaunchKernelGGL((quantize_rows_kernel<T, CONTIG>), grid, block, 0, s, p, bc,
                       (uint32_t)((p.rows + kRowTile - 1) / kRowTile));
  else if (p.square)
    hipLaunchKernelGGL((quantize_tile_kernel<T, CONTIG, true>), grid, block, 0, s, p, bc, br);
  else
    hipLaunchKernelGGL((quantize_tile_kernel<T, CONTIG, false>), grid, block, 0, s, p, bc, br);
}

}  // namespace

int32_t quantize_rows(const QuantizeParams& p) { return rows_only(p) ? kRowTile : 128; }

hipError_t launch_quantize(const QuantizeParams& p, hipStream_t s) {
  const bool contig = p.x_cs == 1;
  switch (p.type) {
    case OT_F16: contig ? go<OT_F16, true>(p, s) : go<OT_F16, false>(p, s); break;
    case OT_BF16: contig ? go<OT_BF16, true>(p, s) : go<OT_BF16, false>(p, s); break;
    case OT_F32: contig ? go<OT_F32, true>(p, s) : go<OT_F32, false>(p, s); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace sl
