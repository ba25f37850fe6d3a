// gated_backward.hip -- what the backward pass of the gated feed-forward block
// does beside its matrix products.  With g = x Wg^T, u = x Wu^T, h = act(g) u:
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu = [dg | du] [Wg ; Wu]
//   dWg = dg^T x,  dWu = du^T x
// The products contract over F and over the rows of x, along which their
// operands do not lie contiguous; the GEMM's ring kernel wants them so (read as
// they lie, by transposing LDS reads, 4096 x 4096 x 8192 takes 222 us, along K 179).  So
// dg and du are written both ways by the pass that makes them, x and the
// weights are transposed once, and every product reads both operands along K.
// dg and du are rounded to the operands' 16 bits, half a step each, as any
// operand of a matrix product here.
#include "activation.hpp"
#include "sl_device.hpp"

namespace sl {
namespace {

constexpr int kTile = 64;              // rows and columns of a tile
constexpr int kPitch = kTile / 2 + 1;  // dwords (pairs of rows) of a tile's column in LDS, off the banks' number

typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));

// eight values of a row from column c (zero from `cols` on)
__device__ __forceinline__ u16x8 load8(const uint16_t* row, int64_t cs, int64_t c, int64_t cols) {
  if (cs == 1 && c + 8 <= cols) return *(const u16x8u*)(row + c);
  u16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < cols) v[e] = row[(c + e) * cs];
  return v;
}

// A thread's values of two neighbouring rows (2 pair, 2 pair + 1), columns
// 8 l .. + 7, into the tile's columns: pair p of column c at c kPitch + p.  A
// wave's 64 lanes (8 column groups, 8 pairs) write one e to 64 banks.
__device__ __forceinline__ void put_columns(uint32_t* lds, int32_t l, int32_t pair, const u16x8& r0, const u16x8& r1) {
#pragma unroll
  for (int e = 0; e < 8; ++e) lds[(8 * l + e) * kPitch + pair] = (uint32_t)r0[e] | (uint32_t)r1[e] << 16;
}
// rows 8 k .. + 7 of column c
__device__ __forceinline__ u32x4 get_column(const uint32_t* lds, int32_t c, int32_t k) {
  const uint32_t* at = lds + c * kPitch + 4 * k;
  return u32x4{at[0], at[1], at[2], at[3]};
}

__global__ __launch_bounds__(kPackThreads) void gated_slope_kernel(const GatedSlopeParams p, uint32_t tiles_f, uint32_t tiles_m) {
  __shared__ uint32_t lds[2][kTile * kPitch];
  const uint32_t id = blockIdx.x;
  const int64_t tf = id % tiles_f, tm = id / tiles_f % tiles_m, b = id / tiles_f / tiles_m;
  const int32_t l = threadIdx.x & 7, pair = threadIdx.x >> 3;
  const int64_t f0 = tf * kTile + 8 * l;
  u16x8 dg[2], du[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = tm * kTile + 2 * pair + i;
    u16x8 g = {0, 0, 0, 0, 0, 0, 0, 0}, u = g, d = g;
    if (m < p.M) {
      g = load8(p.g + b * p.g_bs + m * p.g_rs, p.g_cs, f0, p.F);
      u = load8(p.u + b * p.u_bs + m * p.u_rs, p.u_cs, f0, p.F);
      d = load8(p.dh + b * p.dh_bs + m * p.dh_rs, p.dh_cs, f0, p.F);
    }
    auto value = [&](uint16_t v) { return p.type == OT_F16 ? to_f32<DT_F16>(v) : to_f32<DT_BF16>(v); };
    auto code = [&](float v) { return p.type == OT_F16 ? from_f32<DT_F16>(v) : from_f32<DT_BF16>(v); };
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a, slope;
      activate_with_slope(p.act, value(g[e]), a, slope);
      const float dh = value(d[e]);
      // padding is zero whatever the activation makes of it
      const bool in = m < p.M && f0 + e < p.F;
      dg[i][e] = in ? code(dh * value(u[e]) * slope) : (uint16_t)0;
      du[i][e] = in ? code(dh * a) : (uint16_t)0;
    }
    if (p.rows && m < p.M) {
      uint16_t* out = p.rows + (b * p.M + m) * 2 * p.Fp + f0;
      *(u16x8*)out = dg[i];
      *(u16x8*)(out + p.Fp) = du[i];
    }
  }
  if (!p.t) return;
  put_columns(lds[0], l, pair, dg[0], dg[1]);
  put_columns(lds[1], l, pair, du[0], du[1]);
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t c = 32 * i + pair;
      const int64_t f = tf * kTile + c;
      if (f < p.F) *(u32x4*)(p.t + b * p.t_bs + s * p.t_us + f * p.t_rs + tm * kTile + 8 * l) = get_column(lds[s], c, l);
    }
}

// x's rows lie apart and its columns together: a tile is read along the rows'
// index and stored along the columns'
__global__ __launch_bounds__(kPackThreads) void pack_transposing_kernel(const PackParams p, uint32_t tiles_c, uint32_t tiles_r) {
  __shared__ uint32_t lds[kTile * kPitch];
  const uint32_t id = blockIdx.x;
  const int64_t tr = id % tiles_r, tc = id / tiles_r % tiles_c, b = id / tiles_r / tiles_c;
  const int32_t l = threadIdx.x & 7, pair = threadIdx.x >> 3;
  const int64_t r0 = tr * kTile + 8 * l, c0 = tc * kTile + 2 * pair;
  u16x8 v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i] = u16x8{0, 0, 0, 0, 0, 0, 0, 0};
    if (c0 + i < p.cols) v[i] = load8(p.x + b * p.x_bs + (c0 + i) * p.x_cs, p.x_rs, r0, p.rows);
  }
  put_columns(lds, l, pair, v[0], v[1]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t r = 32 * i + pair;
    const int64_t row = tr * kTile + r, col = tc * kTile + 8 * l;
    if (row < p.rows && col < p.width) *(u32x4*)(p.out + b * p.out_bs + row * p.out_rs + col) = get_column(lds, r, l);
  }
}

// rows of x contiguous (off 16 bytes) or of any strides: 2048 values of a row
// to a workgroup
__global__ __launch_bounds__(kPackThreads) void pack_rows_kernel(const PackParams p, uint32_t tiles_c) {
  const uint32_t id = blockIdx.x;
  const int64_t c = (int64_t)(id % tiles_c) * (8 * kPackThreads) + 8 * threadIdx.x;
  const int64_t r = id / tiles_c % p.rows, b = id / tiles_c / p.rows;
  if (c < p.width) *(u16x8*)(p.out + b * p.out_bs + r * p.out_rs + c) = load8(p.x + b * p.x_bs + r * p.x_rs, p.x_cs, c, p.cols);
}

int64_t tiles(int64_t n) { return (n + kTile - 1) / kTile; }
bool transposing(const PackParams& p) { return p.x_rs == 1 && p.x_cs != 1; }

}  // namespace

int64_t gated_slope_groups(const GatedSlopeParams& p) { return p.batch * tiles(p.F) * tiles(p.M); }

hipError_t launch_gated_slope(const GatedSlopeParams& p, hipStream_t s) {
  hipLaunchKernelGGL(gated_slope_kernel, dim3((uint32_t)gated_slope_groups(p)), dim3(kPackThreads), 0, s, p, (uint32_t)tiles(p.F),
                     (uint32_t)tiles(p.M));
  return hipGetLastError();
}

int64_t pack_groups(const PackParams& p) {
  return transposing(p) ? p.batch * tiles(p.rows) * tiles(p.width) : p.batch * p.rows * ((p.width + 8 * kPackThreads - 1) / (8 * kPackThreads));
}

hipError_t launch_pack(const PackParams& p, hipStream_t s) {
  const dim3 grid((uint32_t)pack_groups(p)), block(kPackThreads);
  if (transposing(p))
    hipLaunchKernelGGL(pack_transposing_kernel, grid, block, 0, s, p, (uint32_t)tiles(p.width), (uint32_t)tiles(p.rows));
  else
    hipLaunchKernelGGL(pack_rows_kernel, grid, block, 0, s, p, (uint32_t)((p.width + 8 * kPackThreads - 1) / (8 * kPackThreads)));
  return hipGetLastError();
}

}  // namespace sl
