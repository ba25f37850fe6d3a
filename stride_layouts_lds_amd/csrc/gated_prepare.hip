// gated_prepare.hip -- what the gated feed-forward block's calls do ahead of
// their products, in one launch.
//
// Forward: operands whose rows are not K-contiguous on 16-byte boundaries are
// copied to such rows.  Backward, with g = x Wg^T, u = x Wu^T, h = act(g) u:
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu = [dg | du] [Wg ; Wu],  dWg = dg^T x,  dWu = du^T x
// The products contract over F and over the rows of x, along which their
// operands do not lie contiguous.  Where a product reads x or the weights as they lie
// (gated_backward.hip) it takes [dg | du] as rows; where it wants rows along
// the contracted axis, dg and du are written the other way too, and x or the
// weights transposed.  dg and du are rounded to the operands' 16 bits, half a step
// each, as any operand of a matrix product here: the gradients' errors are 2.4e-3 (bf16)
// and 2.9e-4 (fp16) of their norm, 1.7e-3 and 2.1e-4 with dg and du in 32 bits, which would take pairs
// of 16-bit values and twice the products.
//
// Bound by memory: 64 x 64 tiles, read along the axis that is contiguous in
// memory, turned in LDS.  dg and du of 4096 x 8192 as rows: 64 us, 5.2 TB/s.  Of small
// calls 3 us are the launch (one tile 3.7 us; 512 x 1024, both ways, with transposes for
// 512 columns of x 8).  (All of a thread's loads ahead of its tests for the edges
// changed nothing.)
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

template <int OT, int ACT>
__device__ __forceinline__ void slopes(const u16x8& g, const u16x8& u, const u16x8& d, u16x8& dg, u16x8& du) {
  constexpr int DT = OT == OT_F16 ? DT_F16 : DT_BF16;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a, slope;
    activate_with_slope(ACT, to_f32<DT>(g[e]), a, slope);
    const float dh = to_f32<DT>(d[e]);
    dg[e] = from_f32<DT>(dh * to_f32<DT>(u[e]) * slope);
    du[e] = from_f32<DT>(dh * a);
  }
}
template <int OT>
__device__ __forceinline__ void slopes_by_act(int32_t act, const u16x8& g, const u16x8& u, const u16x8& d, u16x8& dg, u16x8& du) {
  switch (act) {
    case ACT_SILU: slopes<OT, ACT_SILU>(g, u, d, dg, du); break;
    case ACT_GELU: slopes<OT, ACT_GELU>(g, u, d, dg, du); break;
    case ACT_GELU_TANH: slopes<OT, ACT_GELU_TANH>(g, u, d, dg, du); break;
    default: slopes<OT, ACT_RELU>(g, u, d, dg, du);
  }
}

__device__ __forceinline__ void slope_tile(const GatedSlopeParams& p, uint32_t id, uint32_t (*lds)[kTile * kPitch]) {
  const uint32_t tiles_f = (uint32_t)(p.Fp / kTile), tiles_m = (uint32_t)(p.Mp / kTile);
  const int64_t tf = id % tiles_f, tm = id / tiles_f % tiles_m, b = id / tiles_f / tiles_m;
  const int32_t l = threadIdx.x & 7, pair = threadIdx.x >> 3;
  const int64_t f0 = tf * kTile + 8 * l;
  u16x8 g[2], u[2], d[2], dg[2], du[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = tm * kTile + 2 * pair + i;
    g[i] = u[i] = d[i] = u16x8{0, 0, 0, 0, 0, 0, 0, 0};
    if (m < p.M) {
      g[i] = load8(p.g + b * p.g_bs + m * p.g_rs, p.g_cs, f0, p.F);
      u[i] = load8(p.u + b * p.u_bs + m * p.u_rs, p.u_cs, f0, p.F);
      d[i] = load8(p.dh + b * p.dh_bs + m * p.dh_rs, p.dh_cs, f0, p.F);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = tm * kTile + 2 * pair + i;
    if (p.type == OT_F16) slopes_by_act<OT_F16>(p.act, g[i], u[i], d[i], dg[i], du[i]);
    else slopes_by_act<OT_BF16>(p.act, g[i], u[i], d[i], dg[i], du[i]);
    // (where dh is zero, as in the padding, so are dg and du: act and act' of zero are finite)
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

// x's columns contiguous: rows copied.  Otherwise a tile is read along the
// rows' index and stored along the columns'.
__device__ __forceinline__ void pack_tile(const PackParams& p, uint32_t id, uint32_t* lds) {
  const uint32_t tiles_c = (uint32_t)((p.width + kTile - 1) / kTile), tiles_r = (uint32_t)((p.rows + kTile - 1) / kTile);
  const bool straight = p.x_cs == 1;
  // neighbouring workgroups along the axis that is contiguous in x
  const int64_t tc = straight ? id % tiles_c : id / tiles_r % tiles_c, tr = straight ? id / tiles_c % tiles_r : id % tiles_r;
  const int64_t b = id / tiles_c / tiles_r;
  const int32_t l = threadIdx.x & 7, pair = threadIdx.x >> 3;
  const uint16_t* x = p.x + b * p.x_bs;
  uint16_t* out = p.out + b * p.out_bs;
  if (straight) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = tr * kTile + 32 * i + pair, c = tc * kTile + 8 * l;
      if (r < p.rows && c < p.width) *(u16x8*)(out + r * p.out_rs + c) = load8(x + r * p.x_rs, 1, c, p.cols);
    }
    return;
  }
  const int64_t r0 = tr * kTile + 8 * l, c0 = tc * kTile + 2 * pair;
  u16x8 v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i] = u16x8{0, 0, 0, 0, 0, 0, 0, 0};
    if (c0 + i < p.cols) v[i] = load8(x + (c0 + i) * p.x_cs, p.x_rs, r0, p.rows);
  }
  put_columns(lds, l, pair, v[0], v[1]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t r = 32 * i + pair;
    const int64_t row = tr * kTile + r, col = tc * kTile + 8 * l;
    if (row < p.rows && col < p.width) *(u32x4*)(out + row * p.out_rs + col) = get_column(lds, r, l);
  }
}

__global__ __launch_bounds__(kPrepareThreads) void gated_prepare_kernel(const GatedPrepareParams p) {
  __shared__ uint32_t lds[2][kTile * kPitch];
  const uint32_t id = blockIdx.x;
  if (id < p.first[1]) slope_tile(p.slope, id, lds);
  else if (id < p.first[2]) pack_tile(p.pack[0], id - (uint32_t)p.first[1], lds[0]);
  else if (id < p.first[3]) pack_tile(p.pack[1], id - (uint32_t)p.first[2], lds[0]);
  else pack_tile(p.pack[2], id - (uint32_t)p.first[3], lds[0]);
}

int64_t tiles(int64_t n) { return (n + kTile - 1) / kTile; }

}  // namespace

int64_t gated_prepare_groups(GatedPrepareParams* p) {
  p->first[0] = 0;
  p->first[1] = p->slope.batch * tiles(p->slope.F) * tiles(p->slope.M);
  for (int i = 0; i < 3; ++i) p->first[i + 2] = p->first[i + 1] + p->pack[i].batch * tiles(p->pack[i].rows) * tiles(p->pack[i].width);
  return p->first[4];
}

hipError_t launch_gated_prepare(const GatedPrepareParams& p, hipStream_t s) {
  if (!p.first[4]) return hipSuccess;
  hipLaunchKernelGGL(gated_prepare_kernel, dim3((uint32_t)p.first[4]), dim3(kPrepareThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace sl
