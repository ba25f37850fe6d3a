// dense.hpp -- the kernels of a product of K-contiguous rows, for the int8
// product (gemm_i8.hip) and the gated pair of products (gated.hip):
//
//   sums[m,n] = sum_k A[m,k] B[n,k]
//
// on fp16, bf16 or int8 values, handed on in fp32 (int8: exact int32) to what
// makes the result of them.  A row's K-tile is 128 bytes (64 or 128 values)
// and a matrix instruction takes 64 of them, 16 a lane, so that one kernel
// serves every kind: only the instruction differs.
//
// The gated pair (GATED) is one product whose B rows come from two matrices
// in turn, a few 16-row fragments of the one and then of the other, so that a
// lane's accumulators hold g and u of the same (m, n): the activation and the
// product with u cost no traffic, and A is read once for both.
//
// Tiles (dense_plan):
//   256 x 256, 256 x 192, 256 x 128, 128 x 128   4 waves, accumulators in AGPRs, LDS a ring
//   DT_STREAM  32 or 64 rows of A, the waves of a workgroup splitting K
//   DT_SKINNY  up to 16 rows, K-tiles straight from memory into registers
#pragma once
#include "sl_ops.hpp"

#include "sl_device.hpp"

namespace sl {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// One step of 64 bytes of K on a 16 x 16 result.  int8 sums are int32 in the
// accumulator's registers, which travel as floats' bits.
template <int EK>
__device__ __forceinline__ floatx4 dense_mfma(const u32x4& a, const u32x4& b, const floatx4& c) {
  if constexpr (EK == EK_I8)
    return __builtin_bit_cast(floatx4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b),
                                                                             __builtin_bit_cast(i32x4, c), 0, 0, 0));
  else
    return mfma16<EK == EK_F16 ? DT_F16 : DT_BF16>(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c);
}
// the same on an accumulator held in AGPRs (as mfma_acc of gemm_f16.hip: the
// compiler inserts no wait states before the result is read)
template <int EK>
__device__ __forceinline__ void dense_mfma_agpr(floatx4& c, const u32x4& a, const u32x4& b) {
  if constexpr (EK == EK_I8)
    asm("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else if constexpr (EK == EK_F16)
    asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// two waves' sums
template <int EK>
__device__ __forceinline__ floatx4 dense_add(floatx4 a, floatx4 b) {
  if constexpr (EK == EK_I8) return __builtin_bit_cast(floatx4, __builtin_bit_cast(i32x4, a) + __builtin_bit_cast(i32x4, b));
  else return floatx4{a[0] + b[0], a[1] + b[1], a[2] + b[2], a[3] + b[3]};
}
// sums as fp32 (int32 rounded to nearest: 2^-24)
template <int EK>
__device__ __forceinline__ floatx4 dense_value(floatx4 v) {
  if constexpr (EK == EK_I8) {
    const i32x4 i = __builtin_bit_cast(i32x4, v);
    return floatx4{(float)i[0], (float)i[1], (float)i[2], (float)i[3]};
  } else {
    return v;
  }
}

// HBM -> LDS copies of a K-tile of ROWS rows, 128 bytes each, in the
// XOR-swizzled layout of lds_offset (LoaderKVec's, which see).  G > 0: rows of
// two matrices in turn, G of the one and G of the other; which one a copy
// reads depends on its number alone.  Rows past the valid ones, and K past its
// end, read zero: their offsets are out of range whatever the strides.
template <int ROWS, int NT, int G>
struct RowLoader {
  static constexpr int WAVES = NT / 64, RB = kRowBytes;
  static constexpr int CPR = RB / 16, RPI = 64 / CPR;  // 16-byte chunks of a row, rows of a copy
  static constexpr int ITERS = ROWS / (RPI * WAVES);
  static constexpr int SRC = G > 0 ? 2 : 1;
  static_assert(ITERS >= 1 && ROWS % (RPI * WAVES) == 0, "copies of whole waves");
  static_assert(G == 0 || G % (RPI * WAVES) == 0, "a copy reads one matrix");
  static constexpr int src(int j) { return G > 0 ? (j * WAVES * RPI / (G > 0 ? G : 1)) & 1 : 0; }

  __amdgpu_buffer_rsrc_t rsrc[SRC];
  int32_t K, wave, lane;
  uint32_t voff[ITERS];

  // `rows` valid rows of each matrix from base[s]
  __device__ __forceinline__ RowLoader(const uint8_t* const (&base)[SRC], const int64_t (&rs)[SRC], int32_t rows, int64_t K_, int32_t wave_,
                                       int32_t lane_)
      : K((int32_t)K_), wave(wave_), lane(lane_) {
#pragma unroll
    for (int s = 0; s < SRC; ++s) rsrc[s] = make_rsrc(base[s], rows > 0 ? (uint32_t)((int64_t)(rows - 1) * rs[s] + K_) : 0u);
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
      const int32_t R = tile_row(j);
      const int32_t r = G > 0 ? R / (2 * (G > 0 ? G : 1)) * G + R % (G > 0 ? G : 1) : R;
      voff[j] = r < rows ? (uint32_t)(r * rs[src(j)] + 16 * chunk(j)) : kOutOfRange;
    }
  }
  __device__ __forceinline__ int32_t tile_row(int j) const { return (j * WAVES + wave) * RPI + lane / CPR; }
  __device__ __forceinline__ int32_t chunk(int j) const { return (lane & (CPR - 1)) ^ swz(tile_row(j), 0, RB); }

  // From here on the copies are of the last K-tile, of which `bytes` lie inside K
  // (128 or fewer): the chunks past them read zero.
  __device__ __forceinline__ void last_tile(int32_t bytes) {
#pragma unroll
    for (int j = 0; j < ITERS; ++j) voff[j] = 16 * chunk(j) < bytes ? voff[j] : kOutOfRange;
  }

  // copy j of a K-tile that lies inside K, or of the last one after last_tile.
  // The lane's offset is voff[j] and the K-tile's start goes into the scalar
  // offset: no vector arithmetic next to the products.  (Elements are copied to locals
  // first: the host compilation pass drops the launch stubs of kernels that
  // index a member array inside the builtin's argument list.)
  __device__ __forceinline__ void issue_full(int32_t t, char* lds, int j) const {
    const uint32_t v = voff[j];
    const uint32_t s = (uint32_t)t * RB;
    const __amdgpu_buffer_rsrc_t from = rsrc[src(j)];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void_t*)(lds + (j * WAVES + wave) * 1024), 16, v, s, 0, 0);
  }
  // copy j of any K-tile (counted in 32 bits without a sign: K is below 2^31, a K-tile
  // requested ahead of the last one may start past that)
  __device__ __forceinline__ void issue_one(int32_t t, char* lds, int j) const {
    const uint32_t s = (uint32_t)t * RB;
    const uint32_t at = voff[j] == kOutOfRange || s + (uint32_t)(16 * chunk(j)) >= (uint32_t)K ? kOutOfRange : voff[j] + s;
    const __amdgpu_buffer_rsrc_t from = rsrc[src(j)];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void_t*)(lds + (j * WAVES + wave) * 1024), 16, at, 0, 0, 0);
  }
  __device__ __forceinline__ void issue(int32_t t, char* lds) const {
#pragma unroll
    for (int j = 0; j < ITERS; ++j) issue_one(t, lds, j);
  }
};

// The product that a workgroup belongs to, its number among that one's
// workgroups, and theirs.
__device__ __forceinline__ const DenseParams& dense_product(const DenseParams& p, uint32_t& id, uint32_t& total) {
  id = blockIdx.x, total = gridDim.x;
  return p;
}
__device__ __forceinline__ const DenseParams& dense_product(const DensePair& p, uint32_t& id, uint32_t& total) {
  const bool second = blockIdx.x >= p.first;
  id = blockIdx.x - (second ? p.first : 0u), total = second ? gridDim.x - p.first : p.first;
  return second ? p.p[1] : p.p[0];
}

// rows of the gated pair that a tile of BN rows of B holds of each matrix
template <bool GATED, int BN>
constexpr int kResultCols = GATED ? BN / 2 : BN;

template <bool GATED, int BN, int NT, int G>
__device__ __forceinline__ RowLoader<BN, NT, G> dense_b_loader(const DenseParams& p, int64_t batch, int64_t n0, int32_t cols, int32_t wave,
                                                               int32_t lane) {
  if constexpr (GATED) {
    const uint8_t* const base[2] = {p.b[0] + batch * p.b_bs[0] + n0 * p.b_rs[0], p.b[1] + batch * p.b_bs[1] + n0 * p.b_rs[1]};
    const int64_t rs[2] = {p.b_rs[0], p.b_rs[1]};
    return RowLoader<BN, NT, G>(base, rs, cols, p.K, wave, lane);
  } else {
    const uint8_t* const base[1] = {p.b[0] + (batch >> p.b_shift) * p.b_bs[0] + n0 * p.b_rs[0]};
    const int64_t rs[1] = {p.b_rs[0]};
    return RowLoader<BN, NT, G>(base, rs, cols, p.K, wave, lane);
  }
}
template <int BM, int NT>
__device__ __forceinline__ RowLoader<BM, NT, 0> dense_a_loader(const DenseParams& p, int64_t batch, int64_t m0, int32_t rows, int32_t wave,
                                                               int32_t lane) {
  const uint8_t* const base[1] = {p.a + batch * p.a_bs + m0 * p.a_rs};
  const int64_t rs[1] = {p.a_rs};
  return RowLoader<BM, NT, 0>(base, rs, rows, p.K, wave, lane);
}

// a lane's 16 bytes of slice ks (64 bytes of K) of the 16 rows from row0
__device__ __forceinline__ u32x4 dense_frag(const char* tile, int32_t lane, int32_t row0, int32_t ks) {
  return *(const u32x4*)(tile + fragment_lds_offset(MFMA16_F16, lane, 0, row0, ks, 0));
}

// ---------------------------------------------------------------------------
// What becomes of the sums: EPI::finish(batch, m, n, v) takes four consecutive
// columns of one row, for the gated pair those of both products, with m < M
// and n < N; columns from N on are not stored.  EPI::rows: see dense_rows.
// Defined by the including file.
// ---------------------------------------------------------------------------

// four values to a 16- or 32-bit row, `valid` of them
__device__ __forceinline__ void dense_store(void* base, int32_t type, int64_t off, int64_t cs, bool vec, int64_t valid, floatx4 v) {
  if (type == OT_F32) {
    float* d = (float*)base + off;
    if (vec && valid >= 4) {
      *(floatx4*)d = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < valid) d[r * cs] = v[r];
    }
    return;
  }
  const u16x4 w = type == OT_F16 ? u16x4{from_f32<DT_F16>(v[0]), from_f32<DT_F16>(v[1]), from_f32<DT_F16>(v[2]), from_f32<DT_F16>(v[3])}
                                 : u16x4{from_f32<DT_BF16>(v[0]), from_f32<DT_BF16>(v[1]), from_f32<DT_BF16>(v[2]), from_f32<DT_BF16>(v[3])};
  uint16_t* d = (uint16_t*)base + off;
  if (vec && valid >= 4) {
    *(u16x4*)d = w;
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < valid) d[r * cs] = w[r];
  }
}
__device__ __forceinline__ floatx4 dense_load(const void* base, int32_t type, int64_t off, int64_t cs, bool vec, int64_t valid) {
  floatx4 v = {0.f, 0.f, 0.f, 0.f};
  if (type == OT_F32) {
    const float* d = (const float*)base + off;
    if (vec && valid >= 4) return *(const floatx4*)d;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < valid) v[r] = d[r * cs];
    return v;
  }
  const uint16_t* d = (const uint16_t*)base + off;
  u16x4 w = {0, 0, 0, 0};
  if (vec && valid >= 4) {
    w = *(const u16x4*)d;
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < valid) w[r] = d[r * cs];
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = type == OT_F16 ? to_f32<DT_F16>(w[r]) : to_f32<DT_BF16>(w[r]);
  return v;
}

// V consecutive values of a row that starts on a boundary of V of them (16-bit types: one,
// four or eight; fp32: one or four).
template <int OT, int V>
__device__ __forceinline__ void dense_store_cols(void* at, const float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (OT == OT_F32) *(float*)at = v[0];
    else *(uint16_t*)at = from_f32<OT == OT_F16 ? DT_F16 : DT_BF16>(v[0]);
  } else if constexpr (OT == OT_F32) {
    typedef float floats __attribute__((ext_vector_type(V)));
    floats w;
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = v[e];
    *(floats*)at = w;
  } else {
    typedef uint16_t halves __attribute__((ext_vector_type(V)));
    halves w;
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = from_f32<OT == OT_F16 ? DT_F16 : DT_BF16>(v[e]);
    *(halves*)at = w;
  }
}
template <int OT, int V>
__device__ __forceinline__ void dense_load_cols(const void* at, float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (OT == OT_F32) v[0] = *(const float*)at;
    else v[0] = to_f32<OT == OT_F16 ? DT_F16 : DT_BF16>(*(const uint16_t*)at);
  } else if constexpr (OT == OT_F32) {
    typedef float floats __attribute__((ext_vector_type(V)));
    const floats w = *(const floats*)at;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = w[e];
  } else {
    typedef uint16_t halves __attribute__((ext_vector_type(V)));
    const halves w = *(const halves*)at;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = to_f32<OT == OT_F16 ? DT_F16 : DT_BF16>(w[e]);
  }
}

// A wave's 64 x COLS block of sums (COLS = 128, 96 or 64) from its region of LDS,
// in the chunk order of rows_chunk (96 columns in rows of 128), row after row: whole
// rows of the block are stored together.  GATED: the first half of the columns are
// g, the others u.
//
// Contiguous outputs go V columns a lane: EPI::rows<RPI, V>(batch, m, n, count, get)
// finishes columns n .. n + V - 1 of rows m, m + RPI, ... as far as `count` of
// them, get(it, s, v) being the sums of the it-th, s 0: g or the product's, 1: u.
// V is eight (DF_ROWS8) or four (DF_ROWS4) where every row starts on a boundary of so many,
// else one (DF_ROWS): an access off its boundaries is taken apart by the hardware (us, int8 528
// x 870 x 48 + C 20 by eights and 8 by ones; 528 x 868 x 48, rows on 8 bytes, 12 by eights, 8 by
// ones, 7 by fours; 4000 x 3004 x 2064 + C 66, 47 and 40).  (Of eights, where eight lanes have a row, a wave's LDS reads pair lanes 0-7 with 16-23, 8-15 with 24-31 and so
// on: the rows of a pair differ in the lowest bit, so that their chunks, all even or all
// odd in a row, lie on different banks.)  Other outputs, and the columns next to N
// where those are no V: EPI::finish.
template <int COLS>
constexpr int kRowsPitch = COLS == 96 ? 128 : COLS;
template <int EK, bool GATED, int COLS, class EPI>
__device__ __forceinline__ void dense_rows(const EPI& epi, const DenseParams& p, int64_t batch, int64_t m_base, int64_t n_base, int32_t lane,
                                           const char* region) {
  static_assert(!GATED || COLS != 96, "halves of whole lanes");
  constexpr int OUT = GATED ? COLS / 2 : COLS;  // columns of the result
  constexpr int PITCH = kRowsPitch<COLS>;
  auto quad = [&](int32_t r, int32_t q) { return dense_value<EK>(*(const floatx4*)(region + rows_chunk<PITCH>(r, q))); };
  auto by = [&](auto columns, bool whole) {
    constexpr int V = decltype(columns)::value;
    constexpr int PAD = GATED ? PITCH / 2 : PITCH;  // (of 96 columns a quarter of the lanes is idle)
    constexpr int LPR = PAD / V < 64 ? PAD / V : 64, RPI = 64 / LPR;  // lanes to a row, rows at once
    const int32_t group = lane / LPR;
    // (the row bit that pairs of lane groups differ in goes last)
    const int32_t r0 = V == 8 && LPR == 8 ? (group & 4) | (group & 1) << 1 | (group & 2) >> 1 : group;
    const int64_t m = m_base + r0;
    const int32_t count = m < p.M ? (int32_t)(p.M - m > 64 ? 64 / RPI : (p.M - m + RPI - 1) / RPI) : 0;
#pragma unroll 1
    for (int32_t c = V * (lane % LPR); c < OUT; c += V * LPR) {
      const int64_t n = n_base + c;
      if (n >= p.N || count == 0) return;
      if (whole && n + V <= p.N) {
        auto get = [&](int32_t it, int s, float(&v)[V]) {
          const int32_t r = RPI * it + r0, at = c + (s ? OUT : 0);
          if constexpr (V == 1) {
            const char* from = region + rows_chunk<PITCH>(r, at / 4) + 4 * (at % 4);
            if constexpr (EK == EK_I8) v[0] = (float)*(const int32_t*)from;
            else v[0] = *(const float*)from;
          } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
              const floatx4 a = quad(r, at / 4 + i);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[4 * i + e] = a[e];
            }
          }
        };
        epi.template rows<RPI, V>(p, batch, m, n, count, get);
      } else if constexpr (V > 1) {
#pragma unroll 1
        for (int it = 0; it < V / 4 * count; ++it) {
          const int32_t r = RPI * (it / (V / 4)) + r0, q = c / 4 + it % (V / 4);
          const int64_t nq = n + 4 * (it % (V / 4));
          if (nq >= p.N) continue;
          if constexpr (GATED) epi.finish(p, batch, m_base + r, nq, quad(r, q), quad(r, q + OUT / 4));
          else epi.finish(p, batch, m_base + r, nq, quad(r, q));
        }
      }
    }
  };
  if (p.flags & DF_ROWS8) by(std::integral_constant<int, 8>{}, true);
  else if ((p.flags & (DF_ROWS | DF_ROWS4)) == DF_ROWS) by(std::integral_constant<int, 1>{}, true);
  else by(std::integral_constant<int, 4>{}, p.flags & DF_ROWS4);
}

// ---------------------------------------------------------------------------
// Large tiles, on the schedule of gemm_f16_w4r_kernel (gemm_f16.hip), which see:
// four waves, each FM x FN instruction tiles with its accumulators in AGPRs,
// LDS a ring of S operand K-tiles, operand tile q (A of K-tile q / 2 for even q, B for
// odd q) in slot q % S.  Per K-tile: reads of its first slice beside the last
// products of the K-tile before, the first slice's products beside the reads of
// the second, half of the second's, one barrier.  A copy has a K-tile of compute or
// more to land.
//   8 x 8  256 x 256, one workgroup to a CU
//   8 x 6  256 x 192, the same
//   8 x 4  256 x 128, the same
//   4 x 4  128 x 128, two to a CU
// AHEAD K-tiles more on their way (dense_plan) take a CU's LDS.  The gated pair's wave
// holds 8 FN rows of each matrix.  int8 8192^3 takes 383 to 395 us (2.8 POP/s), gated bf16 4096 x
// 8192 x 4096 with both projections kept 396 to 412 us (1.36 PFLOP/s), back to back on several
// cards: the matrix cores are busy 70% of the time, at 1.9 GHz (power).
// ---------------------------------------------------------------------------
template <int EK, bool GATED, int FM, int FN, int AHEAD, class EPI, class PRODUCTS>
__global__ __launch_bounds__(256, FM == 8 || AHEAD > 0 ? 1 : 2) void dense_ring_kernel(const PRODUCTS products_) {
  uint32_t id, total;
  const DenseParams& p = dense_product(products_, id, total);
  constexpr int ROWS_A = 32 * FM, ROWS_B = 32 * FN, SLOT = (FM > FN ? ROWS_A : ROWS_B) * kRowBytes;
  constexpr int BN = kResultCols<GATED, ROWS_B>;
  constexpr int NR = FM + FN;      // fragment reads of a slice
  constexpr int NH = FM / 2 * FN;  // products of half a slice
  constexpr int S = kRing + 2 * AHEAD;  // operand K-tiles in LDS
  __shared__ __attribute__((aligned(1024))) char smem[S * SLOT];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TileCoord tc = map_tile((int32_t)id, (int32_t)total, p.tiles_m, p.tiles_n, p.group_m, p.batch);
  const int64_t m0 = (int64_t)tc.tm * ROWS_A, n0 = (int64_t)tc.tn * BN;
  const int32_t rows_a = (int32_t)(p.M - m0 < ROWS_A ? p.M - m0 : ROWS_A);
  const int32_t cols = (int32_t)(p.N - n0 < BN ? p.N - n0 : BN);
  auto la = dense_a_loader<ROWS_A, 256>(p, tc.batch, m0, rows_a, wave, lane);
  auto lb = dense_b_loader<GATED, ROWS_B, 256, GATED ? 8 * FN : 0>(p, tc.batch, n0, cols, wave, lane);
  static_assert(decltype(la)::ITERS == FM && decltype(lb)::ITERS == FN, "copy layout");

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int32_t a_row0 = (wave & 1) * 16 * FM, b_row0 = (wave >> 1) * 16 * FN;
  const int32_t T = p.k_tiles;  // at least 1
  __builtin_assume(T >= 1);
  auto slot = [&](int32_t q) { return smem + q * SLOT; };
  auto copy_a = [&](int32_t u, char* dst, int j) { la.issue_full(u, dst, j); };
  auto copy_b = [&](int32_t u, char* dst, int j) { lb.issue_full(u, dst, j); };
  const int32_t last_bytes = (int32_t)p.K - (T - 1) * kRowBytes;
  u32x4 fa0[FM], fb0[FN], fa1[FM], fb1[FN];
  typedef __attribute__((address_space(3))) const u32x4 lds_u4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)smem;
  uint32_t offA[2][2], offB[2][2], bA[2][2], bB[2][2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      offA[ks][par] = lds0 + (uint32_t)fragment_lds_offset(MFMA16_F16, lane, 0, a_row0 + 16 * par, ks, 0);
      offB[ks][par] = lds0 + (uint32_t)fragment_lds_offset(MFMA16_F16, lane, 0, b_row0 + 16 * par, ks, 0);
    }
  auto bases = [&](int32_t qa, int32_t qb) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        bA[ks][par] = offA[ks][par] + (uint32_t)(qa * SLOT);
        bB[ks][par] = offB[ks][par] + (uint32_t)(qb * SLOT);
      }
    // computed here, not next to the reads
    asm volatile("" : "+v"(bA[0][0]), "+v"(bA[0][1]), "+v"(bA[1][0]), "+v"(bA[1][1]));
    asm volatile("" : "+v"(bB[0][0]), "+v"(bB[0][1]), "+v"(bB[1][0]), "+v"(bB[1][1]));
  };
  // B's fragments first
  auto read = [&](int r, int ks, u32x4(&fa)[FM], u32x4(&fb)[FN]) {
    if (r < FN)
      fb[r] = *(lds_u4*)(uintptr_t)(bB[ks][r & 1] + 4096u * (uint32_t)(r >> 1));
    else
      fa[r - FN] = *(lds_u4*)(uintptr_t)(bA[ks][(r - FN) & 1] + 4096u * (uint32_t)((r - FN) >> 1));
  };
  // products [e0, e1) of the block's rows from i0 on
  auto products = [&](int i0, int e0, int e1, const u32x4(&fa)[FM], const u32x4(&fb)[FN]) {
#pragma unroll
    for (int e = e0; e < e1; ++e) dense_mfma_agpr<EK>(acc[i0 + e / FN][e % FN], fb[e % FN], fa[i0 + e / FN]);
  };
  // ahead of a copy of K-tile u: the last one ends at K, those behind it read zeros
  auto ends_a = [&](int32_t u) {
    if (u >= T - 1) la.last_tile(u == T - 1 ? last_bytes : 0);
  };
  auto ends_b = [&](int32_t u) {
    if (u >= T - 1) lb.last_tile(u == T - 1 ? last_bytes : 0);
  };
#pragma unroll
  for (int u = 0; u <= AHEAD + 1; ++u) {
    ends_a(u);
#pragma unroll
    for (int j = 0; j < FM; ++j) copy_a(u, slot(2 * u), j);
    ends_b(u);
#pragma unroll
    for (int j = 0; j < FN && u <= AHEAD; ++j) copy_b(u, slot(2 * u + 1), j);
  }
  ends_a(AHEAD + 2);
  // the first K-tile's first part computes with zero fragments (adds nothing)
#pragma unroll
  for (int i = 0; i < FM; ++i) fa1[i] = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < FN; ++j) fb1[j] = u32x4{0, 0, 0, 0};
  constexpr int FLIGHT = FM * (AHEAD + 1) + FN * AHEAD;  // copies of the K-tiles behind the next one
  wait_vmem_n<FLIGHT>();
  phase_barrier();
  int32_t sa = 0;  // slot of A(t); B(t) in the next one
  int32_t t = 0;
  bases(0, 1);
  // one copy of the loop body: a peeled or unswitched copy would give the
  // accumulators a second path to what follows
#pragma clang loop unroll(disable)
  do {
    const int32_t s3 = sa < 2 ? sa + S - 2 : sa - 2, s4 = sa == 0 ? S - 1 : sa - 1;
#pragma unroll
    for (int g = 0; g < NR; ++g) {
      read(g, 0, fa0, fb0);
#pragma unroll
      for (int j = g * FN / NR; j < (g + 1) * FN / NR; ++j) copy_b(t + AHEAD + 1, slot(s3), j);
      products(FM / 2, g * NH / NR, (g + 1) * NH / NR, fa1, fb1);  // K-tile t - 1's
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int g = 0; g < NR; ++g) {
      read(g, 1, fa1, fb1);
#pragma unroll
      for (int j = g * FM / NR; j < (g + 1) * FM / NR; ++j) copy_a(t + AHEAD + 2, slot(s4), j);
      products(0, g * 2 * NH / NR, (g + 1) * 2 * NH / NR, fa0, fb0);
      __builtin_amdgcn_sched_barrier(0);
    }
    products(0, 0, NH, fa1, fb1);
    const int32_t na = sa + 2 >= S ? sa + 2 - S : sa + 2;
    bases(na, na == S - 1 ? 0 : na + 1);
    ends_b(t + AHEAD + 2);
    ends_a(t + AHEAD + 3);
    wait_vmem_n<FLIGHT>();  // K-tile t + 1 has landed
    phase_barrier();
    sa = na;
  } while (++t < T);
  products(FM / 2, 0, NH, fa1, fb1);
  wait_vmem();
  // the products are inline assembly: an idle of 32 cycles between the last
  // of them and the first read of an accumulator, which the two statements
  // that re-define them all hold in place
  auto pin = [&] {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; j += 2) asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
  };
  pin();
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  pin();
  // every wave's copies have landed and its reads of the ring are done
  __syncthreads();
  constexpr int COLS = 16 * FN;
  constexpr int PITCH = kRowsPitch<COLS>;
  char* region = smem + wave * (64 * PITCH * 4);
  static_assert(4 * 64 * PITCH * 4 <= S * SLOT, "the sums fit");
  const EPI epi(p, tc.batch);
  const int64_t n_base = n0 + kResultCols<GATED, COLS> * (wave >> 1);
#pragma unroll
  for (int h = 0; h < FM / 4; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) *(floatx4*)(region + rows_chunk<PITCH>(16 * i + (lane & 15), 4 * j + (lane >> 4))) = acc[4 * h + i][j];
    dense_rows<EK, GATED, COLS>(epi, p, tc.batch, m0 + a_row0 + 64 * h, n_base, lane, region);
  }
}

// The sums of a workgroup's W waves, each of FM x FN instruction tiles, meet
// in LDS and the waves finish a tile (gated: a pair of tiles) each in turn.
template <int EK, bool GATED, int FM, int FN, int W, class EPI>
__device__ __forceinline__ void dense_join(const DenseParams& p, int64_t batch, int64_t m0, int64_t n0, int32_t lane, int32_t wave,
                                           const floatx4 (&acc)[FM][FN], floatx4* part) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) part[((wave * FM + i) * FN + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  const EPI epi(p, batch);
  constexpr int OUT = GATED ? FN / 2 : FN;
  auto total = [&](int32_t tile) {
    floatx4 v = part[tile * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v = dense_add<EK>(v, part[(w * FM * FN + tile) * 64 + lane]);
    return dense_value<EK>(v);
  };
  for (int32_t e = wave; e < FM * OUT; e += W) {
    const int32_t i = e / OUT, j = e % OUT;
    const int64_t m = m0 + 16 * i + (lane & 15), n = n0 + 16 * j + 4 * (lane >> 4);
    if (m >= p.M || n >= p.N) continue;
    if constexpr (GATED) epi.finish(p, batch, m, n, total(i * FN + j), total(i * FN + OUT + j));
    else epi.finish(p, batch, m, n, total(i * FN + j));
  }
}

// Up to 16 rows of A: B is read once and bounds the call.  A workgroup owns
// 16 FN rows of B (gated: 8 FN of each matrix); wave w of eight takes the
// K-tiles w, w + 8, ... straight from memory into registers, DEPTH requested
// ahead.  int8 1 x 4096 x 8192: 8.4 us, 4.0 TB/s; gated bf16 1 x 8192 x 4096: 25 us, 5.3.
template <int EK, bool GATED, int FN, class EPI, class PRODUCTS>
__global__ __launch_bounds__(kDenseSkinnyWaves * 64) void dense_skinny_kernel(const PRODUCTS products_) {
  uint32_t id, total;
  const DenseParams& p = dense_product(products_, id, total);
  constexpr int W = kDenseSkinnyWaves, DEPTH = 4;
  constexpr int OUT = GATED ? FN / 2 : FN;
  __shared__ floatx4 part[W * FN * 64];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tn = id % p.tiles_n, tm = id / p.tiles_n % p.tiles_m, batch = id / p.tiles_n / p.tiles_m;
  const int64_t m0 = tm * 16, n0 = tn * (16 * OUT);
  const int32_t rows = (int32_t)(p.M - m0 < 16 ? p.M - m0 : 16);
  const int32_t cols = (int32_t)(p.N - n0 < 16 * OUT ? p.N - n0 : 16 * OUT);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + batch * p.a_bs + m0 * p.a_rs, (uint32_t)((rows - 1) * p.a_rs + p.K));
  __amdgpu_buffer_rsrc_t rb[GATED ? 2 : 1];
#pragma unroll
  for (int s = 0; s < (GATED ? 2 : 1); ++s)
    rb[s] = make_rsrc(p.b[s] + (batch >> p.b_shift) * p.b_bs[s] + n0 * p.b_rs[s], (uint32_t)((cols - 1) * p.b_rs[s] + p.K));
  const uint32_t kl = 16 * (lane >> 4), K = (uint32_t)p.K;
  const uint32_t off_a = (lane & 15) < rows ? (uint32_t)((lane & 15) * p.a_rs + kl) : kOutOfRange;
  uint32_t off_b[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int32_t r = 16 * (j % OUT) + (lane & 15);
    off_b[j] = r < cols ? (uint32_t)(r * p.b_rs[j / OUT] + kl) : kOutOfRange;
  }
  struct Regs {
    u32x4 a[2], b[FN][2];
  };
  auto load = [&](int32_t t, Regs& x) {
    const uint32_t k = (uint32_t)t * kRowBytes;  // (may pass 2^31, as in RowLoader::issue_one)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = k + 64 * h;
      const bool in = at + kl < K;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        x.b[j][h] = __builtin_amdgcn_raw_buffer_load_b128(rb[j / OUT], in && off_b[j] != kOutOfRange ? off_b[j] + at : kOutOfRange, 0, 0);
      x.a[h] = __builtin_amdgcn_raw_buffer_load_b128(ra, in && off_a != kOutOfRange ? off_a + at : kOutOfRange, 0, 0);
    }
  };
  floatx4 acc[1][FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[0][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int32_t T = p.k_tiles;
  if (wave < T) {
    Regs x[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(wave + d * W, x[d]);
    for (int32_t t = wave; t < T; t += DEPTH * W) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[0][j] = dense_mfma<EK>(x[d].b[j][h], x[d].a[h], acc[0][j]);  // past K: zeros
        load(t + (d + DEPTH) * W, x[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  dense_join<EK, GATED, 1, FN, W, EPI>(p, batch, m0, n0, lane, wave, acc, part);
}

// 17 to 64 rows of A, 16 FM of them: the same with each wave's K-tiles copied
// straight into its own part of LDS, STAGES deep; no barrier until the sums
// meet.  Also for more rows, 16 FM to a workgroup, where 128 x 128 tiles would
// be few.  Gated int8 48 x 8192 x 4096: 15 us, 4.5 TB/s.
template <int EK, bool GATED, int FM, int FN, int STAGES, class EPI, class PRODUCTS>
__global__ __launch_bounds__(kDenseStreamWaves * 64, 1) void dense_stream_kernel(const PRODUCTS products_) {
  uint32_t id, total;
  const DenseParams& p = dense_product(products_, id, total);
  constexpr int W = kDenseStreamWaves;
  constexpr int OUT = GATED ? FN / 2 : FN;
  constexpr int ABYTES = 16 * FM * kRowBytes, STAGE = ABYTES + 16 * FN * kRowBytes;
  __shared__ __attribute__((aligned(1024))) char smem[W * STAGES * STAGE];
  static_assert(W * FM * FN * 1024 <= (int)sizeof smem, "the sums fit");
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tn = id % p.tiles_n, tm = id / p.tiles_n % p.tiles_m, batch = id / p.tiles_n / p.tiles_m;
  const int64_t m0 = tm * (16 * FM), n0 = tn * (16 * OUT);
  const int32_t rows = (int32_t)(p.M - m0 < 16 * FM ? p.M - m0 : 16 * FM);
  const int32_t cols = (int32_t)(p.N - n0 < 16 * OUT ? p.N - n0 : 16 * OUT);
  const auto la = dense_a_loader<16 * FM, 64>(p, batch, m0, rows, 0, lane);
  const auto lb = dense_b_loader<GATED, 16 * FN, 64, GATED ? 16 * OUT : 0>(p, batch, n0, cols, 0, lane);
  constexpr int LOADS = decltype(la)::ITERS + decltype(lb)::ITERS;
  char* ring = smem + wave * (STAGES * STAGE);
  const int32_t T = p.k_tiles;
  auto request = [&](int32_t t, int d) {
    la.issue(t, ring + d * STAGE);  // past the last K-tile: zeros
    lb.issue(t, ring + d * STAGE + ABYTES);
  };
  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (wave < T) {
#pragma unroll
    for (int d = 0; d < STAGES - 1; ++d) request(wave + d * W, d);
    for (int32_t t = wave; t < T; t += STAGES * W) {
#pragma unroll
      for (int d = 0; d < STAGES; ++d) {
        // into the stage of the K-tile before, whose reads are done
        asm volatile("" ::: "memory");
        request(t + (d + STAGES - 1) * W, (d + STAGES - 1) % STAGES);
        wait_vmem_n<(STAGES - 1) * LOADS>();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const char* at = ring + d * STAGE;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          u32x4 fa[FM], fb[FN];
#pragma unroll
          for (int j = 0; j < FN; ++j) fb[j] = dense_frag(at + ABYTES, lane, 16 * j, ks);
#pragma unroll
          for (int i = 0; i < FM; ++i) fa[i] = dense_frag(at, lane, 16 * i, ks);
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = dense_mfma<EK>(fb[j], fa[i], acc[i][j]);  // past K: zeros
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this K-tile's reads
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  wait_vmem();
  __syncthreads();
  dense_join<EK, GATED, FM, FN, W, EPI>(p, batch, m0, n0, lane, wave, acc, (floatx4*)smem);
}

__host__ inline int64_t dense_groups(const DenseParams& p) { return (int64_t)p.batch * p.tiles_m * p.tiles_n; }
__host__ inline int64_t dense_groups(const DensePair& p) { return dense_groups(p.p[0]) + dense_groups(p.p[1]); }

template <int EK, bool GATED, class EPI, class PRODUCTS>
hipError_t dense_launch(const PRODUCTS& p, const DensePlan& plan, hipStream_t s) {
  const dim3 grid((uint32_t)dense_groups(p)), block(plan.threads);
  auto stream = [&](auto fm, auto fn, auto stages) {
    hipLaunchKernelGGL((dense_stream_kernel<EK, GATED, decltype(fm)::value, decltype(fn)::value, decltype(stages)::value, EPI, PRODUCTS>), grid,
                       block, 0, s, p);
  };
  typedef std::integral_constant<int, 2> c2;
  typedef std::integral_constant<int, 3> c3;
  typedef std::integral_constant<int, 4> c4;
  switch (plan.tile) {
    case DT_256x256: hipLaunchKernelGGL((dense_ring_kernel<EK, GATED, 8, 8, 0, EPI, PRODUCTS>), grid, block, 0, s, p); break;
    case DT_256x192:  // no plan of the gated pair or of two products
      if constexpr (GATED || std::is_same<PRODUCTS, DensePair>::value) return hipErrorInvalidValue;
      else hipLaunchKernelGGL((dense_ring_kernel<EK, GATED, 8, 6, 0, EPI, PRODUCTS>), grid, block, 0, s, p);
      break;
    case DT_256x128: hipLaunchKernelGGL((dense_ring_kernel<EK, GATED, 8, 4, 0, EPI, PRODUCTS>), grid, block, 0, s, p); break;
    case DT_128x128:
      if (plan.stages == kDeepRing) hipLaunchKernelGGL((dense_ring_kernel<EK, GATED, 4, 4, (kDeepRing - kRing) / 2, EPI, PRODUCTS>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((dense_ring_kernel<EK, GATED, 4, 4, 0, EPI, PRODUCTS>), grid, block, 0, s, p);
      break;
    case DT_STREAM:
      if (plan.bm == 64) plan.bn == 32 ? stream(c4{}, c2{}, c3{}) : stream(c4{}, c4{}, c2{});
      else if (plan.bn == 32) stream(c2{}, c2{}, c4{});
      else if constexpr (std::is_same<PRODUCTS, DensePair>::value) return hipErrorInvalidValue;  // no plan of two products
      else stream(c2{}, c4{}, c3{});
      break;
    case DT_SKINNY:
      if constexpr (std::is_same<PRODUCTS, DensePair>::value) return hipErrorInvalidValue;  // no plan of two products
      else if (plan.bn == 32) hipLaunchKernelGGL((dense_skinny_kernel<EK, GATED, 2, EPI, PRODUCTS>), grid, block, 0, s, p);
      else if constexpr (GATED) return hipErrorInvalidValue;
      else hipLaunchKernelGGL((dense_skinny_kernel<EK, GATED, 1, EPI, PRODUCTS>), grid, block, 0, s, p);
      break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace sl
