// gemm_block.hip -- the block-scaled product on E4M3 codes with fp32 scales
// per 128 K:
//   D[m,n] = C[m,n] + sum_j SA[m,j] SB[n,j] sum_{k in block j} A[m,k] B[n,k]
// where a scale row covers one row of its operand or 128 of them.
//
// The matrix core sums one K block of 128 on a zero accumulator; its result,
// times the block's scale, is added to the running fp32 sum by the vector
// unit (the hardware's own scale operands are powers of two and cannot hold
// these).  A lane of the 16 x 16 result holds four consecutive n of one m, so
// with SB constant over 128 rows of B that is one multiply-add per value on
// top of one scale product per 16 rows of A.
//
// 16-bit results: one 128-wide step of the 8-bit instruction per K block.  It
// aligns a block's products to the largest and drops bits below about 2^-16
// of it (measured on normally distributed codes: 1.5e-5 of the result, every
// 8-bit instruction alike), a tenth of fp16's rounding.  fp32 results would
// show that, so for them the codes become fp16 in registers (exact) and four
// steps of the fp16 instruction, at half the rate, sum the block (measured
// 1e-8 of the result).
#include <type_traits>

#include "sl_ops.hpp"

#include "sl_device.hpp"

namespace sl {
namespace {

constexpr int32_t kE4M3 = 0;  // CBSZ / BLGP format code

// A lane's 32 codes of one K block, as the instruction takes them.
struct FragF8 {
  i32x8 v;
  __device__ __forceinline__ FragF8() {}
  __device__ __forceinline__ FragF8(const u32x4& lo, const u32x4& hi)
      : v{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]} {}
};
struct FragF16 {
  half8 v[4];
  __device__ __forceinline__ FragF16() {}
  __device__ __forceinline__ FragF16(const u32x4& lo, const u32x4& hi) {
    typedef _Float16 half2v __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w0 = q < 2 ? lo[2 * q] : hi[2 * q - 4], w1 = q < 2 ? lo[2 * q + 1] : hi[2 * q - 3];
      const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false);
      const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true);
      const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false);
      const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true);
      v[q] = half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
  }
};
template <int OT>
struct FragOf {
  typedef FragF8 type;
};
template <>
struct FragOf<OT_F32> {
  typedef FragF16 type;
};

__device__ __forceinline__ floatx4 mfma_block(const FragF8& a, const FragF8& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, floatx4{0.f, 0.f, 0.f, 0.f}, kE4M3, kE4M3, 0, 0, 0, 0);
}
// the order of K inside a block is free as long as both operands share it
__device__ __forceinline__ floatx4 mfma_block(const FragF16& a, const FragF16& b) {
  floatx4 t = mfma16<DT_F16>(a.v[0], b.v[0], floatx4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
  for (int q = 1; q < 4; ++q) t = mfma16<DT_F16>(a.v[q], b.v[q], t);
  return t;
}

template <int OT>
__device__ __forceinline__ float block_load(const void* p, int64_t off) {
  if constexpr (OT == OT_F32)
    return ((const float*)p)[off];
  else
    return to_f32<OT == OT_F16 ? DT_F16 : DT_BF16>(((const uint16_t*)p)[off]);
}
template <int OT>
__device__ __forceinline__ void block_store(void* p, int64_t off, float v) {
  if constexpr (OT == OT_F32)
    ((float*)p)[off] = v;
  else
    ((uint16_t*)p)[off] = from_f32<OT == OT_F16 ? DT_F16 : DT_BF16>(v);
}

// D(m, n .. n + 3) = v + C, where in range
template <int OT>
__device__ __forceinline__ void block_store_quad(const BlockGemmParams& p, int64_t batch, int64_t m, int64_t n, floatx4 v) {
  if (m >= p.M || n >= p.N) return;
  const bool whole = n + 4 <= p.N;
  if (p.flags & BF_HAS_C) {
    const int64_t off = batch * p.c_bs + m * p.c_rs + n * p.c_cs;
    if (whole && (p.flags & BF_C_VEC)) {
      if constexpr (OT == OT_F32) {
        const floatx4 c = *(const floatx4*)((const float*)p.c + off);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += c[r];
      } else {
        const u16x4 c = *(const u16x4*)((const uint16_t*)p.c + off);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += to_f32<OT == OT_F16 ? DT_F16 : DT_BF16>(c[r]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < p.N) v[r] += block_load<OT>(p.c, off + r * p.c_cs);
    }
  }
  const int64_t off = batch * p.d_bs + m * p.d_rs + n * p.d_cs;
  if (whole && (p.flags & BF_D_VEC)) {
    if constexpr (OT == OT_F32) {
      *(floatx4*)((float*)p.d + off) = v;
    } else {
      constexpr int DT = OT == OT_F16 ? DT_F16 : DT_BF16;
      *(u16x4*)((uint16_t*)p.d + off) = u16x4{from_f32<DT>(v[0]), from_f32<DT>(v[1]), from_f32<DT>(v[2]), from_f32<DT>(v[3])};
    }
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < p.N) block_store<OT>(p.d, off + r * p.d_cs, v[r]);
  }
}

// A lane holds the scale of one row of its wave's A or B (of the operand's
// last row, past it: those results are not stored); the lanes that need it
// take it from there.
__device__ __forceinline__ const float* row_scale(const float* base, int64_t row, int64_t rows, int32_t shift, int64_t rs) {
  return base + ((row < rows ? row : rows - 1) >> shift) * rs;
}
__device__ __forceinline__ float from_lane(float v, int32_t l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(4 * l, __builtin_bit_cast(int32_t, v)));
}

// how a tile reads SB: one scale for the wave's columns (128 x 128 blocks), or
// one per row of B
constexpr int SB_SQUARE = 0, SB_ROWS = 1;

// BM x BN output tiles, the K-tiles of 128 bytes per row brought straight
// into LDS, STAGES deep: two, and two workgroups to a CU, or, where there is
// not more than one for each, four.  Measured: 4096 x 4096 x 8192 + C into
// fp32 300 us a pass (916 TFLOP/s; 360 vector instructions a K-tile beside 64
// MFMAs; MFMA busy 40%), 1024 x 2048 x 4096 into bf16 30 us.
template <int BM, int BN, int WM, int WN, int STAGES, int SBK, int OT>
__global__ __launch_bounds__(WM* WN * 64, STAGES == 2 ? 2 : 1) void gemm_block_kernel(const BlockGemmParams p) {
  typedef typename FragOf<OT>::type Frag;
  constexpr int NT = WM * WN * 64;
  constexpr int TM = BM / WM, TN = BN / WN;
  constexpr int FM = TM / 16, FN = TN / 16;
  static_assert(128 % TN == 0, "a wave's columns lie in one square block");
  constexpr int ABYTES = BM * kRowBytes, BBYTES = BN * kRowBytes;
  constexpr int STAGE = ABYTES + BBYTES;
  __shared__ __attribute__((aligned(1024))) char smem[STAGES * STAGE];

  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t wm = wave % WM, wn = wave / WM;
  const TileCoord tc = map_tile(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, p.batch);
  const int64_t m0 = (int64_t)tc.tm * BM, n0 = (int64_t)tc.tn * BN;
  const int32_t rows_a = (int32_t)(p.M - m0 < BM ? p.M - m0 : BM);
  const int32_t rows_b = (int32_t)(p.N - n0 < BN ? p.N - n0 : BN);
  LoaderKVec<BM, NT, 0, 1> la(p.a + tc.batch * p.a_bs + m0 * p.a_rs, rows_a, p.a_rs, 1, p.K, wave, lane);
  LoaderKVec<BN, NT, 0, 1> lb(p.b + tc.batch * p.b_bs + n0 * p.b_rs, rows_b, p.b_rs, 1, p.K, wave, lane);
  const int32_t a_row0 = wm * TM, b_row0 = wn * TN;

  static_assert(TM == 64 && TN == 64, "a lane holds one row's scale");
  const float* sa_p = row_scale(p.sa + tc.batch * p.sa_bs, m0 + a_row0 + lane, p.M, p.a_shift, p.sa_rs);
  const float* sb_p = row_scale(p.sb + tc.batch * p.sb_bs, n0 + b_row0 + lane, p.N, p.b_shift, p.sb_rs);

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  const int32_t T = p.k_blocks;
  // Copies of a request.  Its two scale loads are not counted on: the compiler
  // may move them among the copies, and a count that holds in any order leaves
  // no more operations in flight than there are copies behind the K-tile.
  constexpr int LOADS = decltype(la)::ITERS + decltype(lb)::ITERS;
  float sa_own[STAGES], sb_own[STAGES];
  auto request = [&](int32_t t, int d) {
    const int64_t at = t < T ? t : T - 1;
    sa_own[d] = sa_p[at * p.sa_ks], sb_own[d] = sb_p[at * p.sb_ks];
    la.issue(t, smem + d * STAGE);  // past the last K-tile: zeros, not read
    lb.issue(t, smem + d * STAGE + ABYTES);
  };
  auto multiply = [&](int d) {
    const char* cur = smem + d * STAGE;
    auto read = [&](const char* at, int32_t row0) {
      return Frag(*(const u32x4*)(at + fragment_lds_offset(MFMA16_F8, lane, 0, row0, 0, 0)),
                  *(const u32x4*)(at + fragment_lds_offset(MFMA16_F8, lane, 1, row0, 0, 0)));
    };
    Frag bf[FN], af[2];
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = read(cur + ABYTES, b_row0 + 16 * j);
    af[0] = read(cur, a_row0);
    float sav[FM], sb[SBK == SB_ROWS ? FN : 1][4];
#pragma unroll
    for (int i = 0; i < FM; ++i) sav[i] = from_lane(sa_own[d], 16 * i + (lane & 15));
    if constexpr (SBK == SB_ROWS) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) sb[j][r] = from_lane(sb_own[d], 16 * j + 4 * (lane >> 4) + r);
    } else {
      sb[0][0] = sb_own[d];  // the wave's columns lie in one block
    }
    // product e of the wave's 16, its sums scaled and added LAG products later
    constexpr int LAG = OT == OT_F32 ? 1 : 3;
    floatx4 sums[LAG + 1];
    float sai = 0.f;
#pragma unroll
    for (int e = 0; e < FM * FN + LAG; ++e) {
      const int i = e / FN, j = e % FN;
      if (e < FM * FN) {
        if (j == 0 && i + 1 < FM) af[(i + 1) & 1] = read(cur, a_row0 + 16 * (i + 1));
        sums[e % (LAG + 1)] = mfma_block(bf[j], af[i & 1]);
      }
      if (e >= LAG) {
        const int u = (e - LAG) / FN, w = (e - LAG) % FN;
        if (w == 0) sai = SBK == SB_ROWS ? sav[u] : sav[u] * sb[0][0];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s = SBK == SB_ROWS ? sai * sb[SBK == SB_ROWS ? w : 0][SBK == SB_ROWS ? r : 0] : sai;
          acc[u][w][r] = __builtin_fmaf(sums[(e - LAG) % (LAG + 1)][r], s, acc[u][w][r]);
        }
      }
      // left to itself, the compiler moved each read next to its use (1024 x
      // 2048 x 4096: 39 us; 30 in this order.  With fp16 fragments its own
      // order is 4% faster)
      if constexpr (OT != OT_F32) __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (T > 0) {
#pragma unroll
    for (int d = 0; d < STAGES - 1; ++d) request(d, d);
    for (int32_t t = 0; t < T; t += STAGES) {
#pragma unroll
      for (int d = 0; d < STAGES; ++d) {
        wait_vmem_n<(STAGES - 2) * LOADS>();  // K-tile t + d has landed
        phase_barrier();                      // for every wave, and the one before is no longer read
        request(t + d + STAGES - 1, (d + STAGES - 1) % STAGES);
        if (t + d < T) multiply(d);
      }
    }
    wait_vmem();
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      block_store_quad<OT>(p, tc.batch, m0 + a_row0 + 16 * i + (lane & 15), n0 + b_row0 + 16 * j + 4 * (lane >> 4), acc[i][j]);
}

// 256 x 256 tiles for 16-bit results: 8 waves, two per SIMD, each 128 x 64,
// and five slots for operand K-tiles (32 KiB each) in LDS: A and B of K-tiles
// t and t + 1, and a free one.  One barrier, in the middle of K-tile t: K-tile
// t + 1 has landed then, so the first fragments of t + 1 are read while t's
// last products run, and the copies of t + 2 (A into the free slot, B into
// B(t)'s, which is in registers) have a whole K-tile to land.  A block's sums
// are scaled and added while the next ones run in the matrix core.  Measured:
// 8192^3, bf16 D, square blocks of B: 520 to 535 us a pass, 2.05 to 2.12 PFLOP/s
// (MXFP8: 403); MFMA busy 45%, 5.9 vector instructions beside each.
template <int SBK, int OT>
__global__ __launch_bounds__(512, 2) void gemm_block_ring_kernel(const BlockGemmParams p) {
  typedef FragF8 Frag;
  constexpr int FM = 8, FN = 4, SLOT = 256 * kRowBytes;
  __shared__ __attribute__((aligned(1024))) char smem[5 * SLOT];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TileCoord tc = map_tile(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, p.batch);
  const int64_t m0 = (int64_t)tc.tm * 256, n0 = (int64_t)tc.tn * 256;
  const int32_t rows_a = (int32_t)(p.M - m0 < 256 ? p.M - m0 : 256);
  const int32_t rows_b = (int32_t)(p.N - n0 < 256 ? p.N - n0 : 256);
  const LoaderKVec<256, 512, 0, 1> la(p.a + tc.batch * p.a_bs + m0 * p.a_rs, rows_a, p.a_rs, 1, p.K, wave, lane);
  const LoaderKVec<256, 512, 0, 1> lb(p.b + tc.batch * p.b_bs + n0 * p.b_rs, rows_b, p.b_rs, 1, p.K, wave, lane);
  constexpr int LOADS = decltype(la)::ITERS;
  const int32_t a_row0 = wave % 2 * 128, b_row0 = wave / 2 * 64;

  // A lane holds the scales of rows lane and lane + 64 of the wave's A and of
  // row lane of its B.
  const float* sa_base = p.sa + tc.batch * p.sa_bs;
  const float* sa0 = row_scale(sa_base, m0 + a_row0 + lane, p.M, p.a_shift, p.sa_rs);
  const float* sa1 = row_scale(sa_base, m0 + a_row0 + 64 + lane, p.M, p.a_shift, p.sa_rs);
  const float* sb0 = row_scale(p.sb + tc.batch * p.sb_bs, n0 + b_row0 + (SBK == SB_ROWS ? lane : 0), p.N, p.b_shift, p.sb_rs);
  struct Scales {
    float a[2], b;
  };
  const int32_t T = p.k_blocks;
  auto load_scales = [&](Scales& s, bool more) {
    s.a[0] = *sa0, s.a[1] = *sa1, s.b = *sb0;
    if (more) sa0 += p.sa_ks, sa1 += p.sa_ks, sb0 += p.sb_ks;
  };

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (T > 0) {
    auto read = [&](int32_t slot, int32_t row0) {
      const char* at = smem + slot * SLOT;
      return Frag(*(const u32x4*)(at + fragment_lds_offset(MFMA16_F8, lane, 0, row0, 0, 0)),
                  *(const u32x4*)(at + fragment_lds_offset(MFMA16_F8, lane, 1, row0, 0, 0)));
    };
    Scales cur, nxt;
    load_scales(cur, T > 1);
    la.issue(0, smem);
    lb.issue(0, smem + SLOT);
    la.issue(1, smem + 2 * SLOT);
    lb.issue(1, smem + 3 * SLOT);
    wait_vmem_n<2 * LOADS>();
    phase_barrier();
    // slots of A(t), B(t), A(t + 1), B(t + 1), and the free one
    int32_t sa = 0, sb = 1, na = 2, nb = 3, fr = 4;
    Frag bf[FN], af[2];
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = read(sb, b_row0 + 16 * j);
    af[0] = read(sa, a_row0);
    for (int32_t t = 0; t < T; ++t) {
      float sbv[SBK == SB_ROWS ? FN * 4 : 1];
      if constexpr (SBK == SB_ROWS) {
#pragma unroll
        for (int j = 0; j < FN * 4; ++j) sbv[j] = from_lane(cur.b, 16 * (j / 4) + 4 * (lane >> 4) + j % 4);
      } else {
        sbv[0] = cur.b;
      }
      auto a_scale = [&](int i) { return from_lane(cur.a[i / 4], 16 * (i % 4) + (lane & 15)); };
      float sav[3], sai = 0.f;
      sav[0] = a_scale(0);
      // product e of the wave's 32, its sums added LAG products later
      constexpr int LAG = 3;
      floatx4 sums[LAG + 1];
#pragma unroll
      for (int e = 0; e < FM * FN + LAG; ++e) {
        const int i = e / FN, j = e % FN;
        if (e == FM * FN / 2) {
          // K-tile t + 1 has landed, for every wave, and B(t), read whole,
          // is free.  LDS reads may be in flight: those of A(t), which is
          // not, and the compiler waits for them where they are used.
          __builtin_amdgcn_sched_barrier(0);
          wait_vmem();
          asm volatile("s_barrier" ::: "memory");
          load_scales(nxt, t + 2 < T);
          la.issue(t + 2, smem + fr * SLOT);
          lb.issue(t + 2, smem + sb * SLOT);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (e < FM * FN) {
          if (j == 0) {
            af[(i + 1) & 1] = i + 1 < FM ? read(sa, a_row0 + 16 * (i + 1)) : read(na, a_row0);
            if (i + 1 < FM) sav[(i + 1) % 3] = a_scale(i + 1);
          }
          sums[e % (LAG + 1)] = mfma_block(bf[j], af[i & 1]);
          if (i + 1 == FM) bf[j] = read(nb, b_row0 + 16 * j);
        }
        if (e >= LAG) {
          const int u = (e - LAG) / FN, w = (e - LAG) % FN;
          if (w == 0) sai = SBK == SB_ROWS ? sav[u % 3] : sav[u % 3] * sbv[0];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float s = SBK == SB_ROWS ? sai * sbv[SBK == SB_ROWS ? 4 * w + r : 0] : sai;
            acc[u][w][r] = __builtin_fmaf(sums[(e - LAG) % (LAG + 1)][r], s, acc[u][w][r]);
          }
        }
        // left to itself, the compiler moved each read next to its use
        __builtin_amdgcn_sched_barrier(0);
      }
      cur = nxt;
      const int32_t was_a = sa, was_b = sb;
      sa = na, sb = nb, na = fr, nb = was_b, fr = was_a;
    }
    wait_vmem();
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      block_store_quad<OT>(p, tc.batch, m0 + a_row0 + 16 * i + (lane & 15), n0 + b_row0 + 16 * j + 4 * (lane >> 4), acc[i][j]);
}

// Up to 16 rows of A: the weight B is read once and bounds the call.  A
// workgroup of 8 waves owns 16 FN rows of B; wave w takes the
// K blocks w, w + 8, ... straight from memory into registers (four lanes read
// 64 consecutive bytes of a row; the order of K inside a block is free as
// long as A and B share it), and the waves' sums meet in LDS.
template <int FN, int SBK, int OT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void gemm_block_skinny_kernel(const BlockGemmParams p) {
  constexpr int FM = 1;
  __shared__ __attribute__((aligned(16))) float part[kSkinnyWaves - 1][FM * FN][64][4];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t id = blockIdx.x;
  const int32_t tn = id % p.tiles_n, tm = id / p.tiles_n % p.tiles_m;
  const int64_t batch = id / p.tiles_n / p.tiles_m;
  const int64_t m0 = (int64_t)tm * kSkinnyRows, n0 = (int64_t)tn * (16 * FN);
  const int32_t rows_a = (int32_t)(p.M - m0 < 16 * FM ? p.M - m0 : 16 * FM);
  const int32_t rows_b = (int32_t)(p.N - n0 < 16 * FN ? p.N - n0 : 16 * FN);
  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(p.a + batch * p.a_bs + m0 * p.a_rs, (uint32_t)((rows_a - 1) * p.a_rs + p.K));
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(p.b + batch * p.b_bs + n0 * p.b_rs, (uint32_t)((rows_b - 1) * p.b_rs + p.K));
  const int32_t kl = 16 * (lane >> 4);
  uint32_t off_a[FM], off_b[FN];
  const float* sa_p[FM];
  constexpr int NSB = SBK == SB_ROWS ? FN : 0;  // square blocks: one scale for the workgroup's columns
  int64_t sb_off[SBK == SB_ROWS ? FN : 1][4];
  sb_off[0][0] = (n0 >> p.b_shift) * p.sb_rs;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int32_t r = 16 * i + (lane & 15);
    off_a[i] = r < rows_a ? (uint32_t)(r * p.a_rs + kl) : kOutOfRange;
    const int64_t m = m0 + (r < rows_a ? r : rows_a - 1);
    sa_p[i] = p.sa + batch * p.sa_bs + (m >> p.a_shift) * p.sa_rs;
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int32_t r = 16 * j + (lane & 15);
    off_b[j] = r < rows_b ? (uint32_t)(r * p.b_rs + kl) : kOutOfRange;
#pragma unroll
    for (int e = 0; e < (SBK == SB_ROWS ? 4 : 0); ++e) {
      const int32_t n = 16 * j + 4 * (lane >> 4) + e;
      sb_off[j][e] = ((n0 + (n < rows_b ? n : rows_b - 1)) >> p.b_shift) * p.sb_rs;
    }
  }
  const float* sb_base = p.sb + batch * p.sb_bs;

  struct Regs {
    u32x4 a[FM][2], b[FN][2];
    float sa[FM], sb[SBK == SB_ROWS ? FN : 1][4];
  };
  const int32_t T = p.k_blocks;
  auto load = [&](int32_t t, Regs& x) {
    const int32_t k = t * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = t < T && k + kl + 64 * h < p.K;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        x.b[j][h] = __builtin_amdgcn_raw_buffer_load_b128(
            rb, in && off_b[j] != kOutOfRange ? off_b[j] + (uint32_t)(k + 64 * h) : kOutOfRange, 0, 0);
#pragma unroll
      for (int i = 0; i < FM; ++i)
        x.a[i][h] = __builtin_amdgcn_raw_buffer_load_b128(
            ra, in && off_a[i] != kOutOfRange ? off_a[i] + (uint32_t)(k + 64 * h) : kOutOfRange, 0, 0);
    }
    const int64_t ts = t < T ? t : T - 1;
#pragma unroll
    for (int i = 0; i < FM; ++i) x.sa[i] = t < T ? sa_p[i][ts * p.sa_ks] : 0.f;  // past the last block: adds 0
    if constexpr (SBK == SB_SQUARE) x.sb[0][0] = t < T ? sb_base[sb_off[0][0] + ts * p.sb_ks] : 0.f;
#pragma unroll
    for (int j = 0; j < NSB; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x.sb[j][e] = t < T ? sb_base[sb_off[j][e] + ts * p.sb_ks] : 0.f;
  };
  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](const Regs& x) {
    typedef typename FragOf<OT>::type Frag;
    Frag bf[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = Frag(x.b[j][0], x.b[j][1]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const Frag af(x.a[i][0], x.a[i][1]);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const floatx4 t4 = mfma_block(bf[j], af);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(t4[e], x.sa[i] * x.sb[SBK == SB_ROWS ? j : 0][SBK == SB_ROWS ? e : 0], acc[i][j][e]);
      }
    }
  };
  // DEPTH blocks requested ahead: a wave has few of them (8 at K = 8192), and
  // two ahead left the call waiting for memory
  constexpr int DEPTH = 4;
  if (wave < T) {
    Regs x[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(wave + d * kSkinnyWaves, x[d]);
    for (int32_t t = wave; t < T; t += DEPTH * kSkinnyWaves) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        step(x[d]);
        load(t + (d + DEPTH) * kSkinnyWaves, x[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) *(floatx4*)part[wave - 1][i * FN + j][lane] = acc[i][j];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      floatx4 v = acc[i][j];
      for (int w = 0; w < kSkinnyWaves - 1; ++w) {
        const floatx4 o = *(const floatx4*)part[w][i * FN + j][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += o[e];
      }
      block_store_quad<OT>(p, batch, m0 + 16 * i + (lane & 15), n0 + 16 * j + 4 * (lane >> 4), v);
    }
}

// 17 to 64 rows of A: the same with the K blocks of a wave copied straight
// into its own part of LDS, STAGES deep (in registers two blocks filled the
// file: 48 x 8192 x 8192 took 26 us, here 23, 2.9 TB/s).  Four waves split K;
// no barrier until their sums meet.  Also for more rows, 64 to a workgroup,
// where 128 x 128 tiles would be few.
template <int FM, int FN, int SBK, int OT>
__global__ __launch_bounds__(kStreamWaves * 64, 1) void gemm_block_stream_kernel(const BlockGemmParams p) {
  typedef typename FragOf<OT>::type Frag;
  constexpr int STAGES = FM == 4 ? 3 : 4;
  constexpr int ABYTES = 16 * FM * kRowBytes, STAGE = ABYTES + 16 * FN * kRowBytes;
  __shared__ __attribute__((aligned(1024))) char smem[kStreamWaves * STAGES * STAGE];
  static_assert((kStreamWaves - 1) * FM * FN * 1024 <= (int)sizeof smem, "the sums fit");
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t id = blockIdx.x;
  const int32_t tn = id % p.tiles_n, tm = id / p.tiles_n % p.tiles_m;
  const int64_t batch = id / p.tiles_n / p.tiles_m;
  const int64_t m0 = (int64_t)tm * kSkinnyRows, n0 = (int64_t)tn * (16 * FN);
  const int32_t rows_a = (int32_t)(p.M - m0 < 16 * FM ? p.M - m0 : 16 * FM);
  const int32_t rows_b = (int32_t)(p.N - n0 < 16 * FN ? p.N - n0 : 16 * FN);
  const LoaderKVec<16 * FM, 64, 0, 1> la(p.a + batch * p.a_bs + m0 * p.a_rs, rows_a, p.a_rs, 1, p.K, 0, lane);
  const LoaderKVec<16 * FN, 64, 0, 1> lb(p.b + batch * p.b_bs + n0 * p.b_rs, rows_b, p.b_rs, 1, p.K, 0, lane);
  constexpr int LOADS = decltype(la)::ITERS + decltype(lb)::ITERS;  // copies of a request: as in gemm_block_kernel
  const float* sa_p = row_scale(p.sa + batch * p.sa_bs, m0 + lane, p.M, p.a_shift, p.sa_rs);
  const float* sb_p = row_scale(p.sb + batch * p.sb_bs, n0 + (lane & (16 * FN - 1)), p.N, p.b_shift, p.sb_rs);
  char* ring = smem + wave * (STAGES * STAGE);
  const int32_t T = p.k_blocks;
  float sa[STAGES], sb[STAGES];  // of the rows `lane` of A and B
  auto request = [&](int32_t t, int d) {
    const int64_t at = t < T ? t : T - 1;
    sa[d] = sa_p[at * p.sa_ks];
    sb[d] = sb_p[at * p.sb_ks];
    la.issue(t, ring + d * STAGE);  // past the last block: zeros
    lb.issue(t, ring + d * STAGE + ABYTES);
  };
  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](int32_t t, int d) {
    const char* at = ring + d * STAGE;
    auto read = [&](const char* x, int32_t row0) {
      return Frag(*(const u32x4*)(x + fragment_lds_offset(MFMA16_F8, lane, 0, row0, 0, 0)),
                  *(const u32x4*)(x + fragment_lds_offset(MFMA16_F8, lane, 1, row0, 0, 0)));
    };
    Frag bf[FN];
    float sbv[FN][4];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      bf[j] = read(at + ABYTES, 16 * j);
#pragma unroll
      for (int r = 0; r < 4; ++r) sbv[j][r] = SBK == SB_ROWS ? from_lane(sb[d], 16 * j + 4 * (lane >> 4) + r) : sb[d];
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const Frag af = read(at, 16 * i);
      const float sai = from_lane(sa[d], 16 * i + (lane & 15));
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const floatx4 t4 = mfma_block(bf[j], af);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(t4[r], sai * sbv[j][r], acc[i][j][r]);
      }
    }
  };
  if (wave < T) {
#pragma unroll
    for (int d = 0; d < STAGES - 1; ++d) request(wave + d * kStreamWaves, d);
    for (int32_t t = wave; t < T; t += STAGES * kStreamWaves) {
#pragma unroll
      for (int d = 0; d < STAGES; ++d) {
        // into the stage of the block before, whose reads are done
        asm volatile("" ::: "memory");
        request(t + (d + STAGES - 1) * kStreamWaves, (d + STAGES - 1) % STAGES);
        wait_vmem_n<(STAGES - 1) * LOADS>();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (t + d * kStreamWaves < T) step(t + d * kStreamWaves, d);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this block's reads
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  wait_vmem();
  __syncthreads();
  floatx4* part = (floatx4*)smem;  // [wave - 1][tile][lane]
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) part[((wave - 1) * FM * FN + i * FN + j) * 64 + lane] = acc[i][j];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      floatx4 v = acc[i][j];
#pragma unroll
      for (int w = 0; w < kStreamWaves - 1; ++w) {
        const floatx4 o = part[(w * FM * FN + i * FN + j) * 64 + lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += o[r];
      }
      block_store_quad<OT>(p, batch, m0 + 16 * i + (lane & 15), n0 + 16 * j + 4 * (lane >> 4), v);
    }
}

template <int OT>
hipError_t go(const BlockGemmParams& p, int32_t tile, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.batch * p.tiles_m * p.tiles_n));
  const bool square = p.b_shift != 0;
  if (tile == BT_256x256 && OT != OT_F32) {
    constexpr int OT2 = OT == OT_F32 ? OT_F16 : OT;  // fp32 results have no such tile
    if (square) hipLaunchKernelGGL((gemm_block_ring_kernel<SB_SQUARE, OT2>), grid, dim3(512), 0, s, p);
    else hipLaunchKernelGGL((gemm_block_ring_kernel<SB_ROWS, OT2>), grid, dim3(512), 0, s, p);
  } else if (tile == BT_128x128 && grid.x > 256) {
    if (square) hipLaunchKernelGGL((gemm_block_kernel<128, 128, 2, 2, 2, SB_SQUARE, OT>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((gemm_block_kernel<128, 128, 2, 2, 2, SB_ROWS, OT>), grid, dim3(256), 0, s, p);
  } else if (tile == BT_128x128) {
    if (square) hipLaunchKernelGGL((gemm_block_kernel<128, 128, 2, 2, 4, SB_SQUARE, OT>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((gemm_block_kernel<128, 128, 2, 2, 4, SB_ROWS, OT>), grid, dim3(256), 0, s, p);
  } else if (tile == BT_SKINNY) {
    const bool wide = skinny_cols(p.M, p.N, p.batch) == 32;
    auto skinny = [&](auto fm_c, auto fn_c, auto sb_c) {
      constexpr int FM = decltype(fm_c)::value, FN = decltype(fn_c)::value, SBK = decltype(sb_c)::value;
      if constexpr (FM == 1)
        hipLaunchKernelGGL((gemm_block_skinny_kernel<FN, SBK, OT>), grid, dim3(kSkinnyWaves * 64), 0, s, p);
      else
        hipLaunchKernelGGL((gemm_block_stream_kernel<FM, FN, SBK, OT>), grid, dim3(kStreamWaves * 64), 0, s, p);
    };
    auto by_cols = [&](auto fm_c, auto sb_c) {
      wide ? skinny(fm_c, std::integral_constant<int, 2>{}, sb_c) : skinny(fm_c, std::integral_constant<int, 1>{}, sb_c);
    };
    auto by_rows = [&](auto sb_c) {
      if (p.M <= 16) by_cols(std::integral_constant<int, 1>{}, sb_c);
      else if (p.M <= 32) by_cols(std::integral_constant<int, 2>{}, sb_c);
      else by_cols(std::integral_constant<int, 4>{}, sb_c);
    };
    square ? by_rows(std::integral_constant<int, SB_SQUARE>{}) : by_rows(std::integral_constant<int, SB_ROWS>{});
  } else {
    return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_block(const BlockGemmParams& p, int32_t tile, hipStream_t s) {
  switch (p.type) {
    case OT_F16: return go<OT_F16>(p, tile, s);
    case OT_BF16: return go<OT_BF16>(p, tile, s);
    case OT_F32: return go<OT_F32>(p, tile, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sl
