// gated_backward.hip -- the matrix products of the gated feed-forward block's
// backward pass:
//   dx = [dg | du] [Wg ; Wu],   dWg = dg^T x,   dWu = du^T x
// the weights' gradients as one product of a batch of pairs.  Two ways:
//
// grad_ring_kernel and grad_tile read x, the weights and, for the weights' gradients, dg
// and du as they lie, the contracted axis across the rows, through transposing LDS
// reads.  The dense kernels read along the contracted axis, from transposes that
// gated_prepare.hip makes first: for few rows, and where a transpose costs less than
// it gains.
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
  template <int RPI, int V, class GET>
  __device__ __forceinline__ void rows(const DenseParams& p, int64_t batch, int64_t m, int64_t n, int32_t count, const GET& get) const {
    uint16_t* d = (uint16_t*)p.kept[s] + (batch >> p.b_shift) * p.kept_bs[s] + m * p.kept_rs[s] + n;
#pragma unroll 4
    for (int it = 0; it < count; ++it) {
      float v[V];
      get(it, 0, v);
      dense_store_cols<OT, V>(d, v);
      d += RPI * p.kept_rs[s];
    }
  }
};

// A K-tile of an operand whose rows are contracted over: 64 rows of W of its
// columns into the M-major LDS tile (mn_lds_offset), copy j of a wave 512 / W rows.
template <int W>
struct AcrossLoader {
  static constexpr int CPR = W / 8, RPC = 64 / CPR, ITERS = 16 / RPC;  // 16-byte chunks of a row, rows of a copy, copies
  int32_t wave, lane, cols;
  uint32_t step;         // bytes between rows
  uint32_t voff[ITERS];  // the lane's offset in copy j of a K-tile
  // `cols` valid columns, a multiple of 8, of rows `step_` bytes apart
  __device__ __forceinline__ AcrossLoader(int32_t cols_, int64_t step_, int32_t wave_, int32_t lane_)
      : wave(wave_), lane(lane_), cols(cols_), step((uint32_t)step_) {
    rows(64);
  }
  // of the K-tiles copied from here on `valid` rows are there (others read zero)
  __device__ __forceinline__ void rows(int32_t valid) {
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
      const int32_t k = RPC * (4 * j + wave) + lane / CPR, c = lane % CPR ^ mn_swz(k);
      voff[j] = k < valid && 8 * c < cols ? (uint32_t)k * step + (uint32_t)(16 * c) : kOutOfRange;
    }
  }
};

// A copy's operands as inline assembly takes them.
__device__ __forceinline__ u32x4 rsrc_words(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b), (uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32) & 0xFFFF),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), (uint32_t)kRsrcWord3};
}

// 32 products (four rows of a wave's block), beside the first of them NF
// fragments read by transposing reads, with the wait for these in the same
// statement, and beside the others NC copies into LDS, 4096 apart from `to` on, which
// return nothing and are waited for by count.  As builtins the reads would
// each get a wait for every copy in flight in front (the GEMM's ring kernel, built
// that way, took 424 us at 4096 x 4096 x 8192 where its 8-wave kernel takes
// 222), and copies between the statements leave the matrix core without work (4096 x
// 4096 x 16384 in 410 us, so 386).  A fragment is two reads of 8 bytes a lane,
// 2048 apart: k0 and k1 are their offsets.
#define SL_READ(n) "ds_read_b64_tr_b16 %[l" #n "], %[t" #n "] offset:%[k0]\n\tds_read_b64_tr_b16 %[h" #n "], %[t" #n "] offset:%[k1]\n\t"
#define SL_TO(n) "s_add_i32 m0, %[m], " #n " * 4096\n\t"
#define SL_COPY(n) "buffer_load_dwordx4 %[v" #n "], %[rs], %[so] offen lds\n\t"
#define SL_MFMA(op, c, b, a) op " %[c" #c "], %[b" #b "], %[a" #a "], %[c" #c "]\n\t"
#define SL_PRODUCTS(op, r0, r1, r2, r3, r4, r5, r6, r7, c8, c9, c10, c11, c12, c13, c14, c15, c16, c17, c18, c19, c20, c21, c22, c23) \
  r0 SL_MFMA(op, 0, 0, 0) r1 SL_MFMA(op, 1, 1, 0) r2 SL_MFMA(op, 2, 2, 0) r3 SL_MFMA(op, 3, 3, 0)                              \
  r4 SL_MFMA(op, 4, 4, 0) r5 SL_MFMA(op, 5, 5, 0) r6 SL_MFMA(op, 6, 6, 0) r7 SL_MFMA(op, 7, 7, 0)                              \
  c8 SL_MFMA(op, 8, 0, 1) c9 SL_MFMA(op, 9, 1, 1) c10 SL_MFMA(op, 10, 2, 1) c11 SL_MFMA(op, 11, 3, 1)                          \
  c12 SL_MFMA(op, 12, 4, 1) c13 SL_MFMA(op, 13, 5, 1) c14 SL_MFMA(op, 14, 6, 1) c15 SL_MFMA(op, 15, 7, 1)                      \
  c16 SL_MFMA(op, 16, 0, 2) c17 SL_MFMA(op, 17, 1, 2) c18 SL_MFMA(op, 18, 2, 2) c19 SL_MFMA(op, 19, 3, 2)                      \
  c20 SL_MFMA(op, 20, 4, 2) c21 SL_MFMA(op, 21, 5, 2) c22 SL_MFMA(op, 22, 6, 2) c23 SL_MFMA(op, 23, 7, 2)                      \
  SL_MFMA(op, 24, 0, 3) SL_MFMA(op, 25, 1, 3) SL_MFMA(op, 26, 2, 3) SL_MFMA(op, 27, 3, 3) SL_MFMA(op, 28, 4, 3)                \
  SL_MFMA(op, 29, 5, 3) SL_MFMA(op, 30, 6, 3) SL_MFMA(op, 31, 7, 3) "s_waitcnt lgkmcnt(0)"
#define SL_ALL(...) SL_PRODUCTS(__VA_ARGS__)
#define SL_READS8 SL_READ(0), SL_READ(1), SL_READ(2), SL_READ(3), SL_READ(4), SL_READ(5), SL_READ(6), SL_READ(7)
#define SL_READS4 SL_READ(0), "", SL_READ(1), "", SL_READ(2), "", SL_READ(3), ""
#define SL_COPIES8                                                                                                             \
  SL_TO(0), SL_COPY(0), SL_TO(1), SL_COPY(1), SL_TO(2), SL_COPY(2), SL_TO(3), SL_COPY(3), SL_TO(4), SL_COPY(4), SL_TO(5),      \
      SL_COPY(5), SL_TO(6), SL_COPY(6), SL_TO(7), SL_COPY(7)
#define SL_COPIES4                                                                                                             \
  SL_TO(0), SL_COPY(0), "", "", SL_TO(1), SL_COPY(1), "", "", SL_TO(2), SL_COPY(2), "", "", SL_TO(3), SL_COPY(3), "", ""
#define SL_COPIES0 "", "", "", "", "", "", "", "", "", "", "", "", "", "", "", ""
#define SL_ROW(i, n0, n1, n2, n3, n4, n5, n6, n7)                                                                              \
  [c##n0] "+a"(acc[i][0]), [c##n1] "+a"(acc[i][1]), [c##n2] "+a"(acc[i][2]), [c##n3] "+a"(acc[i][3]), [c##n4] "+a"(acc[i][4]), \
      [c##n5] "+a"(acc[i][5]), [c##n6] "+a"(acc[i][6]), [c##n7] "+a"(acc[i][7])
#define SL_ACC                                                                                                                 \
  SL_ROW(I0, 0, 1, 2, 3, 4, 5, 6, 7), SL_ROW(I0 + 1, 8, 9, 10, 11, 12, 13, 14, 15),                                            \
      SL_ROW(I0 + 2, 16, 17, 18, 19, 20, 21, 22, 23), SL_ROW(I0 + 3, 24, 25, 26, 27, 28, 29, 30, 31)
#define SL_OPERANDS                                                                                                            \
  [b0] "v"(fb[0]), [b1] "v"(fb[1]), [b2] "v"(fb[2]), [b3] "v"(fb[3]), [b4] "v"(fb[4]), [b5] "v"(fb[5]), [b6] "v"(fb[6]),       \
      [b7] "v"(fb[7]), [a0] "v"(fa[I0]), [a1] "v"(fa[I0 + 1]), [a2] "v"(fa[I0 + 2]), [a3] "v"(fa[I0 + 3]), [k0] "n"(K0),       \
      [k1] "n"(K0 + 2048)
#define SL_COPY4 [m] "s"(copy.to), [rs] "s"(copy.rsrc), [so] "s"(copy.start), [v0] "v"(voff[0]), [v1] "v"(voff[1]), [v2] "v"(voff[2]), [v3] "v"(voff[3])
#define SL_COPY8 SL_COPY4, [v4] "v"(voff[4]), [v5] "v"(voff[5]), [v6] "v"(voff[6]), [v7] "v"(voff[7])
#define SL_OUT(n) [l##n] "=&v"(o[n][0]), [h##n] "=&v"(o[n][1])
#define SL_OUT4 SL_OUT(0), SL_OUT(1), SL_OUT(2), SL_OUT(3)
#define SL_OUT8 SL_OUT4, SL_OUT(4), SL_OUT(5), SL_OUT(6), SL_OUT(7)
#define SL_AT(n) [t##n] "v"(at[n])
#define SL_AT4 SL_AT(0), SL_AT(1), SL_AT(2), SL_AT(3)
#define SL_AT8 SL_AT4, SL_AT(4), SL_AT(5), SL_AT(6), SL_AT(7)
#define SL_STATEMENT(op)                                                                                                       \
  if constexpr (NF == 8 && NC == 8)                                                                                            \
    asm volatile(SL_ALL(op, SL_READS8, SL_COPIES8) : SL_ACC, SL_OUT8 : SL_OPERANDS, SL_COPY8, SL_AT8 : "memory", "m0", "scc"); \
  else if constexpr (NF == 8 && NC == 4)                                                                                       \
    asm volatile(SL_ALL(op, SL_READS8, SL_COPIES4) : SL_ACC, SL_OUT8 : SL_OPERANDS, SL_COPY4, SL_AT8 : "memory", "m0", "scc"); \
  else if constexpr (NF == 8)                                                                                                  \
    asm volatile(SL_ALL(op, SL_READS8, SL_COPIES0) : SL_ACC, SL_OUT8 : SL_OPERANDS, SL_AT8 : "memory");                        \
  else if constexpr (NC == 8)                                                                                                  \
    asm volatile(SL_ALL(op, SL_READS4, SL_COPIES8) : SL_ACC, SL_OUT4 : SL_OPERANDS, SL_COPY8, SL_AT4 : "memory", "m0", "scc"); \
  else if constexpr (NC == 4)                                                                                                  \
    asm volatile(SL_ALL(op, SL_READS4, SL_COPIES4) : SL_ACC, SL_OUT4 : SL_OPERANDS, SL_COPY4, SL_AT4 : "memory", "m0", "scc"); \
  else                                                                                                                         \
    asm volatile(SL_ALL(op, SL_READS4, SL_COPIES0) : SL_ACC, SL_OUT4 : SL_OPERANDS, SL_AT4 : "memory");

struct Copies {
  uint32_t to;     // LDS address of the first (4096 to the next)
  u32x4 rsrc;
  uint32_t start;  // scalar offset
};
// rows I0 to I0 + 3 of the block; fragments at[0 .. NF - 1] + K0 into to[];
// copies with lane offsets voff[0 .. NC - 1]
template <int EK, int I0, int NF, int NC, int K0>
__device__ __forceinline__ void products_reads_copies(floatx4 (&acc)[8][8], const u32x4 (&fb)[8], const u32x4 (&fa)[8], const uint32_t* at,
                                                      u32x4* to, const Copies& copy, const uint32_t* voff) {
  u32x2 o[NF][2];
  if constexpr (EK == EK_F16) {
    SL_STATEMENT("v_mfma_f32_16x16x32_f16")
  } else {
    SL_STATEMENT("v_mfma_f32_16x16x32_bf16")
  }
#pragma unroll
  for (int n = 0; n < NF; ++n) to[n] = __builtin_shufflevector(o[n][0], o[n][1], 0, 1, 2, 3);
}
#undef SL_STATEMENT

// The same for a wave's 4 x 4 block: its 16 products, NF = 4 or 8 fragments (B's
// four, then A's) and four copies.
#define SL_PRODUCTS16(op, r0, r1, r2, r3, r4, r5, r6, r7, c8, c9, c10, c11, c12, c13, c14, c15)                     \
  r0 SL_MFMA(op, 0, 0, 0) r1 SL_MFMA(op, 1, 1, 0) r2 SL_MFMA(op, 2, 2, 0) r3 SL_MFMA(op, 3, 3, 0)                   \
  r4 SL_MFMA(op, 4, 0, 1) r5 SL_MFMA(op, 5, 1, 1) r6 SL_MFMA(op, 6, 2, 1) r7 SL_MFMA(op, 7, 3, 1)                   \
  c8 SL_MFMA(op, 8, 0, 2) c9 SL_MFMA(op, 9, 1, 2) c10 SL_MFMA(op, 10, 2, 2) c11 SL_MFMA(op, 11, 3, 2)               \
  c12 SL_MFMA(op, 12, 0, 3) c13 SL_MFMA(op, 13, 1, 3) c14 SL_MFMA(op, 14, 2, 3) c15 SL_MFMA(op, 15, 3, 3) "s_waitcnt lgkmcnt(0)"
#define SL_ALL16(...) SL_PRODUCTS16(__VA_ARGS__)
#define SL_FIRST4 SL_READ(0), SL_READ(1), SL_READ(2), SL_READ(3), "", "", "", ""
#define SL_COPIES16 SL_TO(0), SL_COPY(0), SL_TO(1), SL_COPY(1), SL_TO(2), SL_COPY(2), SL_TO(3), SL_COPY(3)
#define SL_ROW4(i, n0, n1, n2, n3) [c##n0] "+a"(acc[i][0]), [c##n1] "+a"(acc[i][1]), [c##n2] "+a"(acc[i][2]), [c##n3] "+a"(acc[i][3])
#define SL_ACC16 SL_ROW4(0, 0, 1, 2, 3), SL_ROW4(1, 4, 5, 6, 7), SL_ROW4(2, 8, 9, 10, 11), SL_ROW4(3, 12, 13, 14, 15)
#define SL_OPERANDS16                                                                                                        \
  [b0] "v"(fb[0]), [b1] "v"(fb[1]), [b2] "v"(fb[2]), [b3] "v"(fb[3]), [a0] "v"(fa[0]), [a1] "v"(fa[1]), [a2] "v"(fa[2]),      \
      [a3] "v"(fa[3]), [k0] "n"(K0), [k1] "n"(K0 + 1024)
#define SL_STATEMENT16(op)                                                                                                   \
  if constexpr (NF == 8)                                                                                                     \
    asm volatile(SL_ALL16(op, SL_READS8, SL_COPIES16) : SL_ACC16, SL_OUT8 : SL_OPERANDS16, SL_COPY4, SL_AT8 : "memory", "m0", "scc"); \
  else                                                                                                                       \
    asm volatile(SL_ALL16(op, SL_FIRST4, SL_COPIES16) : SL_ACC16, SL_OUT4 : SL_OPERANDS16, SL_COPY4, SL_AT4 : "memory", "m0", "scc");
template <int EK, int NF, int K0>
__device__ __forceinline__ void products16(floatx4 (&acc)[4][4], const u32x4 (&fb)[4], const u32x4 (&fa)[4], const uint32_t (&at)[8],
                                           u32x4 (&to_b)[4], u32x4 (&to_a)[4], const Copies& copy, const uint32_t (&voff)[4]) {
  u32x2 o[NF][2];
  if constexpr (EK == EK_F16) {
    SL_STATEMENT16("v_mfma_f32_16x16x32_f16")
  } else {
    SL_STATEMENT16("v_mfma_f32_16x16x32_bf16")
  }
#pragma unroll
  for (int n = 0; n < NF; ++n) (n < 4 ? to_b[n & 3] : to_a[n & 3]) = __builtin_shufflevector(o[n][0], o[n][1], 0, 1, 2, 3);
}
#undef SL_STATEMENT16
#undef SL_OPERANDS16
#undef SL_ACC16
#undef SL_ROW4
#undef SL_COPIES16
#undef SL_FIRST4
#undef SL_ALL16
#undef SL_PRODUCTS16
#undef SL_AT8
#undef SL_AT4
#undef SL_AT
#undef SL_OUT8
#undef SL_OUT4
#undef SL_OUT
#undef SL_COPY8
#undef SL_COPY4
#undef SL_OPERANDS
#undef SL_ACC
#undef SL_ROW
#undef SL_COPIES0
#undef SL_COPIES4
#undef SL_COPIES8
#undef SL_READS4
#undef SL_READS8
#undef SL_ALL
#undef SL_PRODUCTS
#undef SL_MFMA
#undef SL_COPY
#undef SL_TO
#undef SL_READ

// 256 x 256 on the schedule of dense_ring_kernel (dense.hpp), which see, with B
// (x, or the weights one after the other) and, ACROSS, A (dg and du) as they lie.  4096 x
// 4096 x 16384 (dx of F = 8192) 372 us, 1.48 PFLOP/s, the matrix cores busy 72%; 16384 x
// 4096 x 4096 (both weights) 403 us, 66%; at 1.8 GHz (power).
template <int EK, bool ACROSS>
__global__ __launch_bounds__(256, 1) void grad_ring_kernel(const GradParams g) {
  constexpr int F = 8, SLOT = 256 * kRowBytes;
  const DenseParams& p = g.d;
  __shared__ __attribute__((aligned(1024))) char smem[5 * SLOT];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TileCoord tc = map_tile(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, p.batch);
  const int64_t m0 = (int64_t)tc.tm * 256, n0 = (int64_t)tc.tn * 256;
  const int32_t rows_a = (int32_t)(p.M - m0 < 256 ? p.M - m0 : 256), rows_b = (int32_t)(p.N - n0 < 256 ? p.N - n0 : 256);
  const int64_t matrix = tc.batch >> p.b_shift;
  const int32_t second = tc.batch & p.b_shift;
  const uint8_t* a = p.a + matrix * p.a_bs + second * g.a_second + (ACROSS ? 2 * m0 : m0 * p.a_rs);
  // (columns of A past the result's rows hold zeros)
  const int32_t part = (int32_t)g.rows, parts = g.parts;  // rows of B to a part, parts
  const int32_t PT = (part + 63) / 64, T = parts * PT;    // K-tiles
  __builtin_assume(T >= 1);
  const uint8_t* const a_base[1] = {a};
  const int64_t a_rs[1] = {p.a_rs};
  RowLoader<256, 256, 0> la(a_base, a_rs, ACROSS ? 0 : rows_a, ACROSS ? 0 : (int64_t)T * kRowBytes, wave, lane);
  AcrossLoader<256> xa(ACROSS ? (rows_a + 7) / 8 * 8 : 0, p.a_rs, wave, lane), xb(rows_b, p.b_rs[0], wave, lane);
  const uint32_t a_bytes = ACROSS ? (uint32_t)((part - 1) * p.a_rs + 512) : (uint32_t)((rows_a - 1) * p.a_rs + (int64_t)T * kRowBytes);
  const uint32_t b_bytes = (uint32_t)((part - 1) * p.b_rs[0] + 2 * rows_b);
  const u32x4 ra = rsrc_words(a, a_bytes);
  const uint8_t* const b0 = p.b[0] + matrix * p.b_bs[0] + 2 * n0;
  const uint8_t* const b1 = p.b[1] + matrix * p.b_bs[1] + 2 * n0;
  const u32x4 rb0 = rsrc_words(b0, b_bytes), rb1 = rsrc_words(b1, b_bytes);
  floatx4 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int32_t a_row0 = (wave & 1) * 128, b_row0 = (wave >> 1) * 128;
  auto kt = [&](int32_t u) { return u < T ? u : T - 1; };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)smem;
  // the last K-tile of a part may have fewer than 64 rows: the loaders know
  // before its copies
  const int32_t last = part - 64 * (PT - 1);
  auto before_a = [&](int32_t u) {
    if (ACROSS && last < 64 && u == T - 1) xa.rows(last);
  };
  auto before_b = [&](int32_t u) {
    if (last < 64 && u < T) {
      const int32_t at = u >= PT ? u - PT : u;
      if (at == PT - 1) xb.rows(last);
      else if (at == 0 && u > 0) xb.rows(64);
    }
  };
  // K-tile u's copies into slot q: their lane offsets are the loaders'
  auto copies_a = [&](int32_t u, int32_t q) {
    return Copies{lds0 + (uint32_t)(q * SLOT + wave * 1024), ra, (uint32_t)kt(u) * (ACROSS ? 64u * xa.step : (uint32_t)kRowBytes)};
  };
  auto copies_b = [&](int32_t u, int32_t q) {
    const int32_t v = kt(u);
    return Copies{lds0 + (uint32_t)(q * SLOT + wave * 1024), v >= PT ? rb1 : rb0, (uint32_t)(v >= PT ? v - PT : v) * 64u * xb.step};
  };
  const uint32_t* const va = ACROSS ? xa.voff : la.voff;
  const uint32_t* const vb = xb.voff;
  // all eight at once, ahead of the loop
  auto copy_all = [&](const uint8_t* base, uint32_t bytes, const uint32_t* voff, const Copies& c) {
    const __amdgpu_buffer_rsrc_t from = make_rsrc(base, bytes);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t v = voff[j];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void_t*)(uintptr_t)(c.to + 4096u * (uint32_t)j), 16, v, c.start, 0, 0);
    }
  };
  u32x4 fa0[F], fb0[F], fa1[F], fb1[F];
  typedef __attribute__((address_space(3))) const u32x4 lds_u4;
  // LDS addresses: of an operand read across, one for each fragment (slices
  // 16384 apart); of A read along its rows, for either slice and parity of the
  // fragment (pairs of fragments 4096 apart)
  uint32_t offB[F], tb[F], offA[F], ta[F];
#pragma unroll
  for (int j = 0; j < F; ++j) {
    offB[j] = lds0 + (uint32_t)tr_read_offset(lane, 0, b_row0 + 16 * j, 0, 256);
    offA[j] = ACROSS ? lds0 + (uint32_t)tr_read_offset(lane, 0, a_row0 + 16 * j, 0, 256)
                     : lds0 + (uint32_t)fragment_lds_offset(MFMA16_F16, lane, 0, a_row0 + 16 * (j & 1), j >> 1 & 1, 0);
  }
  auto bases = [&](int32_t qa, int32_t qb) {
#pragma unroll
    for (int j = 0; j < F; ++j) {
      tb[j] = offB[j] + (uint32_t)(qb * SLOT);
      if (ACROSS || j < 4) ta[j] = offA[j] + (uint32_t)(qa * SLOT);
    }
  };
  // A's fragments from i on, along its rows
  auto read_a = [&](int i, int n, int ks, u32x4(&fa)[F]) {
    if constexpr (!ACROSS) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= i && e < i + n) fa[e] = *(lds_u4*)(uintptr_t)(ta[2 * ks + (e & 1)] + 4096u * (uint32_t)(e >> 1));
    }
  };
  before_a(0), before_b(0);
  copy_all(a, a_bytes, va, copies_a(0, 0));
  copy_all(b0, b_bytes, vb, copies_b(0, 1));
  before_a(1);
  copy_all(a, a_bytes, va, copies_a(1, 2));
  before_b(1), before_a(2);
  // the first K-tile's first products are of zero fragments (add nothing)
#pragma unroll
  for (int i = 0; i < F; ++i) fa1[i] = fb1[i] = u32x4{0, 0, 0, 0};
  wait_vmem_n<8>();
  phase_barrier();
  int32_t sa = 0;  // slot of A(t); B(t) in the next one
  int32_t t = 0;
  bases(0, 1);
#pragma clang loop unroll(disable)
  do {
    const int32_t s3 = sa + 3 >= 5 ? sa - 2 : sa + 3, s4 = sa == 0 ? 4 : sa - 1;
    // K-tile t - 1's second slice; slice 0 read; B(t + 1) copied, early.  Then
    // its first slice; slice 1 read; A(t + 2) copied.
#define SL_STEP(half, ks, a, b, to_a, to_b, nc, copy, voff)                                                           \
  read_a(4 * half, 4, ks, to_a);                                                                                       \
  __builtin_amdgcn_sched_barrier(0);                                                                                   \
  products_reads_copies<EK, 4 * half, ACROSS ? 8 : 4, nc, 16384 * ks>(acc, b, a, ACROSS && half ? ta : tb + (half ? 4 : 0), \
                                                                      ACROSS && half ? to_a : to_b + (half ? 4 : 0), copy, voff); \
  __builtin_amdgcn_sched_barrier(0);
    const Copies to_b = copies_b(t + 1, s3);
    SL_STEP(0, 0, fa1, fb1, fa0, fb0, 8, to_b, vb)
    SL_STEP(1, 0, fa1, fb1, fa0, fb0, 0, to_b, vb)
    Copies to_a = copies_a(t + 2, s4);
    SL_STEP(0, 1, fa0, fb0, fa1, fb1, 4, to_a, va)
    to_a.to += 4 * 4096;
    SL_STEP(1, 1, fa0, fb0, fa1, fb1, 4, to_a, va + 4)
#undef SL_STEP
    const int32_t na = sa + 2 >= 5 ? sa - 3 : sa + 2;
    bases(na, na == 4 ? 0 : na + 1);
    before_b(t + 2), before_a(t + 3);  // the next copies
    wait_vmem_n<8>();  // in flight after this: A(t + 2)
    phase_barrier();
    sa = na;
  } while (++t < T);
#pragma unroll
  for (int e = 0; e < 64; ++e) dense_mfma_agpr<EK>(acc[e / F][e % F], fb1[e % F], fa1[e / F]);
  wait_vmem();
  // as in dense_ring_kernel: an idle between the last product and the first
  // read of an accumulator
  auto pin = [&] {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; j += 2) asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
  };
  pin();
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  pin();
  __syncthreads();
  char* region = smem + wave * 32768;
  const Gradient<EK == EK_F16 ? OT_F16 : OT_BF16> epi(p, tc.batch);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) *(floatx4*)(region + rows_chunk(16 * i + (lane & 15), 4 * j + (lane >> 4))) = acc[4 * h + i][j];
    dense_rows<EK, false, 128>(epi, p, tc.batch, m0 + a_row0 + 64 * h, n0 + b_row0, lane, region);
  }
}

// 128 x 128 tiles of the same, two workgroups to a CU.  Bound by LDS: a K-tile takes 0.5 us
// alone on its CU, where the dense kernel's, whose reads are 16 bytes a lane and not 8, takes
// 0.35.
template <int EK, bool ACROSS>
__device__ __forceinline__ void grad_tile(const GradParams& g, uint32_t id, uint32_t total, char* smem) {
  constexpr int F = 4, W = 128, SLOT = W * kRowBytes;
  const DenseParams& p = g.d;
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TileCoord tc = map_tile((int32_t)id, (int32_t)total, p.tiles_m, p.tiles_n, p.group_m, p.batch);
  const int64_t m0 = (int64_t)tc.tm * W, n0 = (int64_t)tc.tn * W;
  const int32_t rows_a = (int32_t)(p.M - m0 < W ? p.M - m0 : W), rows_b = (int32_t)(p.N - n0 < W ? p.N - n0 : W);
  const int64_t matrix = tc.batch >> p.b_shift;
  const int32_t second = tc.batch & p.b_shift;
  const uint8_t* a = p.a + matrix * p.a_bs + second * g.a_second + (ACROSS ? 2 * m0 : m0 * p.a_rs);
  // (columns of A past the result's rows hold zeros)
  const int32_t part = (int32_t)g.rows, parts = g.parts;  // rows of B to a part, parts
  const int32_t PT = (part + 63) / 64, T = parts * PT;    // K-tiles
  __builtin_assume(T >= 1);
  const uint8_t* const a_base[1] = {a};
  const int64_t a_rs[1] = {p.a_rs};
  RowLoader<W, 256, 0> la(a_base, a_rs, ACROSS ? 0 : rows_a, ACROSS ? 0 : (int64_t)T * kRowBytes, wave, lane);
  AcrossLoader<W> xa(ACROSS ? (rows_a + 7) / 8 * 8 : 0, p.a_rs, wave, lane), xb(rows_b, p.b_rs[0], wave, lane);
  const uint32_t a_bytes = ACROSS ? (uint32_t)((part - 1) * p.a_rs + 2 * W) : (uint32_t)((rows_a - 1) * p.a_rs + (int64_t)T * kRowBytes);
  const uint32_t b_bytes = (uint32_t)((part - 1) * p.b_rs[0] + 2 * rows_b);
  const u32x4 ra = rsrc_words(a, a_bytes);
  const uint8_t* const b0 = p.b[0] + matrix * p.b_bs[0] + 2 * n0;
  const uint8_t* const b1 = p.b[1] + matrix * p.b_bs[1] + 2 * n0;
  const u32x4 rb0 = rsrc_words(b0, b_bytes), rb1 = rsrc_words(b1, b_bytes);
  floatx4 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int32_t a_row0 = (wave & 1) * 64, b_row0 = (wave >> 1) * 64;
  auto kt = [&](int32_t u) { return u < T ? u : T - 1; };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)smem;
  // ahead of K-tile u's copies: the last one of a part may have fewer than 64 rows, and
  // those past the last read zeros
  const int32_t last = part - 64 * (PT - 1);
  auto before_a = [&](int32_t u) {
    if constexpr (ACROSS) {
      if (u >= T - 1) xa.rows(u == T - 1 ? last : 0);
    } else {
      if (u >= T) la.last_tile(0);
    }
  };
  auto before_b = [&](int32_t u) {
    const int32_t at = u >= PT ? u - PT : u;
    if (u >= T) xb.rows(0);
    else if (at == PT - 1) xb.rows(last);
    else if (at == 0 && u > 0) xb.rows(64);
  };
  auto copies_a = [&](int32_t u, int32_t q) {
    return Copies{lds0 + (uint32_t)(q * SLOT + wave * 1024), ra, (uint32_t)kt(u) * (ACROSS ? 64u * xa.step : (uint32_t)kRowBytes)};
  };
  auto copies_b = [&](int32_t u, int32_t q) {
    const int32_t v = kt(u);
    return Copies{lds0 + (uint32_t)(q * SLOT + wave * 1024), v >= PT ? rb1 : rb0, (uint32_t)(v >= PT ? v - PT : v) * 64u * xb.step};
  };
  const uint32_t(&va)[4] = ACROSS ? xa.voff : la.voff;
  const uint32_t(&vb)[4] = xb.voff;
  // all four at once, ahead of the loop
  auto copy_all = [&](const uint8_t* base, uint32_t bytes, const uint32_t(&voff)[4], const Copies& c) {
    const __amdgpu_buffer_rsrc_t from = make_rsrc(base, bytes);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = voff[j];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void_t*)(uintptr_t)(c.to + 4096u * (uint32_t)j), 16, v, c.start, 0, 0);
    }
  };
  u32x4 fa0[F], fb0[F], fa1[F], fb1[F];
  typedef __attribute__((address_space(3))) const u32x4 lds_u4;
  // LDS addresses: of an operand read across, one for each fragment (slices 8192
  // apart); of A read along its rows, for either slice and parity of the fragment (pairs
  // of fragments 4096 apart)
  uint32_t off[8], at[8];  // B's, then A's
#pragma unroll
  for (int j = 0; j < F; ++j) {
    off[j] = lds0 + (uint32_t)tr_read_offset(lane, 0, b_row0 + 16 * j, 0, W);
    off[F + j] = ACROSS ? lds0 + (uint32_t)tr_read_offset(lane, 0, a_row0 + 16 * j, 0, W)
                        : lds0 + (uint32_t)fragment_lds_offset(MFMA16_F16, lane, 0, a_row0 + 16 * (j & 1), j >> 1, 0);
  }
  auto bases = [&](int32_t qa, int32_t qb) {
#pragma unroll
    for (int j = 0; j < F; ++j) at[j] = off[j] + (uint32_t)(qb * SLOT), at[F + j] = off[F + j] + (uint32_t)(qa * SLOT);
  };
  auto read_a = [&](int ks, u32x4(&fa)[F]) {
    if constexpr (!ACROSS) {
#pragma unroll
      for (int e = 0; e < F; ++e) fa[e] = *(lds_u4*)(uintptr_t)(at[F + 2 * ks + (e & 1)] + 4096u * (uint32_t)(e >> 1));
    }
  };
  before_a(0), before_b(0);
  copy_all(a, a_bytes, va, copies_a(0, 0));
  copy_all(b0, b_bytes, vb, copies_b(0, 1));
  before_a(1);
  copy_all(a, a_bytes, va, copies_a(1, 2));
  before_b(1), before_a(2);
  // the first K-tile's first products are of zero fragments (add nothing)
#pragma unroll
  for (int i = 0; i < F; ++i) fa1[i] = fb1[i] = u32x4{0, 0, 0, 0};
  wait_vmem_n<4>();
  phase_barrier();
  int32_t sa = 0;  // slot of A(t); B(t) in the next one
  int32_t t = 0;
  bases(0, 1);
#pragma clang loop unroll(disable)
  do {
    const int32_t s3 = sa + 3 >= 5 ? sa - 2 : sa + 3, s4 = sa == 0 ? 4 : sa - 1;
    // K-tile t - 1's second slice; slice 0 read; B(t + 1) copied.  Then its first
    // slice; slice 1 read; A(t + 2) copied.
    read_a(0, fa0);
    __builtin_amdgcn_sched_barrier(0);
    products16<EK, ACROSS ? 8 : 4, 0>(acc, fb1, fa1, at, fb0, fa0, copies_b(t + 1, s3), vb);
    __builtin_amdgcn_sched_barrier(0);
    read_a(1, fa1);
    __builtin_amdgcn_sched_barrier(0);
    products16<EK, ACROSS ? 8 : 4, 8192>(acc, fb0, fa0, at, fb1, fa1, copies_a(t + 2, s4), va);
    __builtin_amdgcn_sched_barrier(0);
    const int32_t na = sa + 2 >= 5 ? sa - 3 : sa + 2;
    bases(na, na == 4 ? 0 : na + 1);
    before_b(t + 2), before_a(t + 3);  // the next copies
    wait_vmem_n<4>();  // in flight after this: A(t + 2)
    phase_barrier();
    sa = na;
  } while (++t < T);
#pragma unroll
  for (int e = 0; e < 16; ++e) dense_mfma_agpr<EK>(acc[e / F][e % F], fb1[e % F], fa1[e / F]);
  wait_vmem();
  auto pin = [&] {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; j += 2) asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
  };
  pin();
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  pin();
  __syncthreads();
  char* region = smem + wave * 16384;
  const Gradient<EK == EK_F16 ? OT_F16 : OT_BF16> epi(p, tc.batch);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) *(floatx4*)(region + rows_chunk<64>(16 * i + (lane & 15), 4 * j + (lane >> 4))) = acc[i][j];
  dense_rows<EK, false, 64>(epi, p, tc.batch, m0 + a_row0, n0 + b_row0, lane, region);
}

template <int EK, bool ACROSS>
__global__ __launch_bounds__(256, 2) void grad_tile_kernel(const GradParams g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRing * 128 * kRowBytes];
  grad_tile<EK, ACROSS>(g, blockIdx.x, gridDim.x, smem);
}
// x's gradient and the weights' in one launch
template <int EK>
__global__ __launch_bounds__(256, 2) void grad_pair_kernel(const GradPair g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRing * 128 * kRowBytes];
  if (blockIdx.x < g.first) grad_tile<EK, false>(g.dx, blockIdx.x, g.first, smem);
  else grad_tile<EK, true>(g.dw, blockIdx.x - g.first, gridDim.x - g.first, smem);
}

// x's gradient of few rows, 16 FM to a tile: the weights are read as they lie, from
// memory once, and bound the call.  A wave takes 32 rows of a weight and 128 of its
// columns straight into registers, a lane eight values of each of eight rows: turned
// within the lane, eight fragments (fragment j holds columns j, 8 + j, 16 + j, ...), so that neither LDS nor
// copies are needed.  The eight waves of a workgroup and `splits` workgroups share the
// rows; waves' sums meet in LDS, workgroups' in the workspace (grad_few_join_kernel), always
// in one order.  Two weights of 8192 x 4096 (134 MB) for one row: 24 us, 5.5 TB/s; for 64 rows 29.
constexpr int kFewWaves = 8, kFewPitch = 132;  // floats of a row of sums in LDS, off the banks' number
template <int EK, int FM>
__global__ __launch_bounds__(kFewWaves * 64, 1) void grad_few_kernel(const GradParams g) {
  constexpr int DEPTH = FM == 4 ? 2 : FM == 2 ? 3 : 4, C = 8;  // steps requested ahead, fragments of columns
  const DenseParams& p = g.d;
  __shared__ __attribute__((aligned(16))) float part[kFewWaves][16][kFewPitch];
  const int32_t lane = threadIdx.x & 63, l0 = lane & 15, l1 = lane >> 4;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // An XCD's workgroups: whole rows of a share of the weights, and the tiles that read the
  // same of them next to each other.
  const uint32_t per = gridDim.x / 8, id = gridDim.x % 8 == 0 ? blockIdx.x % 8 * per + blockIdx.x / 8 : blockIdx.x;
  const uint32_t tm = id % (uint32_t)p.tiles_m, share = id / (uint32_t)p.tiles_m;
  const uint32_t tiles = (uint32_t)p.batch * (uint32_t)p.tiles_n, split = share / tiles, tile = share % tiles;
  const int64_t batch = tile / (uint32_t)p.tiles_n, n0 = (int64_t)(tile % (uint32_t)p.tiles_n) * 128, m0 = (int64_t)tm * (16 * FM);
  const int32_t F = (int32_t)g.rows, steps = (F + 31) / 32;  // of either weight
  const int32_t cols = (int32_t)(p.N - n0 < 128 ? p.N - n0 : 128);
  const int32_t rows = (int32_t)(p.M - m0 < 16 * FM ? p.M - m0 : 16 * FM);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + batch * p.a_bs + m0 * p.a_rs, (uint32_t)((rows - 1) * p.a_rs + p.K));
  const uint32_t b_bytes = (uint32_t)((F - 1) * p.b_rs[0] + 2 * cols), step = (uint32_t)p.b_rs[0];
  const __amdgpu_buffer_rsrc_t rb0 = make_rsrc(p.b[0] + batch * p.b_bs[0] + 2 * n0, b_bytes);
  const __amdgpu_buffer_rsrc_t rb1 = make_rsrc(p.b[1] + batch * p.b_bs[1] + 2 * n0, b_bytes);
  const uint32_t off_b = 8 * l0 < cols ? (uint32_t)(8 * l1) * step + (uint32_t)(16 * l0) : kOutOfRange;
  uint32_t off_a[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) off_a[i] = 16 * i + l0 < rows ? (uint32_t)((16 * i + l0) * p.a_rs + 16 * l1) : kOutOfRange;
  struct Regs {
    u32x4 a[FM], b[8];
  };
  // step t of both weights'; past the last one zeros
  auto load = [&](int32_t t, Regs& x) {
    const bool second = t >= steps;
    const int32_t f0 = 32 * (second ? t - steps : t);
    const int32_t left = t < 2 * steps ? F - f0 : 0;  // rows there are
    const __amdgpu_buffer_rsrc_t rb = second ? rb1 : rb0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x.b[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, off_b != kOutOfRange && 8 * l1 + i < left ? off_b + (uint32_t)(f0 + i) * step : kOutOfRange, 0, 0);
#pragma unroll
    for (int i = 0; i < FM; ++i)
      x.a[i] = __builtin_amdgcn_raw_buffer_load_b128(
          ra, off_a[i] != kOutOfRange && left > 0 ? off_a[i] + (uint32_t)(2 * f0) + (second ? (uint32_t)p.K / 2 : 0u) : kOutOfRange, 0, 0);
  };
  floatx4 acc[FM][C];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int32_t first = (int32_t)split * kFewWaves + wave, stride = g.splits * kFewWaves;
  if (first < 2 * steps) {
    Regs x[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(first + d * stride, x[d]);
    for (int32_t t = first; t < 2 * steps; t += DEPTH * stride) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
          u32x4 fb;  // column j of the lane's eight rows
#pragma unroll
          for (int i = 0; i < 4; ++i)
            fb[i] = __builtin_amdgcn_perm(x[d].b[2 * i + 1][j / 2], x[d].b[2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int i = 0; i < FM; ++i) acc[i][j] = dense_mfma<EK>(fb, x[d].a[i], acc[i][j]);  // past the last row: zeros
        }
        load(t + (d + DEPTH) * stride, x[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // the lane's values r of the eight fragments are eight columns of one row
  const Gradient<EK == EK_F16 ? OT_F16 : OT_BF16> epi(p, batch);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* at = &part[wave][l0][8 * (4 * l1 + r)];
      *(floatx4*)at = floatx4{acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]};
      *((floatx4*)at + 1) = floatx4{acc[i][4][r], acc[i][5][r], acc[i][6][r], acc[i][7][r]};
    }
    __syncthreads();
    const int32_t row = threadIdx.x / 32, c = 4 * (threadIdx.x % 32);
    floatx4 v = *(const floatx4*)&part[0][row][c];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) {
      const floatx4 u = *(const floatx4*)&part[w][row][c];
      v = floatx4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
    }
    const int64_t m = m0 + 16 * i + row, n = n0 + c;
    if (16 * i + row >= rows || n >= p.N) continue;
    if (g.splits == 1) epi.finish(p, batch, m, n, v);
    else *(floatx4*)(g.partial + (((int64_t)split * p.batch + batch) * p.M + m) * p.N + n) = v;
  }
}
// the sums of `splits` workgroups, four columns to a thread (N a multiple of 8)
template <int EK>
__global__ __launch_bounds__(256) void grad_few_join_kernel(const GradParams g) {
  const DenseParams& p = g.d;
  const int64_t quads = p.N / 4, all = p.batch * p.M * quads, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= all) return;
  const floatx4* at = (const floatx4*)g.partial + id;
  floatx4 v = *at;
  for (int32_t s = 1; s < g.splits; ++s) {
    const floatx4 u = at[s * all];
    v = floatx4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
  }
  const int64_t n = id % quads * 4, m = id / quads % p.M, batch = id / quads / p.M;
  const Gradient<EK == EK_F16 ? OT_F16 : OT_BF16> epi(p, batch);
  epi.finish(p, batch, m, n, v);
}

}  // namespace

hipError_t launch_grad_few(const GradParams& g, int32_t kind, hipStream_t s) {
  const dim3 grid((uint32_t)(dense_groups(g.d) * g.splits)), block(kFewWaves * 64);
  auto few = [&](auto fm) {
    constexpr int FM = decltype(fm)::value;
    if (kind == EK_F16) hipLaunchKernelGGL((grad_few_kernel<EK_F16, FM>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_few_kernel<EK_BF16, FM>), grid, block, 0, s, g);
  };
  if (g.d.M <= 16) few(std::integral_constant<int, 1>{});
  else if (g.d.M <= 32) few(std::integral_constant<int, 2>{});
  else few(std::integral_constant<int, 4>{});
  if (g.splits > 1) {
    const dim3 join((uint32_t)((g.d.batch * g.d.M * (g.d.N / 4) + 255) / 256));
    if (kind == EK_F16) hipLaunchKernelGGL((grad_few_join_kernel<EK_F16>), join, dim3(256), 0, s, g);
    else hipLaunchKernelGGL((grad_few_join_kernel<EK_BF16>), join, dim3(256), 0, s, g);
  }
  return hipGetLastError();
}

hipError_t launch_grad_ring(const GradParams& g, int32_t kind, bool across, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)g.d.batch * g.d.tiles_m * g.d.tiles_n)), block(256);
  if (kind == EK_F16) {
    if (across) hipLaunchKernelGGL((grad_ring_kernel<EK_F16, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_ring_kernel<EK_F16, false>), grid, block, 0, s, g);
  } else {
    if (across) hipLaunchKernelGGL((grad_ring_kernel<EK_BF16, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_ring_kernel<EK_BF16, false>), grid, block, 0, s, g);
  }
  return hipGetLastError();
}

hipError_t launch_grad_tiles(const GradParams& g, int32_t kind, bool across, hipStream_t s) {
  const dim3 grid((uint32_t)dense_groups(g.d)), block(256);
  if (kind == EK_F16) {
    if (across) hipLaunchKernelGGL((grad_tile_kernel<EK_F16, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_tile_kernel<EK_F16, false>), grid, block, 0, s, g);
  } else {
    if (across) hipLaunchKernelGGL((grad_tile_kernel<EK_BF16, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_tile_kernel<EK_BF16, false>), grid, block, 0, s, g);
  }
  return hipGetLastError();
}
hipError_t launch_grad_tiles(const GradPair& g, int32_t kind, hipStream_t s) {
  const dim3 grid((uint32_t)(g.first + dense_groups(g.dw.d))), block(256);
  if (kind == EK_F16) hipLaunchKernelGGL((grad_pair_kernel<EK_F16>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((grad_pair_kernel<EK_BF16>), grid, block, 0, s, g);
  return hipGetLastError();
}

template <class PRODUCTS>
static hipError_t products_of(const PRODUCTS& p, int32_t kind, const DensePlan& plan, hipStream_t s) {
  if (kind == EK_F16) return dense_launch<EK_F16, false, Gradient<OT_F16>>(p, plan, s);
  return dense_launch<EK_BF16, false, Gradient<OT_BF16>>(p, plan, s);
}
hipError_t launch_gated_products(const DenseParams& p, int32_t kind, const DensePlan& plan, hipStream_t s) { return products_of(p, kind, plan, s); }
hipError_t launch_gated_products(const DensePair& p, int32_t kind, const DensePlan& plan, hipStream_t s) { return products_of(p, kind, plan, s); }

}  // namespace sl
