// sl_ops.hpp -- parameters and launchers of the operators next to the GEMM:
// block quantisation to E4M3, the block-scaled 8-bit product, the
// orthogonalised update, row quantisation to int8, the int8 product, and the
// gated feed-forward block with its backward pass.  Shared by the host side
// (api_ops.cpp, api_gated.cpp) and their kernel translation units.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sl {

constexpr int32_t kScaleBlock = 128;  // K elements (and rows, for square blocks) that share one scale

// element types of the operators' inputs and outputs (template arguments)
constexpr int OT_F16 = 0;
constexpr int OT_BF16 = 1;
constexpr int OT_F32 = 2;

// ---------------------------------------------------------------------------
// Quantisation of x (batch, rows, cols) to E4M3 codes and fp32 scales:
// along the columns (q, s) and / or along the rows, transposed (qt, st).
// ---------------------------------------------------------------------------
struct QuantizeParams {
  const void* x;
  int64_t rows, cols, x_bs, x_rs, x_cs;
  int32_t type;        // OT_*
  int32_t square;      // 1: blocks of 128 x 128, else 1 x 128
  int32_t batch;
  // q[b][r][c] at q + b q_bs + r q_rs + c, columns [cols, q_cols) zero; s of
  // block row i, block j at s + b s_bs + i s_rs + j s_cs
  uint8_t* q;          // may be NULL
  float* s;
  int64_t q_cols, q_bs, q_rs, s_bs, s_rs, s_cs;
  // the transpose's: qt[b][c][r], rows [rows, qt_cols) zero
  uint8_t* qt;         // may be NULL
  float* st;
  int64_t qt_cols, qt_bs, qt_rs, st_bs, st_rs, st_cs;
};
constexpr int32_t kQuantizeThreads = 256;
int32_t quantize_rows(const QuantizeParams& p);  // of a workgroup; 128 columns
hipError_t launch_quantize(const QuantizeParams& p, hipStream_t stream);

// ---------------------------------------------------------------------------
// The block-scaled product D = C + (A SA) (B SB)^T on E4M3 codes with fp32
// scales per 128 K: row r of A takes scale row r >> a_shift (0: one per row,
// 7: one per 128 rows), B the same.
// ---------------------------------------------------------------------------
struct BlockGemmParams {
  const uint8_t* a;  // (b, m, k) at a + b a_bs + m a_rs + k
  const uint8_t* b;
  const void* c;     // may be NULL
  void* d;
  const float* sa;   // (b, row, K block) at sa + b sa_bs + row sa_rs + block sa_ks
  const float* sb;
  int64_t M, N, K;
  int64_t a_rs, a_bs, b_rs, b_bs;
  int64_t c_rs, c_cs, c_bs, d_rs, d_cs, d_bs;
  int64_t sa_rs, sa_ks, sa_bs, sb_rs, sb_ks, sb_bs;
  int32_t a_shift, b_shift;
  int32_t type;      // OT_* of C and D
  int32_t batch, tiles_m, tiles_n, group_m;
  int32_t k_blocks;  // ceil(K / 128)
  int32_t flags;     // BF_*
};
constexpr int32_t BF_HAS_C = 1;
constexpr int32_t BF_D_VEC = 2;   // four consecutive n of D in one aligned access
constexpr int32_t BF_C_VEC = 4;   // ... of C

// tile configurations of the product (rows of A x rows of B)
enum BlockTile : int32_t {
  BT_256x256 = 0,  // 8 waves, each 128 x 64
  BT_128x128 = 1,  // 4 waves, each 64 x 64
  BT_SKINNY = 2,   // 64 rows of A x 16 or 32 of B, the waves of a workgroup splitting K
};
struct BlockTileShape {
  int32_t bm, bn, wm, wn;
};
constexpr BlockTileShape kBlockTiles[3] = {{256, 256, 2, 4}, {128, 128, 2, 2}, {64, 32, 1, 1}};
constexpr int32_t kSkinnyRows = 64;   // most rows of A of one skinny workgroup
constexpr int32_t kSkinnyWaves = 8;    // up to 16 rows of A
constexpr int32_t kStreamWaves = 4;    // 17 to 64
// rows of B of a skinny workgroup: 32 when that still gives every CU one
inline int32_t skinny_cols(int64_t M, int64_t N, int64_t batch) {
  return batch * ((M + kSkinnyRows - 1) / kSkinnyRows) * ((N + 31) / 32) >= 256 ? 32 : 16;
}
hipError_t launch_gemm_block(const BlockGemmParams& p, int32_t tile, hipStream_t stream);

// ---------------------------------------------------------------------------
// The orthogonalised update.  x is taken with m <= n (a tall x by its
// strides, transposed); the matrices of the iteration are one or two planes of
// fp16 in the workspace, their sizes padded with zeros to multiples of 64.
// ---------------------------------------------------------------------------
struct OrthoParams {
  const void* x;               // (b, i, j), i < m, j < n
  void* d;
  int64_t m, n;                // m <= n
  int64_t x_bs, x_rs, x_cs, d_bs, d_rs, d_cs;
  int32_t x_type, d_type;      // OT_*
  int32_t batch, steps;
  const float* coefficients;   // 3 per step (host)
  char* ws;
};
constexpr int32_t kOrthoMaxSteps = 64;
size_t orthogonalize_workspace(const OrthoParams& p);
bool orthogonalize_grid_ok(const OrthoParams& p);
hipError_t launch_orthogonalize(const OrthoParams& p, hipStream_t stream);

// Through the Gram matrix the steps go in cycles: those from `first` on that
// one cycle takes.  ortho_gram.hip: up to kGramRows rows.
int32_t ortho_cycle(const OrthoParams& p, int32_t first);
constexpr int64_t kGramRows = 128;
struct OrthoGramPlan {
  int32_t rows;          // m padded: 32, 64, 96 or 128
  int32_t splits, cols;  // ranges of columns, and the columns of one
};
OrthoGramPlan ortho_gram_plan(int64_t m, int64_t n);
size_t ortho_gram_workspace(const OrthoParams& p);
hipError_t launch_ortho_gram(const OrthoParams& p, hipStream_t stream);

// ---------------------------------------------------------------------------
// Row quantisation of x (batch, rows, cols) to int8 codes with one fp32 scale
// per row: q[b][r][c] at q + b q_bs + r q_rs + c, columns [cols, q_cols) zero;
// s of row r at s + b s_bs + r s_rs.
// ---------------------------------------------------------------------------
struct QuantizeRowsParams {
  const void* x;
  int64_t rows, cols, x_bs, x_rs, x_cs;
  int8_t* q;
  float* s;
  int64_t q_cols, q_bs, q_rs, s_bs, s_rs;
  int32_t type;   // OT_*
  int32_t batch;
};
int64_t quantize_rows_groups(const QuantizeRowsParams& p);
int32_t quantize_rows_threads(const QuantizeRowsParams& p);  // of a workgroup
hipError_t launch_quantize_rows(const QuantizeRowsParams& p, hipStream_t stream);

// ---------------------------------------------------------------------------
// Products of K-contiguous rows (dense.hpp): the int8 product
//   D[m,n] = C[m,n] + sa[m] sb[n] sum_k A[m,k] B[n,k]
// and the gated pair, with B's rows n and those of a second matrix,
//   h[m,n] = act(g) u,  g = sum_k A[m,k] B0[n,k],  u = sum_k A[m,k] B1[n,k]
// (times the scales for int8), g and u kept where asked.
// ---------------------------------------------------------------------------
constexpr int EK_F16 = 0;   // the operands' element kinds (template arguments)
constexpr int EK_BF16 = 1;
constexpr int EK_I8 = 2;

constexpr int32_t ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3;  // sl_activation - 1

struct DenseParams {
  // rows of K bytes: row m of A at a + b a_bs + m a_rs (bytes), row n of matrix
  // s of B the same
  const uint8_t* a;
  const uint8_t* b[2];
  int64_t a_rs, a_bs, b_rs[2], b_bs[2];
  int64_t M, N, K;          // N: columns of the result; K in bytes, a multiple of 16
  // int8: one scale per row of A and of each B
  const float* sa;
  const float* sb[2];
  int64_t sa_rs, sa_bs, sb_rs[2], sb_bs[2];
  const void* c;            // may be NULL (the product alone)
  void* d;                  // the product's D, or h
  void* kept[2];            // g and u; may be NULL
  int64_t c_rs, c_cs, c_bs, d_rs, d_cs, d_bs, kept_rs[2], kept_cs[2], kept_bs[2];
  int32_t type;             // OT_* of C, D, g and u
  int32_t act;              // ACT_*
  int32_t b_shift;          // matrix b of the batch takes B's matrix b >> b_shift
  int32_t batch, tiles_m, tiles_n, group_m;
  int32_t k_tiles;          // ceil(K / 128)
  int32_t flags;            // DF_*
};
constexpr int32_t DF_D_VEC = 1;     // four consecutive n of D in one aligned access
constexpr int32_t DF_C_VEC = 2;     // ... of C
constexpr int32_t DF_KEPT_VEC = 4;  // ... of g, and 8: of u
constexpr int32_t DF_ROWS = 16;     // the columns of C and of every output contiguous
constexpr int32_t DF_ROWS4 = 32;    // ... and rows of them start on boundaries of four
constexpr int32_t DF_ROWS8 = 64;    // ... of eight, and are of 16-bit types

// tile configurations: rows of A x rows of B (for the gated pair, of both
// matrices together)
enum DenseTile : int32_t {
  DT_256x256 = 0,  // 4 waves, each 128 x 128
  DT_256x192 = 1,  // 4 waves, each 128 x 96
  DT_256x128 = 2,  // 4 waves, each 128 x 64
  DT_128x128 = 3,  // 4 waves, each 64 x 64; two workgroups to a CU, or one of the deep ring's
  DT_STREAM = 4,   // 32 or 64 rows of A, 4 waves that split K
  DT_SKINNY = 5,   // 16 rows of A, 8 waves that split K
};
constexpr int32_t kDenseSkinnyWaves = 8, kDenseStreamWaves = 4;
constexpr int32_t kRing = 5, kDeepRing = 9;  // operand K-tiles in the ring of the first four
struct DensePlan {
  int32_t tile;
  int32_t bm, bn;       // rows of A and of B of a workgroup
  int32_t threads, lds;
  int32_t stages;       // LDS K-tiles of a wave of DT_STREAM, operand K-tiles of a ring
  double us;            // what the model of dense_plan gives it
};
// `gated`: bn / 2 columns of the result to a workgroup
DensePlan dense_plan(bool gated, int64_t batch, int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_i8(const DenseParams& p, const DensePlan& plan, hipStream_t stream);
hipError_t launch_gated(const DenseParams& p, int32_t kind, const DensePlan& plan, hipStream_t stream);

// ---------------------------------------------------------------------------
// What the gated block's calls do ahead of their products (gated_prepare.hip),
// one launch.  16-bit matrices copied to rows of contiguous values: out row r
// (of `out_rs` values; columns [cols, width) zero) from x's row r, any strides.
// ---------------------------------------------------------------------------
struct PackParams {
  const uint16_t* x;
  uint16_t* out;
  int64_t rows, cols, width;   // rows 0: no copy; width a multiple of 8
  int64_t x_bs, x_rs, x_cs, out_bs, out_rs;  // out_rs, out_bs multiples of 8
  int32_t batch;
};

// dg = dh u act'(g) and du = dh act(g), each rounded to 16 bits, as rows
// (dg's columns at 0, du's at Fp of a row of 2 Fp) and as columns (row f of
// dg's transpose at t + f t_rs, of du's at t + t_us more); padding zero.
struct GatedSlopeParams {
  const uint16_t *g, *u, *dh;
  int64_t M, F, Fp, Mp;        // padded to multiples of 64
  int64_t g_bs, g_rs, g_cs, u_bs, u_rs, u_cs, dh_bs, dh_rs, dh_cs;
  uint16_t* rows;              // may be NULL; row m of batch b at rows + (b M + m) 2 Fp
  uint16_t* t;                 // may be NULL
  int64_t t_bs, t_rs, t_us;
  int32_t type, act, batch;    // batch 0: nothing to do
};
struct GatedPrepareParams {
  GatedSlopeParams slope;
  PackParams pack[3];
  int64_t first[5];            // workgroups of the slopes, the copies; set by gated_prepare_groups
};
constexpr int32_t kPrepareThreads = 256;
int64_t gated_prepare_groups(GatedPrepareParams* p);
hipError_t launch_gated_prepare(const GatedPrepareParams& p, hipStream_t stream);

// The products of the backward pass: 16-bit D = A B^T as DenseParams states it,
// D in kept[0]; with pairs (b_shift 1) matrix 2 i + s of the batch takes B's
// matrix i and goes to matrix i of kept[s].  One of them, or two in one launch:
// the first `first` workgroups are p[0]'s.
struct DensePair {
  DenseParams p[2];
  uint32_t first;
};
DensePlan dense_pair_plan(const DenseParams& p, const DenseParams& q);
hipError_t launch_gated_products(const DenseParams& p, int32_t kind, const DensePlan& plan, hipStream_t stream);
hipError_t launch_gated_products(const DensePair& p, int32_t kind, const DensePlan& plan, hipStream_t stream);

// The same products with B's rows (and, across, A's) contracted over: B is
// `parts` matrices (b[0], b[1]) of `rows` rows of N contiguous values one after
// the other, b_rs[0] bytes apart, N a multiple of 8, on 16-byte boundaries.  A: along its rows
// (K-contiguous, each part's values padded with zeros to a multiple of 64), or
// across, `rows` rows of M contiguous values, padded with zeros to a multiple of 64;
// the odd matrices of pairs a_second bytes on.
struct GradParams {
  DenseParams d;
  int64_t rows, a_second;
  int32_t parts;
  int32_t splits;  // launch_grad_few: workgroups that share the rows of B; more than one leave
  float* partial;  // their sums here, [split][batch][M][N]
};
// x's gradient, A along its rows, by the first `first` workgroups, and the weights'
struct GradPair {
  GradParams dx, dw;
  uint32_t first;
};
hipError_t launch_grad_ring(const GradParams& g, int32_t kind, bool across, hipStream_t stream);  // 256 x 256 tiles
hipError_t launch_grad_tiles(const GradParams& g, int32_t kind, bool across, hipStream_t stream); // 128 x 128 tiles
constexpr int32_t kFewRows = 64, kFewThreads = 512;
hipError_t launch_grad_few(const GradParams& g, int32_t kind, hipStream_t stream);  // x's, few rows: kFewRows x 128 tiles
hipError_t launch_grad_tiles(const GradPair& g, int32_t kind, hipStream_t stream);

template <int T>
struct OrthoElem {
  typedef uint16_t type;
};
template <>
struct OrthoElem<OT_F32> {
  typedef uint32_t type;
};

}  // namespace sl
