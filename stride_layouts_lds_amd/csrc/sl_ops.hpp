// sl_ops.hpp -- parameters and launchers of the operators next to the GEMM:
// block quantisation to E4M3, the block-scaled 8-bit product, and the
// orthogonalised update.  Shared by the host side (api_ops.cpp) and their
// kernel translation units.
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

template <int T>
struct OrthoElem {
  typedef uint16_t type;
};
template <>
struct OrthoElem<OT_F32> {
  typedef uint32_t type;
};

}  // namespace sl
