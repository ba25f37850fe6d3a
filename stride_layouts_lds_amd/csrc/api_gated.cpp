// api_gated.cpp -- host side of the gated feed-forward block and its backward
// pass, of the int8 form of sl_gemm and of sl_quantize_rows.  Every check runs
// before any HIP call.
#include <cmath>
#include <initializer_list>

#include "api_common.hpp"
#include "api_ops.hpp"
#include "sl_kernels.hpp"

namespace sl {

// The tile (dense.hpp), by the least time of a plain model: rounds of workgroups
// over the CUs times (start and end of a workgroup + K-tiles of 128 bytes x one's
// time), in us, fitted to calls with each tile forced.  Some of them, gated bf16
// (M x F, K 256 / 1024 / 4096; 256 x 256, 256 x 128, 128 x 128, streamed):
//   256 x 1024   14 26 73     9 16 42     6 10 26     5  7  13
//   512 x 1024   14 26 73     9 16 43     6 10 33     6  8  18
//   1000 x 2000  14 26 74     9 16 43     7 11 37     22 36 101
//   1000 x 2500  19 31 78     12 18 45    9 17 47     27 43 130
//   2048 x 2048  15 27 75     10 20 56    9 19 58     42 55 130
//   4096 x 2048  17 32 96     19 39 112   16 35 113   83 108 259
//   4096 x 8192  59 126 372   68 145 432  53 129 446  324 458 1586
// int8 (256 x 256, 256 x 192, 128 x 128): 4000 x 3000 x 256 / 2064 / 8192 16 14 13, 35 33 39,
// 83 79 93; 3000 x 3000 x 2048 31 26 29; 4096 x 6144 x 4096 100 89 96; 8192 x 8192 x 2048
// 133 155 141.  Up to 64 rows of A the streamed tiles read B once, and where that bounds the
// call they stay (int8 16 of 17 x 8192 x 4096 120 us, in larger tiles 126; 64 x 8192 x 4096 is
// read at 4.4 TB/s).  Elsewhere many workgroups only start and end (int8, streamed and in 128 x 128
// tiles: 16 of 17 x 8192 x 128 31 and 10, 16 of 64 x 8192 x 256 45 and 15, 16 of 16 x 8192 x 1024 61
// and 26; gated bf16 64 of 33 x 4096 x 64 148 and 35).  From 17 rows on a larger tile has to be
// a fifth better than streamed ones in parts of a round: a last round that is not full costs less than
// one (gated bf16 2 of 24 x 3744 x 1216 11 us streamed, by the model 15, and 13).
//
// A 128 x 128 tile alone on its CU waits for its copies where many K-tiles meet many
// others': the deep ring has two K-tiles more on their way (gated bf16 512 x 1024 x 4096 33 ->
// 27, 1000 x 1900 x 4096 37 -> 32, x 2048 23 -> 21; int8 2048 x 1024 x 8192 34 -> 28), and
// takes longer to fill where there are few (256 x 1024 x 2048 14.9 -> 15.7, 512 x 1024 x 1024
// 10.0 -> 10.4).
static DensePlan ring_plan(int32_t tile, int32_t bm, int32_t bn, int32_t slots) {
  return {tile, bm, bn, 256, slots * std::max(bm, bn) * 128, slots, 0.0};
}
// 128 x 128 tiles of a product (rows of B: N): alone on their CU the more of them the
// longer a K-tile takes, two to a CU by rounds; and 256 x 256 ones.
static double alone_k(double tiles, bool deep) { return 0.33 + (deep ? 0.1 : 0.2) * tiles / kCUs; }
static double dense_small_us(double tiles, double T, bool deep) {
  if (tiles > kCUs) return 2.4 + std::ceil(tiles / (2 * kCUs)) * (3.4 + 0.8 * T);
  return (deep ? 4.8 : 4.4) + alone_k(tiles, deep) * T;
}
static double dense_large_us(int64_t batch, int64_t M, int64_t N, int64_t K) {
  using host::ceil_div;
  const double tiles = (double)batch * (double)ceil_div(M, 256) * (double)ceil_div(N, 256);
  return std::ceil(tiles / kCUs) * (10.2 + 1.3 * (double)ceil_div(K, 128));
}
DensePlan dense_plan(bool gated, int64_t batch, int64_t M, int64_t N, int64_t K) {
  using host::ceil_div;
  const int64_t B = gated ? 2 * N : N;  // rows of B: a gated tile's columns of the result are half of its rows of B
  const double T = (double)ceil_div(K, 128);
  const int32_t bm = M <= 32 ? 32 : 64;
  const int32_t bn = batch * ceil_div(M, bm) * ceil_div(B, 64) >= kCUs ? 64 : 32;
  const int32_t stages = bm == 32 ? (bn == 32 ? 4 : 3) : (bn == 32 ? 3 : 2);
  DensePlan best = {DT_STREAM, bm, bn, kDenseStreamWaves * 64, kDenseStreamWaves * stages * (bm + bn) * 128, stages, 0.0};
  const double groups = (double)batch * (double)ceil_div(M, bm) * (double)ceil_div(B, bn), one = 5.0 + T * (bn == 64 ? 0.2 : 0.13);
  best.us = std::ceil(groups / kCUs) * one;
  double limit = M <= 64 ? 0.8 * std::max(1.0, groups / kCUs) * one : best.us;  // what a larger tile has to be below
  if (M <= 16) {
    const int32_t cols = gated || batch * ceil_div(N, 32) >= kCUs ? 32 : 16;
    const double rounds = (double)batch * (double)ceil_div(B, cols) / (2.0 * kCUs);  // two workgroups to a CU
    best = {DT_SKINNY, 16, cols, kDenseSkinnyWaves * 64, kDenseSkinnyWaves * cols / 16 * 1024, 0, std::ceil(rounds) * (3.0 + 0.1 * T)};
    limit = best.us;
  }
  const bool once = M <= 64 && best.us <= (double)batch * (double)B * (double)K / 4.5e6;  // one pass over B bounds it
  if (K == 0 || once) return best;
  auto tiles = [&](int64_t rows_a, int64_t rows_b) { return (double)batch * (double)ceil_div(M, rows_a) * (double)ceil_div(B, rows_b); };
  const double t2 = tiles(128, 128);
  const bool deep = t2 <= kCUs && t2 * T >= 3500.0;
  DensePlan large[4] = {ring_plan(DT_256x256, 256, 256, kRing), ring_plan(DT_256x192, 256, 192, kRing),
                        ring_plan(DT_256x128, 256, 128, kRing), ring_plan(DT_128x128, 128, 128, deep ? kDeepRing : kRing)};
  large[0].us = dense_large_us(batch, M, B, K);
  large[1].us = gated ? best.us : std::ceil(tiles(256, 192) / kCUs) * (8.6 + 1.1 * T);
  large[2].us = std::ceil(tiles(256, 128) / kCUs) * (7.0 + 0.77 * T);
  large[3].us = dense_small_us(t2, T, deep);
  for (const DensePlan& t : large)
    if (t.us < limit) best = t, limit = t.us;
  return best;
}

// 128 x 128 tiles of the backward pass on operands as they lie: transposing reads take
// LDS twice as long, which bounds these tiles (1024 x 2048 x 1024's dx 37 us, with
// copies, made in 3 us more, 18; 8 of 300 x 1000 x 520's 21 and 15.5; two to a CU 2048 tiles of 8
// K-tiles 43 both ways).
static double lying_k(double tiles) { return 0.5 + 0.11 * tiles / kCUs; }
static double grad_tiles_us(double tiles, double T) {
  return tiles > kCUs ? 2.4 + std::ceil(tiles / (2 * kCUs)) * (3.4 + 0.85 * T) : 4.4 + lying_k(tiles) * T;
}

// Two products in one launch, by the same model: the workgroups' times over the
// slots there are, or the longest one's.
namespace {
struct PairTile {
  DensePlan plan;
  double slots, start, k;
};
double pair_us(const PairTile& t, const DenseParams& p, const DenseParams& q, bool lying) {
  using host::ceil_div;
  double work[2], T[2], groups = 0.0;
  for (int i = 0; i < 2; ++i) {
    const DenseParams& x = i ? q : p;
    if (x.K == 0 && t.plan.tile != DT_STREAM) return 1e30;  // the others want a K-tile
    const double n = (double)x.batch * (double)ceil_div(x.M, t.plan.bm) * (double)ceil_div(x.N, t.plan.bn);
    T[i] = (double)ceil_div(x.K, 128), work[i] = n * (t.start + t.k * T[i]) / t.slots, groups += n;
  }
  double longest = 0.0;
  for (int i = 0; i < 2; ++i) {
    double k = t.k;
    if (t.plan.tile == DT_128x128 && groups <= kCUs) k = lying ? lying_k(groups) : alone_k(groups, false);
    // as they lie: faster while no neighbour is there (400 x 1000 x 2304's two 30 us, 512 x 8192 x 4096's 260)
    else if (lying) k = 0.65 + 0.35 * std::min(1.0, work[1 - i] / (t.start + 0.65 * T[i]));
    longest = std::max(longest, t.start + k * T[i]);
  }
  return std::max(work[0] + work[1], longest);
}
PairTile pair_128x128() { return {ring_plan(DT_128x128, 128, 128, kRing), 2 * kCUs, 4.4, 0.8}; }
}  // namespace
DensePlan dense_pair_plan(const DenseParams& p, const DenseParams& q) {
  const PairTile tiles[6] = {{ring_plan(DT_256x256, 256, 256, kRing), kCUs, 10.2, 1.3},
                             {ring_plan(DT_256x128, 256, 128, kRing), kCUs, 7.0, 0.77},
                             pair_128x128(),
                             {{DT_STREAM, 64, 64, 256, 4 * 2 * 128 * 128, 2, 0.0}, kCUs, 5.0, 0.2},
                             {{DT_STREAM, 64, 32, 256, 4 * 3 * 96 * 128, 3, 0.0}, kCUs, 5.0, 0.13},
                             {{DT_STREAM, 32, 32, 256, 4 * 4 * 64 * 128, 4, 0.0}, kCUs, 4.5, 0.1}};
  DensePlan best = tiles[0].plan;
  best.us = 1e300;
  for (const PairTile& t : tiles) {
    const double cost = pair_us(t, p, q, false);
    if (cost < best.us) best = t.plan, best.us = cost;
  }
  return best;
}

namespace host {

// K (and the batch's stride) of rows that the kernels read as they lie
static bool rows_ready(const View& v, int64_t batch, int64_t es) {
  const int64_t vec = 16 / es;
  return (v.cs == 1 || v.cols <= 1) && v.cols % vec == 0 && (v.rows <= 1 || v.rs % vec == 0) && (uintptr_t)v.t->data % 16 == 0 &&
         (v.t->layout.rank == 2 || batch <= 1 || v.bs % vec == 0) && ((std::min<int64_t>(v.rows, 256) - 1) * v.rs + v.cols) * es < kLim;
}
static bool quad_rows(const View& v, int64_t batch) {
  return v.cs == 1 && (v.rows <= 1 || v.rs % 4 == 0) && (uintptr_t)v.t->data % (4 * elem_size(v.t->dtype)) == 0 &&
         (batch <= 1 || batch_stride(v) % 4 == 0);
}

// how a product's kernel may write (and read C) along the rows of these, all of one type
static int32_t row_flags(std::initializer_list<const View*> outs, int64_t batch) {
  bool rows = true, four = true, eight = true;
  for (const View* v : outs) {
    rows = rows && v->cs == 1, four = four && quad_rows(*v, batch);
    eight = eight && elem_size(v->t->dtype) == 2 && (v->rows <= 1 || v->rs % 8 == 0) && (uintptr_t)v->t->data % 16 == 0 &&
            (batch <= 1 || batch_stride(*v) % 8 == 0);
  }
  return !rows ? 0 : DF_ROWS | (four ? DF_ROWS4 : 0) | (four && eight ? DF_ROWS8 : 0);
}

// one scale per row: (batch?, rows, 1) f32
static sl_status scale_view(const char* name, const sl_tensor& t, int64_t rows, int64_t batch, View* v) {
  sl_status s;
  if (t.dtype != SL_F32) return fail(SL_ERR_DTYPE, "%s must be f32", name);
  if ((s = make_view(name, t, v)) != SL_OK) return s;
  if (v->rows != rows || v->cols != 1)
    return fail(SL_ERR_SHAPE, "%s is (%lld,%lld), expected (%lld,1)", name, (long long)v->rows, (long long)v->cols, (long long)rows);
  if (t.layout.rank == 3 && v->batch != batch)
    return fail(SL_ERR_SHAPE, "%s has batch %lld, expected %lld", name, (long long)v->batch, (long long)batch);
  return SL_OK;
}

constexpr int64_t kInt8MaxK = 131072;  // 128 x 128 x K < 2^31

// the tiles of a plan in p and whether they fit a grid
static sl_status place_tiles(DenseParams* p, const DensePlan& t, bool gated) {
  const int64_t cols = gated ? t.bn / 2 : t.bn;
  const int64_t tm = ceil_div(p->M, t.bm), tn = ceil_div(p->N, cols);
  if (!grid_fits(p->batch, tm, tn, t.threads))
    return fail(SL_ERR_SHAPE, "too many output tiles (batch %d of %lld x %lld)", p->batch, (long long)tm, (long long)tn);
  p->tiles_m = (int32_t)tm, p->tiles_n = (int32_t)tn, p->group_m = 8;
  p->k_tiles = (int32_t)ceil_div(p->K, 128);
  return SL_OK;
}

sl_status plan_int8(const sl_gemm_args* args, RowsPlan* out) {
  g_msg.clear();
  if (args->b.dtype != SL_I8) return fail(SL_ERR_DTYPE, "b must be i8 when a is");
  const int32_t type = op_type(args->d.dtype);
  if (type < 0) return fail(SL_ERR_DTYPE, "d must be f16, bf16 or f32");
  const bool has_c = args->c.data != nullptr;
  if (has_c && args->c.dtype != args->d.dtype) return fail(SL_ERR_DTYPE, "c must have d's dtype");
  View A, B, C{}, D, SA, SB;
  sl_status s;
  if ((s = make_view("a", args->a, &A)) != SL_OK) return s;
  if ((s = make_view("b", args->b, &B)) != SL_OK) return s;
  if ((s = make_view("d", args->d, &D)) != SL_OK) return s;
  if (has_c && (s = make_view("c", args->c, &C)) != SL_OK) return s;
  const int64_t batch = D.batch, M = A.rows, K = A.cols, N = B.rows;
  if (B.cols != K) return fail(SL_ERR_SHAPE, "b is (%lld,%lld) but a has K=%lld", (long long)B.rows, (long long)B.cols, (long long)K);
  if (D.rows != M || D.cols != N)
    return fail(SL_ERR_SHAPE, "d is (%lld,%lld), expected (%lld,%lld)", (long long)D.rows, (long long)D.cols, (long long)M, (long long)N);
  if (has_c && (C.rows != M || C.cols != N))
    return fail(SL_ERR_SHAPE, "c is (%lld,%lld), expected (%lld,%lld)", (long long)C.rows, (long long)C.cols, (long long)M, (long long)N);
  if ((s = scale_view("sfa", args->sfa, M, batch, &SA)) != SL_OK) return s;
  if ((s = scale_view("sfb", args->sfb, N, batch, &SB)) != SL_OK) return s;
  const View* all[6] = {&A, &B, has_c ? &C : nullptr, &D, &SA, &SB};
  const char* names[6] = {"a", "b", "c", "d", "sfa", "sfb"};
  for (int i = 0; i < 3; ++i)
    if (all[i] && all[i]->t->layout.rank == 3 && all[i]->batch != batch)
      return fail(SL_ERR_SHAPE, "%s has batch %lld, d has %lld", names[i], (long long)all[i]->batch, (long long)batch);
  if (M >= kLim || N >= kLim || batch >= kLim) return fail(SL_ERR_SHAPE, "a dimension exceeds 2^31-1");
  if (K >= kInt8MaxK) return fail(SL_ERR_SHAPE, "K is %lld, below %lld are summed exactly", (long long)K, (long long)kInt8MaxK);
  RowsPlan& P = *out;
  memset(&P, 0, sizeof P);
  P.pub.kernel = K_I8;
  P.pub.batch = batch, P.pub.m = M, P.pub.n = N, P.pub.k = K;
  P.pub.split_k = 1;
  P.empty = batch == 0 || M == 0 || N == 0;
  if (P.empty) return SL_OK;
  for (int i = 0; i < 6; ++i) {
    if (!all[i] || (!all[i]->t->data && i < 2 && K == 0)) continue;
    if ((s = check_data(names[i], *all[i]->t)) != SL_OK) return s;
  }
  if (!injective(D, batch)) return fail(SL_ERR_LAYOUT, "d's strides map distinct elements to one address");
  for (int i = 0; i < 6; ++i) {
    if (!all[i] || i == 3 || (i < 2 && K == 0)) continue;
    if (i == 2 && args->c.data == args->d.data && same_layout(args->c, args->d)) continue;
    if (overlap(*all[i], D, batch)) return fail(SL_ERR_ALIAS, "d overlaps %s", names[i]);
  }
  if (K > 0 && (K % 16 != 0 || !code_rows(A, batch) || !code_rows(B, batch)))
    return fail(SL_ERR_LAYOUT, "i8 operands must be K-contiguous with 16-byte aligned rows and K %% 16 == 0");
  for (const View* X : {&A, &B})
    if ((std::min<int64_t>(X->rows, 256) - 1) * X->rs + K >= kLim)
      return fail(SL_ERR_SHAPE, "a 256-row tile of an operand spans 2^31 bytes or more");
  DenseParams& p = P.p;
  p.a = (const uint8_t*)args->a.data, p.b[0] = (const uint8_t*)args->b.data;
  p.a_rs = A.rs, p.a_bs = batch_stride(A), p.b_rs[0] = B.rs, p.b_bs[0] = batch_stride(B);
  p.M = M, p.N = N, p.K = K;
  p.sa = (const float*)args->sfa.data, p.sb[0] = (const float*)args->sfb.data;
  p.sa_rs = SA.rs, p.sa_bs = batch_stride(SA), p.sb_rs[0] = SB.rs, p.sb_bs[0] = batch_stride(SB);
  p.c = has_c ? args->c.data : nullptr, p.d = args->d.data;
  if (has_c) p.c_rs = C.rs, p.c_cs = C.cs, p.c_bs = batch_stride(C);
  p.d_rs = D.rs, p.d_cs = D.cs, p.d_bs = batch_stride(D);
  p.type = type, p.batch = (int32_t)batch;
  p.flags = (quad_rows(D, batch) ? DF_D_VEC : 0) | (has_c && quad_rows(C, batch) ? DF_C_VEC : 0) |
            row_flags({&D, has_c ? &C : &D}, batch);
  P.tile = dense_plan(false, batch, M, N, K);
  if ((s = place_tiles(&p, P.tile, false)) != SL_OK) return s;
  P.pub.a_load = P.pub.b_load = LOAD_KVEC;
  P.pub.tile_m = P.tile.bm, P.pub.tile_n = P.tile.bn, P.pub.tile_k = 128;
  P.pub.threads = P.tile.threads, P.pub.lds_bytes = P.tile.lds;
  P.pub.workgroups = batch * p.tiles_m * p.tiles_n;
  return SL_OK;
}

sl_status run_int8(const sl_gemm_args* args, void* stream) {
  RowsPlan P;
  sl_status s = plan_int8(args, &P);
  if (s != SL_OK) return s;
  if (P.empty) return SL_OK;
  if ((s = check_arch()) != SL_OK) return s;
  const hipError_t e = launch_gemm_i8(P.p, P.tile, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SL_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return SL_OK;
}

}  // namespace host
}  // namespace sl

using namespace sl::host;

extern "C" {

sl_status sl_quantize_rows(const sl_quantize_rows_args* args, void* stream) {
  g_msg.clear();
  if (!args) return fail(SL_ERR_NULL, "args is NULL");
  const int32_t type = op_type(args->x.dtype);
  if (type < 0) return fail(SL_ERR_DTYPE, "x must be f16, bf16 or f32");
  if (args->q.dtype != SL_I8) return fail(SL_ERR_DTYPE, "q must be i8");
  View X, Q, S;
  sl_status s;
  if ((s = make_view("x", args->x, &X)) != SL_OK) return s;
  if ((s = make_view("q", args->q, &Q)) != SL_OK) return s;
  if ((s = scale_view("s", args->s, X.rows, X.batch, &S)) != SL_OK) return s;
  const int64_t batch = X.batch, R = X.rows, C = X.cols;
  if (Q.batch != batch || S.batch != batch) return fail(SL_ERR_SHAPE, "q and s must have x's batch of %lld", (long long)batch);
  if (R >= kLim - 128 || C >= kLim - 128 || batch >= kLim) return fail(SL_ERR_SHAPE, "a dimension exceeds 2^31-129");
  if (Q.rows != R || Q.cols < C || Q.cols > 128 * ceil_div(C, 128))
    return fail(SL_ERR_SHAPE, "q is (%lld,%lld), expected %lld rows of %lld to %lld codes", (long long)Q.rows, (long long)Q.cols,
                (long long)R, (long long)C, (long long)(128 * ceil_div(C, 128)));
  if (batch == 0 || R == 0) return SL_OK;
  if ((s = check_data("s", args->s)) != SL_OK) return s;
  if (!injective(S, batch)) return fail(SL_ERR_LAYOUT, "s's strides map distinct elements to one address");
  if (C > 0) {
    if ((s = check_data("x", args->x)) != SL_OK) return s;
    if ((s = check_data("q", args->q)) != SL_OK) return s;
    if (!code_rows(Q, batch)) return fail(SL_ERR_LAYOUT, "q must be contiguous along its last axis with 16-byte aligned rows");
    if (!injective(Q, batch)) return fail(SL_ERR_LAYOUT, "q's strides map distinct elements to one address");
    if (overlap(Q, X, batch)) return fail(SL_ERR_ALIAS, "q overlaps x");
    if (overlap(S, X, batch)) return fail(SL_ERR_ALIAS, "s overlaps x");
    if (overlap(S, Q, batch)) return fail(SL_ERR_ALIAS, "s overlaps q");
  }
  sl::QuantizeRowsParams p{};
  p.x = args->x.data, p.q = (int8_t*)args->q.data, p.s = (float*)args->s.data;
  p.rows = R, p.cols = C, p.x_bs = batch_stride(X), p.x_rs = X.rs, p.x_cs = X.cs;
  p.q_cols = Q.cols, p.q_bs = batch_stride(Q), p.q_rs = Q.rs, p.s_bs = batch_stride(S), p.s_rs = S.rs;
  p.type = type, p.batch = (int32_t)batch;
  if (!grid_fits(batch, R, 1, 1) || !grid_fits(sl::quantize_rows_groups(p), 1, 1, sl::quantize_rows_threads(p)))
    return fail(SL_ERR_SHAPE, "too many rows (batch %lld of %lld)", (long long)batch, (long long)R);
  if ((s = check_arch()) != SL_OK) return s;
  const hipError_t e = sl::launch_quantize_rows(p, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SL_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return SL_OK;
}

}  // extern "C"

namespace {

constexpr int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// the caller's workspace against what a plan needs and the operands
sl_status check_workspace(void* ws, int64_t given, int64_t needed, const View* const* views, const char* const* names, int n) {
  if (!needed) return SL_OK;
  if (!ws) return fail(SL_ERR_NULL, "workspace is NULL, %lld bytes are needed", (long long)needed);
  if (given < needed) return fail(SL_ERR_SHAPE, "workspace of %lld bytes, %lld are needed", (long long)given, (long long)needed);
  const uintptr_t lo = (uintptr_t)ws, hi = lo + (uintptr_t)needed;
  if (lo % 16) return fail(SL_ERR_ALIGN, "workspace is not on a 16-byte boundary");
  for (int i = 0; i < n; ++i) {
    if (!views[i] || !views[i]->t->data) continue;
    uintptr_t l, h;
    byte_range(*views[i], views[i]->batch, &l, &h);
    if (l < hi && lo < h) return fail(SL_ERR_ALIAS, "workspace overlaps %s", names[i]);
  }
  return SL_OK;
}

bool has_values(const View& v) { return v.batch > 0 && v.rows > 0 && v.cols > 0; }

// Two views hold no element in common: their address ranges are apart, or they
// are alike and one lies between the rows or columns of the other (the two
// halves of a matrix that holds both).
bool apart(const View& a, const View& b) {
  uintptr_t al, ah, bl, bh;
  byte_range(a, a.batch, &al, &ah);
  byte_range(b, b.batch, &bl, &bh);
  if (ah <= bl || bh <= al) return true;
  if (a.t->dtype != b.t->dtype || a.batch != b.batch || a.rows != b.rows || a.cols != b.cols || a.bs != b.bs || a.rs != b.rs || a.cs != b.cs)
    return false;
  const int64_t es = elem_size(a.t->dtype);
  const uintptr_t off = al > bl ? al - bl : bl - al;
  if (off % es) return false;
  struct Dim {
    int64_t n, s;
  } d[4] = {{a.batch, a.bs}, {a.rows, a.rs}, {a.cols, a.cs}, {2, (int64_t)(off / es)}};
  std::sort(d, d + 4, [](const Dim& x, const Dim& y) { return x.s < y.s; });
  int64_t span = 0;
  for (const Dim& x : d) {
    if (x.n <= 1) continue;
    if (x.s <= span) return false;
    span += x.s * (x.n - 1);
  }
  return true;
}

// The data of every view that is there and holds values, and the outputs (from
// `first` on) apart from everything else.
sl_status check_operands(const View* const* views, const char* const* names, int n, int first) {
  sl_status s;
  for (int i = 0; i < n; ++i)
    if (views[i] && has_values(*views[i]) && (s = check_data(names[i], *views[i]->t)) != SL_OK) return s;
  for (int i = first; i < n; ++i) {
    if (!views[i] || !has_values(*views[i])) continue;
    if (!injective(*views[i], views[i]->batch)) return fail(SL_ERR_LAYOUT, "%s's strides map distinct elements to one address", names[i]);
    for (int j = 0; j < i; ++j) {
      if (!views[j] || !has_values(*views[j])) continue;
      if (!apart(*views[i], *views[j])) return fail(SL_ERR_ALIAS, "%s overlaps %s", names[i], names[j]);
    }
  }
  return SL_OK;
}

bool valid_activation(int32_t a) { return a >= SL_SILU && a <= SL_RELU; }

// shape (batch?, rows, cols) of a view: rank 3 with this batch, or rank 2 where
// that is allowed
sl_status check_shape(const char* name, const View& v, int64_t batch, int64_t rows, int64_t cols, bool shared, bool rank3) {
  if (v.rows != rows || v.cols != cols)
    return fail(SL_ERR_SHAPE, "%s is (%lld,%lld), expected (%lld,%lld)", name, (long long)v.rows, (long long)v.cols, (long long)rows,
                (long long)cols);
  if (v.t->layout.rank == 2 ? rank3 && !shared : !rank3 || v.batch != batch)
    return fail(SL_ERR_SHAPE, "%s has another batch than the result's %lld", name, (long long)batch);
  return SL_OK;
}

// A batch whose matrices follow each other is one matrix of all their rows.
bool follows(const View& v) { return v.bs == v.rows * v.rs || v.rows == 1; }
View flattened(View v) {
  if (v.rows == 1) v.rs = v.bs;
  v.rows *= v.batch, v.batch = 1, v.bs = 0;
  return v;
}

struct GatedPlan {
  sl::DenseParams p;
  sl::DensePlan tile;
  int32_t kind;
  sl::GatedPrepareParams prepare;  // copies of x, w_gate, w_up; rows 0: read as it lies
  int64_t offset[3], ws_bytes;
  bool empty;
  View v[9];
};

// batch strides count for rank 3 alone
int64_t bstride(const View& v) { return v.batch > 1 ? v.bs : 0; }

sl_status plan_gated(const sl_gated_args* args, GatedPlan* out) {
  g_msg.clear();
  if (!args) return fail(SL_ERR_NULL, "args is NULL");
  GatedPlan& P = *out;
  memset((void*)&P, 0, sizeof P);
  const bool i8 = args->x.dtype == SL_I8;
  if (args->x.dtype != SL_F16 && args->x.dtype != SL_BF16 && !i8) return fail(SL_ERR_DTYPE, "x must be f16, bf16 or i8");
  if (args->w_gate.dtype != args->x.dtype || args->w_up.dtype != args->x.dtype)
    return fail(SL_ERR_DTYPE, "w_gate and w_up must have x's dtype");
  const int32_t type = op_type(args->h.dtype);
  if (type < 0 || (!i8 && args->h.dtype != args->x.dtype))
    return fail(SL_ERR_DTYPE, i8 ? "h must be f16, bf16 or f32" : "h must have x's dtype");
  const bool keep = args->gate.data || args->up.data;
  if (keep && (args->gate.dtype != args->h.dtype || args->up.dtype != args->h.dtype))
    return fail(SL_ERR_DTYPE, "gate and up must have h's dtype");
  if (!i8 && (args->sx.data || args->s_gate.data || args->s_up.data)) return fail(SL_ERR_DTYPE, "scales given for 16-bit operands");
  if (!valid_activation(args->activation)) return fail(SL_ERR_ARG, "activation %d", args->activation);
  enum { X, WG, WU, SX, SG, SU, H, G, U, COUNT };
  static const char* const names[COUNT] = {"x", "w_gate", "w_up", "sx", "s_gate", "s_up", "h", "gate", "up"};
  const sl_tensor* t[COUNT] = {&args->x, &args->w_gate, &args->w_up, &args->sx, &args->s_gate, &args->s_up, &args->h, &args->gate, &args->up};
  View* v = P.v;
  const View* used[COUNT];
  sl_status s;
  for (int i = 0; i < COUNT; ++i) {
    used[i] = nullptr;
    if ((i >= SX && i <= SU && !i8) || (i >= G && !keep)) continue;
    if ((s = make_view(names[i], *t[i], &v[i])) != SL_OK) return s;
    used[i] = &v[i];
  }
  const bool rank3 = args->h.layout.rank == 3;
  const int64_t batch = v[H].batch, M = v[H].rows, F = v[H].cols, K = v[X].cols;
  if ((s = check_shape("x", v[X], batch, M, K, true, rank3)) != SL_OK) return s;
  for (int i : {(int)WG, (int)WU})
    if ((s = check_shape(names[i], v[i], batch, F, K, true, rank3)) != SL_OK) return s;
  for (int i : {(int)G, (int)U})
    if (used[i] && (s = check_shape(names[i], v[i], batch, M, F, false, rank3)) != SL_OK) return s;
  if (i8) {
    if ((s = scale_view("sx", args->sx, M, batch, &v[SX])) != SL_OK) return s;
    if ((s = scale_view("s_gate", args->s_gate, F, batch, &v[SG])) != SL_OK) return s;
    if ((s = scale_view("s_up", args->s_up, F, batch, &v[SU])) != SL_OK) return s;
  }
  if (M >= kLim || F >= kLim / 2 || K >= kLim / 2 || batch >= kLim) return fail(SL_ERR_SHAPE, "a dimension exceeds its limit");
  if (i8 && K >= kInt8MaxK) return fail(SL_ERR_SHAPE, "K is %lld, below %lld are summed exactly", (long long)K, (long long)kInt8MaxK);
  P.empty = batch == 0 || M == 0 || F == 0;
  if (P.empty) return SL_OK;
  if (keep && (!args->gate.data || !args->up.data)) return fail(SL_ERR_NULL, "gate and up are kept together");
  if ((s = check_operands(used, names, COUNT, H)) != SL_OK) return s;

  // one matrix of all tokens where the weights are shared: a token of each of
  // many sequences is a batch of one row each
  auto shared = [&](int i) { return !used[i] || v[i].t->layout.rank == 2 || v[i].bs == 0; };
  bool flat = batch > 1 && shared(WG) && shared(WU) && shared(SG) && shared(SU) && batch * M < kLim;
  for (int i : {(int)X, (int)SX, (int)H, (int)G, (int)U}) flat = flat && (!used[i] || (v[i].t->layout.rank == 3 && follows(v[i])));
  View w[COUNT];
  for (int i = 0; i < COUNT; ++i) {
    w[i] = v[i];
    if (!used[i]) continue;
    if (flat && (i == X || i == SX || i >= H)) w[i] = flattened(v[i]);
    else if (flat) w[i].batch = 1, w[i].bs = 0;
    else if (w[i].t->layout.rank == 2) w[i].bs = 0;
  }
  sl::DenseParams& p = P.p;
  p.batch = (int32_t)(flat ? 1 : batch);
  p.M = flat ? batch * M : M, p.N = F;
  const int64_t es = i8 ? 1 : 2;
  int64_t k_bytes = K * es;
  const uint8_t* data[3] = {(const uint8_t*)args->x.data, (const uint8_t*)args->w_gate.data, (const uint8_t*)args->w_up.data};
  int64_t rs[3], bs[3];
  for (int i = 0; i < 3; ++i) rs[i] = w[i].rs * es, bs[i] = bstride(w[i]) * es;
  if (i8) {
    for (int i = 0; i < 3; ++i)
      if (K > 0 && (K % 16 != 0 || !code_rows(w[i], w[i].batch)))
        return fail(SL_ERR_LAYOUT, "i8 operands must be K-contiguous with 16-byte aligned rows and K %% 16 == 0");
    for (int i = 0; i < 3; ++i)
      if ((std::min<int64_t>(w[i].rows, 256) - 1) * w[i].rs + K >= kLim)
        return fail(SL_ERR_SHAPE, "a 256-row tile of an operand spans 2^31 bytes or more");
  } else if (K > 0) {
    const int64_t Kp = round_up(K, 8);
    for (int i = 0; i < 3; ++i) {
      if (rows_ready(w[i], w[i].batch, 2)) continue;
      if ((std::min<int64_t>(w[i].rows, 256)) * Kp * 2 >= kLim) return fail(SL_ERR_SHAPE, "a 256-row tile of an operand spans 2^31 bytes or more");
      sl::PackParams& q = P.prepare.pack[i];
      q.x = (const uint16_t*)data[i];
      q.rows = w[i].rows, q.cols = K, q.width = Kp;
      q.batch = (int32_t)(bstride(w[i]) ? w[i].batch : 1);
      q.x_bs = bstride(w[i]), q.x_rs = w[i].rs, q.x_cs = w[i].cs, q.out_rs = Kp, q.out_bs = w[i].rows * Kp;
      if (!grid_fits(q.batch, ceil_div(q.rows, 64), ceil_div(Kp, 64), sl::kPrepareThreads))
        return fail(SL_ERR_SHAPE, "%s is too large to be copied", names[i]);
      P.offset[i] = P.ws_bytes;
      P.ws_bytes += round_up(q.batch * q.out_bs * 2, 256);
      rs[i] = Kp * 2, bs[i] = q.batch > 1 ? q.out_bs * 2 : 0;
    }
    k_bytes = Kp * 2;
  }
  if (!grid_fits(sl::gated_prepare_groups(&P.prepare), 1, 1, sl::kPrepareThreads))
    return fail(SL_ERR_SHAPE, "the operands are too large to be copied");
  p.K = k_bytes;
  p.a = data[0], p.a_rs = rs[0], p.a_bs = bs[0];
  for (int i = 0; i < 2; ++i) p.b[i] = data[1 + i], p.b_rs[i] = rs[1 + i], p.b_bs[i] = bs[1 + i];
  if (i8) {
    p.sa = (const float*)args->sx.data, p.sa_rs = w[SX].rs, p.sa_bs = bstride(w[SX]);
    p.sb[0] = (const float*)args->s_gate.data, p.sb_rs[0] = w[SG].rs, p.sb_bs[0] = bstride(w[SG]);
    p.sb[1] = (const float*)args->s_up.data, p.sb_rs[1] = w[SU].rs, p.sb_bs[1] = bstride(w[SU]);
  }
  p.d = args->h.data, p.d_rs = w[H].rs, p.d_cs = w[H].cs, p.d_bs = bstride(w[H]);
  p.flags = quad_rows(w[H], p.batch) ? sl::DF_D_VEC : 0;
  p.flags |= row_flags({&w[H], &w[keep ? G : H], &w[keep ? U : H]}, p.batch);
  if (keep)
    for (int i = 0; i < 2; ++i) {
      const View& k = w[G + i];
      p.kept[i] = t[G + i]->data, p.kept_rs[i] = k.rs, p.kept_cs[i] = k.cs, p.kept_bs[i] = bstride(k);
      if (quad_rows(k, p.batch)) p.flags |= sl::DF_KEPT_VEC << i;
    }
  p.type = type, p.act = args->activation - SL_SILU;
  P.kind = i8 ? sl::EK_I8 : args->x.dtype == SL_F16 ? sl::EK_F16 : sl::EK_BF16;
  P.tile = sl::dense_plan(true, p.batch, p.M, F, k_bytes);
  return place_tiles(&p, P.tile, true);
}

}  // namespace

extern "C" {

sl_status sl_gated_workspace_bytes(const sl_gated_args* args, int64_t* bytes) {
  g_msg.clear();
  if (!bytes) return fail(SL_ERR_NULL, "bytes is NULL");
  GatedPlan P;
  const sl_status s = plan_gated(args, &P);
  if (s == SL_OK) *bytes = P.ws_bytes;
  return s;
}

sl_status sl_gated(const sl_gated_args* args, void* stream) {
  GatedPlan P;
  sl_status s = plan_gated(args, &P);
  if (s != SL_OK) return s;
  if (P.empty) return SL_OK;
  const bool i8 = args->x.dtype == SL_I8, keep = args->gate.data != nullptr;
  const View* views[9] = {&P.v[0], &P.v[1], &P.v[2], i8 ? &P.v[3] : nullptr, i8 ? &P.v[4] : nullptr, i8 ? &P.v[5] : nullptr, &P.v[6],
                          keep ? &P.v[7] : nullptr, keep ? &P.v[8] : nullptr};
  const char* const names[9] = {"x", "w_gate", "w_up", "sx", "s_gate", "s_up", "h", "gate", "up"};
  if ((s = check_workspace(args->workspace, args->workspace_bytes, P.ws_bytes, views, names, 9)) != SL_OK) return s;
  if ((s = check_arch()) != SL_OK) return s;
  for (int i = 0; i < 3; ++i) {
    if (!P.prepare.pack[i].rows) continue;
    P.prepare.pack[i].out = (uint16_t*)((char*)args->workspace + P.offset[i]);
    (i == 0 ? P.p.a : P.p.b[i - 1]) = (const uint8_t*)P.prepare.pack[i].out;
  }
  hipError_t e = sl::launch_gated_prepare(P.prepare, (hipStream_t)stream);
  if (e == hipSuccess) e = sl::launch_gated(P.p, P.kind, P.tile, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SL_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return SL_OK;
}

}  // extern "C"

namespace {

struct BackwardPlan {
  sl::GatedPrepareParams prepare;  // copies: x's transpose, w_gate's, w_up's
  sl::GradParams dx, dw;
  sl::DensePlan dx_tile, dw_tile;
  bool pair;                       // both in one launch
  int32_t kind;
  bool want_dx, want_dw, launch;
  bool dx_lies, dw_lies;           // on operands as they lie (launch_grad_ring, launch_grad_tiles)
  bool dx_few;                     // on launch_grad_few, as they lie too
  int64_t off_partial;
  int64_t off_rows, off_t, off_xt, off_wt, ws_bytes;
  View v[9];
};

sl_status plan_backward(const sl_gated_backward_args* args, BackwardPlan* out) {
  g_msg.clear();
  if (!args) return fail(SL_ERR_NULL, "args is NULL");
  BackwardPlan& P = *out;
  memset((void*)&P, 0, sizeof P);
  const int32_t dt = args->dh.dtype;
  if (dt != SL_F16 && dt != SL_BF16) return fail(SL_ERR_DTYPE, "dh must be f16 or bf16");
  enum { DH, X, WG, WU, G, U, DX, DWG, DWU, COUNT };
  static const char* const names[COUNT] = {"dh", "x", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up"};
  const sl_tensor* t[COUNT] = {&args->dh, &args->x, &args->w_gate, &args->w_up, &args->gate, &args->up, &args->dx, &args->dw_gate, &args->dw_up};
  View* v = P.v;
  const View* used[COUNT];
  sl_status s;
  P.want_dx = args->dx.data, P.want_dw = args->dw_gate.data || args->dw_up.data;
  if (!valid_activation(args->activation)) return fail(SL_ERR_ARG, "activation %d", args->activation);
  for (int i = 0; i < COUNT; ++i) {
    used[i] = nullptr;
    if ((i == DX && !P.want_dx) || (i >= DWG && !P.want_dw)) continue;
    if (t[i]->dtype != dt) return fail(SL_ERR_DTYPE, "%s must have dh's dtype", names[i]);
    if ((s = make_view(names[i], *t[i], &v[i])) != SL_OK) return s;
    used[i] = &v[i];
  }
  const bool rank3 = args->dh.layout.rank == 3;
  const int64_t batch = v[DH].batch, M = v[DH].rows, F = v[DH].cols, K = v[X].cols;
  if ((s = check_shape("x", v[X], batch, M, K, false, rank3)) != SL_OK) return s;
  for (int i : {(int)WG, (int)WU})
    if ((s = check_shape(names[i], v[i], batch, F, K, true, rank3)) != SL_OK) return s;
  for (int i : {(int)G, (int)U})
    if ((s = check_shape(names[i], v[i], batch, M, F, false, rank3)) != SL_OK) return s;
  if (v[WG].t->layout.rank != v[WU].t->layout.rank) return fail(SL_ERR_SHAPE, "w_gate and w_up must have one rank");
  const bool one_weight = v[WG].t->layout.rank == 2;  // for every matrix of the batch
  if (P.want_dx && (s = check_shape("dx", v[DX], batch, M, K, false, rank3)) != SL_OK) return s;
  for (int i : {(int)DWG, (int)DWU})
    if (P.want_dw && (s = check_shape(names[i], v[i], batch, F, K, false, !one_weight)) != SL_OK) return s;
  if (M >= kLim / 2 || F >= kLim / 4 || K >= kLim / 2 || batch >= kLim) return fail(SL_ERR_SHAPE, "a dimension exceeds its limit");
  if (P.want_dw && K > 0 && F > 0 && (!args->dw_gate.data || !args->dw_up.data)) return fail(SL_ERR_NULL, "dw_gate and dw_up are wanted together");
  P.want_dx = P.want_dx && has_values(v[DX]);
  P.want_dw = P.want_dw && has_values(v[DWG]);
  if (!P.want_dx && !P.want_dw) return SL_OK;
  P.launch = true;
  if ((s = check_operands(used, names, COUNT, DX)) != SL_OK) return s;

  // one matrix of all tokens where the weights are shared
  bool flat = rank3 && one_weight && batch > 0 && batch * M < kLim / 2;
  for (int i : {(int)DH, (int)X, (int)G, (int)U, (int)DX}) flat = flat && (!used[i] || follows(v[i]));
  View w[COUNT];
  for (int i = 0; i < COUNT; ++i) {
    w[i] = v[i];
    if (!used[i]) continue;
    if (flat && i != WG && i != WU && i < DWG) w[i] = flattened(v[i]);
    if (w[i].t->layout.rank == 2) w[i].bs = 0;
  }
  const int64_t n = flat ? 1 : batch, rows = w[DH].rows;  // matrices, and rows of each
  const int64_t Fp = round_up(F, 64), Mp = round_up(rows, 64);
  const bool tokens = n > 0 && rows > 0 && F > 0;
  const int64_t weights = one_weight ? 1 : n;          // matrices of weights
  const int64_t across = one_weight ? n * Mp : Mp;     // values of a row of a transpose over the tokens
  if (across >= kLim / 2 || n * rows >= kLim) return fail(SL_ERR_SHAPE, "too many rows in all");
  if (tokens && !grid_fits(n, ceil_div(rows, 64), ceil_div(F, 64), sl::kPrepareThreads)) return fail(SL_ERR_SHAPE, "dh is too large");

  sl::GatedSlopeParams& g = P.prepare.slope;
  g.g = (const uint16_t*)args->gate.data, g.u = (const uint16_t*)args->up.data, g.dh = (const uint16_t*)args->dh.data;
  g.M = rows, g.F = F, g.Fp = Fp, g.Mp = Mp;
  g.g_bs = bstride(w[G]), g.g_rs = w[G].rs, g.g_cs = w[G].cs;
  g.u_bs = bstride(w[U]), g.u_rs = w[U].rs, g.u_cs = w[U].cs;
  g.dh_bs = bstride(w[DH]), g.dh_rs = w[DH].rs, g.dh_cs = w[DH].cs;
  g.type = dt == SL_F16 ? sl::OT_F16 : sl::OT_BF16, g.act = args->activation - SL_SILU, g.batch = (int32_t)(tokens ? n : 0);
  g.t_bs = one_weight ? Mp : 2 * Fp * Mp, g.t_rs = across, g.t_us = Fp * across;

  auto take = [&](int64_t values) {
    const int64_t at = P.ws_bytes;
    P.ws_bytes += round_up(2 * values, 256);
    return at;
  };
  // a transpose: out row r is x's column r
  auto transpose = [&](sl::PackParams* q, const View& x, int64_t count, int64_t width, int64_t out_bs, int64_t out_rs) -> sl_status {
    q->x = (const uint16_t*)x.t->data;
    q->rows = x.cols, q->cols = x.rows, q->width = width;
    q->x_bs = bstride(x), q->x_rs = x.cs, q->x_cs = x.rs, q->out_bs = out_bs, q->out_rs = out_rs;
    q->batch = (int32_t)count;
    if (!grid_fits(count, ceil_div(q->rows, 64), ceil_div(width, 64), sl::kPrepareThreads))
      return fail(SL_ERR_SHAPE, "an operand is too large to be transposed");
    return SL_OK;
  };
  // a product of `count` matrices (m, k) and (n, k) of the workspace, k values a row
  auto product = [&](sl::DenseParams* p, sl::DensePlan* tile, int64_t count, int64_t m, int64_t n, int64_t k, int64_t a_bs, int64_t b_bs,
                     int shift) {
    p->M = m, p->N = n, p->K = 2 * k, p->batch = (int32_t)count, p->b_shift = shift;
    p->a_rs = p->b_rs[0] = 2 * k, p->a_bs = 2 * a_bs, p->b_bs[0] = 2 * b_bs;
    p->type = g.type;
    *tile = sl::dense_plan(false, count, m, n, 2 * k);
  };
  // the rows of a tile that are there span less than 2^31 bytes, of k values each
  auto fits = [](int64_t rows, int64_t k) { return std::min<int64_t>(rows, 256) * 2 * k < kLim; };
  auto too_long = [] { return fail(SL_ERR_SHAPE, "a 256-row tile of an operand spans 2^31 bytes or more"); };
  auto output = [&](sl::DenseParams* p, int i, const sl_tensor& d, const View& v, int64_t count) {
    p->kept[i] = d.data, p->kept_rs[i] = v.rs, p->kept_cs[i] = v.cs, p->kept_bs[i] = count > 1 ? v.bs : 0;
    if (quad_rows(v, count)) p->flags |= sl::DF_KEPT_VEC << i;
  };
  P.kind = dt == SL_F16 ? sl::EK_F16 : sl::EK_BF16;
  // Operands whose rows lie on 16-byte boundaries can be read as they are; others, and where
  // a better tile saves more than the copies (bytes read and written, at 7 TB/s as
  // long as the caches hold them, else 4.5) cost, are copied.  us as they lie and with copies:
  // 4000 x 500 x 3000's dx 43 and 39, 4096 x 4096 x 2048's two 281 and 248, 8 of 1024 x 1000 x
  // 1024's two 91 and 97, 1024 x 4096 x 4096's 134 and 159, 4000 x 2000 x 3000's 194 and 207, 4096
  // x 8192 x 4096's 871 and 925, 1024 x 8192 x 4096's dx 160 and 219 (251 with the workspace's
  // rows 128 bytes off powers of two).
  auto copied_us = [](double bytes) { return bytes / (bytes < 1.5e8 ? 7e6 : 4.5e6); };
  auto readable = [&](const View& x, const View& y) {
    bool ok = tokens && x.rs == y.rs;
    for (const View* v : {&x, &y})
      ok = ok && v->cs == 1 && v->cols % 8 == 0 && v->rs % 8 == 0 && (uintptr_t)v->t->data % 16 == 0 && bstride(*v) % 8 == 0 &&
           v->rows * v->rs * 2 + 1024 < kLim;
    return ok;
  };
  auto choose = [&](const sl::DenseParams& p, bool ok, bool copy, double copies, sl::DensePlan* tile) {
    sl::DensePlan large = sl::ring_plan(sl::DT_256x256, 256, 256, sl::kRing), small = sl::ring_plan(sl::DT_128x128, 128, 128, sl::kRing);
    large.us = sl::dense_large_us(p.batch, p.M, p.N, p.K);
    small.us = sl::grad_tiles_us((double)p.batch * (double)ceil_div(p.M, 128) * (double)ceil_div(p.N, 128), (double)ceil_div(p.K, 128));
    const sl::DensePlan& best = small.us < large.us ? small : large;
    tile->us += copied_us(copies);
    if (!ok || (copy && best.us > tile->us)) return false;
    *tile = best;
    return true;
  };
  bool dx_ok = false, dw_ok = false, dx_copy = true, dw_copy = true;  // on operands as they lie, with copies: possible
  double dx_copies = 0.0, dw_copies = 0.0;
  if (P.want_dx) {
    if (tokens && !fits(rows, 2 * Fp)) return too_long();  // dg and du
    product(&P.dx.d, &P.dx_tile, n, rows, K, tokens ? 2 * Fp : 0, rows * 2 * Fp, one_weight ? 0 : K * 2 * Fp, 0);
    dx_ok = readable(w[WG], w[WU]), dx_copy = !tokens || fits(K, 2 * Fp);
    if (!dx_ok && !dx_copy) return too_long();
    if (tokens) dx_copies = 8.0 * (double)weights * (double)F * (double)K;
    P.dx_lies = choose(P.dx.d, dx_ok, dx_copy, dx_copies, &P.dx_tile);
    // Few rows: the weights read once (8192 x 4096's two, 134 MB in 24 to 29 us for up to 64 rows) and the
    // workgroups' sums joined, by the same kind of model.  us so and otherwise, from Python: 1 x 8192 x
    // 4096 31 and 69, 64 x 8192 x 4096 35 and 82, 512 x 8192 x 4096 111 and 147; 1 x 2048 x 2048 13
    // and 17; 512 x 4096 x 8192 108 and 76; 40 x 1000 x 520 19 and 13.
    if (dx_ok) {
      sl::DensePlan few = {sl::DT_256x256, sl::kFewRows, 128, sl::kFewThreads, 0, 0, 0.0};
      const double tiles = (double)n * (double)ceil_div(rows, sl::kFewRows) * (double)ceil_div(K, 128), steps = 2.0 * (double)ceil_div(F, 32);
      const double splits = std::max(1.0, std::min(std::floor(sl::kCUs / tiles), std::floor(steps / 32)));
      const double fm = rows <= 16 ? 1.0 : rows <= 32 ? 2.0 : 4.0;
      const double work = std::ceil(tiles * splits / sl::kCUs) * (0.6 * fm + std::ceil(steps / (8.0 * splits)) * (0.3 + 0.3 * fm));
      const double join = splits > 1.0 ? 3.5 + 8.0 * splits * (double)n * (double)rows * (double)K / 4e6 : 0.0;
      few.us = 3.0 + join + std::max(work, 4.0 * (double)n * (double)F * (double)K / 5.5e6);
      P.dx.splits = (int32_t)splits;
      P.dx_few = few.us < P.dx_tile.us;
      if (P.dx_few) P.dx_tile = few, P.dx_lies = true;
    }
  }
  if (P.want_dw) {
    product(&P.dw.d, &P.dw_tile, 2 * weights, F, K, tokens ? across : 0, Fp * across, K * across, 1);
    dw_ok = (!one_weight || n == 1) && rows * 4 * Fp + 1024 < kLim && readable(w[X], w[X]);
    dw_copy = !tokens || fits(std::max(F, K), across);
    if (!dw_ok && !dw_copy) return too_long();
    // (with dx wanted too dg and du are written both ways where they are not read as they lie)
    if (tokens) dw_copies = 4.0 * (double)n * (double)rows * (double)(K + (P.want_dx ? F : 0));
    P.dw_lies = choose(P.dw.d, dw_ok, dw_copy, dw_copies, &P.dw_tile);
  }
  if (P.want_dx && P.want_dw) {
    sl::DensePlan copied = sl::dense_pair_plan(P.dx.d, P.dw.d), lying = sl::ring_plan(sl::DT_128x128, 128, 128, sl::kRing);
    copied.us += dx_copy && dw_copy ? copied_us(dx_copies + dw_copies) : 1e30;
    lying.us = dx_ok && dw_ok ? sl::pair_us(sl::pair_128x128(), P.dx.d, P.dw.d, true) : 1e30;
    const sl::DensePlan& both = lying.us < copied.us ? lying : copied;
    sl::DenseParams x = P.dx.d, y = P.dw.d;
    P.pair = both.us < P.dx_tile.us + P.dw_tile.us && place_tiles(&x, both, false) == SL_OK && place_tiles(&y, both, false) == SL_OK &&
             grid_fits((int64_t)x.batch * x.tiles_m * x.tiles_n + (int64_t)y.batch * y.tiles_m * y.tiles_n, 1, 1, both.threads);
    if (P.pair) P.dx_tile = P.dw_tile = both, P.dx_lies = P.dw_lies = lying.us < copied.us, P.dx_few = false;
    g_msg.clear();
  }
  if (P.want_dx || P.dw_lies) P.off_rows = tokens ? take(n * rows * 2 * Fp) : 0;
  if (P.want_dx) {
    if ((s = place_tiles(&P.dx.d, P.dx_tile, false)) != SL_OK) return s;
    if (P.dx_lies) {
      for (int i = 0; i < 2; ++i) P.dx.d.b[i] = (const uint8_t*)t[WG + i]->data, P.dx.d.b_bs[i] = 2 * bstride(w[WG + i]);
      P.dx.d.b_rs[0] = 2 * w[WG].rs;
      P.dx.rows = F, P.dx.parts = 2;
      if (P.dx_few && P.dx.splits > 1) P.off_partial = take(2 * P.dx.splits * n * rows * K);  // fp32
    } else if (tokens) {
      P.off_wt = take(weights * K * 2 * Fp);
      for (int i = 0; i < 2; ++i)
        if ((s = transpose(&P.prepare.pack[1 + i], w[WG + i], weights, Fp, K * 2 * Fp, 2 * Fp)) != SL_OK) return s;
    }
    output(&P.dx.d, 0, args->dx, w[DX], n);
    P.dx.d.flags |= row_flags({&w[DX]}, n);
  }
  if (P.want_dw) {
    if ((s = place_tiles(&P.dw.d, P.dw_tile, false)) != SL_OK) return s;
    if (P.dw_lies) {
      sl::DenseParams& d = P.dw.d;
      d.a_rs = 4 * Fp, d.a_bs = rows * 4 * Fp;
      for (int i = 0; i < 2; ++i) d.b[i] = (const uint8_t*)args->x.data, d.b_bs[i] = 2 * bstride(w[X]);
      d.b_rs[0] = 2 * w[X].rs;
      P.dw.rows = rows, P.dw.parts = 1, P.dw.a_second = 2 * Fp;
    } else if (tokens) {
      P.off_t = take(one_weight ? 2 * Fp * across : n * 2 * Fp * Mp);
      P.off_xt = take(one_weight ? K * across : n * K * Mp);
      if ((s = transpose(&P.prepare.pack[0], w[X], n, Mp, one_weight ? Mp : K * Mp, across)) != SL_OK) return s;
    }
    for (int i = 0; i < 2; ++i) output(&P.dw.d, i, *t[DWG + i], v[DWG + i], weights);
    P.dw.d.flags |= row_flags({&v[DWG], &v[DWU]}, weights);
  }
  if (!grid_fits(sl::gated_prepare_groups(&P.prepare), 1, 1, sl::kPrepareThreads)) return fail(SL_ERR_SHAPE, "the operands are too large");
  return SL_OK;
}

}  // namespace

extern "C" {

sl_status sl_gated_backward_workspace_bytes(const sl_gated_backward_args* args, int64_t* bytes) {
  g_msg.clear();
  if (!bytes) return fail(SL_ERR_NULL, "bytes is NULL");
  BackwardPlan P;
  const sl_status s = plan_backward(args, &P);
  if (s == SL_OK) *bytes = P.ws_bytes;
  return s;
}

sl_status sl_gated_backward(const sl_gated_backward_args* args, void* stream) {
  BackwardPlan P;
  sl_status s = plan_backward(args, &P);
  if (s != SL_OK) return s;
  if (!P.launch) return SL_OK;
  const View* views[9];
  for (int i = 0; i < 9; ++i) views[i] = P.v[i].t ? &P.v[i] : nullptr;
  static const char* const names[9] = {"dh", "x", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up"};
  if ((s = check_workspace(args->workspace, args->workspace_bytes, P.ws_bytes, views, names, 9)) != SL_OK) return s;
  if ((s = check_arch()) != SL_OK) return s;
  const hipStream_t st = (hipStream_t)stream;
  char* const ws = (char*)args->workspace;
  sl::DenseParams &dx = P.dx.d, &dw = P.dw.d;
  if (P.prepare.slope.batch > 0) {  // (without tokens the products have K = 0 and read nothing)
    uint16_t* const rows = (uint16_t*)(ws + P.off_rows);
    if (P.want_dx || P.dw_lies) P.prepare.slope.rows = rows;
    if (P.want_dx) {
      dx.a = (const uint8_t*)rows;
      if (!P.dx_lies) {
        for (int i = 0; i < 2; ++i) P.prepare.pack[1 + i].out = (uint16_t*)(ws + P.off_wt) + i * P.prepare.slope.Fp;
        dx.b[0] = (const uint8_t*)(ws + P.off_wt);
      }
    }
    if (P.want_dw && P.dw_lies) {
      dw.a = (const uint8_t*)rows;
    } else if (P.want_dw) {
      P.prepare.slope.t = (uint16_t*)(ws + P.off_t);
      P.prepare.pack[0].out = (uint16_t*)(ws + P.off_xt);
      dw.a = (const uint8_t*)(ws + P.off_t), dw.b[0] = (const uint8_t*)(ws + P.off_xt);
    }
  }
  hipError_t e = sl::launch_gated_prepare(P.prepare, st);
  const uint32_t first = (uint32_t)((int64_t)dx.batch * dx.tiles_m * dx.tiles_n);
  if (e == hipSuccess && P.pair)
    e = P.dx_lies ? sl::launch_grad_tiles(sl::GradPair{P.dx, P.dw, first}, P.kind, st)
                  : sl::launch_gated_products(sl::DensePair{{dx, dw}, first}, P.kind, P.dx_tile, st);
  auto one = [&](const sl::GradParams& g, const sl::DensePlan& tile, bool lies, bool across) {
    return !lies ? sl::launch_gated_products(g.d, P.kind, tile, st)
                 : tile.tile == sl::DT_256x256 ? sl::launch_grad_ring(g, P.kind, across, st) : sl::launch_grad_tiles(g, P.kind, across, st);
  };
  if (P.dx_few) {
    P.dx.partial = (float*)(ws + P.off_partial);
    if (e == hipSuccess) e = sl::launch_grad_few(P.dx, P.kind, st);
  }
  if (e == hipSuccess && P.want_dx && !P.pair && !P.dx_few) e = one(P.dx, P.dx_tile, P.dx_lies, false);
  if (e == hipSuccess && P.want_dw && !P.pair) e = one(P.dw, P.dw_tile, P.dw_lies, true);
  if (e != hipSuccess) return fail(SL_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return SL_OK;
}

}  // extern "C"
