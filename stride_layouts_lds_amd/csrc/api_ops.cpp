// api_ops.cpp -- host side of the operators next to the GEMM: the planner of
// the block-scaled 8-bit product (a form of sl_gemm), sl_quantize and
// sl_orthogonalize.  Every check runs before any HIP call.
#include "api_ops.hpp"

#include <cmath>

#include "api_common.hpp"
#include "sl_kernels.hpp"

namespace sl {
namespace host {

// The tile: up to 64 rows of A stream the weight once (the skinny kernels),
// and so do products of up to 64 tiles of 128 x 128, which would leave most
// CUs without work (128 x 512 x 8192: 54 us in those tiles, 14 us streamed in 64
// x 16; 512 x 2048 x 4096, 64 tiles: 30 and 21 us; 640 x 2048 x 4096, 80 tiles:
// 30 both ways; 1024 x 2048 x 4096: 30 and 41, and x 512: 9 and 19.  The rule
// loses where A is tall and B narrow, so that each row of A is read several
// times: 8192 x 100 x 4096 29 and 39);
// otherwise the tile with the least (workgroup rounds over the 256 CUs) x
// (work of a tile), the 128 x 128 tile two to a CU and moving twice the
// operand bytes per product (256 x 256 and 128 x 128 forced: 4096^3 67 and 79 us,
// 3000 x 5000 x 4096 65 and 75, 4000 x 3000 x 2064 39 and 48, 2048 x 4096 x 4096
// 66 and 42, 1536 x 4096 x 4096 66 and 41).  fp32 results: 128 x 128 (the fp16 fragments of
// the larger tile do not fit the registers: 4096 x 4096 x 8192 took 836 us).
static int32_t choose_tile(int64_t batch, int64_t M, int64_t N, int32_t type) {
  if (M <= kSkinnyRows || batch * ceil_div(M, 128) * ceil_div(N, 128) <= 64) return BT_SKINNY;
  if (type == OT_F32) return BT_128x128;
  int32_t best = BT_256x256;
  double least = 1e300;
  for (int32_t t : {(int32_t)BT_256x256, (int32_t)BT_128x128}) {
    const BlockTileShape& s = kBlockTiles[t];
    const int64_t tiles = batch * ceil_div(M, s.bm) * ceil_div(N, s.bn);
    const int64_t per_cu = t == BT_128x128 ? 2 : 1;
    const double cost = (double)ceil_div(tiles, 256 * per_cu) * s.bm * s.bn * per_cu / (t == BT_128x128 ? 0.8 : 1.0);
    if (cost < least) least = cost, best = t;
  }
  return best;
}

sl_status plan_block(const sl_gemm_args* args, BlockPlan* out) {
  g_msg.clear();
  if (args->a.dtype != SL_F8_E4M3 || args->b.dtype != SL_F8_E4M3)
    return fail(SL_ERR_DTYPE, "f32 scales belong to f8_e4m3 a and b");
  if (args->sfa.dtype != SL_F32 || args->sfb.dtype != SL_F32) return fail(SL_ERR_DTYPE, "sfa and sfb must both be f32");
  if (args->block_k != kScaleBlock) return fail(SL_ERR_SHAPE, "block_k must be 128 with f32 scales (got %d)", args->block_k);
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
  if ((s = make_view("sfa", args->sfa, &SA)) != SL_OK) return s;
  if ((s = make_view("sfb", args->sfb, &SB)) != SL_OK) return s;
  const int64_t batch = D.batch, M = A.rows, K = A.cols, N = B.rows, kb = ceil_div(K, kScaleBlock);
  if (B.cols != K) return fail(SL_ERR_SHAPE, "b is (%lld,%lld) but a has K=%lld", (long long)B.rows, (long long)B.cols, (long long)K);
  if (D.rows != M || D.cols != N)
    return fail(SL_ERR_SHAPE, "d is (%lld,%lld), expected (%lld,%lld)", (long long)D.rows, (long long)D.cols, (long long)M, (long long)N);
  if (has_c && (C.rows != M || C.cols != N))
    return fail(SL_ERR_SHAPE, "c is (%lld,%lld), expected (%lld,%lld)", (long long)C.rows, (long long)C.cols, (long long)M, (long long)N);
  const View* all[6] = {&A, &B, has_c ? &C : nullptr, &D, &SA, &SB};
  const char* names[6] = {"a", "b", "c", "d", "sfa", "sfb"};
  for (int i = 0; i < 6; ++i)
    if (all[i] && i != 3 && all[i]->t->layout.rank == 3 && all[i]->batch != batch)
      return fail(SL_ERR_SHAPE, "%s has batch %lld, d has %lld", names[i], (long long)all[i]->batch, (long long)batch);
  // one scale row per row of the operand, or per 128 of them
  auto shift_of = [&](const char* name, const View& S, int64_t rows, int32_t* shift) -> sl_status {
    if (S.cols != kb || (S.rows != rows && S.rows != ceil_div(rows, kScaleBlock)))
      return fail(SL_ERR_SHAPE, "%s is (%lld,%lld), expected (%lld,%lld) or (%lld,%lld)", name, (long long)S.rows, (long long)S.cols,
                  (long long)rows, (long long)kb, (long long)ceil_div(rows, kScaleBlock), (long long)kb);
    *shift = S.rows == rows ? 0 : 7;
    return SL_OK;
  };
  BlockPlan& P = *out;
  memset(&P, 0, sizeof P);
  BlockGemmParams& p = P.p;
  if ((s = shift_of("sfa", SA, M, &p.a_shift)) != SL_OK) return s;
  if ((s = shift_of("sfb", SB, N, &p.b_shift)) != SL_OK) return s;
  if (M >= kLim || N >= kLim || K >= kLim || batch >= kLim) return fail(SL_ERR_SHAPE, "a dimension exceeds 2^31-1");
  P.pub.batch = batch, P.pub.m = M, P.pub.n = N, P.pub.k = K;
  P.pub.kernel = K_BLOCK8;
  P.pub.split_k = 1;
  P.empty = batch == 0 || M == 0 || N == 0;
  if (P.empty) return SL_OK;

  for (int i = 0; i < 6; ++i) {
    if (!all[i] || (!all[i]->t->data && i != 3 && K == 0)) continue;
    if ((s = check_data(names[i], *all[i]->t)) != SL_OK) return s;
  }
  if (!injective(D, batch)) return fail(SL_ERR_LAYOUT, "d's strides map distinct elements to one address");
  for (int i = 0; i < 6; ++i) {
    if (!all[i] || i == 3 || !all[i]->t->data || (i != 2 && K == 0)) continue;
    if (i == 2 && args->c.data == args->d.data && same_layout(args->c, args->d)) continue;
    if (overlap(*all[i], D, batch)) return fail(SL_ERR_ALIAS, "d overlaps %s", names[i]);
  }
  if (K > 0 && (K % 16 != 0 || !code_rows(A, batch) || !code_rows(B, batch)))
    return fail(SL_ERR_LAYOUT, "f8_e4m3 operands must be K-contiguous with 16-byte aligned rows and K %% 16 == 0");
  for (const View* X : {&A, &B})
    if ((std::min<int64_t>(X->rows, 256) - 1) * X->rs + K >= kLim)
      return fail(SL_ERR_SHAPE, "a 256-row tile of an operand spans 2^31 bytes or more");

  p.a = (const uint8_t*)args->a.data, p.b = (const uint8_t*)args->b.data;
  p.c = has_c ? args->c.data : nullptr;
  p.d = args->d.data;
  p.sa = (const float*)args->sfa.data, p.sb = (const float*)args->sfb.data;
  p.M = M, p.N = N, p.K = K;
  p.a_rs = A.rs, p.a_bs = batch_stride(A);
  p.b_rs = B.rs, p.b_bs = batch_stride(B);
  if (has_c) p.c_rs = C.rs, p.c_cs = C.cs, p.c_bs = batch_stride(C);
  p.d_rs = D.rs, p.d_cs = D.cs, p.d_bs = batch_stride(D);
  p.sa_rs = SA.rs, p.sa_ks = SA.cs, p.sa_bs = batch_stride(SA);
  p.sb_rs = SB.rs, p.sb_ks = SB.cs, p.sb_bs = batch_stride(SB);
  p.type = type;
  p.batch = (int32_t)batch;
  p.k_blocks = (int32_t)kb;
  p.group_m = 8;
  // four consecutive outputs as one aligned access
  auto quads = [&](const View& X) {
    return X.cs == 1 && (M == 1 || X.rs % 4 == 0) && (uintptr_t)X.t->data % (4 * elem_size(X.t->dtype)) == 0 &&
           (batch == 1 || batch_stride(X) % 4 == 0);
  };
  p.flags = (has_c ? BF_HAS_C : 0) | (quads(D) ? BF_D_VEC : 0) | (has_c && quads(C) ? BF_C_VEC : 0);

  if (!grid_fits(batch, ceil_div(M, 256), ceil_div(N, 256), 256))  // in the largest tiles
    return fail(SL_ERR_SHAPE, "too many output tiles (batch %lld of %lld x %lld)", (long long)batch, (long long)M, (long long)N);
  P.tile = choose_tile(batch, M, N, type);
  BlockTileShape ts = kBlockTiles[P.tile];
  if (P.tile == BT_SKINNY) ts.bn = skinny_cols(M, N, batch);
  p.tiles_m = (int32_t)ceil_div(M, ts.bm), p.tiles_n = (int32_t)ceil_div(N, ts.bn);
  const int64_t total = batch * p.tiles_m * p.tiles_n;
  P.pub.a_load = P.pub.b_load = LOAD_KVEC;
  P.pub.tile_m = ts.bm, P.pub.tile_n = ts.bn, P.pub.tile_k = kScaleBlock;
  P.pub.threads = P.tile == BT_SKINNY ? (M <= 16 ? kSkinnyWaves : kStreamWaves) * 64 : ts.wm * ts.wn * 64;
  if (!grid_fits(batch, p.tiles_m, p.tiles_n, P.pub.threads))
    return fail(SL_ERR_SHAPE, "too many output tiles (%lld)", (long long)total);
  P.pub.workgroups = total;
  if (P.tile == BT_256x256) P.pub.lds_bytes = 5 * 256 * kScaleBlock;
  else if (P.tile == BT_128x128) P.pub.lds_bytes = (total > 256 ? 2 : 4) * 256 * kScaleBlock;
  else if (M <= 16) P.pub.lds_bytes = (kSkinnyWaves - 1) * (ts.bn / 16) * 1024;
  else P.pub.lds_bytes = kStreamWaves * (M <= 32 ? 4 : 3) * ((M <= 32 ? 32 : 64) + ts.bn) * kScaleBlock;
  return SL_OK;
}

sl_status run_block(const sl_gemm_args* args, void* stream) {
  BlockPlan P;
  sl_status s = plan_block(args, &P);
  if (s != SL_OK) return s;
  if (P.empty) return SL_OK;
  if ((s = check_arch()) != SL_OK) return s;
  const hipError_t e = launch_gemm_block(P.p, P.tile, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SL_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return SL_OK;
}

}  // namespace host
}  // namespace sl

using namespace sl::host;

extern "C" {

sl_status sl_quantize(const sl_quantize_args* args, void* stream) {
  g_msg.clear();
  if (!args) return fail(SL_ERR_NULL, "args is NULL");
  const int32_t type = op_type(args->x.dtype);
  if (type < 0) return fail(SL_ERR_DTYPE, "x must be f16, bf16 or f32");
  const int64_t br = args->block_rows;
  if (br != 1 && br != sl::kScaleBlock) return fail(SL_ERR_ARG, "block_rows must be 1 or 128 (got %lld)", (long long)br);
  const bool direct = args->q.data != nullptr, transposed = args->qt.data != nullptr;
  View X, Q{}, S{}, QT{}, ST{};
  sl_status s;
  if ((s = make_view("x", args->x, &X)) != SL_OK) return s;
  const int64_t batch = X.batch, R = X.rows, C = X.cols;
  // one output: codes (rows, columns padded at most to the block's end) and
  // their scales
  auto output = [&](const char* qn, const char* sn, const sl_tensor& q, const sl_tensor& sc, View* vq, View* vs, int64_t rows,
                    int64_t cols) -> sl_status {
    sl_status e;
    if (q.dtype != SL_F8_E4M3) return fail(SL_ERR_DTYPE, "%s must be f8_e4m3", qn);
    if (sc.dtype != SL_F32) return fail(SL_ERR_DTYPE, "%s must be f32", sn);
    if ((e = make_view(qn, q, vq)) != SL_OK) return e;
    if ((e = make_view(sn, sc, vs)) != SL_OK) return e;
    if (vq->batch != batch || vs->batch != batch)
      return fail(SL_ERR_SHAPE, "%s and %s must have x's batch of %lld", qn, sn, (long long)batch);
    if (vq->rows != rows || vq->cols < cols || vq->cols > 128 * ceil_div(cols, 128))
      return fail(SL_ERR_SHAPE, "%s is (%lld,%lld), expected %lld rows of %lld to %lld codes", qn, (long long)vq->rows,
                  (long long)vq->cols, (long long)rows, (long long)cols, (long long)(128 * ceil_div(cols, 128)));
    if (vs->rows != ceil_div(rows, br) || vs->cols != ceil_div(cols, 128))
      return fail(SL_ERR_SHAPE, "%s is (%lld,%lld), expected (%lld,%lld)", sn, (long long)vs->rows, (long long)vs->cols,
                  (long long)ceil_div(rows, br), (long long)ceil_div(cols, 128));
    return SL_OK;
  };
  if (direct && (s = output("q", "s", args->q, args->s, &Q, &S, R, C)) != SL_OK) return s;
  if (transposed && (s = output("qt", "st", args->qt, args->st, &QT, &ST, C, R)) != SL_OK) return s;
  if (R >= kLim - 128 || C >= kLim - 128 || batch >= kLim) return fail(SL_ERR_SHAPE, "a dimension exceeds 2^31-129");
  if (batch == 0 || R == 0 || C == 0) return SL_OK;
  if (!direct && !transposed) return fail(SL_ERR_NULL, "q.data and qt.data are both NULL");
  const View* outs[4] = {direct ? &Q : nullptr, direct ? &S : nullptr, transposed ? &QT : nullptr, transposed ? &ST : nullptr};
  const char* names[4] = {"q", "s", "qt", "st"};
  if ((s = check_data("x", args->x)) != SL_OK) return s;
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    if ((s = check_data(names[i], *outs[i]->t)) != SL_OK) return s;
    if (i % 2 == 0 && !code_rows(*outs[i], batch))
      return fail(SL_ERR_LAYOUT, "%s must be contiguous along its last axis with 16-byte aligned rows", names[i]);
    if (!injective(*outs[i], batch)) return fail(SL_ERR_LAYOUT, "%s's strides map distinct elements to one address", names[i]);
    if (overlap(*outs[i], X, batch)) return fail(SL_ERR_ALIAS, "%s overlaps x", names[i]);
    for (int j = 0; j < i; ++j)
      if (outs[j] && overlap(*outs[i], *outs[j], batch)) return fail(SL_ERR_ALIAS, "%s overlaps %s", names[i], names[j]);
  }

  sl::QuantizeParams p{};
  p.x = args->x.data;
  p.type = type;
  p.square = br != 1;
  p.batch = (int32_t)batch;
  p.rows = R, p.cols = C, p.x_bs = batch_stride(X), p.x_rs = X.rs, p.x_cs = X.cs;
  if (direct) {
    p.q = (uint8_t*)args->q.data, p.s = (float*)args->s.data;
    p.q_cols = Q.cols, p.q_bs = batch_stride(Q), p.q_rs = Q.rs, p.s_bs = batch_stride(S), p.s_rs = S.rs, p.s_cs = S.cs;
  }
  if (transposed) {
    p.qt = (uint8_t*)args->qt.data, p.st = (float*)args->st.data;
    p.qt_cols = QT.cols, p.qt_bs = batch_stride(QT), p.qt_rs = QT.rs, p.st_bs = batch_stride(ST), p.st_rs = ST.rs, p.st_cs = ST.cs;
  }
  // x stored column after column: the same call on its transpose
  if (p.x_rs == 1 && p.x_cs != 1) {
    std::swap(p.rows, p.cols), std::swap(p.x_rs, p.x_cs), std::swap(p.q, p.qt), std::swap(p.s, p.st);
    std::swap(p.q_cols, p.qt_cols), std::swap(p.q_bs, p.qt_bs), std::swap(p.q_rs, p.qt_rs);
    std::swap(p.s_bs, p.st_bs), std::swap(p.s_rs, p.st_rs), std::swap(p.s_cs, p.st_cs);
  }
  if (!grid_fits(batch, ceil_div(p.rows, sl::quantize_rows(p)), ceil_div(p.cols, 128), sl::kQuantizeThreads))
    return fail(SL_ERR_SHAPE, "too many blocks (batch %lld of %lld x %lld)", (long long)batch, (long long)R, (long long)C);
  if ((s = check_arch()) != SL_OK) return s;
  const hipError_t e = sl::launch_quantize(p, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SL_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return SL_OK;
}

}  // extern "C"

namespace {

constexpr int64_t kOrthoMaxBatch = 65536;
constexpr float kDefaultCoefficients[3] = {3.4445f, -4.7750f, 2.0315f};

struct OrthoPlan {
  sl::OrthoParams p;
  float coefficients[3 * sl::kOrthoMaxSteps];
  size_t ws_bytes;
  bool empty;
  View X, D;
};

sl_status plan_orthogonalize(const sl_orthogonalize_args* args, OrthoPlan* P) {
  g_msg.clear();
  if (!args) return fail(SL_ERR_NULL, "args is NULL");
  sl::OrthoParams& p = P->p;
  p = sl::OrthoParams{};
  P->ws_bytes = 0;
  p.x_type = op_type(args->x.dtype);
  p.d_type = op_type(args->d.dtype);
  if (p.x_type < 0) return fail(SL_ERR_DTYPE, "x must be f16, bf16 or f32");
  if (p.d_type != sl::OT_F16 && p.d_type != sl::OT_BF16) return fail(SL_ERR_DTYPE, "d must be f16 or bf16");
  if (args->steps < 1 || args->steps > sl::kOrthoMaxSteps)
    return fail(SL_ERR_ARG, "steps must be 1 to %d (got %d)", sl::kOrthoMaxSteps, args->steps);
  View &X = P->X, &D = P->D;
  sl_status s;
  if ((s = make_view("x", args->x, &X)) != SL_OK) return s;
  if ((s = make_view("d", args->d, &D)) != SL_OK) return s;
  if (D.rows != X.rows || D.cols != X.cols || D.batch != X.batch)
    return fail(SL_ERR_SHAPE, "d is (%lld,%lld,%lld), x is (%lld,%lld,%lld)", (long long)D.batch, (long long)D.rows,
                (long long)D.cols, (long long)X.batch, (long long)X.rows, (long long)X.cols);
  for (int i = 0; i < 3 * args->steps; ++i) {
    const float c = args->coefficients ? args->coefficients[i] : kDefaultCoefficients[i % 3];
    // (While the iterates' singular values s stay below 2, |a + b s^2 + c s^4| is below 2 / s: nothing that the
    // kernels hold in fp16 grows with b or c.)
    const float most = i % 3 == 0 ? 16.f : 64.f;
    if (!(std::fabs(c) <= most)) return fail(SL_ERR_ARG, "coefficient %d is not within %g in magnitude", i, most);
    P->coefficients[i] = c;
  }
  P->empty = X.batch == 0 || X.rows == 0 || X.cols == 0;
  if (P->empty) return SL_OK;
  const bool tall = X.rows > X.cols;
  p.m = tall ? X.cols : X.rows, p.n = tall ? X.rows : X.cols;
  p.x_bs = batch_stride(X), p.x_rs = tall ? X.cs : X.rs, p.x_cs = tall ? X.rs : X.cs;
  p.d_bs = batch_stride(D), p.d_rs = tall ? D.cs : D.rs, p.d_cs = tall ? D.rs : D.cs;
  if (X.batch >= kOrthoMaxBatch) return fail(SL_ERR_SHAPE, "x has %lld matrices, fewer than %lld are taken", (long long)X.batch, (long long)kOrthoMaxBatch);
  p.batch = (int32_t)X.batch;
  p.steps = args->steps;
  p.x = args->x.data, p.d = args->d.data;
  p.coefficients = P->coefficients;
  if (!sl::orthogonalize_grid_ok(p)) return fail(SL_ERR_SHAPE, "x is too large");
  P->ws_bytes = sl::orthogonalize_workspace(p);
  return SL_OK;
}

}  // namespace

extern "C" {

sl_status sl_orthogonalize_workspace_bytes(const sl_orthogonalize_args* args, int64_t* bytes) {
  g_msg.clear();
  if (!bytes) return fail(SL_ERR_NULL, "bytes is NULL");
  OrthoPlan P;
  const sl_status s = plan_orthogonalize(args, &P);
  if (s == SL_OK) *bytes = (int64_t)P.ws_bytes;
  return s;
}

sl_status sl_orthogonalize(const sl_orthogonalize_args* args, void* stream) {
  OrthoPlan P;
  sl_status s = plan_orthogonalize(args, &P);
  if (s != SL_OK) return s;
  if (P.empty) return SL_OK;
  if ((s = check_data("x", args->x)) != SL_OK) return s;
  if ((s = check_data("d", args->d)) != SL_OK) return s;
  if (!injective(P.D, P.D.batch)) return fail(SL_ERR_LAYOUT, "d's strides map distinct elements to one address");
  // d may be x itself: x is read whole before d is written
  if (!(args->x.data == args->d.data && args->x.dtype == args->d.dtype && same_layout(args->x, args->d)) &&
      overlap(P.X, P.D, P.D.batch))
    return fail(SL_ERR_ALIAS, "d overlaps x");
  if (!args->workspace) return fail(SL_ERR_NULL, "workspace is NULL, %zu bytes are needed", P.ws_bytes);
  if (args->workspace_bytes < 0 || (uint64_t)args->workspace_bytes < (uint64_t)P.ws_bytes)
    return fail(SL_ERR_SHAPE, "workspace of %lld bytes, %zu are needed", (long long)args->workspace_bytes, P.ws_bytes);
  const uintptr_t lo = (uintptr_t)args->workspace, hi = lo + P.ws_bytes;
  if (lo % 16) return fail(SL_ERR_ALIGN, "workspace is not on a 16-byte boundary");
  for (const View* v : {&P.X, &P.D}) {
    uintptr_t l, h;
    byte_range(*v, v->batch, &l, &h);
    if (l < hi && lo < h) return fail(SL_ERR_ALIAS, "workspace overlaps %s", v == &P.X ? "x" : "d");
  }
  if ((s = check_arch()) != SL_OK) return s;
  P.p.ws = (char*)args->workspace;
  const hipError_t e = sl::launch_orthogonalize(P.p, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SL_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
  return SL_OK;
}

}  // extern "C"
