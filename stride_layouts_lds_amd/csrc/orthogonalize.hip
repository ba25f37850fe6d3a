// orthogonalize.hip -- the Newton-Schulz orthogonalisation of an update:
//   X <- x / (|x|_F + 1e-7), then per step
//   G = X X^T,  B = b G + c G^2,  X <- a X + B X,
// x taken with no more rows than columns (a tall one transposed by its
// strides).  Three ways, chosen by way_of() below:
//
//   up to 128 rows     ortho_gram.hip: three launches a cycle of steps
//   Gram matrix        the same iteration on m x m matrices alone (G, P = a I
//                      + b G + c G^2, Q <- P Q, G <- P G P, X <- Q X), every one
//                      a pair of fp16 planes; x times a power of two.  In
//                      cycles of steps: X <- Q X and a new G after as many as
//                      amplify little
//   direct             the formula above, for bf16 results and steps that
//                      amplify little: X a pair of which the products read
//                      the first plane, G and B one plane
//
// All on the fp16 matrix cores with fp32 sums.  A plane holds values times a
// power of two (2^10 for X, G and B of the direct way, 2^12 and 2^6 for the
// other), so nothing overflows while the singular values of every iterate
// stay below 2; a pair is a value rounded to fp16 and what that left, and its
// products are P0 Q0 + P1 Q0 + P0 Q1.  x's sum of squares is held in 64 bits
// and added up in a fixed order.
//
// G, B, P, Q and H = P G are symmetric (polynomials in G): only tiles on and
// above the diagonal are computed, each stored a second time, transposed.
// Every product reads both operands along K: X is kept in both orientations
// (read as it lies, by transposing LDS reads, it cost a product of 8192^3
// half as much again).
#include <utility>

#include "ortho_device.hpp"

namespace sl {
namespace {

constexpr int32_t kNormParts = 256;               // most partial sums of squares of one matrix
constexpr int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

constexpr int kNormWaves = 16;

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (uint32_t w = 0; w < blockDim.x / 64; ++w) v += lds[w];
  return v;
}

// sum of squares of part blockIdx.x of matrix blockIdx.y: lines along x's
// contiguous axis, `across` threads (a power of two) to a line
template <int T>
__global__ __launch_bounds__(64 * kNormWaves) void ortho_norm_kernel(const OrthoParams p, double* parts, int32_t across) {
  __shared__ double lds[kNormWaves];
  const int64_t b = blockIdx.y;
  const bool along_rows = p.x_rs == 1 && p.x_cs != 1;
  const int64_t lines = along_rows ? p.n : p.m, length = along_rows ? p.m : p.n;
  const int64_t u = threadIdx.x & (across - 1), w = threadIdx.x / across, at_once = 64 * kNormWaves / across;
  double s = 0;
  for (int64_t c = 8 * u; c < length; c += 8 * across) {
#pragma unroll 4
    for (int64_t r = blockIdx.x * at_once + w; r < lines; r += gridDim.x * at_once) {
      float v[8];
      ortho_load8<T>(p, b, along_rows ? c : r, along_rows ? r : c, p.n, along_rows, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
    }
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) parts[b * kNormParts + blockIdx.x] = s;
}

// Where value (row, col) of a matrix with rows of `cols` lies.  Pairs: 32
// values of the first plane, then the same 32 of the second, so that one
// 128-byte K-tile of a row holds both planes of 32 values and three products
// come from one copy.
template <int PLANES>
__device__ __forceinline__ int64_t plane_at(int64_t row, int64_t cols, int64_t col) {
  return PLANES == 2 ? row * 2 * cols + (col >> 5) * 64 + (col & 31) : row * cols + col;
}

// What products multiply by, one of each for every matrix: the Gram matrix of
// x's planes to make G's, Q's planes times x's to make d or the planes that X is
// kept in, and the first two of those.  (Direct way: the first two.)
enum OrthoScale : int32_t { kScaleGram, kScaleResult, kScaleKeep, kScaleGramKept, kScaleResultKept, kScaleCount };
struct OrthoScales {
  float v[kScaleCount];
};

// The planes that the products read: m x n and n x m, zero to the padded
// sizes.
// EXACT: x times the power of two that brings |x| to 2^14 (to 2^15): exact in
// fp16 but for what lies 2^-38 below |x|; the transpose is a pair in any case
// (its second plane zero).  Else 2^(10 + e) X_0, X_0 = x / (|x| + 1e-7),
// rounded, and in XL (m x n) what the rounding left.  e, for an X between
// steps, is zero but where |x| lies so far below 1e-7 that no iterate passes 1
// (|X_0| below 2^knee): 2^10 X would fall out of fp16's range there, and
// 2^(10 + e) X stays below 2^15 throughout.
template <int T, int PLANES, bool EXACT>
__global__ __launch_bounds__(256) void ortho_start_kernel(const OrthoParams p, const double* parts, uint16_t* X,
                                                          uint16_t* XT, uint16_t* XL, OrthoScales* scales, int32_t tiles_m,
                                                          int32_t tiles_n, int32_t sums, int32_t knee) {
  constexpr int KEPT = EXACT ? PLANES : 2;
  __shared__ double lds[4];
  __shared__ uint16_t tile[KEPT][64][66];
  const uint32_t id = blockIdx.x;
  const int32_t tn = id % tiles_n, tm = id / tiles_n % tiles_m;
  const int64_t b = id / tiles_n / tiles_m;
  const int64_t mp = 64 * (int64_t)tiles_m, np = 64 * (int64_t)tiles_n;
  const double sum = block_sum((int32_t)threadIdx.x < sums ? parts[b * kNormParts + threadIdx.x] : 0.0, lds);
  const double norm = sqrt(sum), inv = 1.0 / (norm + 1e-7);
  const double x0 = norm * inv;
  const int32_t k = x0 > 0.0 ? ilogb(x0) + 1 : 0;                        // |X_0| < 2^k
  const int32_t e = x0 > 0.0 && k <= knee ? min(5 + knee - k, 100) : 0;  // (NaN: 0)
  const bool writes_scales = tm == 0 && tn == 0 && threadIdx.x == 0;
  double f;
  if constexpr (!EXACT) {
    f = ldexp(inv, 10 + e);
    if (writes_scales) scales[b].v[kScaleGram] = ldexpf(1.f, -2 * e), scales[b].v[kScaleResult] = ldexpf(1.f, -e);
  } else {
    // infinite or NaN norms make every scale NaN
    const int32_t en = norm > 0.0 && norm < __builtin_inf() ? ilogb(norm) : 0;
    f = ldexp(1.0, 14 - en);
    const double fx = norm < __builtin_inf() ? inv / f : __builtin_nan("");
    if (writes_scales) {
      scales[b].v[kScaleGram] = (float)(fx * fx * 4096.0), scales[b].v[kScaleResult] = (float)(fx / 64.0);
      scales[b].v[kScaleKeep] = (float)ldexp(fx / 64.0, 10 + e);
      scales[b].v[kScaleGramKept] = ldexpf(1.f, 12 - 2 * (10 + e)), scales[b].v[kScaleResultKept] = ldexpf(1.f, -6 - (10 + e));
    }
  }
  const int64_t i0 = 64 * (int64_t)tm, j0 = 64 * (int64_t)tn;
  const bool along_rows = p.x_rs == 1 && p.x_cs != 1;
  const int32_t u = threadIdx.x & 7, w = threadIdx.x >> 3;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    // eight along x's contiguous axis
    const int32_t il = along_rows ? 8 * u : 32 * k + w, jl = along_rows ? 32 * k + w : 8 * u;
    float v[8];
    ortho_load8<T>(p, b, i0 + il, j0 + jl, p.n, along_rows, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y = as_computed((float)(v[e] * f));
#pragma unroll
      for (int q = 0; q < KEPT; ++q) {
        const uint16_t h = from_f32<DT_F16>(y);
        tile[q][along_rows ? il + e : il][along_rows ? jl : jl + e] = h;
        y -= to_f32<DT_F16>(h);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int32_t r = 32 * k + w;
#pragma unroll
    for (int q = 0; q < PLANES; ++q) {
      u16x8 row, col;
#pragma unroll
      for (int e = 0; e < 8; ++e) row[e] = tile[q][r][8 * u + e], col[e] = tile[q][8 * u + e][r];
      *(u16x8*)(X + plane_at<PLANES>(b * mp + i0 + r, np, j0 + 8 * u) + 32 * q) = row;
      *(u16x8*)(XT + plane_at<EXACT ? 2 : PLANES>(b * np + j0 + r, mp, i0 + 8 * u) + 32 * q) = col;
    }
    if constexpr (KEPT > PLANES) {
      u16x8 row;
#pragma unroll
      for (int e = 0; e < 8; ++e) row[e] = tile[1][r][8 * u + e];
      *(u16x8*)(XL + (b * mp + i0 + r) * np + j0 + 8 * u) = row;
    }
    if constexpr (EXACT && PLANES == 1) *(u16x8*)(XT + plane_at<2>(b * np + j0 + r, mp, i0 + 8 * u) + 32) = u16x8{0, 0, 0, 0, 0, 0, 0, 0};
  }
}

// D = alpha P Q^T + beta E + diag I (with `scales`, alpha times the matrix's
// own), K contiguous in P and Q.  One or two products of the same P in one
// launch.  The kernels' MODE: P and Q of one plane; pairs, P0 Q0 + P1 Q0 +
// P0 Q1; or pairs with P1 = 0.  OP: planes of E and of the result.
constexpr int kPlain = 0, kPairs = 1, kPlainByPair = 2;
struct OrthoGemm {
  const uint16_t* P;             // (m, k)
  const uint16_t* Q[2];          // (n, k)
  const uint16_t* E;             // (m, n), or NULL
  uint16_t* O[2];                // (m, n); sym: its transpose as well
  uint16_t* low;                 // OP 1: the second plane of E and of O, apart from them and in place, or NULL
  uint16_t* OT;                  // (n, m), or NULL
  int64_t P_bs, Q_bs, E_bs, O_bs;
  int32_t m, n, k;               // padded: multiples of 64
  float alpha[2], beta, diag;    // with scales: alpha and beta times one of the matrix's
  const OrthoScales* scales;     // or NULL
  int32_t scale;                 // which of them
  int32_t sym;
  int32_t products;              // 1 or 2
  int32_t tiles_m, tiles_n, batch;
  int32_t first, parts;          // tiles from this one on, each in parts x parts workgroups
  // the last step's result instead of O
  void* d;
  int64_t rows, cols, d_bs, d_rs, d_cs;
  int32_t d_type;
};

struct OrthoTile {
  int32_t batch, product, tm, tn;
  bool mirror;  // off the diagonal of a symmetric result
  float alpha, beta;
};

// The tile of a workgroup.  Workgroups go to the 8 XCDs in turn: each XCD
// takes a contiguous range of (matrix, product, tile), the tiles of a matrix
// in groups of eight tile rows, so that what runs on one XCD at a time shares
// rows of both operands in its L2 (without it 16 x 1000 x 520's products ran
// at the Infinity Cache's rate).  Symmetric results: the tiles tm <= tn.
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoGemm& g) {
  constexpr uint32_t GR = 8;
  OrthoTile o;
  const uint32_t total = gridDim.x, x = blockIdx.x & 7, q = total >> 3, r = total & 7;
  const uint32_t at = x * q + (x < r ? x : r) + (blockIdx.x >> 3), parts = g.parts * g.parts;
  const uint32_t id = g.first + at / parts, part = at % parts;
  const uint32_t nt = (uint32_t)g.tiles_n, per = g.sym ? nt * (nt + 1) / 2 : nt * (uint32_t)g.tiles_m;
  o.batch = id / (per * g.products);
  uint32_t t = id % (per * g.products);
  o.product = t >= per;
  t -= o.product * per;
  if (g.sym) {
    uint32_t g0 = 0, R, tri;
    for (;; g0 += GR) {
      R = nt - g0 < GR ? nt - g0 : GR, tri = R * (R + 1) / 2;
      const uint32_t count = tri + R * (nt - g0 - R);
      if (t < count) break;
      t -= count;
    }
    if (t < tri) {
      uint32_t c = 0;
      while ((c + 1) * (c + 2) / 2 <= t) ++c;
      o.tn = g0 + c, o.tm = g0 + t - c * (c + 1) / 2;
    } else {
      o.tn = g0 + R + (t - tri) / R, o.tm = g0 + (t - tri) % R;
    }
  } else {
    const uint32_t span = GR * nt, first = t / span * GR, left = g.tiles_m - first;
    const uint32_t R = left < GR ? left : GR, in = t % span;
    o.tm = first + in % R, o.tn = in / R;
  }
  o.mirror = g.sym && o.tm != o.tn;
  o.tm = o.tm * g.parts + part % g.parts, o.tn = o.tn * g.parts + part / g.parts;
  o.alpha = o.product ? g.alpha[1] : g.alpha[0];
  o.beta = g.beta;
  if (g.scales) {
    const float s = g.scales[o.batch].v[g.scale];
    o.alpha *= s, o.beta *= s;
  }
  return o;
}

template <int W>
struct Halves {
  typedef uint16_t vec __attribute__((ext_vector_type(W)));
};
// W consecutive values of E at (m, n ..): both planes, the second zero where
// there is none
template <int OP, int W>
__device__ __forceinline__ void ortho_load(const OrthoGemm& g, const OrthoTile& o, int32_t m, int32_t n,
                                           typename Halves<W>::vec (&x)[2]) {
  typedef typename Halves<W>::vec vec;
  const int64_t at = o.batch * g.E_bs + plane_at<OP>(m, g.n, n);
  x[0] = *(const vec*)(g.E + at);
  if constexpr (OP == 2)
    x[1] = *(const vec*)(g.E + at + 32);
  else if (g.low)
    x[1] = *(const vec*)(g.low + at);
  else
    x[1] = vec{};
}
// W consecutive values of D at (m, n ..) from the sums and E's
template <int W>
__device__ __forceinline__ void ortho_value(const OrthoGemm& g, const OrthoTile& o, int32_t m, int32_t n,
                                            const typename Halves<W>::vec (&x)[2], float (&v)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] *= o.alpha;
  if (g.E) {
#pragma unroll
    for (int q = 1; q >= 0; --q)
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = __builtin_fmaf(o.beta, to_f32<DT_F16>(x[q][e]), v[e]);
  }
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = as_computed(m == n + e ? v[e] + g.diag : v[e]);
}

// ... stored along a row
template <int OP, int W>
__device__ __forceinline__ void ortho_store(uint16_t* row, const float (&v)[W]) {
  typedef uint16_t vec __attribute__((ext_vector_type(W)));
  float r[W];
#pragma unroll
  for (int e = 0; e < W; ++e) r[e] = v[e];
#pragma unroll
  for (int q = 0; q < OP; ++q) {
    vec x;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      x[e] = from_f32<DT_F16>(r[e]);
      r[e] = as_computed(r[e] - to_f32<DT_F16>(x[e]));
    }
    *(vec*)(row + 32 * q) = x;
  }
}
// ... to the result's type, `left` of them, `step` apart
template <int W>
__device__ __forceinline__ void ortho_result(const OrthoGemm& g, uint16_t* d, int64_t step, int64_t left, const float (&v)[W]) {
  typedef uint16_t loose __attribute__((ext_vector_type(W), aligned(2)));
  loose x;
#pragma unroll
  for (int e = 0; e < W; ++e) x[e] = g.d_type == OT_BF16 ? from_f32<DT_BF16>(v[e]) : from_f32<DT_F16>(v[e]);
  if (step == 1 && left >= W) {
    *(loose*)d = x;
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < left) d[e * step] = x[e];
  }
}

// what a tile's second pass, along its columns, stores
__device__ __forceinline__ bool ortho_columns(const OrthoGemm& g, const OrthoTile& o) {
  return g.d ? g.d_rs == 1 && g.d_cs != 1 : o.mirror || g.OT;
}
// W consecutive n of row m
template <int OP, int W>
__device__ __forceinline__ void ortho_row(const OrthoGemm& g, const OrthoTile& o, bool columns, int32_t m, int32_t n,
                                          const typename Halves<W>::vec (&x)[2], float (&v)[W]) {
  ortho_value<W>(g, o, m, n, x, v);
  if (!g.d) {
    const int64_t at = o.batch * g.O_bs + plane_at<OP>(m, g.n, n);
    ortho_store<OP, W>((o.product ? g.O[1] : g.O[0]) + at, v);
    if (OP == 1 && g.low) {
      float left[W];
#pragma unroll
      for (int e = 0; e < W; ++e) left[e] = v[e] - to_f32<DT_F16>(from_f32<DT_F16>(v[e]));
      ortho_store<1, W>(g.low + at, left);
    }
  } else if (!columns && m < g.rows)
    ortho_result<W>(g, (uint16_t*)g.d + o.batch * g.d_bs + m * g.d_rs + n * g.d_cs, g.d_cs, g.cols - n, v);
}
// W consecutive m of column n
template <int OP, int W>
__device__ __forceinline__ void ortho_column(const OrthoGemm& g, const OrthoTile& o, int32_t m, int32_t n, float (&v)[W]) {
  if (!g.d)
    ortho_store<OP, W>((g.OT ? g.OT : o.product ? g.O[1] : g.O[0]) + o.batch * g.O_bs + plane_at<OP>(n, g.m, m), v);
  else if (n < g.cols)
    ortho_result<W>(g, (uint16_t*)g.d + o.batch * g.d_bs + m + n * g.d_cs, 1, g.rows - m, v);
}

// An MFMA whose accumulator stays in AGPRs.  The statement is opaque to the
// compiler: results are read only after agprs_settled.
__device__ __forceinline__ void mfma_agpr(floatx4& c, const half8& a, const half8& b) {
  asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// The MFMAs above are inline assembly, so the compiler inserts no wait states
// before their results are read: empty volatile statements that re-define
// every accumulator hold the MFMAs before an idle of 32 cycles and every read
// after it.
template <int FM, int FN>
__device__ __forceinline__ void agprs_settled(floatx4 (&acc)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; j += 2) asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; j += 2) asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
}

// ---------------------------------------------------------------------------
// Outputs too small for 256 x 256 tiles to fill the chip: BM x BN tiles, KG
// groups of four waves that take the K-tiles in turn (their sums meet in
// LDS), each with a ring of four K-tiles in LDS, so that a copy has two
// K-tiles of compute to land.  Fragments are read while the products before
// theirs run, across the one barrier of a K-tile too.  Measured: 128 x 128
// tiles, 240 workgroups (16 x 520^2 from pairs, 18 K-tiles) 24 us; 64 x 64 tiles,
// 136 workgroups (1024^2 from K = 4096) 15 us, from K = 1024 7.5.
// ---------------------------------------------------------------------------
template <int BM, int BN, int KG, int MODE, int OP>
__global__ __launch_bounds__(256 * KG, KG) void ortho_gemm_kernel(const OrthoGemm g) {
  constexpr int STAGES = 4;
  constexpr int TM = BM / 2, TN = BN / 2, FM = TM / 16, FN = TN / 16;
  constexpr int ABYTES = BM * kRowBytes, BBYTES = BN * kRowBytes, STAGE = ABYTES + BBYTES;
  constexpr int PITCH = BN + 4;  // floats a row of the finished tile
  // sixteen accumulators: left to it, the compiler moved them between
  // register files in every K-tile (and an accumulator comes up again only
  // after fifteen others)
  constexpr bool AGPR = FM * FN >= 16;
  constexpr int LDS = KG * STAGES * STAGE;
  static_assert(BM * PITCH * 4 <= LDS && LDS <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) char smem[LDS];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
  const int32_t group = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const OrthoTile o = ortho_tile(g);
  const int32_t m0 = o.tm * BM, n0 = o.tn * BN;
  if (m0 >= g.m || n0 >= g.n) return;  // a part of a tile at the edge
  const int32_t rows_a = g.m - m0 < BM ? g.m - m0 : BM, rows_b = g.n - n0 < BN ? g.n - n0 : BN;
  const int64_t row = MODE == kPlain ? g.k : 2 * (int64_t)g.k;
  LoaderKVec<BM, 256, 0, 2> la(g.P + o.batch * g.P_bs + m0 * row, rows_a, row, 1, row, wave, lane);
  LoaderKVec<BN, 256, 0, 2> lb((o.product ? g.Q[1] : g.Q[0]) + o.batch * g.Q_bs + n0 * row, rows_b, row, 1, row, wave, lane);
  constexpr int LOADS = decltype(la)::ITERS + decltype(lb)::ITERS;
  const int32_t a_row0 = (wave & 1) * TM, b_row0 = (wave >> 1) * TN;
  char* ring = smem + group * (STAGES * STAGE);

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int32_t T = (int32_t)(row / 64), rounds = (T + KG - 1) / KG;
  constexpr int32_t kPast = 1 << 24;  // a K-tile past every K: zeros
  auto issue = [&](int32_t i) {
    const int32_t t = i * KG + group;
    char* at = ring + (i & (STAGES - 1)) * STAGE;
    la.issue(t < T ? t : kPast, at);
    lb.issue(t < T ? t : kPast, at + ABYTES);
  };
  // the two halves of a K-tile: 32 values each, or the planes of 32 values
  struct Half {
    half8 a[FM], b[FN];
  };
  auto read = [&](int32_t i, int half, Half& h) {
    const char* cur = ring + (i & (STAGES - 1)) * STAGE;
#pragma unroll
    for (int a = 0; a < FM; ++a)
      if (MODE != kPlainByPair || half == 0) h.a[a] = read_frag<LOAD_KVEC, BM, 0>(cur, lane, a_row0 + 16 * a, half);
#pragma unroll
    for (int b = 0; b < FN; ++b) h.b[b] = read_frag<LOAD_KVEC, BN, 0>(cur + ABYTES, lane, b_row0 + 16 * b, half);
  };
  auto multiply = [&](const half8(&x)[FM], const half8(&y)[FN]) {
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        if constexpr (AGPR) mfma_agpr(acc[a][b], y[b], x[a]);
        else acc[a][b] = mfma16<DT_F16>(y[b], x[a], acc[a][b]);
      }
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue(i);
  wait_vmem_n<(STAGES - 2) * LOADS>();
  phase_barrier();
  Half first, second, other;
  read(0, 0, first);
  // K-tile i, its first half in `x`; the next one's goes to `y`
  auto tile = [&](int32_t i, Half& x, Half& y) {
    wait_vmem_n<(STAGES - 3) * LOADS>();  // K-tile i + 1 has landed
    phase_barrier();                      // for every wave, and K-tile i - 1 is no longer read
    issue(i + STAGES - 1);
    read(i, 1, second);
    __builtin_amdgcn_sched_barrier(0);
    multiply(x.a, x.b);
    __builtin_amdgcn_sched_barrier(0);
    read(i + 1, 0, y);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MODE == kPlain) multiply(second.a, second.b);
    if constexpr (MODE == kPairs) multiply(second.a, x.b);
    if constexpr (MODE != kPlain) multiply(x.a, second.b);
    __builtin_amdgcn_sched_barrier(0);
  };
  int32_t i = 0;
#pragma clang loop unroll(disable)
  do {
    tile(i, first, other);
    // (with one group the sum over an odd number of K-tiles ends on a K-tile
    // of zeros)
    tile(i + 1, other, first);
    i += 2;
  } while (i < rounds);
  wait_vmem();
  if constexpr (AGPR) agprs_settled(acc);
  __syncthreads();

  // E's values, all requested before any is used
  const bool columns = ortho_columns(g, o);
  constexpr int PIECES = BM * BN / 8 / (256 * KG);
  auto row_of = [](int q) { return (int32_t)(threadIdx.x + 256 * KG * q) / (BN / 8); };
  auto col_of = [](int q) { return 8 * ((int32_t)(threadIdx.x + 256 * KG * q) % (BN / 8)); };
  u16x8 ev[PIECES][2];
  if (g.E) {
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
      if (m0 + row_of(q) < g.m && n0 + col_of(q) < g.n) ortho_load<OP, 8>(g, o, m0 + row_of(q), n0 + col_of(q), ev[q]);
  }
  // the groups' sums, one after the other, into the finished tile
  float* done = (float*)smem;
#pragma unroll
  for (int k = KG - 1; k >= 0; --k) {
    if (group == k) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          floatx4* to = (floatx4*)(done + (a_row0 + 16 * i + (lane & 15)) * PITCH + b_row0 + 16 * j + 4 * (lane >> 4));
          *to = k < KG - 1 ? *to + acc[i][j] : acc[i][j];
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < PIECES; ++q) {
    const int32_t ml = row_of(q), nl = col_of(q);
    floatx4* at = (floatx4*)(done + ml * PITCH + nl);
    if (m0 + ml >= g.m || n0 + nl >= g.n) continue;
    const floatx4 lo = at[0], hi = at[1];
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    ortho_row<OP, 8>(g, o, columns, m0 + ml, n0 + nl, ev[q], v);
    if (columns) at[0] = floatx4{v[0], v[1], v[2], v[3]}, at[1] = floatx4{v[4], v[5], v[6], v[7]};
  }
  if (!columns) return;
  __syncthreads();
  // sixteen columns by four groups of 8 rows to a wave's reads: two lanes to a bank,
  // and 64 bytes of every column stored together
#pragma unroll
  for (int q = 0; q < PIECES; ++q) {
    const int32_t t = threadIdx.x + 256 * KG * q, ml = 8 * (t / 16 % (BM / 8)), nl = t % 16 + 16 * (t / (2 * BM));
    if (m0 + ml >= g.m || n0 + nl >= g.n) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = done[(ml + e) * PITCH + nl];
    ortho_column<OP, 8>(g, o, m0 + ml, n0 + nl, v);
  }
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles: four waves, one per SIMD, each a 128 x 128 block with its
// accumulators in AGPRs, and a ring of five operand K-tiles in LDS, on the
// schedule of gemm_f16_w4r_kernel (gemm_f16.hip), which see: operand tile q
// (P's K-tile q / 2 for even q, Q's for odd q) in slot q % 5; per K-tile the
// reads of its first half beside the last products of the K-tile before, the
// first half's products beside the reads of the second, all but the last of
// the second half's, one barrier.  Measured: 512 tiles of a symmetric 8192^2
// from K = 8192 in 410 to 450 us (1.2 to 1.3 PFLOP/s; MFMA busy 66%), 1024 tiles
// of an 8192^2 stored in both orientations and with its second plane in 935 to
// 990 us (1.11 to 1.18; 56%).
// ---------------------------------------------------------------------------
template <int MODE, int OP>
__global__ __launch_bounds__(256, 1) void ortho_ring_kernel(const OrthoGemm g) {
  constexpr int F = 8, SLOT = 256 * kRowBytes, LOADS = 8;
  __shared__ __attribute__((aligned(1024))) char smem[5 * SLOT];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const OrthoTile o = ortho_tile(g);
  const int32_t m0 = o.tm * 256, n0 = o.tn * 256;
  const int32_t rows_a = g.m - m0 < 256 ? g.m - m0 : 256, rows_b = g.n - n0 < 256 ? g.n - n0 : 256;
  const int64_t row = MODE == kPlain ? g.k : 2 * (int64_t)g.k;
  LoaderKVec<256, 256, 0, 2> la(g.P + o.batch * g.P_bs + m0 * row, rows_a, row, 1, row, wave, lane);
  LoaderKVec<256, 256, 0, 2> lb((o.product ? g.Q[1] : g.Q[0]) + o.batch * g.Q_bs + n0 * row, rows_b, row, 1, row, wave, lane);
  floatx4 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int32_t a_row0 = (wave & 1) * 128, b_row0 = (wave >> 1) * 128;
  const int32_t T = (int32_t)(row / 64);
  __builtin_assume(T >= 1);
  // past the last K-tile the look-ahead copies repeat it and are not read
  auto kt = [&](int32_t u) { return u < T ? u : T - 1; };
  auto slot = [&](int32_t q) { return smem + q * SLOT; };
  auto copy_a = [&](int32_t u, char* dst, int j) { la.issue_full(kt(u), dst, j); };
  auto copy_b = [&](int32_t u, char* dst, int j) { lb.issue_full(kt(u), dst, j); };
  half8 fa0[F], fb0[F], fa1[F], fb1[F];
  typedef __attribute__((address_space(3))) const half8 lds_h8;
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
  auto read = [&](int r, int ks, half8(&fa)[F], half8(&fb)[F]) {
    if (r < F)
      fb[r] = *(lds_h8*)(uintptr_t)(bB[ks][r & 1] + 4096u * (uint32_t)(r >> 1));
    else
      fa[r - F] = *(lds_h8*)(uintptr_t)(bA[ks][r & 1] + 4096u * (uint32_t)((r - F) >> 1));
  };
#pragma unroll
  for (int j = 0; j < LOADS; ++j) copy_a(0, slot(0), j);
#pragma unroll
  for (int j = 0; j < LOADS; ++j) copy_b(0, slot(1), j);
#pragma unroll
  for (int j = 0; j < LOADS; ++j) copy_a(1, slot(2), j);
  // the first tile's first part computes with zero fragments (adds nothing)
#pragma unroll
  for (int i = 0; i < F; ++i) fa0[i] = fa1[i] = half8{}, fb1[i] = half8{};
  // rows i0 .. i0 + 3 of the block, products of the first (0) or second half,
  // or across them (pairs), step q of 16
  auto products = [&](int i0, int q, const half8(&fa)[F], const half8(&fb)[F]) {
#pragma unroll
    for (int e = 2 * q; e < 2 * q + 2; ++e) mfma_agpr(acc[i0 + e / F][e % F], fb[e % F], fa[i0 + e / F]);
  };
  wait_vmem_n<LOADS>();
  phase_barrier();
  int32_t sa = 0;  // slot of P's K-tile t; Q's in the next one
  int32_t t = 0;
  bases(0, 1);
  // one copy of the loop body: a peeled or unswitched copy would give the
  // accumulators a second path to the epilogue
#pragma clang loop unroll(disable)
  do {
    const int32_t s3 = sa + 3 >= 5 ? sa - 2 : sa + 3, s4 = sa == 0 ? 4 : sa - 1;
    if constexpr (MODE == kPlain) {
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        read(q, 0, fa0, fb0);
        if (!(q & 1)) copy_b(t + 1, slot(s3), q >> 1);
        products(F / 2, q, fa1, fb1);  // K-tile t - 1's
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        read(q, 1, fa1, fb1);
        if (q & 1) copy_a(t + 2, slot(s4), q >> 1);
        products(q < 8 ? 0 : F / 2, 2 * (q & 7), fa0, fb0);
        products(q < 8 ? 0 : F / 2, 2 * (q & 7) + 1, fa0, fb0);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) products(0, q, fa1, fb1);
    } else {
      // P0 of K-tile t - 1 times its Q1, rows 4 to 7, is what is left of it:
      // Q0 and the first rows of P0 are free
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        if (q < 12) read(q, 0, fa0, fb0);
        if (!(q & 1)) copy_b(t + 1, slot(s3), q >> 1);
        products(F / 2, q, fa0, fb1);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        if (q < 4) read(12 + q, 0, fa0, fb0);
        if (q & 1) copy_a(t + 2, slot(s4), q >> 1);
        products(0, q, fa0, fb0);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        if (MODE == kPairs || q < F) read(q, 1, fa1, fb1);
        products(F / 2, q, fa0, fb0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (MODE == kPairs) {
#pragma unroll
        for (int q = 0; q < 32; ++q) products(q < 16 ? 0 : F / 2, q & 15, fa1, fb0);
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) products(0, q, fa0, fb1);
    }
    const int32_t na = sa + 2 >= 5 ? sa - 3 : sa + 2;
    bases(na, na == 4 ? 0 : na + 1);
    wait_vmem_n<LOADS>();  // in flight after this: P's K-tile t + 2
    phase_barrier();
    sa = na;
  } while (++t < T);
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    if constexpr (MODE == kPlain) products(F / 2, q, fa1, fb1);
    else products(F / 2, q, fa0, fb1);
  }
  wait_vmem();
  agprs_settled(acc);
  // every wave's copies have landed and its reads of the ring are done
  __syncthreads();
  // the wave's block through its own 32 KiB of LDS, 64 rows at a time
  const bool columns = ortho_columns(g, o);
  char* region = smem + wave * 32768;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
        *(floatx4*)(region + rows_chunk(16 * i + (lane & 15), 4 * j + (lane >> 4))) = acc[4 * h + i][j];
    const int32_t mb = m0 + a_row0 + 64 * h, nb = n0 + b_row0;
#pragma unroll 8
    for (int it = 0; it < 32; ++it) {
      const int32_t r = 2 * it + (lane >> 5), q = lane & 31;
      floatx4* at = (floatx4*)(region + rows_chunk(r, q));
      if (mb + r >= g.m || nb + 4 * q >= g.n) continue;
      u16x4 e[2];
      if (g.E) ortho_load<OP, 4>(g, o, mb + r, nb + 4 * q, e);
      const floatx4 x = *at;
      float v[4] = {x[0], x[1], x[2], x[3]};
      ortho_row<OP, 4>(g, o, columns, mb + r, nb + 4 * q, e, v);
      if (columns) *at = floatx4{v[0], v[1], v[2], v[3]};
    }
    if (columns) {
#pragma unroll 4
      for (int it = 0; it < 32; ++it) {
        const int32_t n = 4 * it + (lane >> 4), m = 4 * (lane & 15);
        if (mb + m >= g.m || nb + n >= g.n) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *(const float*)(region + rows_chunk(m + e, n >> 2) + 4 * (n & 3));
        ortho_column<OP, 4>(g, o, mb + m, nb + n, v);
      }
    }
  }
}

// Workgroups of tiles of `side`
int64_t ortho_tiles(const OrthoGemm& g, int64_t side) {
  const int64_t tm = (g.m + side - 1) / side, tn = (g.n + side - 1) / side;
  return (g.sym ? tn * (tn + 1) / 2 : tm * tn) * g.batch * g.products;
}

template <int MODE, int OP>
void launch_tiles(OrthoGemm g, int32_t side, int64_t first, int64_t count, hipStream_t s) {
  const dim3 grid((uint32_t)(count * g.parts * g.parts));
  g.first = (int32_t)first;
  g.tiles_m = (g.m + side * g.parts - 1) / (side * g.parts), g.tiles_n = (g.n + side * g.parts - 1) / (side * g.parts);
  if (side == 256)
    hipLaunchKernelGGL((ortho_ring_kernel<MODE, OP>), grid, dim3(256), 0, s, g);
  else if (side == 128)
    hipLaunchKernelGGL((ortho_gemm_kernel<128, 128, 1, MODE, OP>), grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((ortho_gemm_kernel<64, 64, 2, MODE, OP>), grid, dim3(512), 0, s, g);
}

// What a last round of 256 x 256 tiles would leave most CUs without goes to 64
// x 64 tiles: a symmetric 8192 x 8192 result has 528 tiles, and a third round
// for 16 of them took 180 of 596 us.
int64_t whole_tiles(int32_t side, int64_t all) {
  const int64_t rest = all % 256;
  return side == 256 && all > 256 && rest <= 64 ? all - rest : all;
}

// The tile with the least time: rounds over the 256 CUs (a workgroup to each)
// times a tile's start and end and its K-loop (`products` of K values), padding
// included.  The constants are a fit to whole calls with each tile forced, 25
// sizes and batches in fp16 and bf16, most within 10%.  256, 128 and 64 forced, us:
// 256 x (200 x 400) bf16 1056, 865, 1174; 256 x (320 x 640) fp16 2699, 2065, 2505;
// 100 x (300 x 300) fp16 1119, 799, 743; 1024 x 4096 bf16 995, 398, 268;
// 2100 x 2300 bf16 1069, 533, 558; 8192 x 8192 bf16 9626, 13021, 18972.
int32_t choose_side(const OrthoGemm& g, int32_t products) {
  struct {
    int32_t side;
    double start, k;  // us a tile, ns a value of K
  } constexpr tiles[3] = {{256, 27.0, 18.0}, {128, 6.3, 7.3}, {64, 3.1, 2.5}};
  const double k = (double)g.k * products * 1e-3;
  int32_t best = 0;
  double least = 0.0;
  for (const auto& t : tiles) {
    const int64_t all = ortho_tiles(g, t.side), whole = whole_tiles(t.side, all);
    if (all >= (int64_t)1 << 23) continue;  // 512 threads each would not fit a grid
    double cost = (double)((whole + 255) / 256) * (t.start + k * t.k);
    if (whole < all) cost += (double)((16 * (all - whole) + 255) / 256) * (tiles[2].start + k * tiles[2].k);
    if (best == 0 || cost < least) best = t.side, least = cost;
  }
  return best;
}

template <int MODE, int OP>
hipError_t run_gemm(OrthoGemm g, hipStream_t s) {
  const int32_t side = choose_side(g, MODE == kPairs ? 3 : MODE == kPlainByPair ? 2 : 1);
  const int64_t all = ortho_tiles(g, side), whole = whole_tiles(side, all);
  g.parts = 1;
  launch_tiles<MODE, OP>(g, side, 0, whole, s);
  if (whole < all) {
    g.parts = 4;
    launch_tiles<MODE, OP>(g, 64, whole, all - whole, s);
  }
  return hipGetLastError();
}

// planes that hold x on the Gram matrix's way
constexpr int x_planes(int type) { return type == OT_F32 ? 2 : 1; }

template <int T>
hipError_t start(const OrthoParams& p, bool exact, double* parts, uint16_t* X, uint16_t* XT, uint16_t* XL,
                 OrthoScales* scales, int32_t knee, hipStream_t s) {
  const int32_t tm = (int32_t)(pad64(p.m) / 64), tn = (int32_t)(pad64(p.n) / 64);
  const int64_t length = p.x_rs == 1 && p.x_cs != 1 ? p.m : p.n;
  int32_t across = 64 * kNormWaves;
  while (across > 1 && 4 * (int64_t)across >= length) across /= 2;
  // 16384 values to a workgroup
  const int64_t want = (p.m * p.n + 16383) / 16384;
  const int32_t sums = (int32_t)(want < kNormParts ? want : kNormParts);
  hipLaunchKernelGGL(ortho_norm_kernel<T>, dim3(sums, p.batch), dim3(64 * kNormWaves), 0, s, p, parts, across);
  const dim3 grid((uint32_t)((int64_t)p.batch * tm * tn)), block(256);
  if (exact)
    hipLaunchKernelGGL((ortho_start_kernel<T, x_planes(T), true>), grid, block, 0, s, p, parts, X, XT, XL, scales, tm, tn, sums,
                       knee);
  else
    hipLaunchKernelGGL((ortho_start_kernel<T, 1, false>), grid, block, 0, s, p, parts, X, XT, XL, scales, tm, tn, sums, knee);
  return hipGetLastError();
}
hipError_t start(const OrthoParams& p, bool exact, double* parts, uint16_t* X, uint16_t* XT, uint16_t* XL,
                 OrthoScales* scales, int32_t knee, hipStream_t s) {
  switch (p.x_type) {
    case OT_F16: return start<OT_F16>(p, exact, parts, X, XT, XL, scales, knee, s);
    case OT_BF16: return start<OT_BF16>(p, exact, parts, X, XT, XL, scales, knee, s);
    default: return start<OT_F32>(p, exact, parts, X, XT, XL, scales, knee, s);
  }
}

enum Way { kSmallGram, kGram, kDirect };

// How much the steps amplify anywhere: a rounding in X grows in a step by at
// most the largest slope of s -> a s + b s^3 + c s^5 over the singular values
// that can occur, 0 to r, r being 1 at first and then what the step makes of
// it.  (Five default steps: 855, six 3400.)
float slope_of(const OrthoParams& p) {
  float slope = 1.f, r = 1.f;
  for (int32_t t = 0; t < p.steps; ++t) {
    const float a = p.coefficients[3 * t], b = p.coefficients[3 * t + 1], c = p.coefficients[3 * t + 2];
    const float top = r * r;
    float most = fabsf(a), next = 0.f;  // over the ends and where the slope, or the value, turns, in squares of s
    auto slope_at = [&](float g) { return a + g * (3.f * b + 5.f * c * g); };
    auto take_value = [&](float g) {
      if (g > 0.f && g <= top) next = fmaxf(next, fabsf(sqrtf(g) * (a + g * (b + c * g))));
    };
    most = fmaxf(most, fabsf(slope_at(top)));
    take_value(top);
    if (c != 0.f) {
      const float turn = -0.3f * b / c, in = 9.f * b * b - 20.f * a * c;
      if (turn > 0.f && turn < top) most = fmaxf(most, fabsf(slope_at(turn)));
      if (in >= 0.f) take_value((-3.f * b + sqrtf(in)) / (10.f * c)), take_value((-3.f * b - sqrtf(in)) / (10.f * c));
    } else if (b != 0.f) {
      take_value(-a / (3.f * b));
    }
    slope *= fmaxf(1.f, most), r = next;
  }
  return slope;
}

// Where |X_0| is below two to this power no iterate passes 1, and |X| grows
// at most in proportion to |X_0|: by |a| + |b| |X|^2 + |c| |X|^4 a step.
int32_t knee_of(const OrthoParams& p) {
  for (int32_t k = 0; k > -160; --k) {
    double u = ldexp(1.0, k);
    for (int32_t t = 0; t < p.steps && u <= 1.0; ++t)
      u *= fmax(1.0, fabs(p.coefficients[3 * t]) + u * u * (fabs(p.coefficients[3 * t + 1]) + u * u * fabs(p.coefficients[3 * t + 2])));
    if (u <= 1.0) return k;
  }
  return -160;
}

// Up to 128 rows: the Gram matrix's way in few launches.  Otherwise bf16
// results whose steps amplify a rounding of X by no more than kSingleSlope go
// the direct way, 15 m^2 n + 5 m^3 operations for five steps, where they have no
// more than four times as many columns as rows; the Gram matrix's multiplies
// pairs, 42 m^3 + 14 m^2 n in two cycles, and is the more accurate one.  Direct
// and Gram: 1000 x 1000 147 and 215 us, 1024 x 4096 240 and 281, x 8192 371 and
// 367, x 16384 634 and 501, 4096 x 4096 1.7 and 3.7 ms, 8192 x 8192 9.3 and 21.8.
//
// The direct way keeps X as a pair, and a X comes from both planes; what is
// rounded to fp16 is X as a factor, G and B.  (X as one plane was wrong: what
// its rounding leaves in directions where x has nothing grows by a each step,
// 4e-2 of a result of rank 8.)  64-bit simulation of these roundings,
// relative 2-norm, 256 x 256 to 1000 x 1000, five default steps: noise 1.1e-3
// to 1.4e-3, rank 1 to 64 1e-4 to 1e-3, singular values over two or four decades
// 7e-4 to 1.2e-3, a few equal rows among zeros up to 2.8e-3; a bf16 result's own
// rounding is 1.7e-3.  Steps that amplify more (slope 3e4: 1e-2 of a result of
// rank 8) and fp16 results (own rounding 2.1e-4) take the pairs.
constexpr float kSingleSlope = 1024.f;
constexpr int64_t kDirectColumns = 4;  // times the rows
Way way_of(const OrthoParams& p) {
  if (p.m <= kGramRows) return kSmallGram;
  // (not <= kSingleSlope: infinite or NaN as well)
  return p.d_type == OT_F16 || p.n > kDirectColumns * p.m || !(slope_of(p) <= kSingleSlope) ? kGram : kDirect;
}

struct Places {
  size_t scales, x, xt[2], low, mm[5], total;  // byte offsets behind the partial sums
};
Places places(const OrthoParams& p, Way way) {
  const bool gram = way == kGram, cycles = gram && ortho_cycle(p, 0) < p.steps;
  const size_t plane = (size_t)p.batch * pad64(p.m) * pad64(p.n) * 2, mm = (size_t)p.batch * pad64(p.m) * pad64(p.m) * 2;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  Places q;
  q.scales = up((size_t)p.batch * kNormParts * 8);
  q.x = q.scales + up((size_t)p.batch * sizeof(OrthoScales));
  // Gram: X a pair from the second cycle on, its transpose in any case
  q.xt[0] = q.x + plane * (cycles ? 2 : gram ? x_planes(p.x_type) : 1);
  q.xt[1] = q.xt[0] + plane * (gram ? 2 : 1);
  q.low = q.xt[1] + plane * (gram ? (cycles ? 2 : 0) : 1);
  size_t at = q.low + (gram ? 0 : plane);
  for (int i = 0; i < 5; ++i) {
    q.mm[i] = at;
    if (gram || i < 2) at += mm * (gram ? 2 : 1);
  }
  q.total = at;
  return q;
}

void to_result(const OrthoParams& p, OrthoGemm* g) {
  g->d = p.d, g->d_type = p.d_type, g->rows = p.m, g->cols = p.n;
  g->d_bs = p.d_bs, g->d_rs = p.d_rs, g->d_cs = p.d_cs;
}

hipError_t direct(const OrthoParams& p, hipStream_t s) {
  const Places q = places(p, kDirect);
  uint16_t* X = (uint16_t*)(p.ws + q.x);
  uint16_t* XT[2] = {(uint16_t*)(p.ws + q.xt[0]), (uint16_t*)(p.ws + q.xt[1])};
  uint16_t* XL = (uint16_t*)(p.ws + q.low);
  uint16_t *G = (uint16_t*)(p.ws + q.mm[0]), *B = (uint16_t*)(p.ws + q.mm[1]);
  OrthoScales* scales = (OrthoScales*)(p.ws + q.scales);
  const int32_t mp = (int32_t)pad64(p.m), np = (int32_t)pad64(p.n);
  const int64_t mn = (int64_t)mp * np, mm = (int64_t)mp * mp;
  constexpr float kDown = 0x1p-10f;  // what a stored value times it stands for
  hipError_t e = start(p, false, (double*)p.ws, X, XT[0], XL, scales, knee_of(p), s);
  for (int32_t k = 0; k < p.steps && e == hipSuccess; ++k) {
    const float a = p.coefficients[3 * k], b = p.coefficients[3 * k + 1], c = p.coefficients[3 * k + 2];
    // stored values carry 2^10, products of two 2^20
    OrthoGemm g{};
    g.batch = p.batch, g.products = 1;
    g.P = g.Q[0] = X, g.P_bs = g.Q_bs = mn;
    g.m = g.n = mp, g.k = np, g.alpha[0] = kDown, g.sym = 1;
    g.O[0] = G, g.O_bs = mm, g.scales = scales, g.scale = kScaleGram;
    if ((e = run_gemm<kPlain, 1>(g, s)) != hipSuccess) break;
    g.scales = nullptr;
    g.P = g.Q[0] = g.E = G, g.P_bs = g.Q_bs = g.E_bs = mm;
    g.k = mp, g.alpha[0] = c * kDown, g.beta = b;
    g.O[0] = B;
    if ((e = run_gemm<kPlain, 1>(g, s)) != hipSuccess) break;
    g.P = B, g.Q[0] = XT[k & 1], g.E = X, g.Q_bs = g.E_bs = mn;
    g.n = np, g.alpha[0] = kDown, g.beta = a, g.sym = 0;
    g.O[0] = X, g.OT = XT[(k + 1) & 1], g.low = XL, g.O_bs = mn;
    if (k + 1 == p.steps) {
      g.alpha[0] *= kDown, g.beta *= kDown, g.scales = scales, g.scale = kScaleResult;
      to_result(p, &g);
    }
    e = run_gemm<kPlain, 1>(g, s);
  }
  return e;
}

// PX: planes of x
template <int PX>
hipError_t gram(const OrthoParams& p, hipStream_t s) {
  const Places q = places(p, kGram);
  OrthoScales* scales = (OrthoScales*)(p.ws + q.scales);
  uint16_t *X = (uint16_t*)(p.ws + q.x), *XT[2] = {(uint16_t*)(p.ws + q.xt[0]), (uint16_t*)(p.ws + q.xt[1])};
  uint16_t* M[5];
  for (int i = 0; i < 5; ++i) M[i] = (uint16_t*)(p.ws + q.mm[i]);
  uint16_t *G = M[0], *P = M[1], *H = M[2];
  const int32_t mp = (int32_t)pad64(p.m), np = (int32_t)pad64(p.n);
  const int64_t mn = (int64_t)mp * np, mm = (int64_t)mp * mp * 2;
  constexpr float kG = 0x1p12f, kP = 0x1p6f;  // what G's planes, and those of P, H and Q, are multiplied by
  hipError_t e = start(p, true, (double*)p.ws, X, XT[0], nullptr, scales, knee_of(p), s);
  if (e != hipSuccess) return e;
  for (int32_t k = 0, cycle = 0; k < p.steps; ++cycle) {
    const int32_t end = k + ortho_cycle(p, k);
    const bool kept = cycle > 0;  // X is a pair that the cycle before made
    OrthoGemm g{};
    g.batch = p.batch, g.products = 1, g.sym = 1;
    g.P = g.Q[0] = X, g.P_bs = g.Q_bs = mn * (kept ? 2 : PX);
    g.m = g.n = mp, g.k = np, g.alpha[0] = 1.f, g.scales = scales, g.scale = kept ? kScaleGramKept : kScaleGram;
    g.O[0] = G, g.O_bs = mm;
    e = kept || PX == 2 ? run_gemm<kPairs, 2>(g, s) : run_gemm<kPlain, 2>(g, s);
    if (e != hipSuccess) return e;
    g.scales = nullptr, g.P_bs = g.Q_bs = g.E_bs = mm, g.k = mp;
    uint16_t* Q = nullptr;
    for (; k < end; ++k) {
      const float a = p.coefficients[3 * k], b = p.coefficients[3 * k + 1], c = p.coefficients[3 * k + 2];
      const bool first = Q == nullptr, last = k + 1 == end;
      // P = a I + b G + c G^2; the cycle's first is Q as well
      uint16_t* Pk = first ? M[3] : P;
      g.P = g.Q[0] = g.E = G, g.alpha[0] = c * (kP / (kG * kG)), g.beta = b * (kP / kG), g.diag = a * kP;
      g.O[0] = Pk;
      if ((e = run_gemm<kPairs, 2>(g, s)) != hipSuccess) return e;
      g.E = nullptr, g.diag = 0.f;
      uint16_t* next = Q == M[3] ? M[4] : M[3];
      g.P = Pk;
      g.products = (last ? 0 : 1) + (first ? 0 : 1);
      int i = 0;
      if (!last) g.Q[i] = G, g.O[i] = H, g.alpha[i] = 1.f / kG, ++i;
      if (!first) g.Q[i] = Q, g.O[i] = next, g.alpha[i] = 1.f / kP;
      if (g.products > 0 && (e = run_gemm<kPairs, 2>(g, s)) != hipSuccess) return e;
      g.products = 1;
      Q = first ? M[3] : next;
      if (last) continue;
      g.P = H, g.Q[0] = Pk, g.O[0] = G, g.alpha[0] = kG / (kP * kP);
      if ((e = run_gemm<kPairs, 2>(g, s)) != hipSuccess) return e;
    }
    // the transpose of Q X: X^T Q, Q being symmetric, so that the pair is the
    // second operand
    g.P = XT[cycle & 1], g.P_bs = 2 * mn, g.Q[0] = Q, g.Q_bs = mm;
    g.m = np, g.sym = 0, g.alpha[0] = 1.f, g.scales = scales;
    if (k == p.steps) {
      g.scale = kept ? kScaleResultKept : kScaleResult;
      to_result(p, &g);
      std::swap(g.rows, g.cols), std::swap(g.d_rs, g.d_cs);
      return kept || PX == 2 ? run_gemm<kPairs, 1>(g, s) : run_gemm<kPlainByPair, 1>(g, s);
    }
    g.O[0] = XT[(cycle + 1) & 1], g.OT = X, g.O_bs = 2 * mn;
    if (kept) g.scales = nullptr, g.alpha[0] = 1.f / kP;
    else g.scale = kScaleKeep;
    e = kept || PX == 2 ? run_gemm<kPairs, 2>(g, s) : run_gemm<kPlainByPair, 2>(g, s);
    if (e != hipSuccess) return e;
  }
  return e;
}

}  // namespace

// As many steps as multiply to 48 in their a's.  In directions where X has
// nothing Q grows with that product, next to parts of the size of 1, and G's
// errors there grow by a^2 a step; products of Q, P and G are symmetric only up
// to their rounding, and mirroring them mixes the one into the other.  A 64-bit
// simulation with fp32 sums and mirrored tiles of 32 (96 x 128; the same on the
// card): rank 1 3.2e-2, rank 8 8e-3 for five default steps in one cycle, 1.0e-4
// and 2.3e-5 in cycles of three, about as the iteration itself in 32 bits (7e-5,
// 1.7e-5).
int32_t ortho_cycle(const OrthoParams& p, int32_t first) {
  constexpr float kCycleGrowth = 48.f;
  float growth = 1.f;
  int32_t n = 0;
  for (; first + n < p.steps; ++n) {
    growth *= fmaxf(1.f, fabsf(p.coefficients[3 * (first + n)]));
    if (n > 0 && growth > kCycleGrowth) break;
  }
  return n;
}

size_t orthogonalize_workspace(const OrthoParams& p) {
  const Way way = way_of(p);
  return way == kSmallGram ? ortho_gram_workspace(p) : places(p, way).total;
}

// Every launch fits a grid (fewer than 2^32 work items along its x, 65536
// matrices along its y), and a matrix's planes 32-bit offsets.  The largest
// grids: up to 128 rows, the last launch's 256 threads for each 128 columns
// (the first one's 512 for up to 64 ranges of columns stay below 2^31);
// otherwise the start's 256 threads for each 64 x 64 values (the products' tiles
// are larger, or a few).  Up to 128 rows there is no limit of 32-bit offsets,
// but an X kept between cycles is to stay below 8 GiB of workspace a matrix.
bool orthogonalize_grid_ok(const OrthoParams& p) {
  const int64_t lim = (int64_t)1 << 31;
  if (p.batch >= 65536 || p.m >= lim || p.n >= lim) return false;
  if (way_of(p) == kSmallGram)
    return (double)p.batch * (double)((p.n + 127) / 128) < 0x1p24 &&
           (ortho_cycle(p, 0) == p.steps || (double)p.m * (double)p.n < 0x1p31);
  return (double)p.batch * (double)(pad64(p.m) / 64) * (double)(pad64(p.n) / 64) < 0x1p24 &&
         (double)pad64(p.m) * (double)pad64(p.n) * 4 < 0x1p31;
}

hipError_t launch_orthogonalize(const OrthoParams& p, hipStream_t s) {
  switch (way_of(p)) {
    case kSmallGram: return launch_ortho_gram(p, s);
    case kGram: return x_planes(p.x_type) == 2 ? gram<2>(p, s) : gram<1>(p, s);
    default: return direct(p, s);
  }
}

}  // namespace sl
