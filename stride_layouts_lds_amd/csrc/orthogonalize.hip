// orthogonalize.hip -- the Newton-Schulz orthogonalisation of an update:
//   X <- x / (|x|_F + 1e-7), then per step
//   G = X X^T,  B = b G + c G^2,  X <- a X + B X,
// x taken with no more rows than columns (a tall one transposed by its
// strides).
//
// Three matrix products a step, all on the fp16 matrix cores with fp32 sums.
// Between products X, G and B are kept as fp16 times 2^10 (one plane), or for
// fp16 results as that and what the rounding left (two): X's and G's values
// stay below 2 and B's below 64 in magnitude for iterates of spectral norm
// below 1.4, so nothing overflows, and a value keeps fp16's 11 bits down to
// 2^-24.  x's sum of squares is held in 64 bits and added up in a fixed order.
//
// Every product reads both operands along their contiguous axis: G and B are
// symmetric, and the product that makes X writes it in both orientations, so
// none of them gathers.  G and G^2 are symmetric, so only the tiles on and
// above the diagonal are computed; each is stored a second time, transposed.
#include "sl_ops.hpp"

#include "sl_device.hpp"

namespace sl {
namespace {

constexpr float kDown = 0x1p-10f;  // what a stored value times it stands for
constexpr int32_t kNormParts = 256;               // partial sums of squares of one matrix
constexpr int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

template <int T>
__device__ __forceinline__ float load_any(const void* p, int64_t off) {
  if constexpr (T == OT_F32)
    return ((const float*)p)[off];
  else
    return to_f32<T == OT_F16 ? DT_F16 : DT_BF16>(((const uint16_t*)p)[off]);
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((lds[0] + lds[1]) + lds[2]) + lds[3];
}

// sum of squares of part blockIdx.x of matrix blockIdx.y: the 64 x 64 tiles
// blockIdx.x, + kNormParts, ...
template <int T>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const OrthoParams p, double* parts) {
  __shared__ double lds[4];
  const int64_t b = blockIdx.y;
  const int32_t tiles_n = (int32_t)((p.n + 63) / 64), tiles = (int32_t)((p.m + 63) / 64) * tiles_n;
  const bool along_rows = p.x_rs == 1 && p.x_cs != 1;  // the lanes' axis: the contiguous one
  const int32_t u = threadIdx.x & 63, w = threadIdx.x >> 6;
  double s = 0;
  for (int32_t t = blockIdx.x; t < tiles; t += kNormParts) {
    const int64_t i0 = (int64_t)(t / tiles_n) * 64, j0 = (int64_t)(t % tiles_n) * 64;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int64_t i = i0 + (along_rows ? u : 4 * k + w), j = j0 + (along_rows ? 4 * k + w : u);
      if (i < p.m && j < p.n) {
        const double v = load_any<T>(p.x, b * p.x_bs + i * p.x_rs + j * p.x_cs);
        s += v * v;
      }
    }
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) parts[b * kNormParts + blockIdx.x] = s;
}

// X = 2^10 x / (|x| + 1e-7) as fp16, m x n and n x m, zero to the padded
// sizes; with two planes also what the rounding left
template <int T, int PLANES>
__global__ __launch_bounds__(256) void ortho_start_kernel(const OrthoParams p, const double* parts, uint16_t* X,
                                                          uint16_t* XT, int32_t tiles_m, int32_t tiles_n) {
  __shared__ double lds[4];
  __shared__ uint16_t tile[PLANES][64][66];
  const uint32_t id = blockIdx.x;
  const int32_t tn = id % tiles_n, tm = id / tiles_n % tiles_m;
  const int64_t b = id / tiles_n / tiles_m;
  const int64_t mp = 64 * (int64_t)tiles_m, np = 64 * (int64_t)tiles_n;
  const double sum = block_sum(parts[b * kNormParts + threadIdx.x], lds);
  const double f = 1024.0 / (sqrt(sum) + 1e-7);
  const int64_t i0 = 64 * (int64_t)tm, j0 = 64 * (int64_t)tn;
  const bool along_rows = p.x_rs == 1 && p.x_cs != 1;
  const int32_t u = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int32_t il = along_rows ? u : 4 * k + w, jl = along_rows ? 4 * k + w : u;
    const int64_t i = i0 + il, j = j0 + jl;
    float v = 0.f;
    if (i < p.m && j < p.n) v = as_computed((float)(load_any<T>(p.x, b * p.x_bs + i * p.x_rs + j * p.x_cs) * f));
#pragma unroll
    for (int q = 0; q < PLANES; ++q) {
      const uint16_t h = from_f32<DT_F16>(v);
      tile[q][il][jl] = h;
      v -= to_f32<DT_F16>(h);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int32_t r = 4 * k + w;
#pragma unroll
    for (int q = 0; q < PLANES; ++q) {
      X[PLANES * (b * mp * np + (i0 + r) * np) + q * np + j0 + u] = tile[q][r][u];
      XT[PLANES * (b * mp * np + (j0 + r) * mp) + q * mp + i0 + u] = tile[q][u][r];
    }
  }
}

// D = alpha P Q^T + beta E on fp16 operands with contiguous K.  `planes` 2: a
// row of every matrix is its values rounded to fp16 and, behind them, what
// that left, so the product is P0 Q0 + P0 Q1 + P1 Q0 and loses 2^-22.
struct OrthoGemm {
  const uint16_t *P, *Q, *E;   // (m, planes k), (n, planes k), (m, planes n)
  int64_t P_bs, Q_bs, E_bs;
  int32_t m, n, k;             // padded: multiples of 64
  float alpha, beta;
  uint16_t* O;                 // (m, planes n), or NULL
  uint16_t* OT;                // (n, planes m), or NULL
  int64_t O_bs;
  int32_t sym;                 // only tiles on and above the diagonal, each stored twice (O = OT)
  int32_t tiles_m, tiles_n, batch;
  // the last step's result instead of O and OT
  void* d;
  int64_t rows, cols, d_bs, d_rs, d_cs;
  int32_t d_type;
};

// the tile of workgroup `id`: row-major, or for symmetric results the pairs
// tm <= tn, column by column
__device__ __forceinline__ void ortho_tile(const OrthoGemm& g, uint32_t id, int32_t& batch, int32_t& tm, int32_t& tn) {
  if (g.sym) {
    const uint32_t per = (uint32_t)g.tiles_n * (g.tiles_n + 1) / 2;
    batch = id / per;
    const uint32_t t = id % per;
    int32_t c = (int32_t)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while ((uint32_t)c * (c + 1) / 2 > t) --c;
    while ((uint32_t)(c + 1) * (c + 2) / 2 <= t) ++c;
    tn = c;
    tm = (int32_t)(t - (uint32_t)c * (c + 1) / 2);
  } else {
    const TileCoord tc = map_tile(id, gridDim.x, g.tiles_m, g.tiles_n, 8, g.batch);
    batch = tc.batch, tm = tc.tm, tn = tc.tn;
  }
}

template <int BM, int BN, int WM, int WN, int PLANES>
__global__ __launch_bounds__(WM* WN * 64) void ortho_gemm_kernel(const OrthoGemm g) {
  constexpr int NT = WM * WN * 64;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int ABYTES = BM * kRowBytes, BBYTES = BN * kRowBytes, STAGE = ABYTES + BBYTES;
  constexpr int PITCH = TM + 8;  // halves per row of the transposing region
  static_assert(WM * WN * TN * PITCH * 2 <= 2 * STAGE, "the transposed tile fits the stages");
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t wm = wave % WM, wn = wave / WM;
  int32_t batch, tm, tn;
  ortho_tile(g, blockIdx.x, batch, tm, tn);
  const int32_t m0 = tm * BM, n0 = tn * BN;
  const int32_t rows_a = g.m - m0 < BM ? g.m - m0 : BM, rows_b = g.n - n0 < BN ? g.n - n0 : BN;
  const int32_t kp = PLANES * g.k;
  LoaderKVec<BM, NT, 0, 2> la(g.P + batch * g.P_bs + (int64_t)m0 * kp, rows_a, kp, 1, kp, wave, lane);
  LoaderKVec<BN, NT, 0, 2> lb(g.Q + batch * g.Q_bs + (int64_t)n0 * kp, rows_b, kp, 1, kp, wave, lane);
  const int32_t a_row0 = wm * TM, b_row0 = wn * TN;
  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  // K-tiles: P0 Q0, with two planes then P0 Q1 and P1 Q0
  const int32_t T1 = g.k / 64, T = PLANES == 2 ? 3 * T1 : T1;
  auto issue = [&](int32_t t, char* at) {  // past the last K-tile: not read
    la.issue(PLANES == 2 && t >= T1 ? t - T1 : t, at);
    lb.issue(PLANES == 2 && t >= 2 * T1 ? t - 2 * T1 : t, at + ABYTES);
  };
  issue(0, smem);
  wait_vmem();
  __syncthreads();
  for (int32_t t = 0; t < T; ++t) {
    char* cur = smem + (t & 1) * STAGE;
    char* nxt = smem + ((t + 1) & 1) * STAGE;
    issue(t + 1, nxt);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      half8 af[FM], bf[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) af[i] = *(const half8*)(cur + fragment_lds_offset(MFMA16_F16, lane, 0, a_row0 + 16 * i, ks, 0));
#pragma unroll
      for (int j = 0; j < FN; ++j)
        bf[j] = *(const half8*)(cur + ABYTES + fragment_lds_offset(MFMA16_F16, lane, 0, b_row0 + 16 * j, ks, 0));
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<DT_F16>(bf[j], af[i], acc[i][j]);
    }
    wait_vmem();
    __syncthreads();
  }

  // lane: m = lane % 16 of tile i, n = 4 (lane / 16) + r of tile j
  const bool mirror = g.sym && tm != tn;
  const bool transposed = g.d ? g.d_rs == 1 && g.d_cs != 1 : g.OT && (!g.sym || mirror);
  uint16_t* region = (uint16_t*)smem + wave * (TN * PITCH);
  const int64_t np = (int64_t)PLANES * g.n, mp = (int64_t)PLANES * g.m;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int32_t m = m0 + a_row0 + 16 * i + (lane & 15);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int32_t n = n0 + b_row0 + 16 * j + 4 * (lane >> 4);
      floatx4 v = acc[i][j];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] *= g.alpha;
      if (g.E && m < g.m && n < g.n) {
#pragma unroll
        for (int q = PLANES - 1; q >= 0; --q) {
          const u16x4 e = *(const u16x4*)(g.E + batch * g.E_bs + m * np + q * g.n + n);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(g.beta, to_f32<DT_F16>(e[r]), v[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = as_computed(v[r]);
    }
  }
#pragma unroll
  for (int q = 0; q < PLANES; ++q) {
    if (q > 0 && g.d) break;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int32_t ml = 16 * i + (lane & 15), m = m0 + a_row0 + ml;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int32_t nl = 16 * j + 4 * (lane >> 4), n = n0 + b_row0 + nl;
        const floatx4 v = acc[i][j];
        u16x4 h;
        if (g.d && g.d_type == OT_BF16) {
          h = u16x4{from_f32<DT_BF16>(v[0]), from_f32<DT_BF16>(v[1]), from_f32<DT_BF16>(v[2]), from_f32<DT_BF16>(v[3])};
        } else {
          h = u16x4{from_f32<DT_F16>(v[0]), from_f32<DT_F16>(v[1]), from_f32<DT_F16>(v[2]), from_f32<DT_F16>(v[3])};
          if (q + 1 < PLANES) {  // the next plane's: what this rounding left
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] = as_computed(v[r] - to_f32<DT_F16>(h[r]));
          }
        }
        if (transposed) {
#pragma unroll
          for (int r = 0; r < 4; ++r) region[(nl + r) * PITCH + ml] = h[r];
        }
        if (g.d) {
          if (!transposed) {
            uint16_t* D = (uint16_t*)g.d + batch * g.d_bs + m * g.d_rs;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (m < g.rows && n + r < g.cols) D[(n + r) * g.d_cs] = h[r];
          }
        } else if (g.O && m < g.m && n < g.n) {
          *(u16x4*)(g.O + batch * g.O_bs + m * np + q * g.n + n) = h;
        }
      }
    }
    if (!transposed) continue;
    // each wave reads back only its own region: the compiler's wait on the
    // LDS writes is enough
    constexpr int LPR = TM / 8, RPI = 64 / LPR;  // lanes per row of the region, rows per instruction
#pragma unroll
    for (int k = 0; k < TN / RPI; ++k) {
      const int32_t nl = RPI * k + lane / LPR, ml = 8 * (lane % LPR);
      const int32_t n = n0 + b_row0 + nl, m = m0 + a_row0 + ml;
      const u16x8 h = *(const u16x8*)(region + nl * PITCH + ml);
      if (g.d) {
        uint16_t* D = (uint16_t*)g.d + batch * g.d_bs + n * g.d_cs + m;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n < g.cols && m + e < g.rows) D[e] = h[e];
      } else if (n < g.n && m < g.m) {
        *(u16x8*)(g.OT + batch * g.O_bs + n * mp + q * g.m + m) = h;
      }
    }
  }
}

hipError_t run_gemm(OrthoGemm g, int32_t planes, hipStream_t s) {
  g.tiles_m = (g.m + 127) / 128, g.tiles_n = (g.n + 127) / 128;
  const int64_t tiles = g.sym ? (int64_t)g.tiles_n * (g.tiles_n + 1) / 2 : (int64_t)g.tiles_m * g.tiles_n;
  const dim3 grid((uint32_t)(tiles * g.batch));
  if (planes == 2)
    hipLaunchKernelGGL((ortho_gemm_kernel<128, 128, 2, 2, 2>), grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((ortho_gemm_kernel<128, 128, 2, 2, 1>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

template <int T>
hipError_t start(int32_t planes, const OrthoParams& p, double* parts, uint16_t* X, uint16_t* XT, int32_t tm, int32_t tn, hipStream_t s) {
  hipLaunchKernelGGL(ortho_norm_kernel<T>, dim3(kNormParts, p.batch), dim3(256), 0, s, p, parts);
  const dim3 grid((uint32_t)((int64_t)p.batch * tm * tn));
  if (planes == 2)
    hipLaunchKernelGGL((ortho_start_kernel<T, 2>), grid, dim3(256), 0, s, p, parts, X, XT, tm, tn);
  else
    hipLaunchKernelGGL((ortho_start_kernel<T, 1>), grid, dim3(256), 0, s, p, parts, X, XT, tm, tn);
  return hipGetLastError();
}

struct Places {
  size_t x, xt0, xt1, g, b, total;  // byte offsets behind the partial sums
};
Places places(int64_t batch, int64_t m, int64_t n, int32_t planes) {
  const size_t mn = (size_t)batch * pad64(m) * pad64(n) * 2 * planes, mm = (size_t)batch * pad64(m) * pad64(m) * 2 * planes;
  Places q;
  q.x = ((size_t)batch * kNormParts * 8 + 255) & ~(size_t)255;
  q.xt0 = q.x + mn;
  q.xt1 = q.xt0 + mn;
  q.g = q.xt1 + mn;
  q.b = q.g + mm;
  q.total = q.b + mm;
  return q;
}

}  // namespace

// fp16 results take two planes: with one, every matrix between products
// rounded to fp16 costs them 1.1e-3 to 1.8e-3 (relative, 2-norm; 64-bit
// simulation at 16 x 16 to 1000 x 1000), five times their own rounding of
// 2.1e-4, with two 3e-7 at three times the products.  A bf16 result's own
// rounding is 1.7e-3.
namespace {
int32_t planes_for(int32_t d_type) { return d_type == OT_F16 ? 2 : 1; }
}  // namespace

// Up to 128 rows the Gram matrix's three launches (96 x 128: 123 us with the
// launches below), unless the steps amplify too much for it.
namespace {
bool through_gram(const OrthoParams& p) {
  float growth = 1.f;
  for (int32_t t = 0; t < p.steps; ++t) growth *= fmaxf(1.f, fabsf(p.coefficients[3 * t]));
  return p.m <= kGramRows && growth <= kGramGrowth;
}
}  // namespace

size_t orthogonalize_workspace(const OrthoParams& p) {
  return through_gram(p) ? ortho_gram_workspace(p) : places(p.batch, p.m, p.n, planes_for(p.d_type)).total;
}

// every launch below fits a grid, and a 128-row tile 32-bit offsets
bool orthogonalize_grid_ok(int64_t batch, int64_t m, int64_t n) {
  const int64_t lim = (int64_t)1 << 31;
  if (batch >= 65536 || m >= lim || n >= lim) return false;
  return (double)batch * (double)(pad64(m) / 64) * (double)(pad64(n) / 64) < 0x1p31 && 256 * pad64(n) * 4 < lim;
}

hipError_t launch_orthogonalize(const OrthoParams& p, hipStream_t s) {
  if (through_gram(p)) return launch_ortho_gram(p, s);
  const int32_t planes = planes_for(p.d_type);
  const Places q = places(p.batch, p.m, p.n, planes);
  double* parts = (double*)p.ws;
  uint16_t* X = (uint16_t*)(p.ws + q.x);
  uint16_t* XT[2] = {(uint16_t*)(p.ws + q.xt0), (uint16_t*)(p.ws + q.xt1)};
  uint16_t* G = (uint16_t*)(p.ws + q.g);
  uint16_t* B = (uint16_t*)(p.ws + q.b);
  const int32_t mp = (int32_t)pad64(p.m), np = (int32_t)pad64(p.n);
  const int64_t mn = (int64_t)mp * np * planes, mm = (int64_t)mp * mp * planes;
  hipError_t e;
  switch (p.x_type) {
    case OT_F16: e = start<OT_F16>(planes, p, parts, X, XT[0], mp / 64, np / 64, s); break;
    case OT_BF16: e = start<OT_BF16>(planes, p, parts, X, XT[0], mp / 64, np / 64, s); break;
    default: e = start<OT_F32>(planes, p, parts, X, XT[0], mp / 64, np / 64, s); break;
  }
  for (int32_t k = 0; k < p.steps && e == hipSuccess; ++k) {
    const float a = p.coefficients[3 * k], b = p.coefficients[3 * k + 1], c = p.coefficients[3 * k + 2];
    const bool last = k + 1 == p.steps;
    // stored values carry 2^10, products of two 2^20
    OrthoGemm g{};
    g.batch = p.batch;
    g.P = X, g.Q = X, g.P_bs = g.Q_bs = mn;
    g.m = g.n = mp, g.k = np, g.alpha = kDown;
    g.O = g.OT = G, g.O_bs = mm, g.sym = 1;
    if ((e = run_gemm(g, planes, s)) != hipSuccess) break;
    g.P = G, g.Q = G, g.E = G, g.P_bs = g.Q_bs = g.E_bs = mm;
    g.k = mp, g.alpha = c * kDown, g.beta = b;
    g.O = g.OT = B;
    if ((e = run_gemm(g, planes, s)) != hipSuccess) break;
    g.P = B, g.Q = XT[k & 1], g.E = X, g.Q_bs = g.E_bs = mn;
    g.n = np, g.alpha = kDown, g.beta = a, g.sym = 0;
    g.O = X, g.OT = XT[(k + 1) & 1], g.O_bs = mn;
    if (last) {
      g.alpha *= kDown, g.beta *= kDown;
      g.d = p.d, g.d_type = p.d_type, g.rows = p.m, g.cols = p.n;
      g.d_bs = p.d_bs, g.d_rs = p.d_rs, g.d_cs = p.d_cs;
    }
    e = run_gemm(g, planes, s);
  }
  return e;
}

}  // namespace sl
