// ortho_gram.hip -- the orthogonalised update of matrices of up to 128 rows
// (x taken with no more rows than columns), through their Gram matrix:
//   G = X X^T,  P = a I + b G + c G^2,  Q <- P Q,  G <- P G P,  d = Q X.
// Every iterate is a polynomial in G times the first X, so the steps run on
// m x m matrices alone and x's n columns are read twice a cycle, as many steps
// as amplify little (ortho_cycle: three default ones); between cycles X is kept
// in fp32.  Three launches a cycle:
//
//   gram    a workgroup per range of columns: x's values times a power of two
//           of its own (exact in fp16; fp32 values as a pair of fp16), their
//           products on the fp16 matrix cores into fp32 partial sums.
//   steps   one workgroup of 8 waves per matrix: sums the partials, takes
//           |x| from G's trace in 64 bits, and runs all steps in LDS.
//   apply   a workgroup per 128 columns: d, or the next X, = Q X.
//
// Between products a matrix is a pair of fp16 planes, its value times a power
// of two and what that rounding left, and a product of pairs is P0 Q0 + P0 Q1
// + P1 Q0: squaring the singular values leaves no bits to spare.  In a
// simulation of these roundings and of fp32 sums, relative 2-norm, five
// default steps in two cycles: noise 4e-6 to 7e-6, singular values over four
// decades 9e-6, rank 8 2e-5, rank 1 1e-4; with one plane 1e-2 and more.
//
// P's products commute, so G and Q stay symmetric, up to their rounding, and
// every operand is read along its rows.  Bound by latency: a step is three dependent rounds of
// products with two barriers each.  Measured at 96 x 128 (bf16, five steps in
// two cycles): gram 6 and 7, steps 17 and 12, apply 7 and 9 us; the steps take
// 0.9 us each at 32 rows, 2.5 at 64, 5.2 at 96 and 10.5 at 128.
#include "ortho_device.hpp"

namespace sl {
namespace {

constexpr float kGScale = 0x1p12f, kPScale = 0x1p6f;  // what the planes of G, and of P, H and Q, are multiplied by
constexpr int32_t kTop = 14;                           // a range's largest magnitude becomes 2^14 to 2^15

__device__ __forceinline__ uint32_t top8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v[e]) & 0x7FFFFFFFu;
    m = m > a ? m : a;
  }
  return m;
}

// the largest over a workgroup of W waves (lds: W words); every wave passes
template <int W>
__device__ __forceinline__ uint32_t block_top(uint32_t m, uint32_t* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
    m = m > o ? m : o;
  }
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) m = m > lds[w] ? m : lds[w];
  return m;
}
// its exponent: -126 for zero and subnormals, 128 for infinities and NaN
__device__ __forceinline__ int32_t top_exponent(uint32_t bits) {
  const int32_t e = (int32_t)(bits >> 23) - 127;
  return e < -126 ? -126 : e;
}

// v times 2^s as fp16, and in the next plane what that left
template <int PX>
__device__ __forceinline__ void to_planes(const float (&v)[8], int32_t s, u16x8 (&h)[PX]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float f = as_computed(__builtin_ldexpf(v[e], s));
#pragma unroll
    for (int q = 0; q < PX; ++q) {
      h[q][e] = from_f32<DT_F16>(f);
      f -= to_f32<DT_F16>(h[q][e]);
    }
  }
}

// tiles on and above the diagonal, column after column
SL_HD constexpr int32_t tri(int32_t tm, int32_t tn) { return tn * (tn + 1) / 2 + tm; }

// ---------------------------------------------------------------------------
// Partial Gram matrices: workgroup (split, matrix), tile (tm, tn)'s 16 x 16
// sums as 64 lanes x 4 floats, and the range's exponent.  Wave w of 8 has the
// tiles of row w.
// ---------------------------------------------------------------------------
template <int T, int MP>
__global__ __launch_bounds__(512) void gram_kernel(const OrthoParams p, const OrthoGramPlan pl, float* parts, int32_t* exps) {
  constexpr int PX = T == OT_F32 ? 2 : 1, R = MP / 16, PPT = (MP * 8 + 511) / 512;
  constexpr int PLANE = MP * kRowBytes;
  __shared__ __attribute__((aligned(16))) char smem[PX * PLANE];
  __shared__ uint32_t tops[8];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t split = blockIdx.x % pl.splits;
  const int64_t b = blockIdx.x / pl.splits;
  const int64_t j0 = (int64_t)split * pl.cols, j1 = j0 + pl.cols < p.n ? j0 + pl.cols : p.n;
  const bool along_rows = p.x_rs == 1 && p.x_cs != 1;

  float v[PPT][8];
  // piece q of a thread: 8 columns of one row, or 8 rows of one column
  auto row_of = [&](int q) { const int32_t t = threadIdx.x + 512 * q; return along_rows ? 8 * (t % (MP / 8)) : t / 8; };
  auto col_of = [&](int q) { const int32_t t = threadIdx.x + 512 * q; return along_rows ? t / (MP / 8) : 8 * (t % 8); };
  auto load = [&](int64_t j) {
#pragma unroll
    for (int q = 0; q < PPT; ++q)
      if (PPT * 512 == MP * 8 || (int)threadIdx.x + 512 * q < MP * 8)
        ortho_load8<T>(p, b, row_of(q), j + col_of(q), j1, along_rows, v[q]);
  };
#pragma unroll
  for (int q = 0; q < PPT; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[q][e] = 0.f;
  uint32_t top = 0;
  for (int64_t j = j0; j < j1; j += 64) {
    load(j);
#pragma unroll
    for (int q = 0; q < PPT; ++q) top = top8(v[q], top);
  }
  const int32_t ex = top_exponent(block_top<8>(top, tops));

  floatx4 acc[R];
#pragma unroll
  for (int t = 0; t < R; ++t) acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
  load(j0);
  for (int64_t j = j0; j < j1; j += 64) {
    __syncthreads();  // the last chunk's reads
#pragma unroll
    for (int q = 0; q < PPT; ++q) {
      if (!(PPT * 512 == MP * 8 || (int)threadIdx.x + 512 * q < MP * 8)) continue;
      u16x8 h[PX];
      to_planes<PX>(v[q], kTop - ex, h);
#pragma unroll
      for (int z = 0; z < PX; ++z) {
        if (!along_rows) {
          *(u16x8*)(smem + z * PLANE + lds_offset(row_of(q), 2 * col_of(q), 0)) = h[z];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) *(uint16_t*)(smem + z * PLANE + lds_offset(row_of(q) + e, 2 * col_of(q), 0)) = h[z][e];
        }
      }
    }
    __syncthreads();
    if (j + 64 < j1) load(j + 64);
    if (wave < R) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        half8 a[PX];
#pragma unroll
        for (int z = 0; z < PX; ++z)
          a[z] = *(const half8*)(smem + z * PLANE + fragment_lds_offset(MFMA16_F16, lane, 0, 16 * wave, ks, 0));
#pragma unroll
        for (int t = 0; t < R; ++t) {
          if (t < wave) continue;
          half8 c[PX];
#pragma unroll
          for (int z = 0; z < PX; ++z)
            c[z] = *(const half8*)(smem + z * PLANE + fragment_lds_offset(MFMA16_F16, lane, 0, 16 * t, ks, 0));
          acc[t] = mfma16<DT_F16>(c[0], a[0], acc[t]);
          if constexpr (PX == 2) {
            acc[t] = mfma16<DT_F16>(c[1], a[0], acc[t]);
            acc[t] = mfma16<DT_F16>(c[0], a[1], acc[t]);
          }
        }
      }
    }
  }
  if (threadIdx.x == 0) exps[blockIdx.x] = ex;
  if (wave < R) {
    float* out = parts + (int64_t)blockIdx.x * (R * (R + 1) / 2) * 256;
#pragma unroll
    for (int t = 0; t < R; ++t)
      if (t >= wave) *(floatx4*)(out + tri(wave, t) * 256 + 4 * lane) = acc[t];
  }
}

// ---------------------------------------------------------------------------
// The steps.  A matrix in LDS: MP rows of MP fp16, its second plane behind
// them, rows 4 MP + 32 bytes apart (an odd multiple of 32: the 16 lanes of
// one pass of a fragment read then cover all banks).
// ---------------------------------------------------------------------------
template <int MP>
struct PairMatrix {
  static constexpr int PITCH = 4 * MP + 32, BYTES = MP * PITCH;
  // the fragment of rows row0 .. + 15, K 32 ks .. + 31, of a matrix in
  // address space AS (3: LDS, 1: memory; a pointer that may be either would
  // make every access wait for both)
  template <int AS>
  static __device__ __forceinline__ half8 frag(const char* p, int32_t lane, int32_t row0, int32_t ks, int32_t plane) {
    typedef const __attribute__((address_space(AS))) half8 elem;
    return *(elem*)(p + (row0 + (lane & 15)) * PITCH + 2 * MP * plane + 64 * ks + 16 * (lane >> 4));
  }
  // four consecutive values of a row, as a pair, and where asked for the
  // mirrored four
  static __device__ __forceinline__ void store_both(char* p, int32_t m, int32_t n, floatx4 v, bool mirror) {
    u16x4 h, l;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = as_computed(v[r]);
      h[r] = from_f32<DT_F16>(x);
      l[r] = from_f32<DT_F16>(x - to_f32<DT_F16>(h[r]));
    }
    *(u16x4*)(p + m * PITCH + 2 * n) = h;
    *(u16x4*)(p + m * PITCH + 2 * MP + 2 * n) = l;
    if (!mirror) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      *(uint16_t*)(p + (n + r) * PITCH + 2 * m) = h[r];
      *(uint16_t*)(p + (n + r) * PITCH + 2 * MP + 2 * m) = l[r];
    }
  }
  static __device__ __forceinline__ floatx4 read(const char* p, int32_t m, int32_t n) {
    const u16x4 h = *(const u16x4*)(p + m * PITCH + 2 * n), l = *(const u16x4*)(p + m * PITCH + 2 * MP + 2 * n);
    floatx4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = to_f32<DT_F16>(h[r]) + to_f32<DT_F16>(l[r]);
    return v;
  }
};

// A product's blocks on and above the diagonal, dealt to the waves in turn
constexpr int kStepWaves = 8;
template <int MP>
struct StepBlock {
  static constexpr int F = MP <= 64 ? 1 : 2, BS = 16 * F, PER = MP / BS, N = PER * (PER + 1) / 2;
  static constexpr int ONE = (N + kStepWaves - 1) / kStepWaves, TWO = (2 * N + kStepWaves - 1) / kStepWaves;  // blocks of a wave
};

// acc = the block of A B^T at rows m0 of A and n0 of B
template <int MP, int F, int BS = 3>
__device__ __forceinline__ void pair_product(const char* A, const char* B, int32_t lane, int32_t m0, int32_t n0, floatx4 (&acc)[F][F]) {
  typedef PairMatrix<MP> M;
  constexpr int KS = MP / 32;
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  // the fragments of KC slices of 32 are requested together: one wave has
  // little else to cover LDS latency with
  constexpr int KC = KS <= 3 ? KS : 2;
#pragma unroll
  for (int k0 = 0; k0 < KS; k0 += KC) {
    half8 a[KC][F][2], b[KC][F][2];
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          a[k][i][z] = M::template frag<3>(A, lane, m0 + 16 * i, k0 + k, z);
          b[k][i][z] = M::template frag<BS>(B, lane, n0 + 16 * i, k0 + k, z);
        }
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
      for (int z = 0; z < 3; ++z)  // P0 Q0, P0 Q1, P1 Q0
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < F; ++j) acc[i][j] = mfma16<DT_F16>(b[k][j][z == 1], a[k][i][z == 2], acc[i][j]);
  }
}

struct StepCoefficients {
  float v[3 * kOrthoMaxSteps];
};

// Q is the third matrix in LDS, or for MP = 128, where three do not fit, the
// result's place in memory: written once a step from P's place in LDS, when P
// is no longer read, and read back by the workgroup that wrote it.
template <int MP>
__global__ __launch_bounds__(64 * kStepWaves) void gram_steps_kernel(const OrthoParams p, const OrthoGramPlan pl, const float* parts,
                                                          const int32_t* exps, const StepCoefficients co, char* q_all,
                                                          double* norms, bool kept) {
  typedef PairMatrix<MP> M;
  typedef StepBlock<MP> S;
  constexpr int R = MP / 16, NT = R * (R + 1) / 2, TPW = (NT + kStepWaves - 1) / kStepWaves;
  constexpr bool Q_LDS = 3 * M::BYTES <= 150 * 1024;
  __shared__ __attribute__((aligned(16))) char smem[(Q_LDS ? 3 : 2) * M::BYTES];
  __shared__ double traces[kStepWaves];
  char* G = smem;                 // G, then H = P G, then the next G
  char* P = smem + M::BYTES;
  const int64_t b = blockIdx.x;
  char* q_out = q_all + b * M::BYTES;
  char* Q = Q_LDS ? smem + 2 * M::BYTES : q_out;
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // the partial sums, at the largest exponent
  int32_t ex = -126;
  for (int32_t s = 0; s < pl.splits; ++s) ex = exps[b * pl.splits + s] > ex ? exps[b * pl.splits + s] : ex;
  floatx4 g[TPW];
  int32_t tm[TPW], tn[TPW];
  double trace = 0;
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
    const int32_t id = wave + kStepWaves * u;
    int32_t c = 0;
    while (tri(0, c + 1) <= id) ++c;
    tn[u] = c, tm[u] = id - tri(0, c);
    g[u] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (id >= NT) continue;
    for (int32_t s = 0; s < pl.splits; ++s) {
      const floatx4 w = *(const floatx4*)(parts + ((b * pl.splits + s) * NT + id) * 256 + 4 * lane);
      const int32_t d = 2 * (exps[b * pl.splits + s] - ex);
#pragma unroll
      for (int r = 0; r < 4; ++r) g[u][r] += __builtin_ldexpf(w[r], d);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (tm[u] == tn[u] && (lane & 15) == 4 * (lane >> 4) + r) trace += (double)g[u][r];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) trace += __shfl_xor(trace, d);
  if (lane == 0) traces[wave] = trace;
  __syncthreads();
  trace = 0;
#pragma unroll
  for (int w = 0; w < kStepWaves; ++w) trace += traces[w];
  const double norm = ldexp(sqrt(trace), ex - kTop);
  const double f = ex < 128 ? (kept ? 1.0 : 1.0 / (norm + 1e-7)) : __builtin_nan("");  // kept: x is an iterate
  if (threadIdx.x == 0) norms[b] = f;
  const double fx = ldexp(f, ex - kTop);
  const float fg = (float)(fx * fx * (double)kGScale);
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
    if (wave + kStepWaves * u >= NT) continue;
    // lane: row lane % 16, columns 4 (lane / 16) .. + 3; and mirrored
    const int32_t m = 16 * tm[u] + (lane & 15), n = 16 * tn[u] + 4 * (lane >> 4);
    floatx4 v = g[u];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] *= fg;
    M::store_both(G, m, n, v, tm[u] != tn[u]);
  }
  __syncthreads();

  // Every product is symmetric: its blocks on and above the diagonal are
  // computed, and those above stored a second time, mirrored.  H = P G and the
  // next Q = P Q are computed at the same time.  Results wait in registers
  // for the barrier after which their place is no longer read.
  constexpr int F = S::F, N = S::N;
  int32_t bm[S::TWO], bn[S::TWO];  // rows and columns of block (wave + 8 u) mod N
#pragma unroll
  for (int u = 0; u < S::TWO; ++u) {
    const int32_t id = (wave + kStepWaves * u) % N;
    int32_t c = 0;
    while (tri(0, c + 1) <= id) ++c;
    bm[u] = (id - tri(0, c)) * S::BS, bn[u] = c * S::BS;
  }
  auto put = [&](char* to, int u, const floatx4 (&x)[F][F], float scale) {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        floatx4 v = x[i][j];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] *= scale;
        M::store_both(to, bm[u] + 16 * i + (lane & 15), bn[u] + 16 * j + 4 * (lane >> 4), v, bm[u] != bn[u]);
      }
  };
  // a matrix in LDS to Q's place in memory
  auto copy_out = [&](const char* from) {
    for (int32_t i = threadIdx.x; i < M::BYTES / 16; i += 64 * kStepWaves) ((u32x4*)q_out)[i] = ((const u32x4*)from)[i];
  };
  floatx4 acc[S::TWO][F][F];
  for (int32_t t = 0; t < p.steps; ++t) {
    const bool last = t + 1 == p.steps;
    const float ca = co.v[3 * t], cb = co.v[3 * t + 1], cc = co.v[3 * t + 2];
#pragma unroll
    for (int u = 0; u < S::ONE; ++u) {
      if (wave + kStepWaves * u >= N) break;
      pair_product<MP, F>(G, G, lane, bm[u], bn[u], acc[u]);
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) {
          const int32_t m = bm[u] + 16 * i + (lane & 15), n = bn[u] + 16 * j + 4 * (lane >> 4);
          const floatx4 e = M::read(G, m, n);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float v = acc[u][i][j][r] * (cc * (kPScale / (kGScale * kGScale)));
            v = __builtin_fmaf(cb * (kPScale / kGScale), e[r], v);
            acc[u][i][j][r] = m == n + r ? v + ca * kPScale : v;
          }
        }
      put(P, u, acc[u], 1.f);
      if (Q_LDS && t == 0) put(Q, u, acc[u], 1.f);
    }
    __syncthreads();
    if (!Q_LDS && t == 0) copy_out(P);
    // blocks 0 .. N - 1 of H, then (from the second step on) those of Q
    const int32_t h = last ? 0 : N, jobs = t > 0 ? h + N : h;
#pragma unroll
    for (int u = 0; u < S::TWO; ++u) {
      const int32_t id = wave + kStepWaves * u;
      if (id < h)
        pair_product<MP, F>(P, G, lane, bm[u], bn[u], acc[u]);
      else if (id < jobs)
        pair_product<MP, F, Q_LDS ? 3 : 1>(P, Q, lane, bm[u], bn[u], acc[u]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < S::TWO; ++u) {
      const int32_t id = wave + kStepWaves * u;
      if (id < h)
        put(G, u, acc[u], 1.f / kGScale);
      else if (id < jobs && (Q_LDS || last))
        put(Q_LDS ? Q : P, u, acc[u], 1.f / kPScale);
    }
    __syncthreads();
    if (last) break;
    floatx4 next[S::ONE][F][F];
#pragma unroll
    for (int u = 0; u < S::ONE; ++u)
      if (wave + kStepWaves * u < N) pair_product<MP, F>(G, P, lane, bm[u], bn[u], next[u]);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < S::ONE; ++u)
      if (wave + kStepWaves * u < N) put(G, u, next[u], kGScale / (kPScale * kPScale));
    if (!Q_LDS && t > 0) {
#pragma unroll
      for (int u = 0; u < S::TWO; ++u) {
        const int32_t id = wave + kStepWaves * u;
        if (id >= h && id < jobs) put(P, u, acc[u], 1.f / kPScale);
      }
      __syncthreads();
      copy_out(P);
    }
    __syncthreads();
  }
  if (Q_LDS || p.steps > 1) copy_out(Q_LDS ? Q : P);
}

// ---------------------------------------------------------------------------
// d = Q X on 128 columns (`keep`: into fp32 rows of `pitch` there, which x may
// be: the workgroup reads its columns first): X's values go, exactly as in gram_kernel, into an
// LDS tile of MP K-rows of 128, read by transposing reads; Q's fragments come
// from memory; the result passes through LDS to be stored along d's
// contiguous axis.
// ---------------------------------------------------------------------------
template <int T, int MP, bool KEEP>
__global__ __launch_bounds__(256) void gram_apply_kernel(const OrthoParams p, const char* q_all, const double* norms,
                                                         uint32_t tiles_n, float* keep, int64_t pitch) {
  typedef PairMatrix<MP> M;
  constexpr int PX = T == OT_F32 ? 2 : 1, PPT = MP * 16 / 256;
  constexpr int WM = MP == 32 ? 1 : 2, WN = 4 / WM, FM = MP / 16 / WM, FN = 8 / WN;
  constexpr int PLANE = MP * 256, DP = 136;  // D tile: halves per row
  constexpr int BYTES = PX * PLANE > MP * DP * 2 ? PX * PLANE : MP * DP * 2;
  __shared__ __attribute__((aligned(16))) char smem[BYTES];
  __shared__ uint32_t tops[4];
  const int32_t lane = threadIdx.x & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t b = blockIdx.x / tiles_n, j0 = (int64_t)(blockIdx.x % tiles_n) * 128;
  const bool along_rows = p.x_rs == 1 && p.x_cs != 1;
  float v[PPT][8];
  auto row_of = [&](int q) { const int32_t t = threadIdx.x + 256 * q; return along_rows ? 8 * (t % (MP / 8)) : t / 16; };
  auto col_of = [&](int q) { const int32_t t = threadIdx.x + 256 * q; return along_rows ? t / (MP / 8) : 8 * (t % 16); };
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < PPT; ++q) ortho_load8<T>(p, b, row_of(q), j0 + col_of(q), p.n, along_rows, v[q]);
  // Q's fragments, all in flight before x's values are used
  const char* Q = q_all + b * M::BYTES;
  const int32_t m0 = wave % WM * (16 * FM), n0 = wave / WM * (16 * FN);
  half8 a[MP / 32][FM][2];
#pragma unroll
  for (int ks = 0; ks < MP / 32; ++ks)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) a[ks][i][z] = M::template frag<1>(Q, lane, m0 + 16 * i, ks, z);
#pragma unroll
  for (int q = 0; q < PPT; ++q) top = top8(v[q], top);
  const int32_t ex = top_exponent(block_top<4>(top, tops));
#pragma unroll
  for (int q = 0; q < PPT; ++q) {
    u16x8 h[PX];
    to_planes<PX>(v[q], kTop - ex, h);
#pragma unroll
    for (int z = 0; z < PX; ++z) {
      if (!along_rows) {
        *(u16x8*)(smem + z * PLANE + mn_lds_offset(row_of(q), col_of(q), 128)) = h[z];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) *(uint16_t*)(smem + z * PLANE + mn_lds_offset(row_of(q) + e, col_of(q), 128)) = h[z][e];
      }
    }
  }
  __syncthreads();
  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < MP / 32; ++ks) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      half8 x[PX];
#pragma unroll
      for (int z = 0; z < PX; ++z) x[z] = read_frag<LOAD_MNDMA, 128, 0>(smem + z * PLANE, lane, n0 + 16 * j, ks);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        acc[i][j] = mfma16<DT_F16>(x[0], a[ks][i][0], acc[i][j]);
        acc[i][j] = mfma16<DT_F16>(x[0], a[ks][i][1], acc[i][j]);
        if constexpr (PX == 2) acc[i][j] = mfma16<DT_F16>(x[1], a[ks][i][0], acc[i][j]);
      }
    }
  }
  const float f = (float)(ldexp(norms[b], ex - kTop) * (1.0 / kPScale));
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int32_t m = m0 + 16 * i + (lane & 15);
        const int64_t n = j0 + n0 + 16 * j + 4 * (lane >> 4);
        if (m < p.m && n < p.n)  // (the row's last quad ends inside the pitch)
          *(floatx4*)(keep + (b * p.m + m) * pitch + n) =
              floatx4{acc[i][j][0] * f, acc[i][j][1] * f, acc[i][j][2] * f, acc[i][j][3] * f};
      }
    return;
  }
  __syncthreads();
  uint16_t* D = (uint16_t*)smem;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      u16x4 h;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float y = acc[i][j][r] * f;
        h[r] = p.d_type == OT_BF16 ? from_f32<DT_BF16>(y) : from_f32<DT_F16>(y);
      }
      *(u16x4*)(D + (m0 + 16 * i + (lane & 15)) * DP + n0 + 16 * j + 4 * (lane >> 4)) = h;
    }
  __syncthreads();
  uint16_t* d = (uint16_t*)p.d + b * p.d_bs;
  const bool d_rows = p.d_rs == 1 && p.d_cs != 1;
  typedef uint16_t out8 __attribute__((ext_vector_type(8), aligned(2)));
#pragma unroll
  for (int q = 0; q < PPT; ++q) {
    // eight consecutive of d's contiguous axis
    const int32_t t = threadIdx.x + 256 * q;
    const int32_t m = d_rows ? 8 * (t % (MP / 8)) : t / 16, n = d_rows ? t / (MP / 8) : 8 * (t % 16);
    if (m >= p.m || j0 + n >= p.n) continue;
    uint16_t* to = d + m * p.d_rs + (j0 + n) * p.d_cs;
    const int64_t step = d_rows ? p.d_rs : p.d_cs, left = d_rows ? p.m - m : p.n - j0 - n;
    uint16_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = D[(d_rows ? m + e : m) * DP + (d_rows ? n : n + e)];
    if (step == 1 && left >= 8) {
      *(out8*)to = out8{w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) to[e * step] = w[e];
    }
  }
}

struct GramPlaces {
  size_t exps, norms, q, x, total;  // byte offsets behind the partial sums
};
constexpr int64_t kept_pitch(int64_t n) { return (n + 3) / 4 * 4; }
GramPlaces gram_places(const OrthoParams& p, const OrthoGramPlan& pl) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  const size_t r = pl.rows / 16, sums = (size_t)p.batch * pl.splits;
  GramPlaces g;
  g.exps = up(sums * (r * (r + 1) / 2) * 1024);
  g.norms = g.exps + up(sums * 4);
  g.q = g.norms + up((size_t)p.batch * 8);
  g.x = g.q + up((size_t)p.batch * pl.rows * (4 * pl.rows + 32));
  g.total = g.x + (ortho_cycle(p, 0) < p.steps ? (size_t)p.batch * p.m * kept_pitch(p.n) * 4 : 0);
  return g;
}

// one cycle of p's steps; `kept`: x is what the cycle before left, `keep`: so is
// what this one makes
template <int T, int MP>
hipError_t go(const OrthoParams& p, const OrthoGramPlan& pl, const GramPlaces& g, bool kept, bool keep, hipStream_t s) {
  float* parts = (float*)p.ws;
  int32_t* exps = (int32_t*)(p.ws + g.exps);
  double* norms = (double*)(p.ws + g.norms);
  char* q = p.ws + g.q;
  float* x = (float*)(p.ws + g.x);
  StepCoefficients co{};
  for (int32_t i = 0; i < 3 * p.steps; ++i) co.v[i] = p.coefficients[i];
  const uint32_t tiles_n = (uint32_t)((p.n + 127) / 128);
  const dim3 columns(tiles_n * p.batch);
  hipLaunchKernelGGL((gram_kernel<T, MP>), dim3((uint32_t)(p.batch * pl.splits)), dim3(512), 0, s, p, pl, parts, exps);
  hipLaunchKernelGGL((gram_steps_kernel<MP>), dim3(p.batch), dim3(64 * kStepWaves), 0, s, p, pl, parts, exps, co, q, norms, kept);
  if (keep)
    hipLaunchKernelGGL((gram_apply_kernel<T, MP, true>), columns, dim3(256), 0, s, p, q, norms, tiles_n, x, kept_pitch(p.n));
  else
    hipLaunchKernelGGL((gram_apply_kernel<T, MP, false>), columns, dim3(256), 0, s, p, q, norms, tiles_n, x, kept_pitch(p.n));
  return hipGetLastError();
}

template <int T>
hipError_t by_rows(const OrthoParams& p, const OrthoGramPlan& pl, const GramPlaces& g, bool kept, bool keep, hipStream_t s) {
  switch (pl.rows) {
    case 32: return go<T, 32>(p, pl, g, kept, keep, s);
    case 64: return go<T, 64>(p, pl, g, kept, keep, s);
    case 96: return go<T, 96>(p, pl, g, kept, keep, s);
    case 128: return go<T, 128>(p, pl, g, kept, keep, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// The ranges of columns: 256 to a workgroup, but no more partial matrices
// than the one workgroup that sums them reads in about two microseconds
// (256 KiB).
OrthoGramPlan ortho_gram_plan(int64_t m, int64_t n) {
  OrthoGramPlan pl;
  pl.rows = (int32_t)((m + 31) / 32 * 32);
  const int32_t most = pl.rows == 32 ? 64 : pl.rows == 64 ? 24 : pl.rows == 96 ? 12 : 8;
  const int64_t want = (n + 255) / 256;
  const int64_t splits = want < most ? want : most;
  const int64_t cols = ((n + splits - 1) / splits + 63) / 64 * 64;
  pl.cols = (int32_t)cols;
  pl.splits = (int32_t)((n + cols - 1) / cols);
  return pl;
}

size_t ortho_gram_workspace(const OrthoParams& p) { return gram_places(p, ortho_gram_plan(p.m, p.n)).total; }

hipError_t launch_ortho_gram(const OrthoParams& p, hipStream_t s) {
  const OrthoGramPlan pl = ortho_gram_plan(p.m, p.n);
  const GramPlaces g = gram_places(p, pl);
  OrthoParams c = p;
  for (int32_t k = 0; k < p.steps; k += c.steps) {
    c.coefficients = p.coefficients + 3 * k;
    c.steps = ortho_cycle(p, k);
    const bool kept = k > 0, keep = k + c.steps < p.steps;
    if (kept) {
      c.x = p.ws + g.x, c.x_type = OT_F32;
      c.x_rs = kept_pitch(p.n), c.x_cs = 1, c.x_bs = p.m * c.x_rs;
    }
    hipError_t e;
    switch (c.x_type) {
      case OT_F16: e = by_rows<OT_F16>(c, pl, g, kept, keep, s); break;
      case OT_BF16: e = by_rows<OT_BF16>(c, pl, g, kept, keep, s); break;
      default: e = by_rows<OT_F32>(c, pl, g, kept, keep, s); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sl
