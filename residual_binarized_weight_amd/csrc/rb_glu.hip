// rb_glu.hip -- the first half of a gated feed-forward block, and its backward.
//
//   G = X Wg^T + bg,  U = X Wu^T + bu,  H = act(G) (.) U        X [M][K], Wg and Wu [N][K] in fp16 or bf16, fp32 sums
//   dG = dH (.) U (.) act'(G),  dU = dH (.) act(G),  dbg and dbu their column sums
//   dX = dG Wg + dU Wu
//
// Kernels of this file:
//   glu_tile_kernel     a tile of batch rows by rows of both weights, on the matrix cores; glu_join_kernel the sums of
//                       split tiles, and the epilogue
//   glu_rows_kernel     up to 4 batch rows, on the vector units: a wave streams a row of each weight
//   glu_few_kernel      small products of 5 to 256 batch rows, on the matrix cores, a block's waves splitting the columns
//   glu_grad_kernel     dG, dU and, per strip of rows, partial column sums; glu_grad_sum_kernel adds them
//   glu_dx_kernel       a tile of dX, both products in one run of sums; glu_dx_join_kernel for split tiles
#include "rb_act.hpp"
#include "rb_internal.h"
#include "rb_tile.hpp"

namespace rb {
namespace {

using tile::f4;
using tile::Source;
using tile::Work;

// Streamed where rows start lines; elsewhere a streamed line that two stores write in part goes to memory twice.
template <typename T>
__device__ __forceinline__ void store_out(T* row, int c, int n, const float (&v)[8], bool line) {
  if (line)
    store8<T, true>(row, c, n, v);
  else
    store8<T>(row, c, n, v);
}

// ---------------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------------
struct GluOut {
  const float *bg, *bu;
  void *G, *U, *H;
  int64_t ldg, ldu, ldh;
  int act;
  bool line_g, line_u, line_h;  // every row starts a 128-byte line
};
__device__ __forceinline__ void add8(const float* b, int n, int N, float (&v)[8]) {
  if (!b) return;
  float t[8];
  widen8<float>(load8_any<float>(b, n, N), t);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += t[j];
}
// columns n .. n + 7 of row m, g and u the products' fp32 sums
template <typename T, typename TH>
__device__ __forceinline__ void finish8(const GluOut& o, float (&g)[8], float (&u)[8], int64_t m, int n, int N) {
  add8(o.bg, n, N, g);
  add8(o.bu, n, N, u);
  if (o.G) store_out<T>(static_cast<T*>(o.G) + m * o.ldg, n, N, g, o.line_g);
  if (o.U) store_out<T>(static_cast<T*>(o.U) + m * o.ldu, n, N, u, o.line_u);
  if (o.act != RB_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = act_value(g[j], o.act);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] *= u[j];
  store_out<TH>(static_cast<TH*>(o.H) + m * o.ldh, n, N, g, o.line_h);
}

// ... and one of them
template <typename T, typename TH>
__device__ __forceinline__ void finish1(const GluOut& o, float g, float u, int64_t m, int n) {
  if (o.bg) g += o.bg[n];
  if (o.bu) u += o.bu[n];
  if (o.G) static_cast<T*>(o.G)[m * o.ldg + n] = Vec8<T>::narrow(g);
  if (o.U) static_cast<T*>(o.U)[m * o.ldu + n] = Vec8<T>::narrow(u);
  if (o.act != RB_ACT_NONE) g = act_value(g, o.act);
  static_cast<TH*>(o.H)[m * o.ldh + n] = Vec8<TH>::narrow(g * u);
}

template <typename T>
struct GluArgs {
  Source<T> src[1];
  int64_t M;
  int N;
  Work work;
  float* part;
  GluOut out;
  uint32_t first;  // of the forms without tiles: the launch's first block of weight rows
};

// Half of a tile's columns are G's and half U's, so that a wave holds both sums of an output and H costs no further pass.
// Bound by the matrix cores at the card's power limit and by the tiles' ends, which nothing overlaps: 2048 x 4096 over
// 2 x 11008 in bf16 323 to 349 us (1.06 to 1.14 PFLOP/s) for both products, G, U and H; the library's product alone takes 426.
// The 256-row tiles' registers are full: one vector register goes to scratch, 57 scalar ones to lanes of vector registers.
template <typename T, typename TH, typename C>
__global__ __launch_bounds__(C::kThreads, 2) void glu_tile_kernel(GluArgs<T> a) {
  extern __shared__ __align__(16) uint8_t t_smem[];
  tile::share(a.work, [&](uint32_t t, int s0, int s1, int slot) {
    const typename C::Where at = C::where(a.work, t, a.M, a.N);
    typename C::Acc acc;
    C::run(a.src, at, a.N, s0, s1, t_smem, acc);
    float* const part = slot < 0 ? nullptr : a.part + (int64_t)slot * C::BM * C::BN;
    C::rows(acc, t_smem, [&](int r, int c, const float* p) {
      float g[8], u[8];
      tile::eight(p, g);
      tile::eight(p + C::kHalfN, u);
      if (part) {
        store8<float>(part + r * C::BN, c, C::BN, g);
        store8<float>(part + r * C::BN, C::kOutN + c, C::BN, u);
      } else if (r < at.mrows && c < at.ncols) {
        finish8<T, TH>(a.out, g, u, at.m0 + r, at.n0 + c, a.N);
      }
    }, [](int, int, const float*) {});
    __syncthreads();
  });
}

// 8 columns of a row of a split tile per thread; its parts are added in the order of the sum
template <typename T, typename TH, typename C>
__global__ __launch_bounds__(256) void glu_join_kernel(GluArgs<T> a) {
  const typename C::Where at = C::where(a.work, a.work.full + blockIdx.x, a.M, a.N);
  const int i = blockIdx.y * 256 + threadIdx.x, r = i / (C::kOutN / 8), c = i % (C::kOutN / 8) * 8;
  if (r >= at.mrows || c >= at.ncols) return;
  float g[8] = {}, u[8] = {};
  tile::parts(a.work, blockIdx.x, [&](uint32_t slot) {
    const float* const p = a.part + ((int64_t)slot * C::BM + r) * C::BN + c;
    float v[8];
    tile::eight(p, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] += v[j];
    tile::eight(p + C::kOutN, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] += v[j];
  });
  finish8<T, TH>(a.out, g, u, at.m0 + r, at.n0 + c, a.N);
}

// Up to 4 batch rows: HBM's rate for the weights is the bound, and the vector units' products are far below it. A
// wave owns a row of each weight, its lanes 8 columns each of a 512-column step; kSteps loads of 1 KB from each row
// are in flight. One launch, no partial sums in memory. One row of 4096 over 2 x 11008 in fp16: 31.5 us, 5.7 TB/s. Two to
// four rows take one form, which does four rows' work (absent ones repeat the first): 39, 40 and 41 us in bf16.
constexpr int kMaxRows = 4;

template <typename T, typename TH, int MR, int kSteps>
__global__ __launch_bounds__(256) void glu_rows_kernel(GluArgs<T> a) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = (int)(a.first + blockIdx.x) * 4 + w;
  if (n >= a.N) return;
  const Source<T>& q = a.src[0];
  const T* const row[2] = {q.B + (int64_t)n * q.ldb, q.B2 + (int64_t)n * q.ldb2};
  float sum[MR][2];
#pragma unroll
  for (int m = 0; m < MR; ++m) sum[m][0] = sum[m][1] = 0.f;
  for (int k0 = 0; k0 < q.R; k0 += 512 * kSteps) {
    typename Vec8<T>::Raw wr[kSteps][2] = {}, xr[kSteps][MR] = {};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = k0 + 512 * s + 8 * lane;
#pragma unroll
      for (int r = 0; r < 2; ++r) load8_long<T>(wr[s][r], row[r], c, q.R);
#pragma unroll
      for (int m = 0; m < MR; ++m) load8_long<T>(xr[s][m], q.A + (m < a.M ? m : 0) * q.lda, c, q.R);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = k0 + 512 * s + 8 * lane;
      if (c < q.R && c + 8 > q.R) {  // the vector at the end of the columns
#pragma unroll
        for (int r = 0; r < 2; ++r) shift_down(wr[s][r], c + 8 - q.R);
#pragma unroll
        for (int m = 0; m < MR; ++m) shift_down(xr[s][m], c + 8 - q.R);
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sum[m][r] = fmaf(Vec8<T>::get(wr[s][r], j), Vec8<T>::get(xr[s][m], j), sum[m][r]);
  }
  // lane m takes row m's sums
  float g = 0.f, u = 0.f;
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    const float x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_dpp(sum[m][0])), 63));
    const float y = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_dpp(sum[m][1])), 63));
    g = lane == m ? x : g;
    u = lane == m ? y : u;
  }
  if (lane < MR && lane < a.M) finish1<T, TH>(a.out, g, u, lane, n);
}

// Small products: one launch on the matrix cores, without partial sums in memory. A block owns 16 rows of each weight by
// 16 batch rows; its 8 waves take the 64-column steps in turn, each with its fragments straight from memory, and join
// in LDS in their order. The fragments' 16-byte pieces cost the address unit a piece each, which bounds the rate.
constexpr int kFewRows = 256;
constexpr double kFewStep = 0.2, kFewStepOdd = 0.5;  // us of a step of 64 columns in 256 blocks

template <typename T, typename TH>
__global__ __launch_bounds__(512) void glu_few_kernel(GluArgs<T> a) {
  constexpr int kWaves = 8, kAhead = 4;  // steps whose loads a wave has in flight
  __shared__ __align__(16) float sums[2][kWaves][256];
  const Source<T>& q = a.src[0];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lr = lane & 15, lj = lane >> 4;
  const int n0 = (int)(a.first + blockIdx.x) * 16;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  // rows past the last one repeat it: their outputs are not stored
  const int64_t n = n0 + lr < a.N ? n0 + lr : a.N - 1;
  const T* const row[3] = {q.B + n * q.ldb, q.B2 + n * q.ldb2, q.A + (m0 + lr < a.M ? m0 + lr : a.M - 1) * q.lda};
  f4 acc[2] = {};
  for (int k0 = w * tile::kTK; k0 < q.R; k0 += kAhead * kWaves * tile::kTK) {
    typename Vec8<T>::Raw f[kAhead][2][3] = {};
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 3; ++i) load8_long<T>(f[s][h][i], row[i], k0 + s * kWaves * tile::kTK + 32 * h + 8 * lj, q.R);
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = k0 + s * kWaves * tile::kTK + 32 * h + 8 * lj;
        if (c < q.R && c + 8 > q.R) {  // the vector at the end of the columns
#pragma unroll
          for (int i = 0; i < 3; ++i) shift_down(f[s][h][i], c + 8 - q.R);
        }
        const tile::u4 x = __builtin_bit_cast(tile::u4, f[s][h][2]);
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i] = tile::mfma(T(0), __builtin_bit_cast(tile::u4, f[s][h][i]), x, acc[i]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) *reinterpret_cast<f4*>(&sums[i][w][lane * 4]) = acc[i];
  __syncthreads();
  // thread 16 m + n: D's lane 16 (n / 4) + m holds weight row n in element n % 4
  if (threadIdx.x >= 256) return;
  const int mm = threadIdx.x >> 4, nn = threadIdx.x & 15, on = n0 + nn;
  const int64_t m = m0 + mm;
  if (m >= a.M || on >= a.N) return;
  float g = 0.f, u = 0.f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int at = ((nn >> 2) * 16 + mm) * 4 + (nn & 3);
    g += sums[0][i][at];
    u += sums[1][i][at];
  }
  finish1<T, TH>(a.out, g, u, m, on);
}

// ---------------------------------------------------------------------------------------------
// the epilogue's backward: a block owns 512 columns (8 per thread over 64 lanes) and a strip of rows, which its 4
// waves take in turn; each thread keeps its columns' sums in fp32. HBM bounds it.
// ---------------------------------------------------------------------------------------------
// A block walks down a strip of rows, 8 columns a thread, and keeps the column sums in registers; bound by HBM (2048 x
// 11008 bf16, 225 MB: 51 us from warm caches, 78 from flushed ones, traced). Sums are joined in a fixed order. Its stores
// are streamed whatever the rows' alignment: a wave writes 1 KB of a row at once, so that few lines are written in two
// parts (odd rows in bf16, us, streamed / only where rows start lines: 2048 x 11007 64 / 68, 2048 x 4095 24 / 26, 512 x 4095
// 7.3 / 8.3, 4096 x 1411 19 / 21).
struct GluGradArgs {
  const void *dH, *G, *U;
  void *dG, *dU;
  float *part_g, *part_u;  // [strips][N], or NULL
  int64_t M, lddh, ldg, ldu, lddg, lddu;
  int N, act, strip;
};
template <typename T, typename TD>
__global__ __launch_bounds__(256) void glu_grad_kernel(GluGradArgs a) {
  __shared__ float s[3][2][512];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = blockIdx.x * 512 + lane * 8;
  const int64_t r0 = (int64_t)blockIdx.y * a.strip;
  const int64_t r1 = r0 + a.strip < a.M ? r0 + a.strip : a.M;
  float sg[8] = {}, su[8] = {};
#pragma unroll 2
  for (int64_t m = r0 + w; m < r1; m += 4) {
    float d[8], g[8], u[8], dg[8], du[8];
    widen8<TD>(load8_any<TD>(static_cast<const TD*>(a.dH) + m * a.lddh, n, a.N), d);
    widen8<T>(load8_any<T>(static_cast<const T*>(a.G) + m * a.ldg, n, a.N), g);
    widen8<T>(load8_any<T>(static_cast<const T*>(a.U) + m * a.ldu, n, a.N), u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dg[j] = d[j] * u[j] * act_slope(g[j], a.act);
      du[j] = d[j] * act_value(g[j], a.act);
      sg[j] += dg[j];
      su[j] += du[j];
    }
    store8<T, true>(static_cast<T*>(a.dG) + m * a.lddg, n, a.N, dg);
    store8<T, true>(static_cast<T*>(a.dU) + m * a.lddu, n, a.N, du);
  }
  if (!a.part_g && !a.part_u) return;
  if (w > 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[w - 1][0][lane * 8 + j] = sg[j], s[w - 1][1][lane * 8 + j] = su[j];
  }
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = lane * 8 + j;
      sg[j] += s[0][0][c] + s[1][0][c] + s[2][0][c];
      su[j] += s[0][1][c] + s[1][1][c] + s[2][1][c];
    }
    if (a.part_g) store8<float>(a.part_g + (int64_t)blockIdx.y * a.N, n, a.N, sg);
    if (a.part_u) store8<float>(a.part_u + (int64_t)blockIdx.y * a.N, n, a.N, su);
  }
}
// 64 columns by 8 interleaved runs of strips; blockIdx.y: which of the two
__global__ __launch_bounds__(512) void glu_grad_sum_kernel(const float* part_g, const float* part_u, int strips, int N,
                                                           float* dbg, float* dbu) {
  __shared__ float s[8][64];
  const float* const part = blockIdx.y ? part_u : part_g;
  if (!part) return;
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float v = 0.f;
  if (c < N) {
#pragma unroll 4
    for (int b = run; b < strips; b += 8) v += part[(int64_t)b * N + c];
  }
  s[run][lane] = v;
  __syncthreads();
  if (run == 0 && c < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    (blockIdx.y ? dbu : dbg)[c] = v;
  }
}

// ---------------------------------------------------------------------------------------------
// the input's gradient
// ---------------------------------------------------------------------------------------------
template <typename T>
struct DxArgs {
  Source<T> src[2];
  int64_t M;
  int N;  // columns of dX
  Work work;
  float* part;
  void* dX;
  int64_t ldx;
  bool line;
};
// dG and dU, and Wg and Wu, follow each other along the sum, so that dX is written once and no product waits for the other;
// the weights' rows lie across the sum and are turned by the transposing LDS reads. 2048 x 4096 over 2 x 11008 bf16: 300 to
// 324 us traced (1.14 to 1.23 PFLOP/s); the library's product of that shape takes 452. The 256-row tiles keep 8 vector
// registers in scratch. Up to 64 rows of it take 42 to 45 us, the weights' 35 at a copy's rate being the floor.
template <typename T, typename TX, typename C>
__global__ __launch_bounds__(C::kThreads, 2) void glu_dx_kernel(DxArgs<T> a) {
  extern __shared__ __align__(16) uint8_t t_smem[];
  tile::share(a.work, [&](uint32_t t, int s0, int s1, int slot) {
    const typename C::Where at = C::where(a.work, t, a.M, a.N);
    typename C::Acc acc;
    C::run(a.src, at, a.N, s0, s1, t_smem, acc);
    float* const part = slot < 0 ? nullptr : a.part + (int64_t)slot * C::BM * C::BN;
    C::rows(acc, t_smem, [&](int r, int c, const float* p) {
      float v[8];
      tile::eight(p, v);
      if (part)
        store8<float>(part + r * C::BN, c, C::BN, v);
      else if (r < at.mrows && c < at.ncols)
        store_out<TX>(static_cast<TX*>(a.dX) + (at.m0 + r) * a.ldx, at.n0 + c, a.N, v, a.line);
    }, [](int, int, const float*) {});
    __syncthreads();
  });
}
template <typename T, typename TX, typename C>
__global__ __launch_bounds__(256) void glu_dx_join_kernel(DxArgs<T> a) {
  const typename C::Where at = C::where(a.work, a.work.full + blockIdx.x, a.M, a.N);
  const int i = blockIdx.y * 256 + threadIdx.x, r = i / (C::kOutN / 8), c = i % (C::kOutN / 8) * 8;
  if (r >= at.mrows || c >= at.ncols) return;
  float v[8] = {};
  tile::parts(a.work, blockIdx.x, [&](uint32_t slot) {
    float p[8];
    tile::eight(a.part + ((int64_t)slot * C::BM + r) * C::BN + c, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += p[j];
  });
  store_out<TX>(static_cast<TX*>(a.dX) + (at.m0 + r) * a.ldx, at.n0 + c, a.N, v, a.line);
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------
// Tiles of 64, 128 and (aligned operands) 256 batch rows by 256 staged rows of the weights.
template <typename T, bool kNN, int kBM, bool kAl> struct Shape;
template <typename T, bool kNN, bool kAl> struct Shape<T, kNN, 64, kAl> {
  typedef tile::Tile<T, 2, 4, 2, 4, kAl ? 3 : 2, kNN, kNN ? 0 : 32, kNN ? 2 : 1, kAl> C;
};
template <typename T, bool kNN, bool kAl> struct Shape<T, kNN, 128, kAl> {
  typedef tile::Tile<T, 4, 2, 2, 8, kAl ? 3 : 2, kNN, kNN ? 0 : 64, kNN ? 2 : 1, kAl> C;
};
template <typename T, bool kNN> struct Shape<T, kNN, 256, true> {
  typedef tile::Tile<T, 4, 2, 4, 8, 2, kNN, kNN ? 0 : 64, kNN ? 2 : 1, true> C;
};

struct Choice {
  int bm;
  tile::Lay lay;
};
// The tile height by estimate: us of a step of a tile of each height when every unit works, measured at 2048 x 16384
// outputs (staged) of 64 steps; the transposing reads of dX's products take a tenth longer. Rows that are not aligned: the
// same from odd rows. 128 rows take 0.97 where 256 take 1.69: what a byte brought to LDS serves.
Choice choose(int64_t M, int64_t out_n, int per_tile, int64_t steps, bool aligned, bool across) {
  struct { int bm; double step; } const kinds[2][3] = {{{64, 0.95}, {128, 1.5}, {0, 0}}, {{64, 0.64}, {128, 0.97}, {256, 1.69}}};
  Choice best{};
  for (const auto& k : kinds[aligned]) {
    if (k.bm == 0) continue;
    const tile::Lay l = tile::lay((M + k.bm - 1) / k.bm, (out_n + per_tile - 1) / per_tile, steps, k.step * (across ? 1.13 : 1.0),
                                  (int64_t)k.bm * 1024);
    if (best.bm == 0 || l.est < best.lay.est) best = Choice{k.bm, l};
  }
  return best;
}
int64_t steps_of(int64_t R) { return (R + tile::kTK - 1) / tile::kTK; }
bool small_ld(int64_t ld) { return ld < (1 << 21); }  // a tile's rows lie within 2^31 bytes, the out-of-range marker

template <typename T, typename TH, int kBM, bool kAl>
hipError_t launch_glu_tile(const GluArgs<T>& a, hipStream_t s) {
  typedef typename Shape<T, false, kBM, kAl>::C C;
  static std::atomic<uint64_t> done;
  hipError_t e = tile::allow_lds(done, glu_tile_kernel<T, TH, C>, C::kLds);
  if (e != hipSuccess) return e;
  glu_tile_kernel<T, TH, C><<<a.work.grid, C::kThreads, C::kLds, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || a.work.full == a.work.tiles) return e;
  glu_join_kernel<T, TH, C><<<dim3(a.work.tiles - a.work.full, C::BM * C::kOutN / 8 / 256), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, typename TH>
hipError_t launch_glu_rows(GluArgs<T> a, hipStream_t s) {
  return launch_in_parts(((int64_t)a.N + 3) / 4, [&](int64_t first, uint32_t blocks) {
    a.first = (uint32_t)first;
    if (a.M == 1)
      glu_rows_kernel<T, TH, 1, 4><<<dim3(blocks), 256, 0, s>>>(a);
    else
      glu_rows_kernel<T, TH, 4, 4><<<dim3(blocks), 256, 0, s>>>(a);
  });
}

// The forms without tiles; both read 8 columns at least. Up to 4 rows the vector units' products cost nothing beside
// the weights. The one-launch form on the matrix cores is taken by its estimate against the tiles', up to the 256 rows
// that the estimate holds for (us, one launch / tiles: 5 x 1000 x 1000 4.1 / 12.5, 16 x 2048 x 2048 8.5 / 15.3, 64 x 1408 x
// 1024 8.6 / 13.3, 64 x 2048 x 2048 14.2 / 17.4, 64 x 4096 x 4096 53 / 27, 256 x 512 x 512 5.6 / 10.8; rows not aligned: 5 x
// 1000 x 1001 7.3 / 15.7, 61 x 1411 x 1027 14.2 / 17.0, 16 x 2047 x 2047 21.4 / 19.4, 128 x 1023 x 1023 21.7 / 17.2). Neither
// estimate has a term for memory's rate, which is the floor where weights are large: 5 to 64 rows of 4096 over 2 x 11008 take
// 49 to 53 us against the 35 that the weights need.
enum class Small { kNone, kRows, kFew };
Small small_form(int64_t M, int64_t N, int64_t K, bool aligned) {
  if (K < 8 || M > kFewRows) return Small::kNone;
  if (M <= kMaxRows) return Small::kRows;
  const double blocks = (double)((N + 15) / 16 * ((M + 15) / 16)), rounds = blocks < 256 ? 1.0 : blocks / 256;
  return 2.6 + rounds * (double)steps_of(K) * (aligned ? kFewStep : kFewStepOdd) < choose(M, N, 128, steps_of(K), aligned, false).lay.est
             ? Small::kFew : Small::kNone;
}

template <typename T, typename TH>
hipError_t launch_glu_product(GluArgs<T> a, void* ws, hipStream_t s) {
  const Source<T>& q = a.src[0];
  const bool al = tile::rows16(q.A, q.lda) && tile::rows16(q.B, q.ldb) && tile::rows16(q.B2, q.ldb2) && q.R % 8 == 0 &&
                  small_ld(q.lda) && small_ld(q.ldb) && small_ld(q.ldb2);
  switch (small_form(a.M, a.N, q.R, al)) {
    case Small::kRows: return launch_glu_rows<T, TH>(a, s);
    case Small::kFew:
      return launch_in_parts(((int64_t)a.N + 15) / 16, [&](int64_t first, uint32_t blocks) {
        a.first = (uint32_t)first;
        glu_few_kernel<T, TH><<<dim3(blocks, (uint32_t)((a.M + 15) / 16)), 512, 0, s>>>(a);
      });
    case Small::kNone: break;
  }
  const Choice c = choose(a.M, a.N, 128, q.steps, al, false);
  a.work = c.lay.work;
  a.part = static_cast<float*>(ws);
  if (c.bm == 256) return launch_glu_tile<T, TH, 256, true>(a, s);
  if (c.bm == 128) return al ? launch_glu_tile<T, TH, 128, true>(a, s) : launch_glu_tile<T, TH, 128, false>(a, s);
  return al ? launch_glu_tile<T, TH, 64, true>(a, s) : launch_glu_tile<T, TH, 64, false>(a, s);
}

template <typename T>
hipError_t launch_glu_typed(const void* X, int64_t M, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu, int64_t ldwu,
                            int64_t N, int64_t K, const GluOut& out, rb_dtype h_dtype, void* ws, hipStream_t s) {
  const GluArgs<T> a{{{static_cast<const T*>(X), static_cast<const T*>(Wg), static_cast<const T*>(Wu), ldx, ldwg, ldwu, (int)K,
                       (int)steps_of(K)}}, M, (int)N, {}, nullptr, out, 0};
  return h_dtype == RB_F32 ? launch_glu_product<T, float>(a, ws, s) : launch_glu_product<T, T>(a, ws, s);
}

template <typename T, typename TX, int kBM, bool kAl>
hipError_t launch_dx_tile(const DxArgs<T>& a, hipStream_t s) {
  typedef typename Shape<T, true, kBM, kAl>::C C;
  static std::atomic<uint64_t> done;
  hipError_t e = tile::allow_lds(done, glu_dx_kernel<T, TX, C>, C::kLds);
  if (e != hipSuccess) return e;
  glu_dx_kernel<T, TX, C><<<a.work.grid, C::kThreads, C::kLds, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || a.work.full == a.work.tiles) return e;
  glu_dx_join_kernel<T, TX, C><<<dim3(a.work.tiles - a.work.full, C::BM * C::kOutN / 8 / 256), 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T, typename TX>
hipError_t launch_dx_product(DxArgs<T> a, void* ws, hipStream_t s) {
  bool al = a.src[0].R % 8 == 0 && a.N % 8 == 0;
  for (const Source<T>& q : a.src)
    al = al && tile::rows16(q.A, q.lda) && tile::rows16(q.B, q.ldb) && small_ld(q.lda) && small_ld(q.ldb);
  const Choice c = choose(a.M, a.N, 256, 2 * a.src[0].steps, al, true);
  a.work = c.lay.work;
  a.part = static_cast<float*>(ws);
  if (c.bm == 256) return launch_dx_tile<T, TX, 256, true>(a, s);
  if (c.bm == 128) return al ? launch_dx_tile<T, TX, 128, true>(a, s) : launch_dx_tile<T, TX, 128, false>(a, s);
  return al ? launch_dx_tile<T, TX, 64, true>(a, s) : launch_dx_tile<T, TX, 64, false>(a, s);
}
template <typename T>
hipError_t launch_dx_typed(const void* dG, int64_t lddg, const void* dU, int64_t lddu, int64_t M, const void* Wg, int64_t ldwg,
                           const void* Wu, int64_t ldwu, int64_t N, int64_t K, void* dX, rb_dtype dx_dtype, int64_t lddx,
                           void* ws, hipStream_t s) {
  const auto side = [&](const void* d, int64_t ldd, const void* w, int64_t ldw) {
    return Source<T>{static_cast<const T*>(d), static_cast<const T*>(w), nullptr, ldd, ldw, 0, (int)N, (int)steps_of(N)};
  };
  const DxArgs<T> a{{side(dG, lddg, Wg, ldwg), side(dU, lddu, Wu, ldwu)}, M, (int)K, {}, nullptr, dX, lddx,
                    tile::lines(dX, lddx, dx_dtype == RB_F32 ? 4 : 2)};
  return dx_dtype == RB_F32 ? launch_dx_product<T, float>(a, ws, s) : launch_dx_product<T, T>(a, ws, s);
}

int grad_strip(int64_t M, int64_t N) {
  if (M <= 8) return 8;
  const int64_t cols = (N + 511) / 512, want = (1024 + cols - 1) / cols;
  const int64_t strip = ((M + want - 1) / want + 3) / 4 * 4;
  return (int)(strip < 4 ? 4 : strip);
}

}  // namespace

size_t glu_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  size_t most = 0;
  for (const bool al : {false, true}) {
    if (small_form(M, N, K, al) != Small::kNone) continue;
    const size_t b = choose(M, N, 128, steps_of(K), al, false).lay.part_bytes;
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_glu(const void* X, rb_dtype a_dtype, int64_t M, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu,
                      int64_t ldwu, int64_t N, int64_t K, const float* bg, const float* bu, int act, void* G, int64_t ldg,
                      void* U, int64_t ldu, void* H, rb_dtype h_dtype, int64_t ldh, void* ws, hipStream_t s) {
  const GluOut out{bg, bu, G, U, H, ldg, ldu, ldh, act, tile::lines(G, ldg, 2), tile::lines(U, ldu, 2),
                   tile::lines(H, ldh, h_dtype == RB_F32 ? 4 : 2)};
  return a_dtype == RB_F16 ? launch_glu_typed<_Float16>(X, M, ldx, Wg, ldwg, Wu, ldwu, N, K, out, h_dtype, ws, s)
                           : launch_glu_typed<__bf16>(X, M, ldx, Wg, ldwg, Wu, ldwu, N, K, out, h_dtype, ws, s);
}

size_t glu_backward_workspace_bytes(int64_t N, int64_t M) {
  const int strip = grad_strip(M, N);
  return M <= strip ? 0 : 2 * (size_t)((M + strip - 1) / strip) * (size_t)N * 4;
}

hipError_t launch_glu_backward(const void* dH, rb_dtype dh_dtype, int64_t M, int64_t N, int64_t lddh, const void* G, int64_t ldg,
                               const void* U, int64_t ldu, rb_dtype a_dtype, int act, void* dG, int64_t lddg, void* dU,
                               int64_t lddu, float* dbg, float* dbu, void* ws, hipStream_t s) {
  const int strip = grad_strip(M, N);
  const int strips = (int)((M + strip - 1) / strip);
  float* const part = static_cast<float*>(ws);
  float* const pg = !dbg ? nullptr : strips == 1 ? dbg : part;
  float* const pu = !dbu ? nullptr : strips == 1 ? dbu : part + (size_t)strips * (size_t)N;
  const GluGradArgs a{dH, G, U, dG, dU, pg, pu, M, lddh, ldg, ldu, lddg, lddu, (int)N, act, strip};
  const dim3 grid((uint32_t)((N + 511) / 512), (uint32_t)strips);
  if (a_dtype == RB_F16) {
    if (dh_dtype == RB_F32)
      glu_grad_kernel<_Float16, float><<<grid, 256, 0, s>>>(a);
    else
      glu_grad_kernel<_Float16, _Float16><<<grid, 256, 0, s>>>(a);
  } else if (dh_dtype == RB_F32) {
    glu_grad_kernel<__bf16, float><<<grid, 256, 0, s>>>(a);
  } else {
    glu_grad_kernel<__bf16, __bf16><<<grid, 256, 0, s>>>(a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || strips == 1 || (!dbg && !dbu)) return e;
  glu_grad_sum_kernel<<<dim3((uint32_t)((N + 63) / 64), 2), 512, 0, s>>>(pg, pu, strips, (int)N, dbg, dbu);
  return hipGetLastError();
}

size_t glu_dx_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  const size_t a = choose(M, K, 256, 2 * steps_of(N), false, true).lay.part_bytes;
  const size_t b = choose(M, K, 256, 2 * steps_of(N), true, true).lay.part_bytes;
  return a > b ? a : b;
}

hipError_t launch_glu_dx(const void* dG, int64_t lddg, const void* dU, int64_t lddu, rb_dtype a_dtype, int64_t M, const void* Wg,
                         int64_t ldwg, const void* Wu, int64_t ldwu, int64_t N, int64_t K, void* dX, rb_dtype dx_dtype,
                         int64_t lddx, void* ws, hipStream_t s) {
  return a_dtype == RB_F16
             ? launch_dx_typed<_Float16>(dG, lddg, dU, lddu, M, Wg, ldwg, Wu, ldwu, N, K, dX, dx_dtype, lddx, ws, s)
             : launch_dx_typed<__bf16>(dG, lddg, dU, lddu, M, Wg, ldwg, Wu, ldwu, N, K, dX, dx_dtype, lddx, ws, s);
}

}  // namespace rb
