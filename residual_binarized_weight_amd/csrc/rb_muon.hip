// rb_muon.hip -- an optimizer step of a matrix by momentum and Newton-Schulz products.
//
//   m <- mu m + s g;  u = s g + mu m (nesterov) or m;  X = u / (|u|_F + eps), as its transpose where it is tall
//   X <- a X + (b A + c A^2) X,  A = X X^T      a few times: the singular values go towards 1
//   (a, b, c) are those published with the method: K. Jordan and others, "Muon: an optimizer for hidden layers in
//   neural networks", 2024
//   W <- W (1 - lr wd) - lr scale X
//
// With n = min(N, K) and m = max(N, K) an iteration is three products: A (symmetric, n x n over m), the polynomial
// B = b A + c A^2 (symmetric, n x n over n) and X' = a X + B X (n x m over n).
//
// Arithmetic. The products take fp16 operands at fixed powers of two and sum in fp32: no entry of X exceeds 1.21 (the
// polynomial's largest value over 0 .. 1.21, where the singular values stay), none of A 1.47, none of B 2.81, so X and
// A are held times 2^15 and B times 2^14, all below fp16's largest, and an entry of X is near 2^15 / sqrt(n m),
// far above its smallest normal one. X itself is held as the sum of two fp16 (22 bits): of the terms of X' only a X
// carries the small singular values on, and each of the iterations multiplies them, and a rounding of X beside
// them, by up to 3.44. With one fp16 the result of a matrix of low rank is off by 15 % (64 x 128 of rank 1) or
// 3.5 % (128 x 256 of rank 16), with bf16 by all of it or 28 %; with two fp16 these are off by 0.07 and 0.08 %, and a
// full-rank one by 0.13 to 0.21 %, the rounding of B and of X inside B X.
//
// Kernels of this file:
//   muon_moment_kernel   m, and partial sums of u^2 (fp64);  muon_start_kernel  X from u and the norm
//   muon_product_kernel  the three products, on the matrix cores;  muon_join_kernel  split tiles
//   muon_few_kernel      the same for small matrices, a block's waves splitting the sum
//   muon_apply_kernel    W and, where asked for, X itself
#include "rb_internal.h"
#include "rb_tile.hpp"

namespace rb {
namespace {

using tile::f4;
using tile::Source;
using tile::Work;
typedef _Float16 half_t;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 32768.f, kScaleA = 32768.f, kScaleB = 16384.f;
constexpr int kMomentBlocks = 1024;

// ---------------------------------------------------------------------------------------------
// momentum and norm
// ---------------------------------------------------------------------------------------------
struct MomentArgs {
  const void* g;
  float* mom;
  int64_t ldg, ldm;
  int64_t N, K;
  float mu, eps;
  int nesterov;
  const float* grad_scale;
  const int32_t* skip;
  double* part;  // [kMomentBlocks] sums of u^2
  half_t *hi, *lo, *t;  // X, n_pad rows of m_pad, and its first half's transpose
  int64_t m_pad, n_pad;
  bool tall;  // X is u^T
};
// 8 elements of u = s g + mu m (or m) from the stored momentum
template <typename TG>
__device__ __forceinline__ void blend8(const MomentArgs& a, float s, int64_t row, int c, const float (&m)[8], float (&u)[8]) {
  if (a.mom && !a.nesterov) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = m[j];
    return;
  }
  widen8<TG>(load8_any<TG>(static_cast<const TG*>(a.g) + row * a.ldg, c, (int)a.K), u);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = a.mom ? fmaf(a.mu, m[j], s * u[j]) : s * u[j];
}

// Bound by HBM at large sizes, by its launch at small ones (256 x 512: 3.4 to 4.3 us traced).
template <typename TG>
__global__ __launch_bounds__(256) void muon_moment_kernel(MomentArgs a) {
  __shared__ double sums[4];
  if (a.skip && *a.skip) return;
  const float s = a.grad_scale ? *a.grad_scale : 1.f;
  const int64_t vecs = (a.K + 7) / 8, all = a.N * vecs;
  double sum = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / vecs;
    const int c = (int)(i - row * vecs) * 8;
    float g[8], m[8], u[8];
    widen8<TG>(load8<TG>(static_cast<const TG*>(a.g) + row * a.ldg, c, (int)a.K), g);
    if (a.mom) {
      float* const mr = a.mom + row * a.ldm;
      widen8<float>(load8<float>(mr, c, (int)a.K), m);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = fmaf(a.mu, m[j], s * g[j]);
      store8<float>(mr, c, (int)a.K, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = a.nesterov ? fmaf(a.mu, m[j], s * g[j]) : m[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = s * g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)u[j] * (double)u[j];
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.part[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// the two fp16 of a value of X
__device__ __forceinline__ void split(float x, half_t& hi, half_t& lo) {
  hi = (half_t)x;
  lo = (half_t)(x - (float)hi);
}

// A block owns 64 x 64 of X; bound by HBM (11008 x 4096: 126 to 140 us traced). The norm is summed from the partial sums
// by every block (8 KB from the cache), in one order.
template <typename TG>
__global__ __launch_bounds__(256) void muon_start_kernel(MomentArgs a) {
  __shared__ double sums[4];
  __shared__ float tilev[64][65];
  if (a.skip && *a.skip) return;
  double sum = 0.0;
  for (int i = threadIdx.x; i < kMomentBlocks; i += 256) sum += a.part[i];
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double inv = (double)kScaleX / (sqrt((sums[0] + sums[1]) + (sums[2] + sums[3])) + (double)a.eps);
  const float s = a.grad_scale ? *a.grad_scale : 1.f;
  // the block's rows and columns of u
  const int64_t r0 = (a.tall ? (int64_t)blockIdx.x : (int64_t)blockIdx.y) * 64;
  const int64_t c0 = (a.tall ? (int64_t)blockIdx.y : (int64_t)blockIdx.x) * 64;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = q * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
    float u[8] = {};
    if (r0 + r < a.N && c0 + c < a.K) {
      float m[8] = {};
      if (a.mom) widen8<float>(load8_any<float>(a.mom + (r0 + r) * a.ldm, (int)c0 + c, (int)a.K), m);
      blend8<TG>(a, s, r0 + r, (int)c0 + c, m, u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) tilev[r][c + j] = (float)((double)u[j] * inv);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = q * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;  // of X, and of its transpose
    half_t hi[8], lo[8], t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float along = tilev[r][c + j], across = tilev[c + j][r];
      split(a.tall ? across : along, hi[j], lo[j]);
      t[j] = (half_t)(a.tall ? along : across);
    }
    const int64_t xr = (int64_t)blockIdx.y * 64, xc = (int64_t)blockIdx.x * 64;
    const int64_t at = (xr + r) * a.m_pad + xc + c;
    *reinterpret_cast<tile::u4*>(a.hi + at) = *reinterpret_cast<const tile::u4*>(hi);
    *reinterpret_cast<tile::u4*>(a.lo + at) = *reinterpret_cast<const tile::u4*>(lo);
    *reinterpret_cast<tile::u4*>(a.t + (xc + r) * a.n_pad + xr + c) = *reinterpret_cast<const tile::u4*>(t);
  }
}

// ---------------------------------------------------------------------------------------------
// the products, all of rows along the sum: X is kept with its first half's transpose, which X' = a X + B X takes (the
// tiles take 1.86 us a step with rows across the sum, read through the transposing LDS reads, and 1.69 with rows along it).
// A symmetric product computes the lower triangle's tiles and writes each twice, the second time turned.
// 11008 x 4096, traced: A 176 to 188 us (+ 35 for the split tiles' join), B 95 to 103 (+ 7), X' 378 to 446, which reads and
// writes 450 MB of X after its sums; the whole step of 5 iterations 4010 to 4128 us (0.75 to 0.78 PFLOP/s). The same tiles reach 1.06 to
// 1.23 PFLOP/s in the gated products; here A makes 0.82 to 0.88 with its join, B on 128-square tiles 0.62 to 0.67, X' 0.83 to
// 0.98, with nothing over its reads and writes.
// ---------------------------------------------------------------------------------------------
enum class Kind { kGram, kPoly, kNext };  // A = X X^T; B = b A + c A A; X' = a X + B X

struct ProductArgs {
  Source<half_t> src[1];
  int M, N;  // of the output
  Work work;
  float* part;
  const half_t* A;         // kPoly: A
  const half_t *hi, *lo;   // kNext: X
  half_t *out, *out_lo;
  half_t* out_t;           // the output's (first half's) transpose: for the symmetric ones the output itself; or NULL
  int64_t ld, ld_t;
  const int32_t* skip;
};

// what an output's 8 columns are made of beside their sums: A, or the two halves of X
struct Beside {
  Vec8<half_t>::Raw a, b;
};
template <Kind kind>
__device__ __forceinline__ Beside beside(const ProductArgs& a, int64_t m, int n) {
  const int64_t at = m * a.ld + n;
  Beside x{};
  if constexpr (kind == Kind::kPoly) x.a = *reinterpret_cast<const Vec8<half_t>::Raw*>(a.A + at);
  if constexpr (kind == Kind::kNext) {
    x.a = *reinterpret_cast<const Vec8<half_t>::Raw*>(a.hi + at);
    x.b = *reinterpret_cast<const Vec8<half_t>::Raw*>(a.lo + at);
  }
  return x;
}
// 8 columns of a row from their sums, into the output's fp16; v becomes what its transpose takes
template <Kind kind>
__device__ __forceinline__ void finish8(const ProductArgs& a, const Beside& x, float (&v)[8], int64_t m, int n) {
  const int64_t at = m * a.ld + n;
  half_t o[8];
  if constexpr (kind == Kind::kGram) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (half_t)(v[j] * (kScaleA / (kScaleX * kScaleX)));
  } else if constexpr (kind == Kind::kPoly) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      o[j] = (half_t)fmaf(kB * (kScaleB / kScaleA), Vec8<half_t>::get(x.a, j), v[j] * (kC * (kScaleB / (kScaleA * kScaleA))));
  } else {
    half_t o2[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      split(fmaf(kA, Vec8<half_t>::get(x.a, j) + Vec8<half_t>::get(x.b, j), v[j] * (1.f / kScaleB)), o[j], o2[j]);
    *reinterpret_cast<tile::u4*>(a.out_lo + at) = *reinterpret_cast<const tile::u4*>(o2);
  }
  *reinterpret_cast<tile::u4*>(a.out + at) = *reinterpret_cast<const tile::u4*>(o);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)o[j];
}
// 8 rows of a column of what finish8 left, as a piece of the transpose
__device__ __forceinline__ void put_turned(const ProductArgs& a, const float* p, int stride, int64_t n, int64_t m) {
  half_t o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = (half_t)p[j * stride];
  *reinterpret_cast<tile::u4*>(a.out_t + n * a.ld_t + m) = *reinterpret_cast<const tile::u4*>(o);
}

// The tile of a symmetric output: those on and below the diagonal, row by row.
__device__ __forceinline__ void place_lower(uint32_t t, uint32_t& m, uint32_t& n) {
  uint32_t r = (uint32_t)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
  while (r * (r + 1) / 2 > t) --r;
  while ((r + 1) * (r + 2) / 2 <= t) ++r;
  m = r, n = t - r * (r + 1) / 2;
}
template <typename C, Kind kind>
__device__ __forceinline__ typename C::Where where(const ProductArgs& a, uint32_t t) {
  if constexpr (kind == Kind::kNext) {
    return C::where(a.work, t, a.M, a.N);
  } else {
    uint32_t m, n;
    place_lower(t, m, n);
    typename C::Where at;
    at.m0 = (int64_t)__builtin_amdgcn_readfirstlane(m) * C::BM;
    at.n0 = (int)__builtin_amdgcn_readfirstlane(n) * C::BN;
    at.mrows = a.M - (int)at.m0 < C::BM ? a.M - (int)at.m0 : C::BM;
    at.ncols = a.N - at.n0 < C::BN ? a.N - at.n0 : C::BN;
    return at;
  }
}

template <typename C, Kind kind>
__global__ __launch_bounds__(C::kThreads, 2) void muon_product_kernel(ProductArgs a) {
  static_assert(C::BM == C::BN, "a symmetric output's tiles mirror each other");
  extern __shared__ __align__(16) uint8_t t_smem[];
  if (a.skip && *a.skip) return;
  tile::share(a.work, [&](uint32_t t, int s0, int s1, int slot) {
    const typename C::Where at = where<C, kind>(a, t);
    typename C::Acc acc;
    C::run(a.src, at, a.N, s0, s1, t_smem, acc);
    float* const part = slot < 0 ? nullptr : a.part + (int64_t)slot * C::BM * C::BN;
    const bool turn = !part && a.out_t && (kind == Kind::kNext || at.m0 != at.n0);
    Beside x[C::kPasses];  // on its way from memory before it is needed
    C::rows_ahead(acc, t_smem, [&](int s, int r, int c) {
      if (!part && r < at.mrows && c < at.ncols) x[s] = beside<kind>(a, at.m0 + r, at.n0 + c);
    }, [&](int s, int r, int c, float* p) {
      float v[8];
      tile::eight(p, v);
      if (part) {
        store8<float>(part + r * C::BN, c, C::BN, v);
      } else if (r < at.mrows && c < at.ncols) {
        finish8<kind>(a, x[s], v, at.m0 + r, at.n0 + c);
        if (turn) {
          *reinterpret_cast<f4*>(p) = (f4){v[0], v[1], v[2], v[3]};
          *reinterpret_cast<f4*>(p + 4) = (f4){v[4], v[5], v[6], v[7]};
        }
      }
    }, [&](int r0, int c0, const float* p) {
      if (!turn || r0 >= at.mrows) return;
      for (int i = threadIdx.x & 63; i < 2 * C::kWaveN; i += 64) {
        const int c = i % C::kWaveN, h = i / C::kWaveN * 8;
        if (c0 + c < at.ncols) put_turned(a, p + h * C::kPad + c, C::kPad, at.n0 + c0 + c, at.m0 + r0 + h);
      }
    });
    __syncthreads();
  });
}

// Split tiles: a block takes 16 rows by kCols columns, 8 columns a thread, and adds the parts in the order of the sum
template <typename C> constexpr int join_cols() { return C::BN < 128 ? C::BN : 128; }
template <typename C, Kind kind>
__global__ __launch_bounds__(2 * join_cols<C>()) void muon_join_kernel(ProductArgs a) {
  constexpr int kCols = join_cols<C>(), kPad = kCols + 4;
  __shared__ __align__(16) float turn[16 * kPad];
  if (a.skip && *a.skip) return;
  const typename C::Where at = where<C, kind>(a, a.work.full + blockIdx.x);
  const int r0 = (int)blockIdx.y / (C::BN / kCols) * 16, c0 = (int)blockIdx.y % (C::BN / kCols) * kCols;
  const int r = threadIdx.x / (kCols / 8), c = threadIdx.x % (kCols / 8) * 8;
  float v[8] = {};
  tile::parts(a.work, blockIdx.x, [&](uint32_t slot) {
    float p[8];
    tile::eight(a.part + ((int64_t)slot * C::BM + r0 + r) * C::BN + c0 + c, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += p[j];
  });
  if (r0 + r < at.mrows && c0 + c < at.ncols) {
    const int64_t m = at.m0 + r0 + r;
    const int n = at.n0 + c0 + c;
    finish8<kind>(a, beside<kind>(a, m, n), v, m, n);
  }
  if (!a.out_t || (kind != Kind::kNext && at.m0 == at.n0) || r0 >= at.mrows) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) turn[r * kPad + c + j] = v[j];
  __syncthreads();
  const int tc = threadIdx.x % kCols, h = threadIdx.x / kCols * 8;
  if (c0 + tc < at.ncols) put_turned(a, turn + h * kPad + tc, kPad, at.n0 + c0 + tc, at.m0 + r0 + h);
}

// Small matrices, whose steps are as many launches as products: a block owns 16 x 16 outputs; its 8 waves take the 64-term
// steps in turn, each with its fragments straight from memory, and join in LDS in their order. Launches and
// latency bound it (a wave has the loads of up to four of its steps in flight at once): 256 x 512, medians traced, 3.8 us for
// A, 3.6 for B and 4.3 for the next X against 5.9, 5.9 and 5.6 on tiles of 64; the whole step 64 to 68 us against 85 to 90. From
// 512 x 512 on the tiles are as fast or faster. Every size is a multiple of 64 here.
template <Kind kind>
__global__ __launch_bounds__(512) void muon_few_kernel(ProductArgs a) {
  constexpr int kWaves = 8, kAhead = 4;  // steps whose loads a wave has in flight
  __shared__ __align__(16) float sums[kWaves][256];
  __shared__ half_t turn[16][17];
  if (a.skip && *a.skip) return;
  const Source<half_t>& q = a.src[0];
  const int lane = threadIdx.x & 63, lr = lane & 15, lj = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  uint32_t tm = blockIdx.y, tn = blockIdx.x;
  if (kind != Kind::kNext) place_lower(blockIdx.x, tm, tn);
  const int64_t m0 = (int64_t)tm * 16, n0 = (int64_t)tn * 16;
  const half_t* const row[2] = {q.B + (n0 + lr) * q.ldb + 8 * lj, q.A + (m0 + lr) * q.lda + 8 * lj};
  f4 acc = {};
  for (int s0 = w; s0 < q.steps; s0 += kAhead * kWaves) {
    tile::u4 f[kAhead][2][2] = {};
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
      if (s0 + s * kWaves < q.steps) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            f[s][h][i] = *reinterpret_cast<const tile::u4*>(row[i] + (int64_t)(s0 + s * kWaves) * tile::kTK + 32 * h);
      }
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = tile::mfma(half_t(0), f[s][h][0], f[s][h][1], acc);
  }
  *reinterpret_cast<f4*>(&sums[w][lane * 4]) = acc;
  __syncthreads();
  // thread 16 m + n: D's lane 16 (n / 4) + m holds column n in element n % 4
  const int r = threadIdx.x >> 4 & 15, c = threadIdx.x & 15;
  const bool mine = threadIdx.x < 256;
  if (mine) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += sums[i][((c >> 2) * 16 + r) * 4 + (c & 3)];
    const int64_t at = (m0 + r) * a.ld + n0 + c;
    half_t o;
    if constexpr (kind == Kind::kGram) {
      o = (half_t)(v * (kScaleA / (kScaleX * kScaleX)));
    } else if constexpr (kind == Kind::kPoly) {
      o = (half_t)fmaf(kB * (kScaleB / kScaleA), (float)a.A[at], v * (kC * (kScaleB / (kScaleA * kScaleA))));
    } else {
      half_t lo;
      split(fmaf(kA, (float)a.hi[at] + (float)a.lo[at], v * (1.f / kScaleB)), o, lo);
      a.out_lo[at] = lo;
    }
    a.out[at] = o;
    turn[r][c] = o;
  }
  if (!a.out_t || (kind != Kind::kNext && m0 == n0)) return;
  __syncthreads();
  if (mine) a.out_t[(n0 + r) * a.ld_t + m0 + c] = turn[c][r];
}

// ---------------------------------------------------------------------------------------------
// the update
// ---------------------------------------------------------------------------------------------
struct ApplyArgs {
  const half_t *hi, *lo;
  int64_t m_pad;
  float* W;
  void* O;
  int64_t ldw, ldo, N, K;
  float keep, rate;  // W <- keep W - rate X
  bool tall;
  const int32_t* skip;
};
// A block owns 64 x 64 of W; a tall matrix reads X's block turned. Bound by HBM (11008 x 4096: 104 us, 541 MB, 5.2 TB/s).
template <typename TO>
__global__ __launch_bounds__(256) void muon_apply_kernel(ApplyArgs a) {
  __shared__ float tilev[64][65];
  if (a.skip && *a.skip) return;
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;  // of W
  const int64_t xr = a.tall ? c0 : r0, xc = a.tall ? r0 : c0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = q * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
    const int64_t at = (xr + r) * a.m_pad + xc + c;
    const Vec8<half_t>::Raw h = *reinterpret_cast<const Vec8<half_t>::Raw*>(a.hi + at);
    const Vec8<half_t>::Raw l = *reinterpret_cast<const Vec8<half_t>::Raw*>(a.lo + at);
#pragma unroll
    for (int j = 0; j < 8; ++j) tilev[r][c + j] = (Vec8<half_t>::get(h, j) + Vec8<half_t>::get(l, j)) * (1.f / kScaleX);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = q * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
    if (r0 + r >= a.N || c0 + c >= a.K) continue;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = a.tall ? tilev[c + j][r] : tilev[r][c + j];
    if (a.O) store8<TO>(static_cast<TO*>(a.O) + (r0 + r) * a.ldo, (int)c0 + c, (int)a.K, x);
    if (a.W) {
      float w[8];
      float* const row = a.W + (r0 + r) * a.ldw;
      widen8<float>(load8<float>(row, (int)c0 + c, (int)a.K), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = fmaf(a.keep, w[j], -a.rate * x[j]);
      store8<float>(row, (int)c0 + c, (int)a.K, w);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------
// Tiles of 64, 128 and 256 square, chosen for each product by estimate: us of a step of such tiles on every unit.
template <int kSize> struct Square;
template <> struct Square<64> { typedef tile::Tile<half_t, 2, 2, 2, 2, 4, false, 0, 1, true> C; };
template <> struct Square<128> { typedef tile::Tile<half_t, 2, 2, 4, 4, 3, false, 0, 1, true> C; };
template <> struct Square<256> { typedef tile::Tile<half_t, 4, 2, 4, 8, 2, false, 0, 1, true> C; };
// Small products go to muon_few_kernel where its estimate, kFewStep us a step of 64 for each round of 256 blocks, is below
// the tiles'. Whole steps with it at 0.2 / 0.3 / 0.4 / 0.5, rounds not yet rounded up: 200 x 2000 90 / 90 / 100 / 100 us (all
// on tiles 110), 512 x 512 116 / 105 / 105 / 100 (101); rounded up, at 0.3: 91 and 100.
struct Choice {
  int size;  // 0: muon_few_kernel
  tile::Lay lay;
};
constexpr double kFewStep = 0.3;
Choice choose(int64_t M, int64_t N, int64_t steps, bool symmetric) {
  constexpr struct { int size; double step; } kinds[3] = {{64, 0.30}, {128, 0.60}, {256, 1.69}};
  Choice best{};
  for (const auto& k : kinds) {
    const int64_t tm = (M + k.size - 1) / k.size, tn = (N + k.size - 1) / k.size;
    const tile::Lay l = tile::lay(symmetric ? 1 : tm, symmetric ? tm * (tm + 1) / 2 : tn, steps, k.step, (int64_t)k.size * k.size * 4);
    if (best.size == 0 || l.est < best.lay.est) best = Choice{k.size, l};
  }
  const int64_t m = M / 16, n = N / 16, blocks = symmetric ? m * (m + 1) / 2 : m * n;
  if (2.6 + (double)((blocks + 255) / 256) * (double)steps * kFewStep < best.lay.est) {
    best.size = 0;
    best.lay.part_bytes = 0;
  }
  return best;
}

// Where everything lies in the workspace; n and m are padded to whole steps with zeros.
struct Buffers {
  int64_t n, m;
  size_t part, x[6], a, b, sums, bytes;
  Choice gram, poly, next;
};
Buffers buffers(int64_t N, int64_t K) {
  Buffers b{};
  b.n = ((N < K ? N : K) + 63) / 64 * 64;
  b.m = ((N < K ? K : N) + 63) / 64 * 64;
  b.gram = choose(b.n, b.n, b.m / 64, true);
  b.poly = choose(b.n, b.n, b.n / 64, true);
  b.next = choose(b.n, b.m, b.n / 64, false);
  const auto take = [&](size_t bytes) {
    const size_t at = b.bytes;
    b.bytes += (bytes + 255) / 256 * 256;
    return at;
  };
  b.part = take(kMomentBlocks * sizeof(double));
  for (size_t& x : b.x) x = take((size_t)b.n * (size_t)b.m * 2);
  b.a = take((size_t)b.n * (size_t)b.n * 2);
  b.b = take((size_t)b.n * (size_t)b.n * 2);
  size_t most = 0;
  for (const Choice* c : {&b.gram, &b.poly, &b.next}) most = c->lay.part_bytes > most ? c->lay.part_bytes : most;
  b.sums = take(most);
  return b;
}

template <int kSize, Kind kind>
hipError_t launch_size(const ProductArgs& a, hipStream_t s) {
  typedef typename Square<kSize>::C C;
  static std::atomic<uint64_t> done;
  hipError_t e = tile::allow_lds(done, muon_product_kernel<C, kind>, C::kLds);
  if (e != hipSuccess) return e;
  muon_product_kernel<C, kind><<<a.work.grid, C::kThreads, C::kLds, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || a.work.full == a.work.tiles) return e;
  constexpr int cols = join_cols<C>();
  muon_join_kernel<C, kind><<<dim3(a.work.tiles - a.work.full, C::BM / 16 * (C::BN / cols)), 2 * cols, 0, s>>>(a);
  return hipGetLastError();
}
template <Kind kind>
hipError_t launch_product(const Choice& c, const ProductArgs& a, hipStream_t s) {
  if (c.size == 0) {
    const uint32_t m = (uint32_t)a.M / 16, n = (uint32_t)a.N / 16;
    muon_few_kernel<kind><<<kind == Kind::kNext ? dim3(n, m) : dim3(m * (m + 1) / 2), 512, 0, s>>>(a);
    return hipGetLastError();
  }
  return c.size == 64 ? launch_size<64, kind>(a, s) : c.size == 128 ? launch_size<128, kind>(a, s) : launch_size<256, kind>(a, s);
}

template <typename TG>
hipError_t launch_start(const MomentArgs& a, hipStream_t s) {
  muon_moment_kernel<TG><<<kMomentBlocks, 256, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  muon_start_kernel<TG><<<dim3((uint32_t)(a.m_pad / 64), (uint32_t)(a.n_pad / 64)), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t muon_workspace_bytes(int64_t N, int64_t K) { return buffers(N, K).bytes; }

hipError_t launch_muon_step(float* W, int64_t ldw, const void* G, rb_dtype g_dtype, int64_t ldg, float* mom, int64_t ldm,
                            int64_t N, int64_t K, double lr, double momentum, int nesterov, double weight_decay,
                            double scale, int steps, double eps, const float* grad_scale, const int32_t* skip, void* O,
                            rb_dtype o_dtype, int64_t ldo, void* ws, hipStream_t s) {
  const Buffers b = buffers(N, K);
  char* const base = static_cast<char*>(ws);
  const auto half_at = [&](size_t at) { return reinterpret_cast<half_t*>(base + at); };
  struct Held { half_t *hi, *lo, *t; } x{half_at(b.x[0]), half_at(b.x[1]), half_at(b.x[2])},
      y{half_at(b.x[3]), half_at(b.x[4]), half_at(b.x[5])};
  half_t *const A = half_at(b.a), *const B = half_at(b.b);
  float* const part = reinterpret_cast<float*>(base + b.sums);
  const MomentArgs m{G, mom, ldg, ldm, N, K, (float)momentum, (float)eps, nesterov, grad_scale, skip,
                     reinterpret_cast<double*>(base + b.part), x.hi, x.lo, x.t, b.m, b.n, N > K};
  hipError_t e = g_dtype == RB_F32 ? launch_start<float>(m, s)
                 : g_dtype == RB_F16 ? launch_start<_Float16>(m, s) : launch_start<__bf16>(m, s);
  if (e != hipSuccess) return e;
  const int n = (int)b.n, cols = (int)b.m;
  for (int i = 0; i < steps; ++i) {
    const ProductArgs gram{{{x.hi, x.hi, nullptr, b.m, b.m, 0, cols, cols / 64}}, n, n, b.gram.lay.work, part, nullptr, nullptr,
                           nullptr, A, nullptr, A, b.n, b.n, skip};
    const ProductArgs poly{{{A, A, nullptr, b.n, b.n, 0, n, n / 64}}, n, n, b.poly.lay.work, part, A, nullptr, nullptr, B,
                           nullptr, B, b.n, b.n, skip};
    const ProductArgs next{{{B, x.t, nullptr, b.n, b.n, 0, n, n / 64}}, n, cols, b.next.lay.work, part, nullptr, x.hi, x.lo,
                           y.hi, y.lo, i + 1 < steps ? y.t : nullptr, b.m, b.n, skip};
    if ((e = launch_product<Kind::kGram>(b.gram, gram, s)) != hipSuccess) return e;
    if ((e = launch_product<Kind::kPoly>(b.poly, poly, s)) != hipSuccess) return e;
    if ((e = launch_product<Kind::kNext>(b.next, next, s)) != hipSuccess) return e;
    const Held t = x;
    x = y, y = t;
  }
  const ApplyArgs p{x.hi, x.lo, b.m, W, O, ldw, ldo, N, K, (float)(1.0 - lr * weight_decay), (float)(lr * scale), N > K, skip};
  const dim3 grid((uint32_t)((K + 63) / 64), (uint32_t)((N + 63) / 64));
  if (o_dtype == RB_F16)
    muon_apply_kernel<_Float16><<<grid, 256, 0, s>>>(p);
  else
    muon_apply_kernel<__bf16><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace rb
