// rb_resnorm.hip -- the norms after one block and before the next, with the block's gate and the
// stream's scale, forward and backward.
//
//   u = norm_post(Y);  S = alpha R + gate u;  X = norm_pre(S)
//   norm(x) = (x - mu) rstd w + b,  rstd = (mean (x - mu)^2 + eps)^(-1/2),  mu = 0 for an rms norm
//
// Every tensor passes once: HBM bounds both directions (a row's arithmetic is some 10 to 25
// operations per element). A row is held in registers by a group of TPR threads, 8 NV
// consecutive columns each (16-byte accesses), and its two norms are reduced there one after the
// other: by DPP inside a wave, through LDS between waves. All sums are fp32; the mean is taken
// before the squares, so a large mean costs no digits.
//
// Measured (bf16, fp32 stream, rms norms, a gate per channel): forward 2048 x 4096 18 to 19 us, 101 MB
// = 5.3 TB/s, about what a copy reaches; one row 3 us. Stores are streamed (nothing here reads them
// again): 23.7 us without.
#include "rb_elem.hpp"
#include "rb_internal.h"
#include <type_traits>

namespace rb {
namespace {

// 8 columns from c of a row of n (0: of a row that is not there) into r; what lies past its end
// becomes 0. LONG: rows of 8 columns and more, without element loads.
template <bool LONG, typename T>
__device__ __forceinline__ void load(typename Vec8<T>::Raw& r, const T* row, int c, int n) {
  if constexpr (LONG) {
    r = typename Vec8<T>::Raw{};
    load8_long<T>(r, row, c, n);
    if (c < n && c + 8 > n) shift_down(r, c + 8 - n);
  } else {
    r = load8<T>(row, c, n);
  }
}
template <bool LONG>
__device__ __forceinline__ void load_vec(float (&v)[8], const float* x, int c, int n) {
  Vec8<float>::Raw r;
  load<LONG, float>(r, x, c, n);
  widen8<float>(r, v);
}

// sum over aligned groups of 16 lanes, in all of them
__device__ __forceinline__ float sum16(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));   // quad [1,0,3,2]
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));   // quad [2,3,0,1]
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));  // row_half_mirror
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));  // row_mirror
  return v;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// totals over the TPR threads that share a row, in all of them: the waves' sums meet in LDS, where
// lane i of every wave reads wave i's. `slot` (a float2 per wave) is this reduction's own area:
// two of them used in turn need one barrier each.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* slot) {
  a = wave_sum_dpp(a);
  b = wave_sum_dpp(b);
  if constexpr (TPR == 64) {
    a = lane_value(a, 63);
    b = lane_value(b, 63);
  } else {
    constexpr int W = TPR / 64;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (lane == 63) slot[wave] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane < W ? slot[wave / W * W + lane] : make_float2(0.f, 0.f);
    a = lane_value(sum16(v.x), 0);
    b = lane_value(sum16(v.y), 0);
  }
}
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float2* slot) {
  float zero = 0.f;
  row_sum2<TPR>(v, zero, slot);
  return v;
}

// (mu, rstd) of the row; slot0 and slot1 are two reductions' LDS areas
template <int TPR, int NV>
__device__ __forceinline__ void row_stats(const float (&x)[NV][8], int c0, int D, int kind, float eps, float2* slot0,
                                          float2* slot1, float& mu, float& rstd) {
  const float inv = 1.f / (float)D;
  mu = 0.f;
  if (kind == RB_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += x[i][j];  // columns past D hold 0
    mu = row_sum<TPR>(s, slot0) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = c0 + i * TPR * 8 + j < D ? x[i][j] - mu : 0.f;
      q += d * d;
    }
  rstd = 1.f / sqrtf(row_sum<TPR>(q, slot1) * inv + eps);
}

struct FwdArgs {
  const void* Y;
  const void* R;
  const void* gate;
  const float *w_post, *b_post, *w_pre, *b_pre;
  void* S;
  void* X;
  float* stats;
  int64_t M, ldy, ldr, ldg, lds, ldx;
  int D, post, pre;
  float alpha, eps;
};

// y = x-hat w + b over the thread's columns
template <bool LONG, int TPR, int NV>
__device__ __forceinline__ void apply_norm(float (&x)[NV][8], int c0, int D, float mu, float rstd, const float* w,
                                           const float* b) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * TPR * 8;
    float wv[8], bv[8];
    load_vec<LONG>(wv, w, c, D);
    if (b) load_vec<LONG>(bv, b, c, D);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float h = (x[i][j] - mu) * rstd * wv[j];
      x[i][j] = b ? h + bv[j] : h;
    }
  }
}

template <typename TA, typename TS, int TPR, int NV, bool LONG>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void resnorm_forward_kernel(FwdArgs a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;  // rows per block
  __shared__ float2 slots[4][16];
  const int t = threadIdx.x % TPR;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);  // rows are scalar: so are their addresses
  const int64_t row = (int64_t)blockIdx.x * kRows + wave / (TPR / 64);
  const bool live = row < a.M;
  const int D = live ? a.D : 0;  // a group past the last row takes part in the barriers only
  const int c0 = t * 8;
  float u[NV][8], r[NV][8];
  typename Vec8<TA>::Raw yr[NV];
  typename Vec8<TS>::Raw rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) load<LONG, TA>(yr[i], static_cast<const TA*>(a.Y) + row * a.ldy, c0 + i * TPR * 8, D);
  if (a.R) {
#pragma unroll
    for (int i = 0; i < NV; ++i) load<LONG, TS>(rr[i], static_cast<const TS*>(a.R) + row * a.ldr, c0 + i * TPR * 8, D);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    widen8<TA>(yr[i], u[i]);
    if (a.R) widen8<TS>(rr[i], r[i]);
  }
  float mu0 = 0.f, rs0 = 0.f, mu1 = 0.f, rs1 = 0.f;
  if (a.post != RB_NORM_NONE) {
    row_stats<TPR, NV>(u, c0, a.D, a.post, a.eps, slots[0], slots[1], mu0, rs0);
    apply_norm<LONG, TPR, NV>(u, c0, D, mu0, rs0, a.w_post, a.b_post);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * TPR * 8;
    if (a.gate) {
      float g[8];
      if (a.ldg) {
        typename Vec8<TA>::Raw gr;
        load<LONG, TA>(gr, static_cast<const TA*>(a.gate) + row * a.ldg, c, D);
        widen8<TA>(gr, g);
      } else {
        load_vec<LONG>(g, static_cast<const float*>(a.gate), c, D);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] *= g[j];
    }
    if (a.R) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] += a.alpha * r[i][j];
    }
    if (a.S) store8<TS, true>(static_cast<TS*>(a.S) + row * a.lds, c, D, u[i]);
  }
  if (a.pre != RB_NORM_NONE) {
    // columns past D hold 0: an absent load gives 0 for every operand above
    row_stats<TPR, NV>(u, c0, a.D, a.pre, a.eps, slots[2], slots[3], mu1, rs1);
    apply_norm<LONG, TPR, NV>(u, c0, D, mu1, rs1, a.w_pre, a.b_pre);
#pragma unroll
    for (int i = 0; i < NV; ++i) store8<TA, true>(static_cast<TA*>(a.X) + row * a.ldx, c0 + i * TPR * 8, D, u[i]);
  }
  if (a.stats && live && t == 0) {
    float* st = a.stats + row * 4;
    st[0] = mu0, st[1] = rs0, st[2] = mu1, st[3] = rs1;
  }
}

// ---------------------------------------------------------------------------------------------
// backward. With d = dy w, xh = (x - mu) rstd, a norm's input gradient is
//   rstd (d - xh mean(d xh) - [layer] mean(d)),  its weights' dw = sum dy xh, db = sum dy;
//   T = dS + pre norm's input gradient;  dR = alpha T;  dgate = u T;  dY from gate T.
// A block walks over rows and keeps the column sums of its rows in registers; at the end its row
// groups are joined through LDS and the block's sums go to the workspace, where a second kernel
// adds them over the blocks in a fixed order.
//
// Measured, bf16 with an fp32 stream, rms norms and a gate per channel, 2048 x 4096: 36 us and 4 for
// the sums, 151 MB = 4.2 TB/s; a row's loads wait while the row before it is reduced, and only the next
// row's are in flight. 1537 x 8191 in bf16, layer norms and a gate per element: 71 us and 8.6, 202 MB =
// 2.8 TB/s; 1024 threads leave 128 registers each, which do not hold a second row. One block per compute
// unit: with two (512 blocks) the first takes 43 us and the sums 6.6.
// ---------------------------------------------------------------------------------------------
struct BwdArgs {
  const void *dX, *dS, *Y, *S, *gate;
  void *dY, *dR, *dgate;  // dgate here: the rows' form only
  float* part;            // [vectors][grid][D]
  int64_t M, lddx, ldds, ldy, lds, ldg, lddy, lddr, lddg;
  int D, post, pre, slot[5];  // slot: a vector's place among the partial sums, -1 where it is not wanted
  float alpha;
};
enum { kDwPre, kDbPre, kDwPost, kDbPost, kDgate };

// A row as it was read: packed, the vector at the row's end not yet shifted. Lanes past the end, and
// tensors that are not there, hold 0 throughout.
template <typename TA, typename TS, int NV> struct RowRaw {
  typename Vec8<TA>::Raw dx[NV], y[NV], g[NV];
  typename Vec8<TS>::Raw ds[NV], s[NV];
};

template <bool LONG, typename TA, typename TS, int TPR, int NV>
__device__ __forceinline__ void load_row(RowRaw<TA, TS, NV>& q, const BwdArgs& a, int64_t row, int c0) {
  if (row >= a.M) {
    q = RowRaw<TA, TS, NV>{};
    return;
  }
  const auto get = [&](auto* p, auto& r, int c) {
    typedef typename std::remove_const<typename std::remove_pointer<decltype(p)>::type>::type T;
    if constexpr (LONG)
      load8_long<T>(r, p, c, a.D);
    else
      r = load8<T>(p, c, a.D);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * TPR * 8;
    if (a.pre != RB_NORM_NONE) {
      get(static_cast<const TA*>(a.dX) + row * a.lddx, q.dx[i], c);
      get(static_cast<const TS*>(a.S) + row * a.lds, q.s[i], c);
    }
    if (a.Y) get(static_cast<const TA*>(a.Y) + row * a.ldy, q.y[i], c);
    if (a.dS) get(static_cast<const TS*>(a.dS) + row * a.ldds, q.ds[i], c);
    if (a.ldg) get(static_cast<const TA*>(a.gate) + row * a.ldg, q.g[i], c);
  }
}

constexpr int bwd_threads(int tpr) { return tpr < 512 ? 512 : tpr; }

// The column sums of rows of 4097 to 8192 columns (a block of 1024 threads, 128 registers each) lie in LDS,
// each word its own thread's; registers hold the others.
constexpr bool sums_in_lds(int tpr, int nv) { return tpr == 1024 && nv == 1; }

template <typename TA, typename TS, int TPR, int NV, bool BIAS, bool LONG>
__global__ __launch_bounds__(bwd_threads(TPR)) void resnorm_backward_kernel(
    BwdArgs a, const float* __restrict__ stats, const float* __restrict__ w_pre, const float* __restrict__ w_post,
    const float* __restrict__ b_post) {
  constexpr int kGroups = bwd_threads(TPR) / TPR;
  constexpr bool kKeep = bwd_threads(TPR) <= 512;  // registers for the vectors and for two rows
  constexpr bool kLds = sums_in_lds(TPR, NV);
  extern __shared__ float join[];  // the groups' sums at the end, [kGroups - 1][D]; or all sums, [vectors][8 NV][TPR]
  __shared__ float2 slots[2][2][16];  // by the round's parity: a slow wave may still read the last round's
  const int t = threadIdx.x % TPR;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);  // rows are scalar: so are their addresses
  const int group = wave / (TPR / 64);
  const int c0 = t * 8;
  const float inv = 1.f / (float)a.D;
  const bool pre = a.pre != RB_NORM_NONE, post = a.post != RB_NORM_NONE, gated = a.gate != nullptr;
  float acc[5][NV][8];
#pragma unroll
  for (int k = 0; k < 5; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[k][i][j] = 0.f;
  if constexpr (kLds) {
    for (int k = 0; k < 4; ++k)
      if (a.slot[k] >= 0)
        for (int j = 0; j < 8 * NV; ++j) join[(a.slot[k] * 8 * NV + j) * TPR + t] = 0.f;
  }
  const auto add = [&](int k, int i, int j, float v) {
    if (kLds && k < 4) {
      if (a.slot[k] >= 0) join[((a.slot[k] * NV + i) * 8 + j) * TPR + t] += v;
    } else {
      acc[k][i][j] += v;
    }
  };

  // the vectors of the thread's columns (0 past the row's end): kept, or read again for every row
  float wpre[NV][8], wpost[NV][8], bpost[NV][8], gvec[NV][8];
  const auto vectors = [&](int which) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * TPR * 8;
      if ((which & 1) && pre) load_vec<LONG>(wpre[i], w_pre, c, a.D);
      if ((which & 2) && post) load_vec<LONG>(wpost[i], w_post, c, a.D);
      if ((which & 2) && b_post) load_vec<LONG>(bpost[i], b_post, c, a.D);
      if ((which & 2) && gated && !a.ldg) load_vec<LONG>(gvec[i], static_cast<const float*>(a.gate), c, a.D);
    }
  };
  if constexpr (kKeep) vectors(3);

  const int64_t stride = (int64_t)gridDim.x * kGroups;
  const auto one_row = [&](RowRaw<TA, TS, NV>& q, int64_t row, int odd) {
    const bool live = row < a.M;
    const int D = live ? a.D : 0;
    const int64_t srow = live ? row : 0;
    const float mu0 = stats[srow * 4], rs0 = stats[srow * 4 + 1], mu1 = stats[srow * 4 + 2], rs1 = stats[srow * 4 + 3];
    if constexpr (LONG) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * TPR * 8;
        if (c < D && c + 8 > D) {
          const int by = c + 8 - D;
          shift_down(q.dx[i], by);
          shift_down(q.s[i], by);
          shift_down(q.y[i], by);
          shift_down(q.ds[i], by);
          shift_down(q.g[i], by);
        }
      }
    }
    float T[NV][8];
    if (pre) {
      if constexpr (!kKeep) vectors(1);
      float c1 = 0.f, c2 = 0.f;
      const float off = -mu1 * rs1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float dx[8], s[8];
        widen8<TA>(q.dx[i], dx);
        widen8<TS>(q.s[i], s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // past the end dx and d are 0, so xh adds nothing
          const float xh = fmaf(s[j], rs1, off), d = dx[j] * wpre[i][j];
          c1 += d;
          c2 = fmaf(d, xh, c2);
          add(kDwPre, i, j, dx[j] * xh);
          if (BIAS) add(kDbPre, i, j, dx[j]);
        }
      }
      row_sum2<TPR>(c1, c2, slots[odd][0]);
      c1 = a.pre == RB_NORM_LAYER ? c1 * inv * rs1 : 0.f;
      c2 *= inv * rs1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float dx[8], s[8], ds[8];
        widen8<TA>(q.dx[i], dx);
        widen8<TS>(q.s[i], s);
        widen8<TS>(q.ds[i], ds);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          T[i][j] = fmaf(-fmaf(s[j], rs1, off), c2, fmaf(dx[j] * wpre[i][j], rs1, ds[j] - c1));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) widen8<TS>(q.ds[i], T[i]);
    }
    if constexpr (!kKeep) vectors(2);
    float e[NV][8], yh[NV][8];
    float c1 = 0.f, c2 = 0.f;
    const float off = -mu0 * rs0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * TPR * 8;
      if (a.dR) {
        float dr[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dr[j] = a.alpha * T[i][j];
        store8<TS, true>(static_cast<TS*>(a.dR) + row * a.lddr, c, D, dr);
      }
      widen8<TA>(q.y[i], yh[i]);
      if (post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) yh[i][j] = fmaf(yh[i][j], rs0, off);
      }
      if (gated) {
        float dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float u = post ? yh[i][j] * wpost[i][j] : yh[i][j];
          if (b_post) u += bpost[i][j];
          dg[j] = u * T[i][j];
        }
        if (a.ldg) {
          if (a.dgate) store8<TA, true>(static_cast<TA*>(a.dgate) + row * a.lddg, c, D, dg);
#pragma unroll
          for (int j = 0; j < 8; ++j) T[i][j] *= Vec8<TA>::get(q.g[i], j);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) add(kDgate, i, j, dg[j]), T[i][j] *= gvec[i][j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) e[i][j] = T[i][j];
      if (post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float du = T[i][j];
          add(kDwPost, i, j, du * yh[i][j]);
          if (BIAS) add(kDbPost, i, j, du);
          e[i][j] = du * wpost[i][j];  // 0 past the row's end
          c1 += e[i][j];
          c2 = fmaf(e[i][j], yh[i][j], c2);
        }
      }
    }
    if constexpr (!kKeep) load_row<LONG, TA, TS, TPR, NV>(q, a, row + stride, c0);
    if (post) {
      row_sum2<TPR>(c1, c2, slots[odd][1]);
      c1 = a.post == RB_NORM_LAYER ? -c1 * inv * rs0 : 0.f;
      c2 *= inv * rs0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) e[i][j] = fmaf(-yh[i][j], c2, fmaf(e[i][j], rs0, c1));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) store8<TA, true>(static_cast<TA*>(a.dY) + row * a.lddy, c0 + i * TPR * 8, D, e[i]);
  };
  // The next row's loads: with registers for two rows issued before this row is begun, otherwise as soon
  // as this row's values are used up. Group 0 has the block's lowest row: while that is live, all groups
  // go on together.
  RowRaw<TA, TS, NV> q[kKeep ? 2 : 1] = {};
  int64_t row = blockIdx.x + (int64_t)gridDim.x * group;
  load_row<LONG, TA, TS, TPR, NV>(q[0], a, row, c0);
  for (int64_t first = blockIdx.x; first < a.M; first += 2 * stride, row += 2 * stride) {
    if (kKeep) load_row<LONG, TA, TS, TPR, NV>(q[kKeep], a, row + stride, c0);
    one_row(q[0], row, 0);
    if (first + stride >= a.M) break;
    if (kKeep) load_row<LONG, TA, TS, TPR, NV>(q[0], a, row + 2 * stride, c0);
    one_row(q[kKeep], row + stride, 1);
  }

#pragma unroll
  for (int k = 0; k < 5; ++k) {
    if (a.slot[k] < 0) continue;
    if (kGroups > 1) {
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) store8<float>(join + (int64_t)(group - 1) * a.D, c0 + i * TPR * 8, a.D, acc[k][i]);
      }
      __syncthreads();
    }
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (kLds && k < 4) {
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[k][i][j] = join[((a.slot[k] * NV + i) * 8 + j) * TPR + t];
        }
        for (int g = 1; g < kGroups; ++g) {
          float o[8];
          widen8<float>(load8<float>(join + (int64_t)(g - 1) * a.D, c0 + i * TPR * 8, a.D), o);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[k][i][j] += o[j];
        }
        store8<float>(a.part + ((int64_t)a.slot[k] * gridDim.x + blockIdx.x) * a.D, c0 + i * TPR * 8, a.D, acc[k][i]);
      }
    }
  }
}

struct SumArgs {
  const float* part;
  float* out[5];  // by slot
  int blocks, D;
};
// column sums over the blocks' partial sums: 64 columns by 8 interleaved runs of blocks
__global__ __launch_bounds__(512) void resnorm_sum_kernel(SumArgs a) {
  __shared__ float s[8][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* p = a.part + (int64_t)blockIdx.y * a.blocks * a.D;
  float v = 0.f;
  if (c < a.D) {
#pragma unroll 4
    for (int b = run; b < a.blocks; b += 8) v += p[(int64_t)b * a.D + c];
  }
  s[run][lane] = v;
  __syncthreads();
  if (run == 0 && c < a.D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    a.out[blockIdx.y][c] = v;
  }
}

constexpr int kBwdGrid = 256;  // one block per compute unit

template <typename TA, typename TS, int TPR, int NV, bool LONG = true>
hipError_t forward(const FwdArgs& a, hipStream_t s) {
  constexpr int threads = TPR < 256 ? 256 : TPR;
  constexpr int rows = TPR < 256 ? 256 / TPR : 1;
  const int64_t grid = (a.M + rows - 1) / rows;
  resnorm_forward_kernel<TA, TS, TPR, NV, LONG><<<dim3((uint32_t)grid), threads, 0, s>>>(a);
  return hipGetLastError();
}

// the fewest threads that hold a row, 8 columns each (16 from 8193 columns on)
template <typename TA, typename TS>
hipError_t forward_width(const FwdArgs& a, hipStream_t s) {
  if (a.D < 8) return forward<TA, TS, 64, 1, false>(a, s);
  if (a.D <= 64 * 8) return forward<TA, TS, 64, 1>(a, s);
  if (a.D <= 128 * 8) return forward<TA, TS, 128, 1>(a, s);
  if (a.D <= 256 * 8) return forward<TA, TS, 256, 1>(a, s);
  if (a.D <= 512 * 8) return forward<TA, TS, 512, 1>(a, s);
  if (a.D <= 1024 * 8) return forward<TA, TS, 1024, 1>(a, s);
  return forward<TA, TS, 1024, 2>(a, s);
}

struct BwdVectors {
  const float *stats, *w_pre, *w_post, *b_post;
};
template <typename TA, typename TS, int TPR, int NV, bool LONG = true>
hipError_t backward(const BwdArgs& a, const BwdVectors& v, int grid, hipStream_t s) {
  const bool bias = a.slot[kDbPre] >= 0 || a.slot[kDbPost] >= 0;
  constexpr int threads = bwd_threads(TPR);
  const size_t lds = sums_in_lds(TPR, NV) ? (size_t)4 * 8 * NV * TPR * 4 : (size_t)(threads / TPR - 1) * a.D * 4;
  if (sums_in_lds(TPR, NV)) {
    static const hipError_t attr[2] = {
        hipFuncSetAttribute((const void*)resnorm_backward_kernel<TA, TS, TPR, NV, false, LONG>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, 4 * 8 * NV * TPR * 4),
        hipFuncSetAttribute((const void*)resnorm_backward_kernel<TA, TS, TPR, NV, true, LONG>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, 4 * 8 * NV * TPR * 4)};
    if (attr[0] != hipSuccess || attr[1] != hipSuccess) return attr[0] != hipSuccess ? attr[0] : attr[1];
  }
  if (bias)
    resnorm_backward_kernel<TA, TS, TPR, NV, true, LONG><<<dim3((uint32_t)grid), threads, lds, s>>>(a, v.stats, v.w_pre, v.w_post, v.b_post);
  else
    resnorm_backward_kernel<TA, TS, TPR, NV, false, LONG><<<dim3((uint32_t)grid), threads, lds, s>>>(a, v.stats, v.w_pre, v.w_post, v.b_post);
  return hipGetLastError();
}
template <typename TA, typename TS>
hipError_t backward_width(const BwdArgs& a, const BwdVectors& v, int grid, hipStream_t s) {
  if (a.D < 8) return backward<TA, TS, 64, 1, false>(a, v, grid, s);
  if (a.D <= 64 * 8) return backward<TA, TS, 64, 1>(a, v, grid, s);
  if (a.D <= 256 * 8) return backward<TA, TS, 256, 1>(a, v, grid, s);
  if (a.D <= 512 * 8) return backward<TA, TS, 512, 1>(a, v, grid, s);
  if (a.D <= 1024 * 8) return backward<TA, TS, 1024, 1>(a, v, grid, s);
  return backward<TA, TS, 1024, 2>(a, v, grid, s);
}

}  // namespace

hipError_t launch_resnorm_forward(const void* Y, rb_dtype a_dtype, int64_t M, int64_t D, int64_t ldy, const void* R,
                                  rb_dtype s_dtype, int64_t ldr, const void* gate, int64_t ldg, float alpha, int post,
                                  const float* w_post, const float* b_post, int pre, const float* w_pre,
                                  const float* b_pre, float eps, void* S, int64_t lds, void* X, int64_t ldx,
                                  float* stats, hipStream_t s) {
  const FwdArgs a{Y, R, gate, w_post, b_post, w_pre, b_pre, S, X, stats, M, ldy, ldr, ldg, lds, ldx, (int)D, post, pre,
                  alpha, eps};
  if (a_dtype == RB_F32) return forward_width<float, float>(a, s);
  if (a_dtype == RB_F16)
    return s_dtype == RB_F32 ? forward_width<_Float16, float>(a, s) : forward_width<_Float16, _Float16>(a, s);
  return s_dtype == RB_F32 ? forward_width<__bf16, float>(a, s) : forward_width<__bf16, __bf16>(a, s);
}

static int resnorm_grid(int64_t M) { return (int)(M < kBwdGrid ? M : kBwdGrid); }

size_t resnorm_backward_workspace_bytes(int64_t D, int64_t M) { return (size_t)5 * resnorm_grid(M) * (size_t)D * 4; }

hipError_t launch_resnorm_backward(const void* dX, rb_dtype a_dtype, int64_t M, int64_t D, int64_t lddx, const void* dS,
                                   rb_dtype s_dtype, int64_t ldds, const void* Y, int64_t ldy, const void* S,
                                   int64_t lds, const float* stats, const void* gate, int64_t ldg, float alpha,
                                   int post, const float* w_post, const float* b_post, int pre, const float* w_pre,
                                   void* dY, int64_t lddy, void* dR, int64_t lddr, void* dgate, int64_t lddg,
                                   float* dw_post, float* db_post, float* dw_pre, float* db_pre, void* ws,
                                   hipStream_t s) {
  const BwdVectors v{stats, w_pre, w_post, b_post};
  BwdArgs a{dX, dS, Y, S, gate, dY, dR, ldg ? dgate : nullptr, static_cast<float*>(ws),
            M, lddx, ldds, ldy, lds, gate ? ldg : 0, lddy, lddr, lddg, (int)D, post, pre, {-1, -1, -1, -1, -1}, alpha};
  SumArgs sum{a.part, {}, resnorm_grid(M), (int)D};
  int vectors = 0;
  const auto want = [&](int k, float* out) {
    if (out) a.slot[k] = vectors, sum.out[vectors++] = out;
  };
  want(kDwPre, dw_pre);
  want(kDbPre, db_pre);
  want(kDwPost, dw_post);
  want(kDbPost, db_post);
  want(kDgate, gate && !ldg ? static_cast<float*>(dgate) : nullptr);
  hipError_t e;
  const int grid = sum.blocks;
  if (a_dtype == RB_F32)
    e = backward_width<float, float>(a, v, grid, s);
  else if (a_dtype == RB_F16)
    e = s_dtype == RB_F32 ? backward_width<_Float16, float>(a, v, grid, s) : backward_width<_Float16, _Float16>(a, v, grid, s);
  else
    e = s_dtype == RB_F32 ? backward_width<__bf16, float>(a, v, grid, s) : backward_width<__bf16, __bf16>(a, v, grid, s);
  if (e != hipSuccess || vectors == 0) return e;
  resnorm_sum_kernel<<<dim3((uint32_t)((D + 63) / 64), (uint32_t)vectors), 512, 0, s>>>(sum);
  return hipGetLastError();
}

}  // namespace rb
