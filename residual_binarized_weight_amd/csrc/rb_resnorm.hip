// rb_resnorm.hip -- the norms after one block and before the next, with the block's gate and the
// stream's scale, forward and backward.
//
//   u = norm_post(Y);  S = alpha R + gate u;  X = norm_pre(S)
//   norm(x) = (x - mu) rstd w + b,  rstd = (mean (x - mu)^2 + eps)^(-1/2),  mu = 0 for an rms norm
//
// Every tensor passes once: HBM bounds both directions (a row's arithmetic is some 10 to 25
// operations per element). A row is held in registers by a group of TPR threads, NV times 8
// consecutive columns each (16-byte accesses), and its two norms are reduced there one after the
// other: by DPP inside a wave, through LDS between waves. All sums are fp32; the mean is taken
// before the squares, so a large mean costs no digits.
//
// Measured (bf16, fp32 stream, rms norms, a gate per channel): forward 2048 x 4096 18 us, 101 MB = 5.5 TB/s,
// about what a copy reaches; one row 3 us. Stores are streamed (nothing here reads them again): 23.7 us
// without. Wide rows, 16 columns per thread from 8193 on: 2048 x 8192 41 us, x 12000 72 us (4.1 TB/s), x 16384 89 us
// (4.5 TB/s). Narrow ones leave lanes without work: 16384 x 512 18 us, 65536 x 128, 16 lanes of 64, 34 us for the
// same bytes (backward 39 and 92).
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
  int64_t row0;  // the launch's first row
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
  const int64_t row = a.row0 + (int64_t)blockIdx.x * kRows + wave / (TPR / 64);
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
  int64_t row0;           // the means' form only: the launch's first row
};
enum { kDwPre, kDbPre, kDwPost, kDbPost, kDgate };

// A row as it was read: packed, the vector at the row's end not yet shifted. Lanes past the end, and
// tensors that are not there, hold 0 throughout.
template <typename TA, typename TS> struct RowRaw {
  typename Vec8<TA>::Raw dx, y, g;
  typename Vec8<TS>::Raw ds, s;
};

template <bool LONG, typename TA, typename TS, int TPR>
__device__ __forceinline__ void load_row(RowRaw<TA, TS>& q, const BwdArgs& a, int64_t row, int c0) {
  if (row >= a.M) {
    q = RowRaw<TA, TS>{};
    return;
  }
  const auto get = [&](auto* p, auto& r) {
    typedef typename std::remove_const<typename std::remove_pointer<decltype(p)>::type>::type T;
    if constexpr (LONG)
      load8_long<T>(r, p, c0, a.D);
    else
      r = load8<T>(p, c0, a.D);
  };
  if (a.pre != RB_NORM_NONE) {
    get(static_cast<const TA*>(a.dX) + row * a.lddx, q.dx);
    get(static_cast<const TS*>(a.S) + row * a.lds, q.s);
  }
  if (a.Y) get(static_cast<const TA*>(a.Y) + row * a.ldy, q.y);
  if (a.dS) get(static_cast<const TS*>(a.dS) + row * a.ldds, q.ds);
  if (a.ldg) get(static_cast<const TA*>(a.gate) + row * a.ldg, q.g);
}

constexpr int bwd_threads(int tpr) { return tpr < 512 ? 512 : tpr; }

// The norms' column sums of rows of more than 4096 columns (a block of 1024 threads, 128 registers each) lie
// in LDS, each word its own thread's; registers hold the others.
constexpr bool sums_in_lds(int tpr) { return tpr == 1024; }

template <typename TA, typename TS, int TPR, bool BIAS, bool LONG>
__global__ __launch_bounds__(bwd_threads(TPR)) void resnorm_backward_kernel(
    BwdArgs a, const float* __restrict__ stats, const float* __restrict__ w_pre, const float* __restrict__ w_post,
    const float* __restrict__ b_post) {
  constexpr int kGroups = bwd_threads(TPR) / TPR;
  constexpr bool kKeep = bwd_threads(TPR) <= 512;  // registers for the vectors and for two rows
  constexpr bool kLds = sums_in_lds(TPR);
  extern __shared__ float join[];  // the groups' sums at the end, [kGroups - 1][D]; or the norms' sums, [vectors][8][TPR]
  __shared__ float2 slots[2][2][16];  // by the round's parity: a slow wave may still read the last round's
  const int t = threadIdx.x % TPR;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);  // rows are scalar: so are their addresses
  const int group = wave / (TPR / 64);
  const int c0 = t * 8;
  const float inv = 1.f / (float)a.D;
  const bool pre = a.pre != RB_NORM_NONE, post = a.post != RB_NORM_NONE, gated = a.gate != nullptr;
  float acc[5][8];
#pragma unroll
  for (int k = 0; k < 5; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[k][j] = 0.f;
  if constexpr (kLds) {
    for (int k = 0; k < 4; ++k)
      if (a.slot[k] >= 0)
        for (int j = 0; j < 8; ++j) join[(a.slot[k] * 8 + j) * TPR + t] = 0.f;
  }
  const auto add = [&](int k, int j, float v) {
    if (kLds && k < 4) {
      if (a.slot[k] >= 0) join[(a.slot[k] * 8 + j) * TPR + t] += v;
    } else {
      acc[k][j] += v;
    }
  };

  // the vectors of the thread's columns (0 past the row's end): kept, or read again for every row
  float wpre[8], wpost[8], bpost[8], gvec[8];
  const auto vectors = [&](int which) {
    if ((which & 1) && pre) load_vec<LONG>(wpre, w_pre, c0, a.D);
    if ((which & 2) && post) load_vec<LONG>(wpost, w_post, c0, a.D);
    if ((which & 2) && b_post) load_vec<LONG>(bpost, b_post, c0, a.D);
    if ((which & 2) && gated && !a.ldg) load_vec<LONG>(gvec, static_cast<const float*>(a.gate), c0, a.D);
  };
  if constexpr (kKeep) vectors(3);

  const int64_t stride = (int64_t)gridDim.x * kGroups;
  const auto one_row = [&](RowRaw<TA, TS>& q, int64_t row, int odd) {
    const bool live = row < a.M;
    const int D = live ? a.D : 0;
    const int64_t srow = live ? row : 0;
    const float mu0 = stats[srow * 4], rs0 = stats[srow * 4 + 1], mu1 = stats[srow * 4 + 2], rs1 = stats[srow * 4 + 3];
    if constexpr (LONG) {
      if (c0 < D && c0 + 8 > D) {
        const int by = c0 + 8 - D;
        shift_down(q.dx, by);
        shift_down(q.s, by);
        shift_down(q.y, by);
        shift_down(q.ds, by);
        shift_down(q.g, by);
      }
    }
    float T[8];
    if (pre) {
      if constexpr (!kKeep) vectors(1);
      float c1 = 0.f, c2 = 0.f;
      const float off = -mu1 * rs1;
      float dx[8], s[8];
      widen8<TA>(q.dx, dx);
      widen8<TS>(q.s, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // past the end dx and d are 0, so xh adds nothing
        const float xh = fmaf(s[j], rs1, off), d = dx[j] * wpre[j];
        c1 += d;
        c2 = fmaf(d, xh, c2);
        add(kDwPre, j, dx[j] * xh);
        if (BIAS) add(kDbPre, j, dx[j]);
      }
      row_sum2<TPR>(c1, c2, slots[odd][0]);
      c1 = a.pre == RB_NORM_LAYER ? c1 * inv * rs1 : 0.f;
      c2 *= inv * rs1;
      float ds[8];
      widen8<TS>(q.ds, ds);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        T[j] = fmaf(-fmaf(s[j], rs1, off), c2, fmaf(dx[j] * wpre[j], rs1, ds[j] - c1));
    } else {
      widen8<TS>(q.ds, T);
    }
    if constexpr (!kKeep) vectors(2);
    float e[8], yh[8];
    float c1 = 0.f, c2 = 0.f;
    const float off = -mu0 * rs0;
    if (a.dR) {
      float dr[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) dr[j] = a.alpha * T[j];
      store8<TS, true>(static_cast<TS*>(a.dR) + row * a.lddr, c0, D, dr);
    }
    widen8<TA>(q.y, yh);
    if (post) {
#pragma unroll
      for (int j = 0; j < 8; ++j) yh[j] = fmaf(yh[j], rs0, off);
    }
    if (gated) {
      float dg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u = post ? yh[j] * wpost[j] : yh[j];
        if (b_post) u += bpost[j];
        dg[j] = u * T[j];
      }
      if (a.ldg) {
        if (a.dgate) store8<TA, true>(static_cast<TA*>(a.dgate) + row * a.lddg, c0, D, dg);
#pragma unroll
        for (int j = 0; j < 8; ++j) T[j] *= Vec8<TA>::get(q.g, j);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) add(kDgate, j, dg[j]), T[j] *= gvec[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = T[j];
    if (post) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float du = T[j];
        add(kDwPost, j, du * yh[j]);
        if (BIAS) add(kDbPost, j, du);
        e[j] = du * wpost[j];  // 0 past the row's end
        c1 += e[j];
        c2 = fmaf(e[j], yh[j], c2);
      }
    }
    if constexpr (!kKeep) load_row<LONG, TA, TS, TPR>(q, a, row + stride, c0);
    if (post) {
      row_sum2<TPR>(c1, c2, slots[odd][1]);
      c1 = a.post == RB_NORM_LAYER ? -c1 * inv * rs0 : 0.f;
      c2 *= inv * rs0;
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = fmaf(-yh[j], c2, fmaf(e[j], rs0, c1));
    }
    store8<TA, true>(static_cast<TA*>(a.dY) + row * a.lddy, c0, D, e);
  };
  // The next row's loads: with registers for two rows issued before this row is begun, otherwise as soon
  // as this row's values are used up. Group 0 has the block's lowest row: while that is live, all groups
  // go on together.
  RowRaw<TA, TS> q[kKeep ? 2 : 1] = {};
  int64_t row = blockIdx.x + (int64_t)gridDim.x * group;
  load_row<LONG, TA, TS, TPR>(q[0], a, row, c0);
  for (int64_t first = blockIdx.x; first < a.M; first += 2 * stride, row += 2 * stride) {
    if (kKeep) load_row<LONG, TA, TS, TPR>(q[kKeep], a, row + stride, c0);
    one_row(q[0], row, 0);
    if (first + stride >= a.M) break;
    if (kKeep) load_row<LONG, TA, TS, TPR>(q[0], a, row + 2 * stride, c0);
    one_row(q[kKeep], row + stride, 1);
  }

#pragma unroll
  for (int k = 0; k < 5; ++k) {
    if (a.slot[k] < 0) continue;
    if (kGroups > 1) {
      __syncthreads();
      if (group > 0) store8<float>(join + (int64_t)(group - 1) * a.D, c0, a.D, acc[k]);
      __syncthreads();
    }
    if (group == 0) {
      if (kLds && k < 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][j] = join[(a.slot[k] * 8 + j) * TPR + t];
      }
      for (int g = 1; g < kGroups; ++g) {
        float o[8];
        widen8<float>(load8<float>(join + (int64_t)(g - 1) * a.D, c0, a.D), o);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][j] += o[j];
      }
      store8<float>(a.part + ((int64_t)a.slot[k] * gridDim.x + blockIdx.x) * a.D, c0, a.D, acc[k]);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// backward of rows of more than 8192 columns, whose column sums fit neither a block's registers nor its LDS
// beside the row: one kernel takes the two norms' means of every row (a row's chunks are read twice, the
// second time from L2), the other walks down strips of rows, 512 columns wide, with the sums in registers.
// Every tensor is read from memory twice, and dY and dR may still replace what they are made of. 2048 x 12000,
// bf16, rms norms and a gate per channel: 152 to 159 us (75 + 79 and 5 for the sums) with an fp32 stream; the row in one
// block of 1024 threads with 16 columns each, sums in spilled registers, took 486. Up to 8192 columns one
// reading is faster: 2048 x 8192 76 us and 6.
// ---------------------------------------------------------------------------------------------
constexpr int kWideColumns = 8192;
constexpr int kWideThreads = 512;
constexpr int kWideStrips = 64;  // by 17 columns of blocks or more

// T of 8 columns of a row, dX there and the pre norm's x-hat; m holds that norm's two means
template <typename TA, typename TS>
__device__ __forceinline__ void stream_grad(const BwdArgs& a, int64_t row, int c, float mu1, float rs1, float2 m,
                                            const float (&w)[8], float (&T)[8], float (&dx)[8], float (&xh)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) T[j] = 0.f;
  if (a.dS) {
    typename Vec8<TS>::Raw r;
    load<true, TS>(r, static_cast<const TS*>(a.dS) + row * a.ldds, c, a.D);
    widen8<TS>(r, T);
  }
  if (a.pre == RB_NORM_NONE) return;
  typename Vec8<TA>::Raw dr;
  typename Vec8<TS>::Raw sr;
  load<true, TA>(dr, static_cast<const TA*>(a.dX) + row * a.lddx, c, a.D);
  load<true, TS>(sr, static_cast<const TS*>(a.S) + row * a.lds, c, a.D);
  widen8<TA>(dr, dx);
  widen8<TS>(sr, xh);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    xh[j] = (xh[j] - mu1) * rs1;
    T[j] += rs1 * (dx[j] * w[j] - m.x - xh[j] * m.y);
  }
}
template <typename TA>
__device__ __forceinline__ void gate_of(const BwdArgs& a, int64_t row, int c, float (&g)[8]) {
  if (a.ldg) {
    typename Vec8<TA>::Raw r;
    load<true, TA>(r, static_cast<const TA*>(a.gate) + row * a.ldg, c, a.D);
    widen8<TA>(r, g);
  } else {
    load_vec<true>(g, static_cast<const float*>(a.gate), c, a.D);
  }
}

template <typename TA, typename TS>
__global__ __launch_bounds__(kWideThreads) void resnorm_backward_means_kernel(BwdArgs a, const float* __restrict__ stats,
                                                                             const float* __restrict__ w_pre,
                                                                             const float* __restrict__ w_post,
                                                                             float4* means) {
  __shared__ float2 slots[2][16];
  const int64_t row = a.row0 + blockIdx.x;
  const float mu0 = stats[row * 4], rs0 = stats[row * 4 + 1], mu1 = stats[row * 4 + 2], rs1 = stats[row * 4 + 3];
  const float inv = 1.f / (float)a.D;
  float2 m1 = make_float2(0.f, 0.f), m0 = m1;
  if (a.pre != RB_NORM_NONE) {
    for (int c = threadIdx.x * 8; c < a.D; c += kWideThreads * 8) {
      typename Vec8<TA>::Raw dr;
      typename Vec8<TS>::Raw sr;
      float w[8], dx[8], s[8];
      load<true, TA>(dr, static_cast<const TA*>(a.dX) + row * a.lddx, c, a.D);
      load<true, TS>(sr, static_cast<const TS*>(a.S) + row * a.lds, c, a.D);
      load_vec<true>(w, w_pre, c, a.D);
      widen8<TA>(dr, dx);
      widen8<TS>(sr, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = dx[j] * w[j];  // 0 past the row's end
        m1.x += d;
        m1.y = fmaf(d, (s[j] - mu1) * rs1, m1.y);
      }
    }
    row_sum2<kWideThreads>(m1.x, m1.y, slots[0]);
    m1.x = a.pre == RB_NORM_LAYER ? m1.x * inv : 0.f;
    m1.y *= inv;
  }
  if (a.post != RB_NORM_NONE) {
    for (int c = threadIdx.x * 8; c < a.D; c += kWideThreads * 8) {
      float w[8] = {}, T[8], dx[8], xh[8], y[8];
      if (a.pre != RB_NORM_NONE) load_vec<true>(w, w_pre, c, a.D);
      stream_grad<TA, TS>(a, row, c, mu1, rs1, m1, w, T, dx, xh);
      if (a.gate) {
        float g[8];
        gate_of<TA>(a, row, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) T[j] *= g[j];
      }
      typename Vec8<TA>::Raw yr;
      load<true, TA>(yr, static_cast<const TA*>(a.Y) + row * a.ldy, c, a.D);
      load_vec<true>(w, w_post, c, a.D);
      widen8<TA>(yr, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = T[j] * w[j];  // 0 past the row's end
        m0.x += e;
        m0.y = fmaf(e, (y[j] - mu0) * rs0, m0.y);
      }
    }
    row_sum2<kWideThreads>(m0.x, m0.y, slots[1]);
    m0.x = a.post == RB_NORM_LAYER ? m0.x * inv : 0.f;
    m0.y *= inv;
  }
  if (threadIdx.x == 0) means[row] = make_float4(m1.x, m1.y, m0.x, m0.y);
}

template <typename TA, typename TS>
__global__ __launch_bounds__(256) void resnorm_backward_strip_kernel(BwdArgs a, const float* __restrict__ stats,
                                                                     const float* __restrict__ w_pre,
                                                                     const float* __restrict__ w_post,
                                                                     const float* __restrict__ b_post,
                                                                     const float4* __restrict__ means, int strip) {
  __shared__ float join[3][512];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c = blockIdx.x * 512 + lane * 8;
  const int64_t r0 = (int64_t)blockIdx.y * strip, r1 = r0 + strip < a.M ? r0 + strip : a.M;
  const bool pre = a.pre != RB_NORM_NONE, post = a.post != RB_NORM_NONE;
  float wpre[8] = {}, wpost[8] = {}, bpost[8] = {}, gate[8] = {}, acc[5][8] = {};
  if (pre) load_vec<true>(wpre, w_pre, c, a.D);
  if (post) load_vec<true>(wpost, w_post, c, a.D);
  if (b_post) load_vec<true>(bpost, b_post, c, a.D);
  if (a.gate && !a.ldg) load_vec<true>(gate, static_cast<const float*>(a.gate), c, a.D);
  for (int64_t row = r0 + w; row < r1; row += 4) {
    const float mu0 = stats[row * 4], rs0 = stats[row * 4 + 1], mu1 = stats[row * 4 + 2], rs1 = stats[row * 4 + 3];
    const float4 m = means[row];
    float T[8], dx[8], xh[8], y[8];
    if (a.Y) {
      typename Vec8<TA>::Raw yr;
      load<true, TA>(yr, static_cast<const TA*>(a.Y) + row * a.ldy, c, a.D);
      widen8<TA>(yr, y);
    }
    if (a.gate && a.ldg) gate_of<TA>(a, row, c, gate);
    stream_grad<TA, TS>(a, row, c, mu1, rs1, make_float2(m.x, m.y), wpre, T, dx, xh);
    if (pre) {
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[kDwPre][j] = fmaf(dx[j], xh[j], acc[kDwPre][j]), acc[kDbPre][j] += dx[j];
    }
    if (a.dR) {
      float dr[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) dr[j] = a.alpha * T[j];
      store8<TS, true>(static_cast<TS*>(a.dR) + row * a.lddr, c, a.D, dr);
    }
    if (post) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (y[j] - mu0) * rs0;
    }
    if (a.gate) {
      float dg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dg[j] = (post ? fmaf(y[j], wpost[j], bpost[j]) : y[j]) * T[j];
        T[j] *= gate[j];
        acc[kDgate][j] += dg[j];
      }
      if (a.dgate) store8<TA, true>(static_cast<TA*>(a.dgate) + row * a.lddg, c, a.D, dg);
    }
    if (post) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[kDwPost][j] = fmaf(T[j], y[j], acc[kDwPost][j]);
        acc[kDbPost][j] += T[j];
        T[j] = rs0 * (T[j] * wpost[j] - m.z - y[j] * m.w);
      }
    }
    store8<TA, true>(static_cast<TA*>(a.dY) + row * a.lddy, c, a.D, T);
  }
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    if (a.slot[k] < 0) continue;
    __syncthreads();
    if (w > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) join[w - 1][lane * 8 + j] = acc[k][j];
    }
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[k][j] += join[0][lane * 8 + j] + join[1][lane * 8 + j] + join[2][lane * 8 + j];
      store8<float>(a.part + ((int64_t)a.slot[k] * gridDim.y + blockIdx.y) * a.D, c, a.D, acc[k]);
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
hipError_t forward(FwdArgs a, hipStream_t s) {
  constexpr int threads = TPR < 256 ? 256 : TPR;
  constexpr int rows = TPR < 256 ? 256 / TPR : 1;
  return launch_in_parts((a.M + rows - 1) / rows, [&](int64_t first, uint32_t blocks) {
    a.row0 = first * rows;
    resnorm_forward_kernel<TA, TS, TPR, NV, LONG><<<dim3(blocks), threads, 0, s>>>(a);
  });
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
template <typename TA, typename TS, int TPR, bool LONG = true>
hipError_t backward(const BwdArgs& a, const BwdVectors& v, int grid, hipStream_t s) {
  const bool bias = a.slot[kDbPre] >= 0 || a.slot[kDbPost] >= 0;
  constexpr int threads = bwd_threads(TPR);
  const size_t lds = sums_in_lds(TPR) ? (size_t)4 * 8 * TPR * 4 : (size_t)(threads / TPR - 1) * a.D * 4;
  if (sums_in_lds(TPR)) {
    static const hipError_t attr[2] = {
        hipFuncSetAttribute((const void*)resnorm_backward_kernel<TA, TS, TPR, false, LONG>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, 4 * 8 * TPR * 4),
        hipFuncSetAttribute((const void*)resnorm_backward_kernel<TA, TS, TPR, true, LONG>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, 4 * 8 * TPR * 4)};
    if (attr[0] != hipSuccess || attr[1] != hipSuccess) return attr[0] != hipSuccess ? attr[0] : attr[1];
  }
  if (bias)
    resnorm_backward_kernel<TA, TS, TPR, true, LONG><<<dim3((uint32_t)grid), threads, lds, s>>>(a, v.stats, v.w_pre, v.w_post, v.b_post);
  else
    resnorm_backward_kernel<TA, TS, TPR, false, LONG><<<dim3((uint32_t)grid), threads, lds, s>>>(a, v.stats, v.w_pre, v.w_post, v.b_post);
  return hipGetLastError();
}
template <typename TA, typename TS>
hipError_t backward_width(const BwdArgs& a, const BwdVectors& v, int grid, hipStream_t s) {
  if (a.D < 8) return backward<TA, TS, 64, false>(a, v, grid, s);
  if (a.D <= 64 * 8) return backward<TA, TS, 64>(a, v, grid, s);
  if (a.D <= 256 * 8) return backward<TA, TS, 256>(a, v, grid, s);
  if (a.D <= 512 * 8) return backward<TA, TS, 512>(a, v, grid, s);
  if (a.D <= kWideColumns) return backward<TA, TS, 1024>(a, v, grid, s);
  float4* const means = reinterpret_cast<float4*>(a.part + ((int64_t)5 * grid * a.D + 3) / 4 * 4);
  const hipError_t e = launch_in_parts(a.M, [&](int64_t first, uint32_t rows) {
    BwdArgs part = a;
    part.row0 = first;
    resnorm_backward_means_kernel<TA, TS><<<dim3(rows), kWideThreads, 0, s>>>(part, v.stats, v.w_pre, v.w_post, means);
  });
  if (e != hipSuccess) return e;
  const int strip = (int)((a.M + grid - 1) / grid);
  resnorm_backward_strip_kernel<TA, TS><<<dim3((uint32_t)((a.D + 511) / 512), (uint32_t)grid), 256, 0, s>>>(
      a, v.stats, v.w_pre, v.w_post, v.b_post, means, strip);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_resnorm_forward(const void* Y, rb_dtype a_dtype, int64_t M, int64_t D, int64_t ldy, const void* R,
                                  rb_dtype s_dtype, int64_t ldr, const void* gate, int64_t ldg, float alpha, int post,
                                  const float* w_post, const float* b_post, int pre, const float* w_pre,
                                  const float* b_pre, float eps, void* S, int64_t lds, void* X, int64_t ldx,
                                  float* stats, hipStream_t s) {
  const FwdArgs a{Y, R, gate, w_post, b_post, w_pre, b_pre, S, X, stats, M, ldy, ldr, ldg, lds, ldx, (int)D, post, pre,
                  alpha, eps, 0};
  if (a_dtype == RB_F32) return forward_width<float, float>(a, s);
  if (a_dtype == RB_F16)
    return s_dtype == RB_F32 ? forward_width<_Float16, float>(a, s) : forward_width<_Float16, _Float16>(a, s);
  return s_dtype == RB_F32 ? forward_width<__bf16, float>(a, s) : forward_width<__bf16, __bf16>(a, s);
}

// the runs of rows whose column sums are made apart: a block each, or strips of 4 rows and more
static int resnorm_grid(int64_t D, int64_t M) {
  if (D <= kWideColumns) return (int)(M < kBwdGrid ? M : kBwdGrid);
  const int64_t strip = (M + kWideStrips - 1) / kWideStrips;
  return (int)((M + (strip < 4 ? 4 : strip) - 1) / (strip < 4 ? 4 : strip));
}

size_t resnorm_backward_workspace_bytes(int64_t D, int64_t M) {
  const size_t sums = ((size_t)5 * resnorm_grid(D, M) * (size_t)D * 4 + 15) / 16 * 16;
  return sums + (D > kWideColumns ? (size_t)M * 16 : 0);
}

hipError_t launch_resnorm_backward(const void* dX, rb_dtype a_dtype, int64_t M, int64_t D, int64_t lddx, const void* dS,
                                   rb_dtype s_dtype, int64_t ldds, const void* Y, int64_t ldy, const void* S,
                                   int64_t lds, const float* stats, const void* gate, int64_t ldg, float alpha,
                                   int post, const float* w_post, const float* b_post, int pre, const float* w_pre,
                                   void* dY, int64_t lddy, void* dR, int64_t lddr, void* dgate, int64_t lddg,
                                   float* dw_post, float* db_post, float* dw_pre, float* db_pre, void* ws,
                                   hipStream_t s) {
  const BwdVectors v{stats, w_pre, w_post, post == RB_NORM_NONE ? nullptr : b_post};  // no norm, no bias in u
  BwdArgs a{dX, dS, Y, S, gate, dY, dR, ldg ? dgate : nullptr, static_cast<float*>(ws),
            M, lddx, ldds, ldy, lds, gate ? ldg : 0, lddy, lddr, lddg, (int)D, post, pre, {-1, -1, -1, -1, -1}, alpha, 0};
  SumArgs sum{a.part, {}, resnorm_grid(D, M), (int)D};
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
