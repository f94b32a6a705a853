// rb_linear.hip -- a coupled-training layer's product with its epilogue, and the epilogue's backward.
//
//   Z = X What^T + b,  Y = act(Z) + R        X [M][K], What [N][K] in fp16 or bf16, fp32 sums
//   dZ = dY act'(Z),   db = column sums of dZ
//
// Kernels of this file:
//   linear_tile_kernel    a tile of batch rows by weight rows per block, on the matrix cores
//   linear_join_kernel    the sums of K chunks, where a tile's columns are split, and the epilogue
//   linear_rows_kernel    up to 4 batch rows, on the vector units: a wave streams whole weight rows
//   linear_few_kernel     small products of 5 to 256 batch rows, on the matrix cores, a block's waves splitting
//                         the columns
//   linear_grad_kernel    dZ and, per strip of rows, partial column sums; linear_grad_sum_kernel adds them
#include "rb_elem.hpp"
#include "rb_internal.h"

namespace rb {
namespace {

typedef _Float16 l_h8 __attribute__((ext_vector_type(8)));
typedef __bf16 l_b8 __attribute__((ext_vector_type(8)));
typedef float l_f4 __attribute__((ext_vector_type(4)));
typedef uint32_t l_u4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) l_u4 l_lds_u4;
typedef __attribute__((address_space(3))) l_f4 l_lds_f4;
typedef __attribute__((address_space(3))) void l_lds_void;

__device__ __forceinline__ l_f4 mfma(_Float16, l_u4 a, l_u4 b, l_f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(l_h8, a), __builtin_bit_cast(l_h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ l_f4 mfma(__bf16, l_u4 a, l_u4 b, l_f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(l_b8, a), __builtin_bit_cast(l_b8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------------------------
// activations, in fp32. Relative to the value their errors are some tens of units of 2^-24 and, in the
// tails, the exponentials' arguments times it (z^2 / 2 for the normal density, 17 at z = -5 for the tanh form).
// ---------------------------------------------------------------------------------------------
constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }
// The normal CDF, e = exp(-z^2 / 2): below zero e r(|z|), above one minus that. 1 + erf loses every digit below zero
// (4 % of the value at z = -5). r, half of exp(x^2) erfc(x), is a polynomial in s = 1 / (1 + 0.3 |z|) without a constant
// term, fitted over |z| = 0 .. 14 by least squares with weights moved towards the largest relative error: 8 units of
// 2^-24 in fp32. The backward of 2048 x 11008 in bf16 takes 34 us with it, 40 with 1 + erff, 47 with erfcf.
__device__ __forceinline__ float normal_cdf(float z, float e) {
  const float s = __builtin_amdgcn_rcpf(fmaf(0.3f, fabsf(z), 1.f));
  float r = fmaf(s, 0.035674576f, -0.15720132f);
  r = fmaf(s, r, 0.20634893f);
  r = fmaf(s, r, -0.053678185f);
  r = fmaf(s, r, 0.12855819f);
  r = fmaf(s, r, 0.09991466f);
  r = fmaf(s, r, 0.12075376f);
  r = fmaf(s, r, 0.11962932f) * s * e;
  return z > 0.f ? 1.f - r : r;
}
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case RB_ACT_RELU: return z < 0.f ? 0.f : z;
    case RB_ACT_GELU: return z * normal_cdf(z, __expf(-0.5f * z * z));
    case RB_ACT_GELU_TANH: return z * logistic(2.f * kGeluA * (z + kGeluB * z * z * z));  // (1 + tanh a) / 2
    case RB_ACT_SILU: return z * logistic(z);
  }
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case RB_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case RB_ACT_GELU: {
      const float e = __expf(-0.5f * z * z);
      return normal_cdf(z, e) + z * 0.3989422804014327f * e;
    }
    case RB_ACT_GELU_TANH: {
      const float g = logistic(2.f * kGeluA * (z + kGeluB * z * z * z));
      // from |z| = 16 on g is 0 or 1 and the second term 0, whatever its factor: z^2 must not overflow there
      return g + z * g * (1.f - g) * 2.f * kGeluA * (1.f + 3.f * kGeluB * fminf(z * z, 256.f));
    }
    case RB_ACT_SILU: {
      const float g = logistic(z);
      return g + z * g * (1.f - g);
    }
  }
  return 1.f;
}

struct Epilogue {
  const float* bias;
  const void* R;
  void* Z;
  void* Y;
  int64_t ldr, ldz, ldy;
  int act;
  bool line_z, line_y;  // every row starts a 128-byte line
};
// Streamed where rows start lines (2048 x 11008 x 4096 with Z 182 us against 186); elsewhere a streamed line that
// two stores write in part goes to memory twice (3441 x 2583 x 640 with bias and Z, bf16: 39 us against 31, with
// operands that are not aligned 48 against 41).
template <typename T>
__device__ __forceinline__ void store_out(T* row, int c, int n, const float (&v)[8], bool line) {
  if (line)
    store8<T, true>(row, c, n, v);
  else
    store8<T>(row, c, n, v);
}
// columns n .. n+7 of row m, v the product's fp32 sums
template <typename TA, typename TY>
__device__ __forceinline__ void finish8(const Epilogue& e, float (&v)[8], int64_t m, int n, int N) {
  if (e.bias) {
    float b[8];
    widen8<float>(load8_any<float>(e.bias, n, N), b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
  }
  if (e.Z) store_out<TA>(static_cast<TA*>(e.Z) + m * e.ldz, n, N, v, e.line_z);
  if (e.act != RB_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_value(v[j], e.act);
  }
  if (e.R) {
    float r[8];
    widen8<TY>(load8_any<TY>(static_cast<const TY*>(e.R) + m * e.ldr, n, N), r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
  store_out<TY>(static_cast<TY*>(e.Y) + m * e.ldy, n, N, v, e.line_y);
}

// ---------------------------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------------------------
// 16 bytes per lane from the buffer to LDS (lane l's at base + 16 l)
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* base, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (l_lds_void*)base, 16, voff, soff, 0, 0);
}

constexpr int kTK = 64;            // columns per step
constexpr int kRowB = kTK * 2;     // bytes of a staged row
constexpr uint32_t kOob = 0x80000000u;
constexpr int kXcds = 8;
constexpr int kPadRow = 68;        // floats of a row in the epilogue's LDS transposition

// s_waitcnt immediates: vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8
constexpr int kWaitLds = 15 | (3 << 14) | (7 << 4);  // lgkmcnt = 0 alone
constexpr int wait_vmcnt(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

struct TileArgs {
  const void *X, *W;
  int64_t ldx, ldw, M;
  int N, K;
  uint32_t tiles_m, tiles, per_xcd;  // tiles: the end of the launch's run
  uint32_t first;                    // its first tile, or block of weight rows
  int chunk_k;    // columns per K chunk, a multiple of kTK
  float* part;    // [chunks][M][N] fp32 sums, or NULL: one chunk, epilogue here
  Epilogue e;
};

// WM x WN waves, each TM x TN accumulators of v_mfma_f32_16x16x32: a tile of 16 WM TM batch rows by
// 16 WN TN weight rows. A step of 64 columns of the tile's rows is one LDS stage of a ring of kS. A
// step is two phases of 32 columns; a phase's fragments are read while the phase before it multiplies.
// In the middle of step s (the second phase's fragments are then in registers, so its stage is free) a
// wave waits for its own loads of step s + 1, the barrier makes everyone's visible, and the loads of
// step s + kS go into the freed stage.
//
// AL: rows of both operands are 16-byte aligned and K is a multiple of 8: the rows go to LDS directly
// (buffer loads, out of range past a tile's rows and past the columns, where they give 0). Otherwise
// they pass through registers one step ahead, by 16-byte loads at any address; the vector that holds the
// end of the columns is read 8 columns before it and shifted.
//
// What bounds it: bringing the operands to LDS. 2048 x 4096 x 11008 (bf16, fp32 stream) takes 176 to 181 us
// from cold memory and 173 with everything in the cache; taken apart, when it took 172 cold, the matrix
// instructions alone took 113, everything but the global loads 128, the loads alone 159 (111 warm). Hence the large
// tiles (a byte brought serves 64 multiply-adds of a 256 x 256 tile, 43 of a 128 x 256 one) and the ring that keeps
// kS - 1 steps in flight. Against the 172: two waves per SIMD; with one (tiles of 4 waves) 192 to 249. 32x32x16
// instructions: 202. Weight fragments straight from memory to registers, 16 bytes a row: 244.
template <typename TA, typename TY, int WM, int WN, int TM, int TN, int kS, bool AL>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_tile_kernel(TileArgs a) {
  constexpr int kWaves = WM * WN;
  constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN;
  constexpr int kStage = (BM + BN) * kRowB;
  constexpr int kPer = (BM + BN) / 8 / kWaves;  // 1 KB groups a wave loads per step
  constexpr int kPerX = BM / 8 / kWaves;
  static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0, "a load instruction has one operand");
  static_assert(AL || kS == 2, "through registers a step is written two steps ahead");
  extern __shared__ __align__(16) uint8_t l_smem[];
  const uint32_t blk = blockIdx.x;
  const uint32_t t = a.first + blk % kXcds * a.per_xcd + blk / kXcds;  // an XCD's blocks take one run of tiles
  if (t >= a.tiles) return;
  const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane(t % a.tiles_m) * BM;
  const int n0 = __builtin_amdgcn_readfirstlane(t / a.tiles_m) * BN;
  const int kb = blockIdx.y * a.chunk_k;
  const int ke = kb + a.chunk_k < a.K ? kb + a.chunk_k : a.K;

  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  const int lr = lane & 15, lj = lane >> 4;

  const int mrows = (int)(a.M - m0 < BM ? a.M - m0 : BM);
  const int nrows = a.N - n0 < BN ? a.N - n0 : BN;

  // 1 KB groups of 8 rows; lane l fills slot l % 8 of row l / 8 with the 16-byte chunk (l % 8) ^ (row % 8),
  // so that the 8 rows of a fragment read's phase lie in 8 bank groups
  const int xc = (lane & 7) ^ (lane >> 3);
  const auto row_of = [&](int i) { return 8 * ((i < kPerX ? i : i - kPerX) * kWaves + w) + (lane >> 3); };
  const __amdgpu_buffer_rsrc_t rx =
      buffer_rsrc(static_cast<const TA*>(a.X) + m0 * a.ldx, AL ? (uint32_t)(mrows * a.ldx * 2) : 0u);
  const __amdgpu_buffer_rsrc_t rw =
      buffer_rsrc(static_cast<const TA*>(a.W) + (int64_t)n0 * a.ldw, AL ? (uint32_t)(nrows * a.ldw * 2) : 0u);
  uint32_t off[kPer];
  const TA* row[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = row_of(i);
    if constexpr (AL) {
      off[i] = (uint32_t)(r * (i < kPerX ? a.ldx : a.ldw) * 2) + 16u * xc;
    } else {
      // a row past the last one repeats it: its outputs are not stored
      row[i] = i < kPerX ? static_cast<const TA*>(a.X) + (m0 + (r < mrows ? r : mrows - 1)) * a.ldx
                         : static_cast<const TA*>(a.W) + (int64_t)(n0 + (r < nrows ? r : nrows - 1)) * a.ldw;
    }
  }
  const auto dma = [&](int s, int stage) {
    const int k0 = kb + s * kTK;
    const bool ok = k0 + 8 * xc < ke;
    uint8_t* const base = l_smem + stage * kStage;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      load_to_lds(i < kPerX ? rx : rw, base + (i * kWaves + w) * 1024, ok ? off[i] : kOob, k0 * 2);
  };
  l_u4 hold[kPer];
  const auto fetch = [&](int s, l_u4 (&hold)[kPer]) {
    const int k0 = kb + s * kTK, c = k0 + 8 * xc;
    if (k0 + kTK <= ke) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        hold[i] = __builtin_bit_cast(l_u4, *reinterpret_cast<const typename Vec8<TA>::Raw*>(row[i] + c));
    } else if (ke >= 8) {
      typename Vec8<TA>::Raw r[kPer] = {};
#pragma unroll
      for (int i = 0; i < kPer; ++i) load8_long<TA>(r[i], row[i], c, ke);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (c < ke && c + 8 > ke) shift_down(r[i], 8 - ke % 8);
        hold[i] = __builtin_bit_cast(l_u4, r[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) hold[i] = __builtin_bit_cast(l_u4, load8<TA>(row[i], c, ke));
    }
  };
  const auto put = [&](int stage, const l_u4 (&hold)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      *reinterpret_cast<l_u4*>(l_smem + stage * kStage + (i * kWaves + w) * 1024 + lane * 16) = hold[i];
  };

  l_f4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = (l_f4){0.f, 0.f, 0.f, 0.f};

  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)l_smem;
  const uint32_t f0 = lr * kRowB + 16u * ((uint32_t)lj ^ (lr & 7u)), f1 = lr * kRowB + 16u * ((4u + lj) ^ (lr & 7u));
  const uint32_t ax = lds0 + wm * TM * 16 * kRowB, aw = lds0 + (BM + wn * TN * 16) * kRowB;
  l_u4 xf[2][TM], wf[2][TN];
  const auto read = [&](int kh, int stage) {  // the fragments of half kh of a stage
#pragma unroll
    for (int j = 0; j < TN; ++j)
      wf[kh][j] = *(l_lds_u4*)(size_t)(aw + stage * kStage + j * 16 * kRowB + (kh ? f1 : f0));
#pragma unroll
    for (int i = 0; i < TM; ++i)
      xf[kh][i] = *(l_lds_u4*)(size_t)(ax + stage * kStage + i * 16 * kRowB + (kh ? f1 : f0));
  };
  const auto multiply = [&](int kh) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma(TA(0), wf[kh][j], xf[kh][i], acc[i][j]);
  };
  constexpr int kR = TM + TN;
  const auto barrier = [] {  // the raw barrier: __syncthreads would also wait for every load in flight
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const int steps = (ke - kb + kTK - 1) / kTK;
  if constexpr (AL) {
#pragma unroll
    for (int s = 0; s < kS; ++s) dma(s, s);
    __builtin_amdgcn_s_waitcnt(wait_vmcnt((kS - 1) * kPer));
  } else {
    l_u4 second[kPer];
    fetch(0, hold);
    fetch(1, second);
    put(0, hold);
    put(1, second);
    fetch(2, hold);
    __builtin_amdgcn_s_waitcnt(kWaitLds);
  }
  barrier();
  read(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  int st = 0;
  for (int s = 0; s < steps; ++s) {
    read(1, st);
    multiply(0);
    // the reads spread over the first products
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
    }
    __builtin_amdgcn_sched_barrier(0);
    const int next = st + 1 == kS ? 0 : st + 1;
    __builtin_amdgcn_s_waitcnt(AL ? wait_vmcnt((kS - 2) * kPer) & kWaitLds : kWaitLds);
    barrier();
    if constexpr (AL) {
      dma(s + kS, st);
    } else {
      put(st, hold);
      fetch(s + 3, hold);
    }
    __builtin_amdgcn_sched_barrier(0);
    read(0, next);
    multiply(1);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    st = next;
  }
  // loads past the last step (out of range, zeros) end before LDS is used again
  __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));
  __syncthreads();

  // 16 rows by 64 columns at a time through the wave's own LDS area, so that 8 lanes hold 64 consecutive
  // columns of a row and whole lines are read and written. D of the product: lane l holds weight rows
  // 4 (l / 16) .. +3 of batch row l % 16.
  float* const turn = reinterpret_cast<float*>(l_smem) + w * (16 * kPadRow);
#pragma unroll 1
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int q = 0; q < TM; ++q)
      if (q == i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<l_f4*>(turn + lr * kPadRow + 16 * j + 4 * lj) = acc[q][j];
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      const int r = 8 * s + (lane >> 3), c = 8 * (lane & 7);
      float v[8];
      const l_f4 lo = *reinterpret_cast<const l_f4*>(turn + r * kPadRow + c);
      const l_f4 hi = *reinterpret_cast<const l_f4*>(turn + r * kPadRow + c + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = lo[j], v[4 + j] = hi[j];
      const int64_t m = m0 + (wm * TM + i) * 16 + r;
      const int n = n0 + wn * 64 + c;
      if (m < a.M && n < a.N) {
        if (a.part)
          store8<float>(a.part + ((int64_t)blockIdx.y * a.M + m) * a.N, n, a.N, v);
        else
          finish8<TA, TY>(a.e, v, m, n, a.N);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  static_assert(TN == 4, "a wave's 64 columns");
}

struct JoinArgs {
  const float* part;
  int64_t M;
  int N, chunks;
  Epilogue e;
};
// 8 columns of a row per thread; the chunks are added in their order
template <typename TA, typename TY>
__global__ __launch_bounds__(256) void linear_join_kernel(JoinArgs a) {
  const int n = (blockIdx.x * 256 + threadIdx.x) * 8;
  const int64_t m = blockIdx.y;
  if (n >= a.N) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int c = 0; c < a.chunks; ++c) {
    float p[8];
    widen8<float>(load8_any<float>(a.part + ((int64_t)c * a.M + m) * a.N, n, a.N), p);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += p[j];
  }
  finish8<TA, TY>(a.e, v, m, n, a.N);
}

// ---------------------------------------------------------------------------------------------
// up to kMaxRows batch rows: HBM's rate for the weights is the bound, and the vector units' products are far
// below it. A wave owns kRows weight rows, its lanes 8 columns each of a 512-column step; kRows x kSteps
// loads of 1 KB are in flight per wave. One launch, no partial sums in memory.
// ---------------------------------------------------------------------------------------------
constexpr int kMaxRows = 4;

template <typename TA, typename TY, int MR, int kRows, int kSteps>
__global__ __launch_bounds__(256) void linear_rows_kernel(TileArgs a) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n0 = ((a.first + blockIdx.x) * 4 + w) * kRows;
  if (n0 >= a.N) return;
  const TA* const X = static_cast<const TA*>(a.X);
  const TA* row[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)  // a row past the last one repeats it: its sums are not stored
    row[r] = static_cast<const TA*>(a.W) + (int64_t)(n0 + r < a.N ? n0 + r : a.N - 1) * a.ldw;
  float sum[MR][kRows];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < kRows; ++r) sum[m][r] = 0.f;
  for (int k0 = 0; k0 < a.K; k0 += 512 * kSteps) {
    typename Vec8<TA>::Raw wr[kSteps][kRows] = {}, xr[kSteps][MR] = {};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = k0 + 512 * s + 8 * lane;
#pragma unroll
      for (int r = 0; r < kRows; ++r) load8_long<TA>(wr[s][r], row[r], c, a.K);
#pragma unroll
      for (int m = 0; m < MR; ++m) load8_long<TA>(xr[s][m], X + (m < a.M ? m : 0) * a.ldx, c, a.K);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = k0 + 512 * s + 8 * lane;
      if (c < a.K && c + 8 > a.K) {  // the vector at the end of the columns
#pragma unroll
        for (int r = 0; r < kRows; ++r) shift_down(wr[s][r], c + 8 - a.K);
#pragma unroll
        for (int m = 0; m < MR; ++m) shift_down(xr[s][m], c + 8 - a.K);
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sum[m][r] = fmaf(Vec8<TA>::get(wr[s][r], j), Vec8<TA>::get(xr[s][m], j), sum[m][r]);
  }
  // lane r + kRows m takes sum (m, r)
  float mine = 0.f;
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_dpp(sum[m][r])), 63));
      mine = lane == m * kRows + r ? v : mine;
    }
  const int m = lane / kRows, n = n0 + lane % kRows;
  if (m >= MR || m >= a.M || n >= a.N) return;
  const Epilogue& e = a.e;
  if (e.bias) mine += e.bias[n];
  if (e.Z) static_cast<TA*>(e.Z)[m * e.ldz + n] = Vec8<TA>::narrow(mine);
  if (e.act != RB_ACT_NONE) mine = act_value(mine, e.act);
  if (e.R) mine += (float)static_cast<const TY*>(e.R)[m * e.ldr + n];
  static_cast<TY*>(e.Y)[m * e.ldy + n] = Vec8<TY>::narrow(mine);
}

// ---------------------------------------------------------------------------------------------
// Small products of 5 to 256 batch rows: one launch on the matrix cores, without partial sums in memory. A
// block owns 16 weight rows by 16 batch rows; its 8 waves take the 64-column steps in turn, each with its
// fragments straight from memory, and join in LDS in their order. The fragments' 16-byte pieces cost the
// address unit a piece each, which bounds the rate: 0.11 us a step for the 256 units at once (4096 columns
// 7.1 us), 0.3 where rows are not 16-byte aligned.
// ---------------------------------------------------------------------------------------------
constexpr int kFewRows = 256;

template <typename TA, typename TY>
__global__ __launch_bounds__(512) void linear_few_kernel(TileArgs a) {
  constexpr int kWaves = 8, kAhead = 4;  // steps whose loads a wave has in flight
  __shared__ __align__(16) float sums[kWaves][256];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lr = lane & 15, lj = lane >> 4;
  const int n0 = blockIdx.x * 16;
  // rows past the last one repeat it: their outputs are not stored
  const TA* const wrow = static_cast<const TA*>(a.W) + (int64_t)(n0 + lr < a.N ? n0 + lr : a.N - 1) * a.ldw;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const TA* const xrow = static_cast<const TA*>(a.X) + (m0 + lr < a.M ? m0 + lr : a.M - 1) * a.ldx;
  l_f4 acc = (l_f4){0.f, 0.f, 0.f, 0.f};
  for (int k0 = w * kTK; k0 < a.K; k0 += kAhead * kWaves * kTK) {
    typename Vec8<TA>::Raw wf[kAhead][2] = {}, xf[kAhead][2] = {};
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = k0 + s * kWaves * kTK + 32 * h + 8 * lj;
        load8_long<TA>(wf[s][h], wrow, c, a.K);
        load8_long<TA>(xf[s][h], xrow, c, a.K);
      }
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = k0 + s * kWaves * kTK + 32 * h + 8 * lj;
        if (c < a.K && c + 8 > a.K) {  // the vector at the end of the columns
          shift_down(wf[s][h], c + 8 - a.K);
          shift_down(xf[s][h], c + 8 - a.K);
        }
        acc = mfma(TA(0), __builtin_bit_cast(l_u4, wf[s][h]), __builtin_bit_cast(l_u4, xf[s][h]), acc);
      }
  }
  *reinterpret_cast<l_f4*>(&sums[w][lane * 4]) = acc;
  __syncthreads();
  // thread 16 m + n: D's lane 16 (n / 4) + m holds weight row n in element n % 4
  if (threadIdx.x >= 256) return;
  const int mm = threadIdx.x >> 4, nn = threadIdx.x & 15, n = n0 + nn;
  const int64_t m = m0 + mm;
  if (m >= a.M || n >= a.N) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) v += sums[i][((nn >> 2) * 16 + mm) * 4 + (nn & 3)];
  const Epilogue& e = a.e;
  if (e.bias) v += e.bias[n];
  if (e.Z) static_cast<TA*>(e.Z)[m * e.ldz + n] = Vec8<TA>::narrow(v);
  if (e.act != RB_ACT_NONE) v = act_value(v, e.act);
  if (e.R) v += (float)static_cast<const TY*>(e.R)[m * e.ldr + n];
  static_cast<TY*>(e.Y)[m * e.ldy + n] = Vec8<TY>::narrow(v);
}

// ---------------------------------------------------------------------------------------------
// the epilogue's backward: a block owns 512 columns (8 per thread over 64 lanes) and a strip of rows,
// which its 4 waves take in turn; each thread keeps its columns' sums in fp32. HBM bounds it: 2048 x
// 11008 in bf16 31.7 us for 135 MB, 4.3 TB/s, of which 4 for the sums.
// ---------------------------------------------------------------------------------------------
struct GradArgs {
  const void *dY, *Z;
  void* dZ;
  float* part;  // [strips][N], or NULL
  int64_t M, lddy, ldz, lddz;
  int N, act, strip;
};
template <typename TA, typename TY>
__global__ __launch_bounds__(256) void linear_grad_kernel(GradArgs a) {
  __shared__ float s[3][512];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = blockIdx.x * 512 + lane * 8;
  const int64_t r0 = (int64_t)blockIdx.y * a.strip;
  const int64_t r1 = r0 + a.strip < a.M ? r0 + a.strip : a.M;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t m = r0 + w; m < r1; m += 4) {
    float d[8], z[8];
    widen8<TY>(load8_any<TY>(static_cast<const TY*>(a.dY) + m * a.lddy, n, a.N), d);
    if (a.act != RB_ACT_NONE) {
      widen8<TA>(load8_any<TA>(static_cast<const TA*>(a.Z) + m * a.ldz, n, a.N), z);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] *= act_slope(z[j], a.act);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += d[j];
    if (a.dZ) store8<TA, true>(static_cast<TA*>(a.dZ) + m * a.lddz, n, a.N, d);
  }
  if (!a.part) return;
  if (w > 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[w - 1][lane * 8 + j] = sum[j];
  }
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += s[0][lane * 8 + j] + s[1][lane * 8 + j] + s[2][lane * 8 + j];
    store8<float>(a.part + (int64_t)blockIdx.y * a.N, n, a.N, sum);
  }
}
// 64 columns by 8 interleaved runs of strips
__global__ __launch_bounds__(512) void linear_grad_sum_kernel(const float* part, int strips, int N, float* db) {
  __shared__ float s[8][64];
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
    db[c] = v;
  }
}

bool tile_aligned(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t K) {
  const auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  // a tile's rows lie within 2^31 bytes, the out-of-range marker
  return a16(X) && a16(W) && ldx % 8 == 0 && ldw % 8 == 0 && K % 8 == 0 && ldx < (1 << 21) && ldw < (1 << 21);
}

// How a product is laid over the GPU's 256 compute units: `bm` batch rows by 256 weight rows per tile
// (32, 64, 128; 256 for the first `big_n` weight rows), the columns in `chunks`.
//
// The layout is chosen by estimate, in us: a step of a tile costs `one` when few units are busy and `all`
// when every unit loads at once; 5 for the launch and the ends of the pipeline; a split costs its partial
// sums' way to memory and back (5 MB / us) and 2 for the join. The figures are fits to measured runs (16..1024
// rows, 1000..4096 weight rows and columns), where the choice is within 10 % of the best of the 15 layouts; one
// layout for all would cost up to twice the time (512 x 4096 x 4096: 32-row tiles 30.6 us, 128-row tiles 47.7 us
// and in 4 chunks 35.4 us; 64 x 4096 x 4096: 28.7 us whole, 14.4 us in 4 chunks).
//
// 256-row tiles move two thirds of the bytes per product that 128-row ones do, but a round of 256 of
// them must be full to pay: whole rounds go to them (kBig a step), the rest to the small tiles. Small tiles alone
// are taken where they are estimated at kClear of that time and less, which is where most of the last row of
// 256-row tiles is empty. Measured, 256-row tiles first / small ones alone: 2048 x 11008 x 4096 170 / 186 us,
// 150 x 65536 x 256 26 / 36, 700 x 24576 x 4096 158 / 178; 2550 x 9640 x 2064 220 / 147, 520 x 24576 x 256 34 / 27,
// 1300 x 11264 x 1024 54 / 46, 2666 x 15176 x 496 120 / 101. Between kClear and equal estimates it goes either way
// (1100 x 14336 x 4096 149 / 129, 3381 x 4824 x 240 38 / 50).
struct Plan {
  int bm, chunks, chunk_k, big_n;
  double est;
};
Plan plan_small_tiles(int64_t M, int64_t N, int64_t K, bool aligned) {
  Plan p{};
  const int64_t steps = (K + kTK - 1) / kTK;
  struct { int bm; double one, all; } const kinds[2][3] = {{{32, 0.79, 0.9}, {64, 1.0, 1.15}, {128, 1.07, 1.3}},
                                                           {{32, 0.36, 0.38}, {64, 0.50, 0.65}, {128, 0.65, 0.95}}};
  for (const auto& k : kinds[aligned]) {
    const int64_t tiles = (M + k.bm - 1) / k.bm * ((N + 255) / 256);
    for (int64_t c = 1; c <= 16 && (c == 1 || (c * 2 <= steps && tiles * c <= 512)); c *= 2) {
      const int64_t blocks = tiles * c, rounds = (blocks + 255) / 256, each = (steps + c - 1) / c;
      const double load = blocks < 256 ? (double)blocks / 256 : 1.0;
      const double est = 5.0 + (double)rounds * (double)(each + 2) * (k.one + (k.all - k.one) * load) +
                         (c > 1 ? 2.0 + (double)c * (double)M * (double)N * 8 / 5e6 : 0.0);
      if (p.bm == 0 || est < p.est) {
        p.est = est;
        p.bm = k.bm;
        p.chunk_k = (int)each * kTK;
      }
    }
  }
  p.chunks = (int)((K + p.chunk_k - 1) / p.chunk_k);
  return p;
}
Plan plan_tiles(int64_t M, int64_t N, int64_t K, bool aligned) {
  constexpr double kBig = 1.6, kClear = 0.87;
  const Plan small = plan_small_tiles(M, N, K, aligned);
  const int64_t tm = (M + 255) / 256, rounds = tm * ((N + 255) / 256) / 256;
  if (!aligned || rounds == 0) return small;
  const int64_t big_n = rounds * 256 / tm * 256 < N ? rounds * 256 / tm * 256 : N;
  Plan p = big_n < N ? plan_small_tiles(M, N - big_n, K, aligned) : Plan{};
  p.big_n = (int)big_n;
  p.est += 5.0 + (double)rounds * (double)((K + kTK - 1) / kTK + 2) * kBig;
  return big_n == 0 || small.est < kClear * p.est ? small : p;
}

// The forms without tiles; both read 8 columns at least. Up to 4 rows the vector units' products cost nothing
// beside the weights. The one-launch form on the matrix cores is taken by its estimate against the tiles', up to
// the 256 rows the estimate was fitted over: it saves the join and the pipeline's ends, and reads each operand
// once per 16 rows of the other (us, one launch / tiles: 64 x 512 x 512 3.0 / 7.2; 64 x 300 x 520 3.1 / 9.1;
// 16 x 4096 x 4096 10.6 / 13.9; 64 x 2048 x 2048 9.7 / 10.7; 128 x 2048 x 2048 16.8 / 12.2; rows not aligned: 48 x
// 1027 x 1411 8.6 / 13.0; 128 x 1027 x 1411 19.6 / 16.1; 20 x 1000 x 4001 21.5 / 12.9).
enum class Small { kNone, kRows, kFew };
Small small_form(int64_t M, int64_t N, int64_t K, bool aligned) {
  if (K < 8 || M > kFewRows) return Small::kNone;
  if (M <= kMaxRows) return Small::kRows;
  const int64_t rounds = ((N + 15) / 16 * ((M + 15) / 16) + 255) / 256, steps = (K + kTK - 1) / kTK;
  const Plan p = plan_tiles(M, N, K, aligned);
  return 2.6 + (double)(rounds * steps) * (aligned ? 0.13 : 0.33) < p.est ? Small::kFew : Small::kNone;
}

template <typename TA, typename TY, int WM, int WN, int TM, int kS, bool AL>
hipError_t launch_tile(TileArgs a, int chunks, hipStream_t s) {
  constexpr int BM = 16 * WM * TM, BN = 64 * WN;
  constexpr int stage = kS * (BM + BN) * kRowB, turn = WM * WN * 16 * kPadRow * 4;
  constexpr int lds = stage > turn ? stage : turn;
  static const hipError_t attr = hipFuncSetAttribute((const void*)linear_tile_kernel<TA, TY, WM, WN, TM, 4, kS, AL>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  const int64_t tm = (a.M + BM - 1) / BM, tiles = tm * ((a.N + BN - 1) / BN);
  if (tiles > 0xffffffffll) return hipErrorInvalidConfiguration;  // outputs of 2^40 elements and more
  a.tiles_m = (uint32_t)tm;
  return launch_in_parts(tiles, [&](int64_t first, uint32_t count) {
    a.first = (uint32_t)first;
    a.tiles = a.first + count;
    a.per_xcd = (count + kXcds - 1) / kXcds;
    linear_tile_kernel<TA, TY, WM, WN, TM, 4, kS, AL>
        <<<dim3(a.per_xcd * kXcds, (uint32_t)chunks), 64 * WM * WN, lds, s>>>(a);
  });
}

// One batch row: a weight row per wave, 8 loads of it in flight (4096 x 4096 fp16: 6.9 us, 4.9 TB/s; 2 rows
// by 4 loads 7.7, 4 by 4 8.1). Up to 4 batch rows: 2 weight rows per wave halve the reads of X (7.4 us;
// 1 by 8 9.3), where that leaves enough waves.
template <typename TA, typename TY>
hipError_t launch_rows(TileArgs a, hipStream_t s) {
  const bool pairs = a.M > 1 && a.N >= 2048;
  return launch_in_parts(pairs ? ((int64_t)a.N + 7) / 8 : ((int64_t)a.N + 3) / 4, [&](int64_t first, uint32_t blocks) {
    a.first = (uint32_t)first;
    if (a.M == 1)
      linear_rows_kernel<TA, TY, 1, 1, 8><<<dim3(blocks), 256, 0, s>>>(a);
    else if (!pairs)
      linear_rows_kernel<TA, TY, 4, 1, 8><<<dim3(blocks), 256, 0, s>>>(a);
    else
      linear_rows_kernel<TA, TY, 4, 2, 4><<<dim3(blocks), 256, 0, s>>>(a);
  });
}

template <typename TA, typename TY>
hipError_t launch_product(TileArgs a, void* ws, hipStream_t s) {
  const bool al = tile_aligned(a.X, a.ldx, a.W, a.ldw, a.K);
  switch (small_form(a.M, a.N, a.K, al)) {
    case Small::kRows: return launch_rows<TA, TY>(a, s);
    case Small::kFew:
      linear_few_kernel<TA, TY><<<dim3((uint32_t)((a.N + 15) / 16), (uint32_t)((a.M + 15) / 16)), 512, 0, s>>>(a);
      return hipGetLastError();
    case Small::kNone: break;
  }
  const Plan p = plan_tiles(a.M, a.N, a.K, al);
  a.chunk_k = (a.K + kTK - 1) / kTK * kTK;
  if (p.big_n > 0) {
    TileArgs b = a;
    b.N = p.big_n;
    const hipError_t e = launch_tile<TA, TY, 2, 4, 8, 2, true>(b, 1, s);
    if (e != hipSuccess || p.big_n == a.N) return e;
    a.N -= p.big_n;
    a.W = static_cast<const TA*>(a.W) + (int64_t)p.big_n * a.ldw;
    if (a.e.bias) a.e.bias += p.big_n;
    if (a.e.R) a.e.R = static_cast<const TY*>(a.e.R) + p.big_n;
    if (a.e.Z) a.e.Z = static_cast<TA*>(a.e.Z) + p.big_n;
    a.e.Y = static_cast<TY*>(a.e.Y) + p.big_n;
  }
  a.chunk_k = p.chunk_k;
  a.part = p.chunks > 1 ? static_cast<float*>(ws) : nullptr;
  hipError_t e;
  if (p.bm == 32)
    e = al ? launch_tile<TA, TY, 1, 4, 2, 3, true>(a, p.chunks, s) : launch_tile<TA, TY, 1, 4, 2, 2, false>(a, p.chunks, s);
  else if (p.bm == 64)
    e = al ? launch_tile<TA, TY, 1, 4, 4, 3, true>(a, p.chunks, s) : launch_tile<TA, TY, 1, 4, 4, 2, false>(a, p.chunks, s);
  else
    e = al ? launch_tile<TA, TY, 2, 4, 4, 3, true>(a, p.chunks, s) : launch_tile<TA, TY, 2, 4, 4, 2, false>(a, p.chunks, s);
  if (e != hipSuccess || p.chunks == 1) return e;
  const JoinArgs j{a.part, a.M, a.N, p.chunks, a.e};
  linear_join_kernel<TA, TY><<<dim3((uint32_t)((a.N + 2047) / 2048), (uint32_t)a.M), 256, 0, s>>>(j);
  return hipGetLastError();
}

// Strips of rows: enough blocks to fill the GPU, few enough partial sums. Up to 8 rows (2 per wave) are one
// strip, whose sums are db itself: 4 x 4096 2.9 us against 4.9 with a second launch, but 16 x 4096 6.0
// against 5.0.
int grad_strip(int64_t M, int64_t N) {
  if (M <= 8) return 8;
  const int64_t cols = (N + 511) / 512, want = (1024 + cols - 1) / cols;
  const int64_t strip = ((M + want - 1) / want + 3) / 4 * 4;
  return (int)(strip < 4 ? 4 : strip);
}

}  // namespace

size_t linear_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  size_t most = 0;
  for (int al = 0; al < 2; ++al) {
    if (small_form(M, N, K, al != 0) != Small::kNone) continue;
    const Plan p = plan_tiles(M, N, K, al != 0);
    const size_t b = p.chunks > 1 ? (size_t)p.chunks * (size_t)M * (size_t)(N - p.big_n) * 4 : 0;
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_linear(const void* X, rb_dtype a_dtype, int64_t M, int64_t ldx, const void* W, int64_t ldw, int64_t N,
                         int64_t K, const float* bias, int act, const void* R, int64_t ldr, void* Z, int64_t ldz,
                         void* Y, rb_dtype y_dtype, int64_t ldy, void* ws, hipStream_t s) {
  const auto lines = [](const void* p, int64_t ld, rb_dtype t) {
    return reinterpret_cast<uintptr_t>(p) % 128 == 0 && ld * (t == RB_F32 ? 4 : 2) % 128 == 0;
  };
  TileArgs a{X, W, ldx, ldw, M, (int)N, (int)K, 0, 0, 0, 0, 0, nullptr,
             {bias, R, Z, Y, ldr, ldz, ldy, act, lines(Z, ldz, a_dtype), lines(Y, ldy, y_dtype)}};
  if (a_dtype == RB_F16)
    return y_dtype == RB_F32 ? launch_product<_Float16, float>(a, ws, s) : launch_product<_Float16, _Float16>(a, ws, s);
  return y_dtype == RB_F32 ? launch_product<__bf16, float>(a, ws, s) : launch_product<__bf16, __bf16>(a, ws, s);
}

size_t linear_backward_workspace_bytes(int64_t N, int64_t M) {
  const int strip = grad_strip(M, N);
  return M <= strip ? 0 : (size_t)((M + strip - 1) / strip) * (size_t)N * 4;
}

hipError_t launch_linear_backward(const void* dY, rb_dtype dy_dtype, int64_t M, int64_t N, int64_t lddy, const void* Z,
                                  rb_dtype a_dtype, int64_t ldz, int act, void* dZ, int64_t lddz, float* db, void* ws,
                                  hipStream_t s) {
  const int strip = grad_strip(M, N);
  const int strips = (int)((M + strip - 1) / strip);
  const GradArgs a{dY, Z, dZ, !db ? nullptr : strips == 1 ? db : static_cast<float*>(ws), M, lddy, ldz, lddz, (int)N, act, strip};
  const dim3 grid((uint32_t)((N + 511) / 512), (uint32_t)strips);
  if (a_dtype == RB_F16) {
    if (dy_dtype == RB_F32)
      linear_grad_kernel<_Float16, float><<<grid, 256, 0, s>>>(a);
    else
      linear_grad_kernel<_Float16, _Float16><<<grid, 256, 0, s>>>(a);
  } else if (dy_dtype == RB_F32) {
    linear_grad_kernel<__bf16, float><<<grid, 256, 0, s>>>(a);
  } else {
    linear_grad_kernel<__bf16, __bf16><<<grid, 256, 0, s>>>(a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !db || strips == 1) return e;
  linear_grad_sum_kernel<<<dim3((uint32_t)((N + 63) / 64)), 512, 0, s>>>(a.part, strips, (int)N, db);
  return hipGetLastError();
}

}  // namespace rb
