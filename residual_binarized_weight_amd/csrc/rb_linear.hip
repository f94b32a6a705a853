// rb_linear.hip -- a coupled-training layer's product with its epilogue, and the epilogue's backward.
//
//   Z = X What^T + b,  Y = act(Z) + R        X [M][K], What [N][K] in fp16 or bf16, fp32 sums
//   dZ = dY act'(Z),   db = column sums of dZ
//
// Kernels of this file:
//   linear_tile_kernel    a tile of 16 MT batch rows by 256 weight rows per block, on the matrix cores
//   linear_join_kernel    the sums of K chunks, where a tile's columns are split, and the epilogue
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
// activations, in fp32: their own error is a few units of 2^-24 of |z|, below every storage type's
// ---------------------------------------------------------------------------------------------
constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case RB_ACT_RELU: return z < 0.f ? 0.f : z;
    case RB_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.7071067811865476f));
    case RB_ACT_GELU_TANH: return z * logistic(2.f * kGeluA * (z + kGeluB * z * z * z));  // (1 + tanh a) / 2
    case RB_ACT_SILU: return z * logistic(z);
  }
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case RB_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case RB_ACT_GELU:
      return 0.5f * (1.f + erff(z * 0.7071067811865476f)) + z * 0.3989422804014327f * __expf(-0.5f * z * z);
    case RB_ACT_GELU_TANH: {
      const float g = logistic(2.f * kGeluA * (z + kGeluB * z * z * z));
      return g + z * g * (1.f - g) * 2.f * kGeluA * (1.f + 3.f * kGeluB * z * z);
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
};
// columns n .. n+7 of row m, v the product's fp32 sums
template <typename TA, typename TY>
__device__ __forceinline__ void finish8(const Epilogue& e, float (&v)[8], int64_t m, int n, int N) {
  if (e.bias) {
    float b[8];
    widen8<float>(load8<float>(e.bias, n, N), b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
  }
  if (e.Z) store8<TA>(static_cast<TA*>(e.Z) + m * e.ldz, n, N, v);
  if (e.act != RB_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_value(v[j], e.act);
  }
  if (e.R) {
    float r[8];
    widen8<TY>(load8<TY>(static_cast<const TY*>(e.R) + m * e.ldr, n, N), r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
  store8<TY>(static_cast<TY*>(e.Y) + m * e.ldy, n, N, v);
}

// ---------------------------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------------------------
// 16 bytes per lane from the buffer to LDS (lane l's at base + 16 l)
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* base, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (l_lds_void*)base, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ l_u4 load_16(__amdgpu_buffer_rsrc_t r, uint32_t voff, int soff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, soff, 0);
}

constexpr int kTN = 256;           // weight rows per tile: 64 per wave
constexpr int kTK = 64;            // columns per step
constexpr int kRowB = kTK * 2;     // bytes of a staged row
constexpr int kStages = 4;         // steps held in LDS: two being read, two arriving
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
  uint32_t tiles_m, tiles, per_xcd;
  int chunk_k;    // columns per K chunk, a multiple of kTK
  float* part;    // [chunks][M][N] fp32 sums, or NULL: one chunk, epilogue here
  Epilogue e;
};

constexpr int tile_lds(int MT, int KG) {
  const int stage = kStages * 16 * MT * kRowB * KG, turn = 4 * KG * 16 * kPadRow * 4;
  const int swap = KG == 2 ? 8 * (MT > 1 ? MT / 2 : 1) * 4096 : 0;
  const int most = stage > turn ? stage : turn;
  return most > swap ? most : swap;
}

// Tile. 4 KG waves; wave w of a group owns weight rows 64 w .. +63 and all 16 MT batch rows (4 x MT
// accumulators of v_mfma_f32_16x16x32). With KG = 2 the two groups take alternate 64-column steps
// of the same tile and join at the end, so that two waves per SIMD share a CU's single tile.
// A weight element is needed by one wave only: it goes straight from L2 to that wave's
// registers (two steps ahead), and LDS carries only the batch rows, which all 4 waves read.
// AL: rows of both operands are 16-byte aligned and K is a multiple of 8, so batch rows go to LDS
// directly. Otherwise they pass through registers, and a step that holds the end of the columns is
// read element by element.
template <typename TA, typename TY, int MT, int KG, bool AL>
__global__ __launch_bounds__(256 * KG, 2) void linear_tile_kernel(TileArgs a) {
  extern __shared__ __align__(16) uint8_t l_smem[];
  const uint32_t blk = blockIdx.x;
  const uint32_t t = blk % kXcds * a.per_xcd + blk / kXcds;  // an XCD's blocks take one run of tiles
  if (t >= a.tiles) return;
  const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane(t % a.tiles_m) * (16 * MT);
  const int n0 = __builtin_amdgcn_readfirstlane(t / a.tiles_m) * kTN;
  const int kb = blockIdx.y * a.chunk_k;
  const int ke = kb + a.chunk_k < a.K ? kb + a.chunk_k : a.K;

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int grp = wv >> 2, w = wv & 3;
  const int lr = lane & 15, lj = lane >> 4;

  const int64_t mrows = a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT;
  const int nrows = a.N - n0 < kTN ? a.N - n0 : kTN;
  const __amdgpu_buffer_rsrc_t rx =
      buffer_rsrc(static_cast<const TA*>(a.X) + m0 * a.ldx, (uint32_t)(mrows * a.ldx * 2));
  const __amdgpu_buffer_rsrc_t rw =
      buffer_rsrc(static_cast<const TA*>(a.W) + (int64_t)n0 * a.ldw, (uint32_t)(nrows * a.ldw * 2));

  uint32_t woff[4];
  const TA* wrow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 64 * w + 16 * i + lr;
    woff[i] = (uint32_t)(r * a.ldw * 2) + 16u * lj;
    // a row past the last one repeats it: its outputs are not stored
    wrow[i] = static_cast<const TA*>(a.W) + (int64_t)(n0 + (r < nrows ? r : nrows - 1)) * a.ldw;
  }

  // batch rows into LDS: 1 KB groups of 8 rows; lane l fills slot l % 8 of row l / 8 with the 16-byte
  // chunk (l % 8) ^ (row % 8), so that the 8 rows of a fragment read's phase lie in 8 bank groups
  constexpr int kGroupsX = 2 * MT;
  constexpr int kPer = kGroupsX >= 4 ? kGroupsX / 4 : 1;
  const int xc = (lane & 7) ^ (lane >> 3);
  uint32_t xoff[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) xoff[i] = (uint32_t)((8 * (w * kPer + i) + (lane >> 3)) * a.ldx * 2) + 16u * xc;
  uint8_t* const area = l_smem + grp * (kStages * 16 * MT * kRowB);
  const auto k_of = [&](int i) { return kb + (i * KG + grp) * kTK; };
  const auto dma = [&](int i) {
    const int k0 = k_of(i);
    const bool ok = k0 + 8 * xc < ke;
    uint8_t* const base = area + (i & (kStages - 1)) * (16 * MT * kRowB);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (kGroupsX < 4 && w >= kGroupsX) break;
      load_to_lds(rx, base + (w * kPer + j) * 1024, ok ? xoff[j] : kOob, k0 * 2);
    }
  };
  // the same through registers: a thread holds chunk slots tid + 256 j of two steps
  constexpr int kHold = MT >= 2 ? MT / 2 : 1;
  l_u4 hold[2][kHold];
  const int gtid = threadIdx.x & 255;
  const auto fetch_x = [&](int i) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int k0 = k_of(i + p);
#pragma unroll
      for (int j = 0; j < kHold; ++j) {
        const int q = gtid + 256 * j, r = q >> 3, c = k0 + 8 * (q & 7);
        if (r >= 16 * MT) continue;
        const TA* row = static_cast<const TA*>(a.X) + (m0 + (r < mrows ? r : (int)mrows - 1)) * a.ldx;
        if (k0 + kTK <= ke)
          hold[p][j] = __builtin_bit_cast(l_u4, *reinterpret_cast<const typename Vec8<TA>::Raw*>(row + c));
        else
          hold[p][j] = __builtin_bit_cast(l_u4, load8<TA>(row, c, ke));
      }
    }
  };
  const auto stage_x = [&](int i) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < kHold; ++j) {
        const int q = gtid + 256 * j, r = q >> 3;
        if (r >= 16 * MT) continue;
        uint8_t* const base = area + ((i + p) & (kStages - 1)) * (16 * MT * kRowB);
        *reinterpret_cast<l_u4*>(base + r * kRowB + 16 * ((q & 7) ^ (r & 7))) = hold[p][j];
      }
  };
  l_u4 wf[2][2][4];  // step parity, half of the step, weight row tile
  const auto load_w = [&](int p, int kh, int i) {
    const int k0 = k_of(i) + 32 * kh;
    if constexpr (!AL) {
      const int c = k0 + 8 * lj;
      if (k0 + 32 <= ke) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          wf[p][kh][j] = __builtin_bit_cast(l_u4, *reinterpret_cast<const typename Vec8<TA>::Raw*>(wrow[j] + c));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) wf[p][kh][j] = __builtin_bit_cast(l_u4, load8<TA>(wrow[j], c, ke));
      }
      return;
    }
    const bool ok = k0 + 8 * lj < ke;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      wf[p][kh][j] = load_16(rw, ok ? woff[j] : kOob, k0 * 2);
  };

  l_f4 acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (l_f4){0.f, 0.f, 0.f, 0.f};

  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)area;
  // fragment row lr + 16 i has lr % 8 in its swizzle whatever i
  const uint32_t fo0 = lr * kRowB + 16u * ((uint32_t)lj ^ (lr & 7u)), fo1 = lr * kRowB + 16u * ((4u + lj) ^ (lr & 7u));
  l_u4 xf[MT];
  const auto read_x = [&](int i, int stage, int kh) {
    xf[i] = *(l_lds_u4*)(size_t)(lds0 + stage * (16 * MT * kRowB) + i * 16 * kRowB + (kh ? fo1 : fo0));
  };

  const int steps = ((ke - kb + kTK - 1) / kTK + KG - 1) / KG;
  const int halves = (steps + 1) / 2;
  if constexpr (AL) {
    dma(0);
    dma(1);
  } else {
    fetch_x(0);
    stage_x(0);
  }
  load_w(0, 0, 0);
  load_w(0, 1, 0);
  load_w(1, 0, 1);
  load_w(1, 1, 1);
  __builtin_amdgcn_sched_barrier(0);
  for (int h = 0; h < halves; ++h) {
    // the 16 weight loads issued after this half's batch rows may still be in flight
    __builtin_amdgcn_s_waitcnt(AL ? wait_vmcnt(16) : kWaitLds);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();  // every wave's rows are in; every wave is done with the other two stages
    asm volatile("" ::: "memory");
    if constexpr (AL) {
      dma(2 * h + 2);
      dma(2 * h + 3);
    } else {
      fetch_x(2 * h + 2);
    }
    __builtin_amdgcn_sched_barrier(0);
    const int st = (h & 1) * 2;
#pragma unroll
    for (int i = 0; i < MT; ++i) read_x(i, st, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        const bool more = p == 0 || kh == 0;  // the other stages' rows are only safe after the next barrier
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma(TA(0), wf[p][kh][j], xf[i], acc[i][j]);
          if (more) read_x(i, st + p + kh, kh ^ 1);
        }
        load_w(p, kh, 2 * h + p + 2);
        // as written: a fragment is read again as soon as its 4 products are issued, the weights once
        // all are, and neither is moved next to its use
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);             // MFMA
          if (more) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    if constexpr (!AL) stage_x(2 * h + 2);
    __builtin_amdgcn_sched_barrier(0);
  }
  // loads past the last step (out of range, zeros) end before LDS is used again
  __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));
  __syncthreads();

  int i0 = 0, i1 = MT;
  if constexpr (KG == 2) {
    // the groups swap halves of the batch rows' tiles and add: group 0 keeps the first half (for MT = 1
    // group 1 gives all to group 0)
    constexpr int kHalf = MT > 1 ? MT / 2 : 1;
    float* const mine = reinterpret_cast<float*>(l_smem) + (size_t)wv * (kHalf * 4 * 256);
    const float* const other = reinterpret_cast<float*>(l_smem) + (size_t)(wv ^ 4) * (kHalf * 4 * 256);
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const l_f4 v = grp == 0 ? acc[MT > 1 ? i + kHalf : i][j] : acc[i][j];
        *reinterpret_cast<l_f4*>(mine + ((i * 4 + j) * 64 + lane) * 4) = v;
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const l_f4 o = *reinterpret_cast<const l_f4*>(other + ((i * 4 + j) * 64 + lane) * 4);
        if (grp == 0) acc[i][j] = acc[i][j] + o;
        if (MT > 1 && grp == 1) acc[i + kHalf][j] = o + acc[i + kHalf][j];
      }
    __syncthreads();
    i0 = grp == 0 ? 0 : kHalf;
    i1 = grp == 0 ? kHalf : MT;
  }

  // 16 rows at a time through the wave's own LDS area, so that 8 lanes hold 64 consecutive columns of
  // a row and whole 128-byte lines are read and written. D of the product: lane l holds weight rows
  // 4 (l / 16) .. +3 of batch row l % 16.
  float* const turn = reinterpret_cast<float*>(l_smem) + wv * (16 * kPadRow);
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
#pragma unroll
    for (int q = 0; q < MT; ++q)
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
      const int64_t m = m0 + 16 * i + r;
      const int n = n0 + 64 * w + c;
      if (m < a.M && n < a.N) {
        if (a.part)
          store8<float>(a.part + ((int64_t)blockIdx.y * a.M + m) * a.N, n, a.N, v);
        else
          finish8<TA, TY>(a.e, v, m, n, a.N);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
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
#pragma unroll 4
  for (int c = 0; c < a.chunks; ++c) {
    float p[8];
    widen8<float>(load8<float>(a.part + ((int64_t)c * a.M + m) * a.N, n, a.N), p);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += p[j];
  }
  finish8<TA, TY>(a.e, v, m, n, a.N);
}

// ---------------------------------------------------------------------------------------------
// the epilogue's backward: a block owns 512 columns (8 per thread over 64 lanes) and a strip of rows,
// which its 4 waves take in turn; each thread keeps its columns' sums in fp32
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
#pragma unroll 2
  for (int64_t m = r0 + w; m < r1; m += 4) {
    float d[8], z[8];
    widen8<TY>(load8<TY>(static_cast<const TY*>(a.dY) + m * a.lddy, n, a.N), d);
    if (a.act != RB_ACT_NONE) {
      widen8<TA>(load8<TA>(static_cast<const TA*>(a.Z) + m * a.ldz, n, a.N), z);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] *= act_slope(z[j], a.act);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += d[j];
    if (a.dZ) store8<TA>(static_cast<TA*>(a.dZ) + m * a.lddz, n, a.N, d);
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

struct Plan {
  int mt, chunks, chunk_k;
  bool two;  // two wave groups per tile
};
// see launch: how many blocks a shape gives
Plan plan_tiles(int64_t M, int64_t N, int64_t K, bool aligned) {
  Plan p;
  p.mt = M <= 16 ? 1 : M <= 32 ? 2 : M <= 64 || !aligned ? 4 : 8;
  const int64_t tiles = (M + 16 * p.mt - 1) / (16 * p.mt) * ((N + kTN - 1) / kTN);
  p.two = p.mt == 8 && tiles < 512;
  const int64_t steps = (K + kTK - 1) / kTK;
  const int64_t want = tiles >= 192 ? 1 : (p.two ? 256 : 512) / tiles;
  const int64_t most = steps / 8 > 1 ? steps / 8 : 1;
  const int64_t chunks = want < most ? want : most;
  p.chunk_k = (int)((steps + chunks - 1) / chunks) * kTK;
  p.chunks = (int)((K + p.chunk_k - 1) / p.chunk_k);
  return p;
}

bool tile_aligned(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t K) {
  const auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  // a tile's rows lie within 2^31 bytes, the out-of-range marker
  return a16(X) && a16(W) && ldx % 8 == 0 && ldw % 8 == 0 && K % 8 == 0 && ldx < (1 << 21) && ldw < (1 << 21);
}

template <typename TA, typename TY, int MT, int KG, bool AL>
hipError_t launch_tile(const TileArgs& a, int chunks, hipStream_t s) {
  constexpr int lds = tile_lds(MT, KG);
  static const hipError_t attr = hipFuncSetAttribute((const void*)linear_tile_kernel<TA, TY, MT, KG, AL>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  linear_tile_kernel<TA, TY, MT, KG, AL>
      <<<dim3(a.per_xcd * kXcds, (uint32_t)chunks), 256 * KG, lds, s>>>(a);
  return hipGetLastError();
}

template <typename TA, typename TY>
hipError_t launch_product(TileArgs a, void* ws, hipStream_t s) {
  const bool al = tile_aligned(a.X, a.ldx, a.W, a.ldw, a.K);
  const Plan p = plan_tiles(a.M, a.N, a.K, al);
  const int64_t tm = (a.M + 16 * p.mt - 1) / (16 * p.mt), tiles = tm * ((a.N + kTN - 1) / kTN);
  if (tiles > 0x70000000) return hipErrorInvalidConfiguration;
  a.tiles_m = (uint32_t)tm;
  a.tiles = (uint32_t)tiles;
  a.per_xcd = (uint32_t)((tiles + kXcds - 1) / kXcds);
  a.chunk_k = p.chunk_k;
  a.part = p.chunks > 1 ? static_cast<float*>(ws) : nullptr;
  hipError_t e;
  if (!al)
    e = p.mt == 1 ? launch_tile<TA, TY, 1, 1, false>(a, p.chunks, s)
                  : p.mt == 2 ? launch_tile<TA, TY, 2, 1, false>(a, p.chunks, s)
                              : launch_tile<TA, TY, 4, 1, false>(a, p.chunks, s);
  else if (p.mt == 1)
    e = launch_tile<TA, TY, 1, 1, true>(a, p.chunks, s);
  else if (p.mt == 2)
    e = launch_tile<TA, TY, 2, 1, true>(a, p.chunks, s);
  else if (p.mt == 4)
    e = launch_tile<TA, TY, 4, 1, true>(a, p.chunks, s);
  else
    e = p.two ? launch_tile<TA, TY, 8, 2, true>(a, p.chunks, s) : launch_tile<TA, TY, 8, 1, true>(a, p.chunks, s);
  if (e != hipSuccess || p.chunks == 1) return e;
  const JoinArgs j{a.part, a.M, a.N, p.chunks, a.e};
  linear_join_kernel<TA, TY><<<dim3((uint32_t)((a.N + 2047) / 2048), (uint32_t)a.M), 256, 0, s>>>(j);
  return hipGetLastError();
}

// strips of rows: enough blocks to fill the GPU, few enough partial sums
int grad_strip(int64_t M, int64_t N) {
  const int64_t cols = (N + 511) / 512, want = (1024 + cols - 1) / cols;
  int64_t strip = (M + want - 1) / want;
  strip = (strip + 3) / 4 * 4;
  return (int)(strip < 4 ? 4 : strip);
}

}  // namespace

size_t linear_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  size_t most = 0;
  for (int al = 0; al < 2; ++al) {
    const Plan p = plan_tiles(M, N, K, al != 0);
    const size_t b = p.chunks > 1 ? (size_t)p.chunks * (size_t)M * (size_t)N * 4 : 0;
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_linear(const void* X, rb_dtype a_dtype, int64_t M, int64_t ldx, const void* W, int64_t ldw, int64_t N,
                         int64_t K, const float* bias, int act, const void* R, int64_t ldr, void* Z, int64_t ldz,
                         void* Y, rb_dtype y_dtype, int64_t ldy, void* ws, hipStream_t s) {
  TileArgs a{X, W, ldx, ldw, M, (int)N, (int)K, 0, 0, 0, 0, nullptr, {bias, R, Z, Y, ldr, ldz, ldy, act}};
  if (a_dtype == RB_F16)
    return y_dtype == RB_F32 ? launch_product<_Float16, float>(a, ws, s) : launch_product<_Float16, _Float16>(a, ws, s);
  return y_dtype == RB_F32 ? launch_product<__bf16, float>(a, ws, s) : launch_product<__bf16, __bf16>(a, ws, s);
}

size_t linear_backward_workspace_bytes(int64_t N, int64_t M) {
  const int strip = grad_strip(M, N);
  return (size_t)((M + strip - 1) / strip) * (size_t)N * 4;
}

hipError_t launch_linear_backward(const void* dY, rb_dtype dy_dtype, int64_t M, int64_t N, int64_t lddy, const void* Z,
                                  rb_dtype a_dtype, int64_t ldz, int act, void* dZ, int64_t lddz, float* db, void* ws,
                                  hipStream_t s) {
  const int strip = grad_strip(M, N);
  const int strips = (int)((M + strip - 1) / strip);
  const GradArgs a{dY, Z, dZ, db ? static_cast<float*>(ws) : nullptr, M, lddy, ldz, lddz, (int)N, act, strip};
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
  if (e != hipSuccess || !db) return e;
  linear_grad_sum_kernel<<<dim3((uint32_t)((N + 63) / 64)), 512, 0, s>>>(a.part, strips, (int)N, db);
  return hipGetLastError();
}

}  // namespace rb
