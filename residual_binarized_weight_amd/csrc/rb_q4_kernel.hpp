// rb_q4_kernel.hpp -- the kernel behind rb_q4_product.hpp; one file per type of x includes it.
#pragma once

#include "rb_q4_product.hpp"

namespace rb {
namespace q4 {
namespace {

using tile::f4;
using tile::u4;

constexpr int kTileN = 16, kTileK = 128;

template <typename T> struct Nib;
template <> struct Nib<_Float16> {  // 16 + q: 0x4c00 with q in bits 9 .. 6
  static constexpr uint32_t kOne = 0x3c003c00u, kMask = 0x03c003c0u, kBase = 0x4c004c00u;
  __device__ static __forceinline__ u4 widen(uint32_t w, uint32_t m, uint32_t b) {
    return (u4){(w << 6 & m) | b, (w << 2 & m) | b, (w >> 2 & m) | b, (w >> 6 & m) | b};
  }
};
template <> struct Nib<__bf16> {  // 16 + q: 0x4180 with q in bits 6 .. 3
  static constexpr uint32_t kOne = 0x3f803f80u, kMask = 0x00780078u, kBase = 0x41804180u;
  __device__ static __forceinline__ u4 widen(uint32_t w, uint32_t m, uint32_t b) {
    return (u4){(w << 3 & m) | b, (w >> 1 & m) | b, (w >> 5 & m) | b, (w >> 9 & m) | b};
  }
};

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u2_by2 __attribute__((ext_vector_type(2), aligned(2)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));

// four rows' scales of a group, n .. n + 3; a row past the last one repeats it (its outputs are not stored)
__device__ __forceinline__ u2 scales4(const _Float16* s, int64_t n, int64_t N) {
  if (n + 4 <= N) return *reinterpret_cast<const u2_by2*>(s + n);
  half4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = s[n + e < N ? n + e : N - 1];
  return __builtin_bit_cast(u2, v);
}

// The columns are taken in chunks of kWaves kSteps tiles. x and the scales of a chunk go to LDS (the scales as fp32 s and
// z - 16 s or -24 s); a wave's codes of a chunk, kSteps loads of 1 KB from each weight, are all in flight at once,
// behind them (a wave's loads return in order). Up to kM batch rows. With 16 of them LDS holds a short chunk only, and
// the next one's loads are in flight while a chunk is multiplied (with groups of 32, and of 64 but for the pair, 2 to 4
// registers go to scratch for that). Up to 4 rows a chunk is as long as the registers for its codes allow: 12288
// columns for 16 waves and 8192 for 8, of a pair 6144 and 4096; the next one's loads start when a chunk is multiplied, so
// that its first tile costs another trip to memory (us, one row, group 128, weights cold, a chunk's end / a tile more:
// 4096 x 12288 9.3 / 10.3, 8192 x 8192 9.8 / 11.2, the pair of 4096 x 6144 8.9 / 9.7 and of 11008 x 4096 12.6 / 14.0; several
// chunks: 8192 x 28672 28.0, 4.3 TB/s, the pair of 28672 x 8192 50.2, 4.8). Bound by the launch's ramp and one trip to memory:
// 4096 x 11008, group 128, 23 MB: 7.6 us cold among other calls (3.1 TB/s); 16 rows, group 32 with offsets 18 us: four
// times the groups, whose staging and sums were not timed apart.
template <typename T, int kGroup, bool kPair, int kM, int kWaves>
struct Kernel {
  static constexpr int kThreads = 64 * kWaves, kMat = kPair ? 2 : 1;
  static constexpr bool kPre = kM > 4;
  static constexpr int kSteps = kM > 4 ? (kPair ? 1 : 2) : kPair ? (kWaves == 16 ? 3 : 4) : kWaves == 16 ? 6 : 8;
  static constexpr int kChunk = kWaves * kSteps;                                   // tiles
  static constexpr int kGroups = kTileK / kGroup, kEach = kGroup / 32;
  static constexpr int kScales = (kChunk * kGroups * 4 + kThreads - 1) / kThreads; // pieces of 4 rows per thread
  static constexpr int kXRow = kChunk * kTileK + 32;                               // elements of a staged row: rows shift by 64 bytes
  static constexpr int kXVecs = (kM * kChunk * (kTileK / 8) + kThreads - 1) / kThreads;  // 16-byte pieces per thread
  static constexpr int kLdsX = kM * kXRow * 2, kLdsScales = kChunk * kGroups * 128;  // bytes of x, of one weight's scales
  static constexpr int kLdsSums = kMat * kWaves * 1024;
  static constexpr int kLdsAll = kLdsX + kMat * kLdsScales;
  static constexpr int kLds = kLdsAll > kLdsSums ? kLdsAll : kLdsSums;
  static_assert(kLds <= 160 * 1024, "LDS of a compute unit");

  u2 sr[kMat][2][kScales];
  u4 xr[kXVecs];

  // x and the scales of the chunk at tile c0, on their way to LDS
  __device__ __forceinline__ void load(const Args& a, int c0, int64_t n0) {
    const int steps = a.steps - c0 < kChunk ? a.steps - c0 : kChunk;
#pragma unroll
    for (int i = 0; i < kXVecs; ++i) {
      const int v = i * kThreads + threadIdx.x, m = v / (kChunk * (kTileK / 8)), c = v % (kChunk * (kTileK / 8)) * 8;
      if (m < a.M && c < steps * kTileK)
        xr[i] = __builtin_bit_cast(u4, load8_any<T>(static_cast<const T*>(a.x) + m * a.ldx, c0 * kTileK + c, a.K));
    }
    const int groups = (a.K + kGroup - 1) / kGroup;
#pragma unroll
    for (int q = 0; q < kMat; ++q)
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        const int v = i * kThreads + threadIdx.x, g = c0 * kGroups + v / 4;
        if (v < steps * kGroups * 4) {  // a last tile's groups past the columns repeat the last one: their x are zero
          const int64_t off = (int64_t)(g < groups ? g : groups - 1) * a.N;
          sr[q][0][i] = scales4(a.w[q].s + off, n0 + 4 * (v & 3), a.N);
          if (a.w[q].z) sr[q][1][i] = scales4(a.w[q].z + off, n0 + 4 * (v & 3), a.N);
        }
      }
  }
  __device__ __forceinline__ void put(const Args& a, int c0, uint8_t* smem) {
    const int steps = a.steps - c0 < kChunk ? a.steps - c0 : kChunk;
#pragma unroll
    for (int i = 0; i < kXVecs; ++i) {
      const int v = i * kThreads + threadIdx.x, m = v / (kChunk * (kTileK / 8)), c = v % (kChunk * (kTileK / 8)) * 8;
      if (m < a.M && c < steps * kTileK) *reinterpret_cast<u4*>(smem + (m * kXRow + c) * 2) = xr[i];
    }
#pragma unroll
    for (int q = 0; q < kMat; ++q)
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        const int v = i * kThreads + threadIdx.x;
        if (v < steps * kGroups * 4) {
          const half4 s = __builtin_bit_cast(half4, sr[q][0][i]);
          const half4 z = a.w[q].z ? __builtin_bit_cast(half4, sr[q][1][i]) : half4{};
          f4 f, off;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = (float)s[e];
            off[e] = a.w[q].z ? fmaf(-16.f, f[e], (float)z[e]) : -24.f * f[e];
          }
          uint8_t* const p = smem + kLdsX + q * kLdsScales + v / 4 * 128 + (v & 3) * 16;
          *reinterpret_cast<f4*>(p) = f;
          *reinterpret_cast<f4*>(p + 64) = off;
        }
      }
  }
  // one tile of 128 columns, the chunk's k-th; m, b: Nib's mask and base, in registers
  __device__ static __forceinline__ void tile128(const Args& a, const u4 (&code)[kMat], const uint8_t* smem, int k, int lane,
                                                 uint32_t m, uint32_t b, f4 (&total)[kMat]) {
    const int lr = lane & 15, lj = lane >> 4;
    const u4 ones = {Nib<T>::kOne, Nib<T>::kOne, Nib<T>::kOne, Nib<T>::kOne};
    const T* const x = reinterpret_cast<const T*>(smem) + (lr < a.M ? lr : 0) * kXRow + k * kTileK + 8 * lj;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      f4 d[kMat] = {}, xs = {};
#pragma unroll
      for (int i = g * kEach; i < (g + 1) * kEach; ++i) {
        const u4 xf = *reinterpret_cast<const u4*>(x + 32 * i);
        xs = tile::mfma(T(0), ones, xf, xs);
#pragma unroll
        for (int q = 0; q < kMat; ++q) d[q] = tile::mfma(T(0), Nib<T>::widen(code[q][i], m, b), xf, d[q]);
      }
#pragma unroll
      for (int q = 0; q < kMat; ++q) {
        const uint8_t* const p = smem + kLdsX + q * kLdsScales + (k * kGroups + g) * 128 + 16 * lj;
        const f4 f = *reinterpret_cast<const f4*>(p), off = *reinterpret_cast<const f4*>(p + 64);
#pragma unroll
        for (int e = 0; e < 4; ++e) total[q][e] = fmaf(f[e], d[q][e], fmaf(off[e], xs[e], total[q][e]));
      }
    }
  }

  __device__ __forceinline__ void run(const Args& a, uint8_t* smem) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    // an XCD's blocks take one run of row tiles: four of them share the lines of the scales, 64 rows each
    const uint32_t run = gridDim.x / tile::kXcds, mine = blockIdx.x % tile::kXcds * run + blockIdx.x / tile::kXcds;
    const int64_t tile_n = a.first + mine, n0 = tile_n * kTileN;
    if (n0 >= a.N) return;
    // one instruction for mask and base needs them in registers: as constants they would be two
    uint32_t m = Nib<T>::kMask, b = Nib<T>::kBase;
    asm("" : "+s"(m));
    asm("" : "+v"(b));
    // codes through a buffer resource over the block's row of tiles: past its end they read 0, without a branch
    const auto codes = [&](int c0, u4 (&code)[kSteps][kMat]) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int q = 0; q < kMat; ++q) {
          const __amdgpu_buffer_rsrc_t r = buffer_rsrc(a.w[q].codes + tile_n * a.steps * 256, (uint32_t)a.steps * 1024u);
          code[i][q] = __builtin_bit_cast(
              u4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)((uint32_t)(c0 + i * kWaves + w) * 1024u + lane * 16u), 0, 0));
        }
    };
    f4 total[kMat] = {};
    u4 code[kSteps][kMat], ahead[kPre ? kSteps : 1][kMat];
    load(a, 0, n0);
    codes(0, code);
    for (int c0 = 0; c0 < a.steps; c0 += kChunk) {
      const int steps = a.steps - c0 < kChunk ? a.steps - c0 : kChunk;
      if (c0 > 0) __syncthreads();
      put(a, c0, smem);
      __syncthreads();
      if constexpr (kPre) {
        if (c0 + kChunk < a.steps) {
          load(a, c0 + kChunk, n0);
          codes(c0 + kChunk, ahead);
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (i * kWaves + w >= steps) break;
        tile128(a, code[i], smem, i * kWaves + w, lane, m, b, total);
        __builtin_amdgcn_sched_barrier(0);  // one tile's registers at a time
      }
      if constexpr (kPre) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int q = 0; q < kMat; ++q) code[i][q] = ahead[i][q];
      } else if (c0 + kChunk < a.steps) {
        load(a, c0 + kChunk, n0);
        codes(c0 + kChunk, code);
      }
    }
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int q = 0; q < kMat; ++q) *reinterpret_cast<f4*>(sums + ((q * kWaves + w) * 64 + lane) * 4) = total[q];
    __syncthreads();
    // thread 16 m + n: D's lane 16 (n / 4) + m holds weight row n in element n % 4
    if (threadIdx.x >= 256) return;
    const int row = threadIdx.x >> 4, nn = threadIdx.x & 15;
    const int64_t n = n0 + nn;
    if (row >= a.M || n >= a.N) return;
    float v[kMat];
#pragma unroll
    for (int q = 0; q < kMat; ++q) {
      v[q] = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) v[q] += sums[((q * kWaves + i) * 64 + (nn >> 2) * 16 + row) * 4 + (nn & 3)];
    }
    const float y = kPair ? act_value(v[0], a.act) * v[kMat - 1] : v[0];
    if (a.wide)
      static_cast<float*>(a.y)[row * a.ldy + n] = y;
    else
      static_cast<T*>(a.y)[row * a.ldy + n] = Vec8<T>::narrow(y);
  }
};
template <typename T, int kGroup, bool kPair, int kM, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void q4_product_kernel(Args a) {
  extern __shared__ __align__(16) uint8_t q_smem[];
  Kernel<T, kGroup, kPair, kM, kWaves> k;
  k.run(a, q_smem);
}

template <typename T, int kGroup, bool kPair, int kM, int kWaves>
hipError_t launch_one(Args a, hipStream_t s) {
  constexpr int lds = Kernel<T, kGroup, kPair, kM, kWaves>::kLds;
  static std::atomic<uint64_t> done;
  if (const hipError_t e = tile::allow_lds(done, q4_product_kernel<T, kGroup, kPair, kM, kWaves>, lds); e != hipSuccess) return e;
  return launch_in_parts((a.N + kTileN - 1) / kTileN, [&](int64_t first, uint32_t blocks) {
    a.first = first;
    const uint32_t grid = (blocks + tile::kXcds - 1) / tile::kXcds * tile::kXcds;
    q4_product_kernel<T, kGroup, kPair, kM, kWaves><<<grid, 64 * kWaves, lds, s>>>(a);
  });
}
// A unit holds 16 waves of these: one block of 16, or two of 8 where there are more blocks than units, which then begin and
// end at different times (us, 16 waves / 8: 4096 x 11008 7.9 / 10.1, the pair of 11008 x 4096 14.8 / 10.9). Of 2 to 4
// rows in groups of 32 and 64, not the pair, the 96 and 80 KB of LDS leave room for one block of 8; neither side
// wins there (4 rows, group 32: 11008 x 4096 15.3 / 14.2, 13824 x 5120 21.3 / 22.1, 28672 x 8192 51.3 / 49.1; group 64: 13.5 / 12.6,
// 18.5 / 19.9, 42.3 / 43.4; in chunks of 6144 columns, of which two blocks fit, 8 waves take 13.5, 20.0, 49.7 and 12.4,
// 18.4, 46.0), so the rule is the same.
template <typename T, int kGroup, bool kPair, int kM>
hipError_t launch_waves(const Args& a, hipStream_t s) {
  return (a.N + kTileN - 1) / kTileN <= tile::kUnits ? launch_one<T, kGroup, kPair, kM, 16>(a, s)
                                                     : launch_one<T, kGroup, kPair, kM, 8>(a, s);
}
template <typename T, int kGroup, bool kPair>
hipError_t launch_rows_of(const Args& a, hipStream_t s) {
  return a.M == 1 ? launch_waves<T, kGroup, kPair, 1>(a, s)
         : a.M <= 4 ? launch_waves<T, kGroup, kPair, 4>(a, s) : launch_one<T, kGroup, kPair, 16, 16>(a, s);
}
template <typename T, bool kPair>
hipError_t launch_group(const Args& a, int group, hipStream_t s) {
  return group == 32 ? launch_rows_of<T, 32, kPair>(a, s)
         : group == 64 ? launch_rows_of<T, 64, kPair>(a, s) : launch_rows_of<T, 128, kPair>(a, s);
}

}  // namespace
}  // namespace q4
}  // namespace rb
