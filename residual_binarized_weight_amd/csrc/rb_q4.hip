// rb_q4.hip -- 4-bit weights with group scales: packing, reading back, and products for decode batches.
//
//   W[n][c] ~ s (q - 8), or s q + z with offsets;  q = 0 .. 15, one s (and z) per row and `group` columns
//   y = W x,  or the gated pair y = act(Wg x) (.) (Wu x),  for up to 16 rows x
//
// The codes lie in tiles of 16 weight rows by 128 columns, 1 KB each, as the matrix instructions' fragments take them:
// lane 16 j + r of a tile holds row r; its word i holds columns 32 i + 8 j .. + 7, column c of those in the four bits
// from 16 (c % 2) + 4 (c / 2) on, so that a shift and a mask leave columns 2 p and 2 p + 1 in the halves of a register.
//
// Kernels of this file: q4_pack_kernel, q4_dequant_kernel (a wave per tile), q4_product_kernel.
#include "rb_act.hpp"
#include "rb_internal.h"
#include "rb_tile.hpp"

namespace rb {
namespace {

using tile::f4;
using tile::u4;

constexpr int kTileN = 16, kTileK = 128;

// ---------------------------------------------------------------------------------------------
// packing and reading back: a wave per tile, lane 16 j + r with 4 x 8 columns of row r
// ---------------------------------------------------------------------------------------------
struct PackArgs {
  const void* W;
  int64_t N, K, ldw, first, all, steps;  // tiles: the launch's first, the end, and those of a row of tiles
  uint32_t* codes;
  _Float16 *s, *z;
  int32_t* status;
};

template <typename TW, int kGroup>
__global__ __launch_bounds__(256) void q4_pack_kernel(PackArgs a) {
  const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
  const int64_t t = (a.first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (t >= a.all) return;
  const int64_t n = t / a.steps * kTileN + r, c0 = t % a.steps * kTileK;
  const int K = (int)(a.K - c0 < kTileK ? a.K - c0 : kTileK);  // the tile's columns that lie inside
  const bool in = n < a.N;
  const TW* const row = static_cast<const TW*>(a.W) + (in ? n : a.N - 1) * a.ldw + c0;
  float w[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) widen8<TW>(load8<TW>(row, 32 * i + 8 * j, K), w[i]);
  u4 words = {0, 0, 0, 0};
  bool bad = false;
  constexpr int kEach = kGroup / 32;  // words of a group
#pragma unroll
  for (int g = 0; g < 4 / kEach; ++g) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = g * kEach; i < (g + 1) * kEach; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (32 * i + 8 * j + e < K) {
          lo = fminf(lo, w[i][e]), hi = fmaxf(hi, w[i][e]);
          bad = bad || !(fabsf(w[i][e]) < INFINITY);
        }
#pragma unroll
    for (int m = 16; m <= 32; m <<= 1) {
      lo = fminf(lo, __shfl_xor(lo, m, RB_WAVE));
      hi = fmaxf(hi, __shfl_xor(hi, m, RB_WAVE));
    }
    // each step in fp32, the scale and the offset rounded to fp16 before they are used
    _Float16 z = 0, s;
    if (a.z) {
      z = (_Float16)lo;
      s = (_Float16)((hi - lo) * (1.f / 15.f));
    } else {
      s = (_Float16)(fmaxf(fabsf(lo), fabsf(hi)) * (1.f / 7.f));
    }
    const float sf = (float)s, zf = (float)z;
    const bool inside = 32 * g * kEach < K;
    bad = bad || (inside && !(sf < INFINITY && fabsf(zf) < INFINITY));
#pragma unroll
    for (int i = g * kEach; i < (g + 1) * kEach; ++i) {
      uint32_t word = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = sf > 0.f ? rintf((w[i][e] - zf) / sf) : 0.f;
        const uint32_t code = a.z ? (uint32_t)(int)fminf(fmaxf(q, 0.f), 15.f) : (uint32_t)((int)fminf(fmaxf(q, -8.f), 7.f) + 8);
        word |= (32 * i + 8 * j + e < K && in ? code : 0u) << (16 * (e & 1) + 4 * (e >> 1));
      }
      words[i] = word;
    }
    if (j == 0 && in && inside) {
      const int64_t at = (c0 / kGroup + g) * a.N + n;
      a.s[at] = s;
      if (a.z) a.z[at] = z;
    }
  }
  *reinterpret_cast<u4*>(a.codes + (t * 64 + lane) * 4) = words;
  if (a.status && bad && in) atomicOr(a.status, 1);
}

struct DequantArgs {
  const uint32_t* codes;
  const _Float16 *s, *z;
  void* W;
  int64_t N, K, ldw, first, all, steps;
  int group;
};
template <typename TW>
__global__ __launch_bounds__(256) void q4_dequant_kernel(DequantArgs a) {
  const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
  const int64_t t = (a.first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (t >= a.all) return;
  const int64_t n = t / a.steps * kTileN + r, c0 = t % a.steps * kTileK;
  const int K = (int)(a.K - c0 < kTileK ? a.K - c0 : kTileK);
  if (n >= a.N) return;
  const u4 words = *reinterpret_cast<const u4*>(a.codes + (t * 64 + lane) * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = 32 * i + 8 * j;
    if (c >= K) break;
    const int64_t at = (c0 + c) / a.group * a.N + n;
    const float s = (float)a.s[at], z = a.z ? (float)a.z[at] : -8.f * s;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(s, (float)(words[i] >> (16 * (e & 1) + 4 * (e >> 1)) & 15u), z);
    store8<TW>(static_cast<TW*>(a.W) + n * a.ldw + c0, c, K, v);
  }
}

// ---------------------------------------------------------------------------------------------
// the product: a block owns 16 weight rows (of both weights of a pair); its 8 waves take the 128-column tiles in turn
// and join in LDS in their order. HBM's rate for the codes is the bound. A code becomes a number of the activations'
// type without arithmetic: in the top four fraction bits above 16, it reads 16 + q. So a group's sum of products is
// s (D - 24 S), or s D + (z - 16 s) S with offsets, with D the matrix instructions' sum over 16 + q and S the sum of the
// group's x, which an instruction with ones for weights gives in the same lanes. All sums are fp32; 16 + q against
// q - 8 costs about two bits of them.
// ---------------------------------------------------------------------------------------------
struct Q4Weights {
  const uint32_t* codes;
  const _Float16 *s, *z;
};
struct Q4Args {
  Q4Weights w[2];
  const void* x;
  void* y;
  int64_t ldx, ldy, N, first;
  int M, K, steps, act;
};

template <typename T> struct Nib;
template <> struct Nib<_Float16> {  // 16 + q: 0x4c00 with q in bits 9 .. 6
  static constexpr uint32_t kOne = 0x3c003c00u;
  __device__ static __forceinline__ u4 widen(uint32_t w) {
    const uint32_t m = 0x03c003c0u, b = 0x4c004c00u;
    return (u4){(w << 6 & m) | b, (w << 2 & m) | b, (w >> 2 & m) | b, (w >> 6 & m) | b};
  }
};
template <> struct Nib<__bf16> {  // 16 + q: 0x4180 with q in bits 6 .. 3
  static constexpr uint32_t kOne = 0x3f803f80u;
  __device__ static __forceinline__ u4 widen(uint32_t w) {
    const uint32_t m = 0x00780078u, b = 0x41804180u;
    return (u4){(w << 3 & m) | b, (w >> 1 & m) | b, (w >> 5 & m) | b, (w >> 9 & m) | b};
  }
};

// four rows' scales, n .. n + 3, of a group
__device__ __forceinline__ f4 scales4(const _Float16* s, int64_t n, int64_t N) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
  typedef _Float16 q4 __attribute__((ext_vector_type(4)));
  if (n + 4 <= N) {
    const u2 v = *reinterpret_cast<const u2*>(s + n);
    const q4 h = __builtin_bit_cast(q4, v);
    return (f4){(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
  }
  f4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)s[n + e < N ? n + e : N - 1];  // a row past the last one repeats it
  return v;
}

template <typename T, typename TY, int kGroup, bool kPair>
__global__ __launch_bounds__(512) void q4_product_kernel(Q4Args a) {
  constexpr int kWaves = 8, kAhead = 2, kMat = kPair ? 2 : 1;
  constexpr int kGroups = kTileK / kGroup, kEach = kGroup / 32;
  __shared__ __align__(16) float sums[kMat][kWaves][256];
  const int lane = threadIdx.x & 63, lr = lane & 15, lj = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t tile_n = a.first + blockIdx.x, n0 = tile_n * kTileN;
  const T* const x = static_cast<const T*>(a.x) + (lr < a.M ? lr : 0) * a.ldx;
  f4 total[kMat];
#pragma unroll
  for (int q = 0; q < kMat; ++q) total[q] = (f4){0.f, 0.f, 0.f, 0.f};
  const u4 ones = {Nib<T>::kOne, Nib<T>::kOne, Nib<T>::kOne, Nib<T>::kOne};
  for (int k0 = w; k0 < a.steps; k0 += kWaves * kAhead) {
    u4 code[kAhead][kMat];
    u4 xf[kAhead][4];
    f4 s[kAhead][kMat][kGroups], z[kAhead][kMat][kGroups];
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      const int k = k0 + p * kWaves;
      if (k >= a.steps) break;
#pragma unroll
      for (int q = 0; q < kMat; ++q) {
        code[p][q] = *reinterpret_cast<const u4*>(a.w[q].codes + ((tile_n * a.steps + k) * 64 + lane) * 4);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          // the last tile's groups past the columns repeat the last one: their x are zero
          const int64_t groups = (a.K + kGroup - 1) / kGroup, at = (int64_t)k * kGroups + g;
          const int64_t off = (at < groups ? at : groups - 1) * a.N;
          s[p][q][g] = scales4(a.w[q].s + off, n0 + 4 * lj, a.N);
          if (a.w[q].z) z[p][q][g] = scales4(a.w[q].z + off, n0 + 4 * lj, a.N);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xf[p][i] = lr < a.M ? __builtin_bit_cast(u4, load8_any<T>(x, k * kTileK + 32 * i + 8 * lj, a.K)) : (u4){0, 0, 0, 0};
    }
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      if (k0 + p * kWaves >= a.steps) break;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f4 d[kMat], xs = (f4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kMat; ++q) d[q] = (f4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = g * kEach; i < (g + 1) * kEach; ++i) {
          xs = tile::mfma(T(0), ones, xf[p][i], xs);
#pragma unroll
          for (int q = 0; q < kMat; ++q) d[q] = tile::mfma(T(0), Nib<T>::widen(code[p][q][i]), xf[p][i], d[q]);
        }
#pragma unroll
        for (int q = 0; q < kMat; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float sc = s[p][q][g][e];
            const float off = a.w[q].z ? z[p][q][g][e] - 16.f * sc : -24.f * sc;
            total[q][e] = fmaf(sc, d[q][e], fmaf(off, xs[e], total[q][e]));
          }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kMat; ++q) *reinterpret_cast<f4*>(&sums[q][w][lane * 4]) = total[q];
  __syncthreads();
  // thread 16 m + n: D's lane 16 (n / 4) + m holds weight row n in element n % 4
  if (threadIdx.x >= 256) return;
  const int m = threadIdx.x >> 4, nn = threadIdx.x & 15;
  const int64_t n = n0 + nn;
  if (m >= a.M || n >= a.N) return;
  float v[kMat];
#pragma unroll
  for (int q = 0; q < kMat; ++q) {
    v[q] = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v[q] += sums[q][i][((nn >> 2) * 16 + m) * 4 + (nn & 3)];
  }
  static_cast<TY*>(a.y)[m * a.ldy + n] = Vec8<TY>::narrow(kPair ? act_value(v[0], a.act) * v[kMat - 1] : v[0]);
}

template <typename T, typename TY, bool kPair>
hipError_t launch_grouped(Q4Args a, int group, hipStream_t s) {
  return launch_in_parts((a.N + kTileN - 1) / kTileN, [&](int64_t first, uint32_t blocks) {
    a.first = first;
    if (group == 32)
      q4_product_kernel<T, TY, 32, kPair><<<blocks, 512, 0, s>>>(a);
    else if (group == 64)
      q4_product_kernel<T, TY, 64, kPair><<<blocks, 512, 0, s>>>(a);
    else
      q4_product_kernel<T, TY, 128, kPair><<<blocks, 512, 0, s>>>(a);
  });
}
template <typename T>
hipError_t launch_typed(const Q4Args& a, int group, bool pair, rb_dtype y_dtype, hipStream_t s) {
  if (pair) return y_dtype == RB_F32 ? launch_grouped<T, float, true>(a, group, s) : launch_grouped<T, T, true>(a, group, s);
  return y_dtype == RB_F32 ? launch_grouped<T, float, false>(a, group, s) : launch_grouped<T, T, false>(a, group, s);
}

template <typename TW>
hipError_t launch_pack_typed(PackArgs a, int group, hipStream_t s) {
  return launch_in_parts((a.all + 3) / 4, [&](int64_t first, uint32_t blocks) {
    a.first = first;
    if (group == 32)
      q4_pack_kernel<TW, 32><<<blocks, 256, 0, s>>>(a);
    else if (group == 64)
      q4_pack_kernel<TW, 64><<<blocks, 256, 0, s>>>(a);
    else
      q4_pack_kernel<TW, 128><<<blocks, 256, 0, s>>>(a);
  });
}

}  // namespace

hipError_t launch_q4_pack(const void* W, rb_dtype w_dtype, int64_t N, int64_t K, int64_t ldw, int group, uint32_t* codes,
                          void* s, void* z, int32_t* status, hipStream_t stream) {
  const int64_t steps = (K + kTileK - 1) / kTileK, all = (N + kTileN - 1) / kTileN * steps;
  const PackArgs a{W, N, K, ldw, 0, all, steps, codes, static_cast<_Float16*>(s), static_cast<_Float16*>(z), status};
  switch (w_dtype) {
    case RB_F32: return launch_pack_typed<float>(a, group, stream);
    case RB_F16: return launch_pack_typed<_Float16>(a, group, stream);
    default: return launch_pack_typed<__bf16>(a, group, stream);
  }
}

hipError_t launch_q4_dequant(const uint32_t* codes, const void* s, const void* z, int64_t N, int64_t K, int group, void* W,
                             rb_dtype w_dtype, int64_t ldw, hipStream_t stream) {
  const int64_t steps = (K + kTileK - 1) / kTileK, all = (N + kTileN - 1) / kTileN * steps;
  DequantArgs a{codes, static_cast<const _Float16*>(s), static_cast<const _Float16*>(z), W, N, K, ldw, 0, all, steps, group};
  return launch_in_parts((all + 3) / 4, [&](int64_t first, uint32_t blocks) {
    a.first = first;
    if (w_dtype == RB_F32)
      q4_dequant_kernel<float><<<blocks, 256, 0, stream>>>(a);
    else if (w_dtype == RB_F16)
      q4_dequant_kernel<_Float16><<<blocks, 256, 0, stream>>>(a);
    else
      q4_dequant_kernel<__bf16><<<blocks, 256, 0, stream>>>(a);
  });
}

hipError_t launch_q4_product(const uint32_t* codes, const void* s, const void* z, const uint32_t* codes2, const void* s2,
                             const void* z2, int64_t N, int64_t K, int group, int act, const void* x, rb_dtype x_dtype,
                             int64_t M, int64_t ldx, void* y, rb_dtype y_dtype, int64_t ldy, hipStream_t stream) {
  const auto half_of = [](const void* p) { return static_cast<const _Float16*>(p); };
  const Q4Args a{{{codes, half_of(s), half_of(z)}, {codes2, half_of(s2), half_of(z2)}}, x, y, ldx, ldy, N, 0, (int)M, (int)K,
                 (int)((K + kTileK - 1) / kTileK), act};
  return x_dtype == RB_F16 ? launch_typed<_Float16>(a, group, codes2 != nullptr, y_dtype, stream)
                           : launch_typed<__bf16>(a, group, codes2 != nullptr, y_dtype, stream);
}

}  // namespace rb
