// rb_q4.hip -- 4-bit weights with group scales: packing, reading back, and products for decode batches.
//
//   W[n][c] ~ s (q - 8), or s q + z with offsets;  q = 0 .. 15, one s (and z) per row and `group` columns
//   y = W x,  or the gated pair y = act(Wg x) (.) (Wu x),  for up to 16 rows x
//
// The codes lie in tiles of 16 weight rows by 128 columns, 1 KB each, as the matrix instructions' fragments take them:
// lane 16 j + r of a tile holds row r; its word i holds columns 32 i + 8 j .. + 7, column c of those in the four bits
// from 16 (c % 2) + 4 (c / 2) on, so that a shift and a mask leave columns 2 p and 2 p + 1 in the halves of a register.
//
// Kernels of this file: q4_pack_kernel, q4_dequant_kernel (a wave per tile). The products: rb_q4_product.hpp.
#include "rb_elem.hpp"
#include "rb_q4_product.hpp"

namespace rb {
namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
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

// Bound by HBM: the codes and scales are an eighth of what is read (4096 x 11008 fp32: 42 to 74 us traced; with the reading back
// into bf16, 22 us, 71 for both). Lanes of a row are 16 apart, so a group's extremes take two exchanges.
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
  const q4::Args a{{{codes, half_of(s), half_of(z)}, {codes2, half_of(s2), half_of(z2)}}, x, y, ldx, ldy, N, 0, (int)M, (int)K,
                 (int)((K + kTileK - 1) / kTileK), act, y_dtype == RB_F32};
  return x_dtype == RB_F16 ? q4::launch_f16(a, group, codes2 != nullptr, stream) : q4::launch_bf16(a, group, codes2 != nullptr, stream);
}

}  // namespace rb
