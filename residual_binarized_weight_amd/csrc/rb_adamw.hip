// rb_adamw.hip -- one optimizer step over many tensors in one launch, states in 32 or 8 bits.
//
//   g' = g grad_scale;  m <- b1 m + (1 - b1) g';  v <- b2 v + (1 - b2) g'^2;  r = sqrt(v)
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (r / sqrt(1 - b2^t) + eps)
//
// Every element is read and written once, so the step is bound by HBM: 28 bytes per element with
// fp32 parameters, gradients and states, 16 with 8-bit states. Measured over three 4096 x 11008
// weights and their scales (135 M elements): 621 us = 6.1 TB/s in 32 bits, 362 us = 6.0 TB/s in 8.
// 256 x 512 with its scales: 6.2 us, a launch and one element's chain of operations.
//
// Split. Tensors are cut into chunks of 4096 elements; a map of the chunks (one 32-bit tensor
// number each, 1/4000 of the traffic) lets one launch serve a 4096 x 11008 weight and its 4096
// row scales alike. A block of 4 waves owns a chunk, a wave 1024 elements of it as 4 groups of
// 256 (4 consecutive elements per lane, 16-byte accesses), and issues all its loads before the
// first use.
//
// 8-bit states. A group of 256 elements shares one scale for m and one for r (the root is held, it
// needs half the exponent range of v): the power of two above the group's largest magnitude, so
// scaling is exact and a state that does not change is stored unchanged. An element is an e4m3
// number, |x| / scale * 256. The 20 fraction bits that do not fit are rounded up with their own
// probability (16 random bits from a hash of seed, step and position): a step changes v by
// (1 - b2), far less than the 1/16 between neighbouring codes, and rounding to nearest would
// freeze it. A nonzero r keeps at least the smallest code, so that an element's m is never
// divided by eps alone because of the rounding.
#include "rb_device.hpp"
#include "rb_internal.h"

#include <cmath>

namespace rb {

namespace {

constexpr int kChunk = 4096;
constexpr int kThreads = 256;
constexpr int kGroup = 256;
constexpr int kPerWave = kChunk / (kThreads / 64);
constexpr int kGroups = kPerWave / kGroup;
constexpr uint32_t kMagic = 0x52424157u;

struct PlanHeader {
  uint32_t magic, bits;
  int64_t count, chunks, reserved[5];
};
struct PlanTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n, first_chunk;
  float lr_mult, weight_decay;
  uint16_t p_dtype, g_dtype;
  uint32_t vec;  // every 4-element access of the tensor is aligned to its size
};
static_assert(sizeof(PlanHeader) == 64 && sizeof(PlanTensor) == 80, "plan layout");

struct StepArgs {
  float beta1, one_beta1, beta2, one_beta2, step_size, lr, rsqrt_bc2, eps;
  uint32_t key;
};

// A bijective mix of 32-bit numbers; the factors are the fractions of the golden ratio and of
// the square root of two.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0x6A09E667u;
  x ^= x >> 16;
  return x;
}

template <typename T> struct Elem4;
// 16-byte accesses marked as streamed (non-temporal): each byte passes once a step, and a step over 45 M
// elements takes 207 us with the mark and 235 without (8-bit states: 115 / 139). Only one whose tensors fit
// the 256 MB cache and are touched by nothing else between two steps loses (8.4 M: 40 / 36 us).
typedef float f4 __attribute__((ext_vector_type(4)));
template <> struct Elem4<float> {
  __device__ static __forceinline__ float4 load(const float* p) {
    const f4 r = __builtin_nontemporal_load(reinterpret_cast<const f4*>(p));
    return make_float4(r[0], r[1], r[2], r[3]);
  }
  __device__ static __forceinline__ void store(float* p, float4 v) {
    __builtin_nontemporal_store((f4){v.x, v.y, v.z, v.w}, reinterpret_cast<f4*>(p));
  }
  __device__ static __forceinline__ float narrow(float v) { return v; }
};
template <> struct Elem4<__half> {
  __device__ static __forceinline__ float4 load(const __half* p) {
    const ushort4 u = *reinterpret_cast<const ushort4*>(p);
    return make_float4(to_f32(__ushort_as_half(u.x)), to_f32(__ushort_as_half(u.y)), to_f32(__ushort_as_half(u.z)),
                       to_f32(__ushort_as_half(u.w)));
  }
  __device__ static __forceinline__ __half narrow(float v) { return __float2half_rn(v); }
  __device__ static __forceinline__ void store(__half* p, float4 v) {
    ushort4 u;
    u.x = __half_as_ushort(narrow(v.x)), u.y = __half_as_ushort(narrow(v.y));
    u.z = __half_as_ushort(narrow(v.z)), u.w = __half_as_ushort(narrow(v.w));
    *reinterpret_cast<ushort4*>(p) = u;
  }
};
template <> struct Elem4<__hip_bfloat16> {
  __device__ static __forceinline__ float4 load(const __hip_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
  }
  __device__ static __forceinline__ __hip_bfloat16 narrow(float v) { return __float2bfloat16(v); }
  __device__ static __forceinline__ void store(__hip_bfloat16* p, float4 v) {
    ushort4 u;
    u.x = __bfloat16_as_ushort(narrow(v.x)), u.y = __bfloat16_as_ushort(narrow(v.y));
    u.z = __bfloat16_as_ushort(narrow(v.z)), u.w = __bfloat16_as_ushort(narrow(v.w));
    *reinterpret_cast<ushort4*>(p) = u;
  }
};

// 4 elements from e on; those past n read as 0 and are not written. FULL: all 4 are there and aligned.
template <bool FULL, typename T>
__device__ __forceinline__ float4 get4(const void* base, int64_t e, int64_t n, bool vec) {
  const T* p = static_cast<const T*>(base) + e;
  if (FULL || (vec && e + 4 <= n)) return Elem4<T>::load(p);
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (e < n) r.x = to_f32(p[0]);
  if (e + 1 < n) r.y = to_f32(p[1]);
  if (e + 2 < n) r.z = to_f32(p[2]);
  if (e + 3 < n) r.w = to_f32(p[3]);
  return r;
}
template <bool FULL, typename T>
__device__ __forceinline__ void put4(void* base, int64_t e, int64_t n, bool vec, float4 v) {
  T* p = static_cast<T*>(base) + e;
  if (FULL || (vec && e + 4 <= n)) {
    Elem4<T>::store(p, v);
    return;
  }
  if (e < n) p[0] = Elem4<T>::narrow(v.x);
  if (e + 1 < n) p[1] = Elem4<T>::narrow(v.y);
  if (e + 2 < n) p[2] = Elem4<T>::narrow(v.z);
  if (e + 3 < n) p[3] = Elem4<T>::narrow(v.w);
}
template <bool FULL>
__device__ __forceinline__ uint32_t get4_codes(const void* base, int64_t e, int64_t n, bool vec) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + e;
  if (FULL || (vec && e + 4 <= n)) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t r = 0;
  for (int j = 0; j < 4; ++j)
    if (e + j < n) r |= (uint32_t)p[j] << (8 * j);
  return r;
}
template <bool FULL>
__device__ __forceinline__ void put4_codes(void* base, int64_t e, int64_t n, bool vec, uint32_t c) {
  uint8_t* p = static_cast<uint8_t*>(base) + e;
  if (FULL || (vec && e + 4 <= n)) {
    *reinterpret_cast<uint32_t*>(p) = c;
    return;
  }
  for (int j = 0; j < 4; ++j)
    if (e + j < n) p[j] = (uint8_t)(c >> (8 * j));
}

typedef float f2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float4 decode4(uint32_t c, float scale) {
  const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  const float s = 0x1p-8f * scale;  // a power of two: the products below are exact
  return make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
}

constexpr uint32_t kInf = 0x7f800000u;
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t finite_mag(float x) { return mag_bits(x) < kInf ? mag_bits(x) : 0u; }
// largest of the wave's non-negative values (as bits: the order is the same)
__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
#define RB_MAX_STEP(ctrl, rows) \
  { \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false); \
    v = v > o ? v : o; \
  }
  RB_MAX_STEP(0xB1, 0xF)   // quad [1,0,3,2]
  RB_MAX_STEP(0x4E, 0xF)   // quad [2,3,0,1]
  RB_MAX_STEP(0x141, 0xF)  // row_half_mirror
  RB_MAX_STEP(0x140, 0xF)  // row_mirror
  RB_MAX_STEP(0x142, 0xA)  // row_bcast:15
  RB_MAX_STEP(0x143, 0x8)  // row_bcast:31
#undef RB_MAX_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// bits of the scale of a group whose largest magnitude is top: the power of two above it, held
// within 2^-99 .. 2^126 so that its inverse is a normal number too
__device__ __forceinline__ uint32_t scale_bits(uint32_t top) {
  const uint32_t lo = (127u - 100u) << 23, hi = (127u + 125u) << 23;
  top = top < lo ? lo : (top > hi ? hi : top);
  return (top & 0x7f800000u) + 0x00800000u;
}
// |x| / scale * 256 as an e4m3 code: times 2^-120 its exponent field is the code's, and the code
// is the upper bits (numbers below 2^-6 become subnormal in both); 16 random bits over the 20 cut
// ones decide the rounding. ROOT: a nonzero x takes the smallest code at least.
// PLAIN: every x of the group is finite and below its scale, so the code is at most 0x78.
template <bool PLAIN, bool ROOT>
__device__ __forceinline__ uint32_t encode(float x, float inv, uint32_t rnd16) {
  const float y = (fabsf(x) * inv) * 0x1p-112f;
  uint32_t c = (__float_as_uint(y) + rnd16 * 16u + 8u) >> 20;
  if (ROOT) c = max(c, x != 0.f ? 1u : 0u);
  if (!PLAIN) {
    c = c > 0x7eu ? 0x7eu : c;
    if (mag_bits(x) >= kInf) c = 0x7fu;
  }
  return ROOT && PLAIN ? c : c | ((__float_as_uint(x) >> 24) & 0x80u);
}
// the codes and scale bits of the lane's 4 values; h0..h3 hold the random bits from bit `shift` on
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4(float x, float y, float z, float w, uint32_t h0, uint32_t h1, uint32_t h2,
                                            uint32_t h3, uint32_t& scale) {
  constexpr int shift = ROOT ? 16 : 0;
  const uint32_t top = wave_max_bits(max(max(mag_bits(x), mag_bits(y)), max(mag_bits(z), mag_bits(w))));
  const auto rnd = [](uint32_t h) { return ROOT ? h >> shift : h & 0xffffu; };
  if (top < (127u + 126u) << 23) {  // the whole group, so the branch is uniform
    scale = scale_bits(top);
    const float inv = __uint_as_float((254u << 23) - scale);
    return encode<true, ROOT>(x, inv, rnd(h0)) | encode<true, ROOT>(y, inv, rnd(h1)) << 8 |
           encode<true, ROOT>(z, inv, rnd(h2)) << 16 | encode<true, ROOT>(w, inv, rnd(h3)) << 24;
  }
  scale = scale_bits(wave_max_bits(max(max(finite_mag(x), finite_mag(y)), max(finite_mag(z), finite_mag(w)))));
  const float inv = __uint_as_float((254u << 23) - scale);
  return encode<false, ROOT>(x, inv, rnd(h0)) | encode<false, ROOT>(y, inv, rnd(h1)) << 8 |
         encode<false, ROOT>(z, inv, rnd(h2)) << 16 | encode<false, ROOT>(w, inv, rnd(h3)) << 24;
}

struct Updated {
  float p, m, v, r;
};
// The operations stand in the formula's order, each rounded once (no contraction), so that a
// plain fp32 evaluation gives the same bits and with them the same 8-bit codes. The quotient alone
// is a product with the hardware reciprocal (1 ulp): it enters p, whose own step is larger.
__device__ __forceinline__ Updated update(float p, float g, float m, float v, const StepArgs& a, float step_size,
                                          float decay) {
#pragma clang fp contract(off)
  Updated o;
  o.m = m * a.beta1 + g * a.one_beta1;
  o.v = v * a.beta2 + (g * g) * a.one_beta2;
  o.r = sqrtf(o.v);
  const float hat = o.m * __builtin_amdgcn_rcpf(o.r * a.rsqrt_bc2 + a.eps);
  o.p = p * decay - step_size * hat;
  return o;
}

template <int BITS, typename TP, typename TG, bool FULL>
__device__ __forceinline__ void wave_step(const PlanTensor& t, int64_t chunk, int wave, int64_t e0, const StepArgs& a, float gscale) {
  const int lane = threadIdx.x & 63;
  const bool vec = t.vec != 0;
  const float step_size = a.step_size * t.lr_mult;
  const float decay = 1.f - a.lr * t.lr_mult * t.weight_decay;
  float4 p[kGroups], g[kGroups], m[kGroups], v[kGroups];
  uint32_t mc[kGroups], vc[kGroups];
  float ms[kGroups], vs[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int64_t e = e0 + i * kGroup + lane * 4;
    g[i] = get4<FULL, TG>(t.g, e, t.n, vec);
    p[i] = get4<FULL, TP>(t.p, e, t.n, vec);
    if (BITS == 32) {
      m[i] = get4<FULL, float>(t.m, e, t.n, vec);
      v[i] = get4<FULL, float>(t.v, e, t.n, vec);
    } else {
      const int64_t row = (e0 >> 8) + i;
      const bool live = FULL || e0 + i * kGroup < t.n;
      mc[i] = get4_codes<FULL>(t.m, e, t.n, vec);
      vc[i] = get4_codes<FULL>(t.v, e, t.n, vec);
      ms[i] = live ? t.m_scale[row] : 1.f;
      vs[i] = live ? t.v_scale[row] : 1.f;
    }
  }
  uint32_t hash0 = 0;
  if (BITS == 8) {
    // positions count over the whole plan; a wave's 1024 lie in one span of 2^32
    const uint64_t pos = (uint64_t)chunk * kChunk + (uint64_t)(wave * kPerWave);
    hash0 = (uint32_t)pos + mix32((uint32_t)(pos >> 32) + a.key);
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int64_t e = e0 + i * kGroup + lane * 4;
    if (BITS == 8) {
      m[i] = decode4(mc[i], ms[i]);
      const float4 r = decode4(vc[i], vs[i]);
      v[i] = make_float4(r.x * r.x, r.y * r.y, r.z * r.z, r.w * r.w);
    }
    const Updated x = update(p[i].x, g[i].x * gscale, m[i].x, v[i].x, a, step_size, decay);
    const Updated y = update(p[i].y, g[i].y * gscale, m[i].y, v[i].y, a, step_size, decay);
    const Updated z = update(p[i].z, g[i].z * gscale, m[i].z, v[i].z, a, step_size, decay);
    const Updated w = update(p[i].w, g[i].w * gscale, m[i].w, v[i].w, a, step_size, decay);
    put4<FULL, TP>(t.p, e, t.n, vec, make_float4(x.p, y.p, z.p, w.p));
    if (BITS == 32) {
      put4<FULL, float>(t.m, e, t.n, vec, make_float4(x.m, y.m, z.m, w.m));
      put4<FULL, float>(t.v, e, t.n, vec, make_float4(x.v, y.v, z.v, w.v));
    } else {
      // elements past n were read as 0 and stay 0: they do not touch the group's scales
      const uint32_t h = hash0 + (uint32_t)(i * kGroup + lane * 4);
      const uint32_t h0 = mix32(h), h1 = mix32(h + 1u), h2 = mix32(h + 2u), h3 = mix32(h + 3u);
      uint32_t mb, vb;
      put4_codes<FULL>(t.m, e, t.n, vec, encode4<false>(x.m, y.m, z.m, w.m, h0, h1, h2, h3, mb));
      put4_codes<FULL>(t.v, e, t.n, vec, encode4<true>(x.r, y.r, z.r, w.r, h0, h1, h2, h3, vb));
      if (lane == 0 && (FULL || e0 + i * kGroup < t.n)) {
        t.m_scale[(e0 >> 8) + i] = __uint_as_float(mb);
        t.v_scale[(e0 >> 8) + i] = __uint_as_float(vb);
      }
    }
  }
}

template <int BITS, typename TP, typename TG>
__device__ __forceinline__ void chunk_step(const PlanTensor& t, int64_t chunk, const StepArgs& a, float gscale) {
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t e0 = (chunk - t.first_chunk) * kChunk + wave * kPerWave;
  if (t.vec && e0 + kPerWave <= t.n)  // all of the wave's elements, without a check at each
    wave_step<BITS, TP, TG, true>(t, chunk, wave, e0, a, gscale);
  else
    wave_step<BITS, TP, TG, false>(t, chunk, wave, e0, a, gscale);
}

template <int BITS>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const uint8_t* __restrict__ plan, StepArgs a,
                                                         const float* __restrict__ grad_scale,
                                                         const int32_t* __restrict__ skip) {
  const PlanHeader* h = reinterpret_cast<const PlanHeader*>(plan);
  const int64_t chunk = blockIdx.x;
  // an image of another kind, or fewer chunks than the caller says: nothing to do
  if (h->magic != kMagic || h->bits != BITS || chunk >= h->chunks) return;
  if (skip && *skip != 0) return;
  const PlanTensor* ts = reinterpret_cast<const PlanTensor*>(plan + sizeof(PlanHeader));
  const uint32_t* map = reinterpret_cast<const uint32_t*>(ts + h->count);
  const PlanTensor t = ts[map[chunk]];
  const float gscale = grad_scale ? *grad_scale : 1.f;
#define RB_CASE(P, G, TP, TG) \
  if (t.p_dtype == P && t.g_dtype == G) return chunk_step<BITS, TP, TG>(t, chunk, a, gscale)
  RB_CASE(RB_F32, RB_F32, float, float);
  RB_CASE(RB_F32, RB_F16, float, __half);
  RB_CASE(RB_F32, RB_BF16, float, __hip_bfloat16);
  RB_CASE(RB_F16, RB_F32, __half, float);
  RB_CASE(RB_F16, RB_F16, __half, __half);
  RB_CASE(RB_BF16, RB_F32, __hip_bfloat16, float);
  RB_CASE(RB_BF16, RB_BF16, __hip_bfloat16, __hip_bfloat16);
#undef RB_CASE
}

}  // namespace

int64_t adamw_chunks(const rb_adamw_tensor* t, int64_t count) {
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) n += t[i].n / kChunk + (t[i].n % kChunk != 0);
  return n;
}

size_t adamw_plan_bytes(const rb_adamw_tensor* t, int64_t count) {
  const size_t b = sizeof(PlanHeader) + (size_t)count * sizeof(PlanTensor) + (size_t)adamw_chunks(t, count) * 4u;
  return (b + 15) / 16 * 16;
}

void adamw_fill_plan(const rb_adamw_tensor* t, int64_t count, int state_bits, void* image) {
  PlanHeader* h = static_cast<PlanHeader*>(image);
  *h = PlanHeader{kMagic, (uint32_t)state_bits, count, adamw_chunks(t, count), {}};
  PlanTensor* ts = reinterpret_cast<PlanTensor*>(h + 1);
  uint32_t* map = reinterpret_cast<uint32_t*>(ts + count);
  int64_t chunk = 0;
  for (int64_t i = 0; i < count; ++i) {
    const auto fits = [](const void* p, int dt) {
      return (reinterpret_cast<uintptr_t>(p) & (dt == RB_F32 ? 15u : 7u)) == 0;
    };
    const auto state_fits = [&](const void* p) {
      return (reinterpret_cast<uintptr_t>(p) & (state_bits == 32 ? 15u : 3u)) == 0;
    };
    const bool vec = fits(t[i].p, t[i].p_dtype) && fits(t[i].g, t[i].g_dtype) && state_fits(t[i].m) && state_fits(t[i].v);
    ts[i] = PlanTensor{t[i].p, t[i].g, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale, t[i].n, chunk, t[i].lr_mult,
                       t[i].weight_decay, (uint16_t)t[i].p_dtype, (uint16_t)t[i].g_dtype, vec ? 1u : 0u};
    const int64_t end = chunk + t[i].n / kChunk + (t[i].n % kChunk != 0);
    for (; chunk < end; ++chunk) map[chunk] = (uint32_t)i;
  }
}

hipError_t launch_adamw_step(const void* plan, int64_t chunks, int state_bits, int64_t step, double lr, double beta1,
                             double beta2, double eps, const float* grad_scale, const int32_t* skip, uint32_t seed,
                             hipStream_t s) {
  if (chunks == 0) return hipSuccess;
  StepArgs a;
  a.beta1 = (float)beta1, a.one_beta1 = (float)(1.0 - beta1);
  a.beta2 = (float)beta2, a.one_beta2 = (float)(1.0 - beta2);
  a.lr = (float)lr, a.eps = (float)eps;
  a.step_size = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  a.rsqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  a.key = mix32(seed + (uint32_t)step * 0x9E3779B1u);
  const uint8_t* image = static_cast<const uint8_t*>(plan);
  if (state_bits == 32)
    adamw_kernel<32><<<dim3((uint32_t)chunks), kThreads, 0, s>>>(image, a, grad_scale, skip);
  else
    adamw_kernel<8><<<dim3((uint32_t)chunks), kThreads, 0, s>>>(image, a, grad_scale, skip);
  return hipGetLastError();
}

}  // namespace rb
