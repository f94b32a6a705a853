// rb_elem.hpp -- 8 consecutive elements of a row in registers, for rows of any alignment.
#pragma once

#include "rb_device.hpp"

namespace rb {

// The storage types of activations and streams. 8 elements are moved by 16-byte accesses whatever
// the row's alignment (gfx950 global accesses need none beyond the element's) and stay packed, two
// 16-bit elements a register, until they are widened.
template <typename T> struct Vec8;

typedef uint32_t u4_by4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4_by2 __attribute__((ext_vector_type(4), aligned(2)));

template <> struct Vec8<float> {
  typedef u4_by4 U4;  // 16 bytes at an element's alignment
  struct __attribute__((packed, aligned(4))) Raw { uint32_t w[8]; };
  __device__ static __forceinline__ float get(const Raw& r, int j) { return __uint_as_float(r.w[j]); }
  __device__ static __forceinline__ void set2(Raw& r, int j, float a, float b) {
    r.w[j] = __float_as_uint(a), r.w[j + 1] = __float_as_uint(b);
  }
  __device__ static __forceinline__ float narrow(float v) { return v; }
};
template <> struct Vec8<_Float16> {
  typedef u4_by2 U4;
  struct __attribute__((packed, aligned(2))) Raw { uint32_t w[4]; };
  __device__ static __forceinline__ float get(const Raw& r, int j) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(r.w[j >> 1] >> (16 * (j & 1))));
  }
  __device__ static __forceinline__ void set2(Raw& r, int j, float a, float b) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    r.w[j >> 1] = __builtin_bit_cast(uint32_t, (h2){(_Float16)a, (_Float16)b});
  }
  __device__ static __forceinline__ _Float16 narrow(float v) { return (_Float16)v; }
};
template <> struct Vec8<__bf16> {
  typedef u4_by2 U4;
  struct __attribute__((packed, aligned(2))) Raw { uint32_t w[4]; };
  __device__ static __forceinline__ float get(const Raw& r, int j) {
    return __uint_as_float(j & 1 ? r.w[j >> 1] & 0xffff0000u : r.w[j >> 1] << 16);
  }
  __device__ static __forceinline__ void set2(Raw& r, int j, float a, float b) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    r.w[j >> 1] = __builtin_bit_cast(uint32_t, (b2){(__bf16)a, (__bf16)b});
  }
  __device__ static __forceinline__ __bf16 narrow(float v) { return (__bf16)v; }
};

// 8 elements to any address of their type. NT marks the store as streamed (non-temporal): it leaves the
// caches to what is read. A norm over 2048 x 4096 takes 18.9 us with the mark and 23.7 without, its backward
// 35.9 / 37.0, the activation's 30.0 / 32.0; the product that reads the result next takes the same time
// either way. (Marked loads: no gain.)
template <bool NT, typename T>
__device__ __forceinline__ void put8(T* p, const typename Vec8<T>::Raw& r) {
  if constexpr (NT) {
    typedef typename Vec8<T>::U4 u4;
#pragma unroll
    for (int k = 0; k < (int)sizeof(r) / 16; ++k)
      __builtin_nontemporal_store((u4){r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]},
                                  reinterpret_cast<u4*>(p) + k);
  } else {
    *reinterpret_cast<typename Vec8<T>::Raw*>(p) = r;
  }
}

// elements c .. c+7 of a row of n; those past n read as 0
template <typename T>
__device__ __forceinline__ typename Vec8<T>::Raw load8(const T* row, int c, int n) {
  typename Vec8<T>::Raw r;
  if (c + 8 <= n) {
    r = *reinterpret_cast<const typename Vec8<T>::Raw*>(row + c);
  } else {
    const T zero = Vec8<T>::narrow(0.f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const T a = c + j < n ? row[c + j] : zero, b = c + j + 1 < n ? row[c + j + 1] : zero;
      Vec8<T>::set2(r, j, (float)a, (float)b);  // widened and narrowed again: the same value
    }
  }
  return r;
}
// The same for a uniform n of 8 or more, without element loads: the vector that holds the end of the
// row is read 8 elements before it and, when it is used, shifted down by the (uniform) rest.
__device__ __forceinline__ void shift_down(Vec8<float>::Raw& r, int by) {
#pragma unroll
  for (int bit = 4; bit >= 1; bit >>= 1)
    if (by & bit) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.w[i] = i + bit < 8 ? r.w[i + bit] : 0u;
    }
}
template <typename Raw>
__device__ __forceinline__ void shift_down(Raw& r, int by) {
#pragma unroll
  for (int bit = 4; bit >= 2; bit >>= 1)
    if (by & bit) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = i + bit / 2 < 4 ? r.w[i + bit / 2] : 0u;
    }
  if (by & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = (r.w[i] >> 16) | (i < 3 ? r.w[i + 1] << 16 : 0u);
  }
}
// elements c .. c+7 into r, or the row's last 8 where those pass its end (to be shifted down by
// c + 8 - n before use); r is left alone from n on
template <typename T>
__device__ __forceinline__ void load8_long(typename Vec8<T>::Raw& r, const T* row, int c, int n) {
  if (c < n) r = *reinterpret_cast<const typename Vec8<T>::Raw*>(row + (c + 8 <= n ? c : n - 8));
}
// load8 for a uniform n: one wide load where n is 8 or more (an element load would hold up the wave)
template <typename T>
__device__ __forceinline__ typename Vec8<T>::Raw load8_any(const T* row, int c, int n) {
  if (n < 8) return load8<T>(row, c, n);
  typename Vec8<T>::Raw r = {};
  load8_long<T>(r, row, c, n);
  if (c < n && c + 8 > n) shift_down(r, c + 8 - n);
  return r;
}
template <typename T, bool NT = false>
__device__ __forceinline__ void store8(T* row, int c, int n, const float (&v)[8]) {
  if (c + 8 <= n) {
    typename Vec8<T>::Raw r;
#pragma unroll
    for (int j = 0; j < 8; j += 2) Vec8<T>::set2(r, j, v[j], v[j + 1]);
    put8<NT, T>(row + c, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < n) row[c + j] = Vec8<T>::narrow(v[j]);
  }
}
template <typename T>
__device__ __forceinline__ void widen8(const typename Vec8<T>::Raw& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = Vec8<T>::get(r, j);
}

}  // namespace rb
