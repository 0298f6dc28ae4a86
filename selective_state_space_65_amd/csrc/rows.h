// rows.h -- loads and stores of consecutive elements of a row whose start need
// only be element-aligned (rows of an odd length start anywhere).  The target
// takes vector accesses at any element alignment, so a whole piece is one
// 16-byte access (two for 8 fp32 values) whatever the row's length; a piece
// that ends past the row is read and written element by element.  Internal:
// not part of the C ABI.
#pragma once

#include "device_common.h"

namespace {

typedef uint32_t words2 __attribute__((ext_vector_type(2)));
typedef uint32_t words4 __attribute__((ext_vector_type(4)));

// 8 bytes at any address.
__device__ __forceinline__ void load_bytes8(const uint8_t* p, uint32_t* lo, uint32_t* hi) {
  words2 w;
  __builtin_memcpy(&w, p, 8);
  *lo = w.x;
  *hi = w.y;
}

__device__ __forceinline__ void load8u(const float* p, float out[8]) {
  words4 a, b;
  __builtin_memcpy(&a, p, 16);
  __builtin_memcpy(&b, p + 4, 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    out[j] = __uint_as_float(a[j]);
    out[4 + j] = __uint_as_float(b[j]);
  }
}

__device__ __forceinline__ void load8u(const bf16_t* p, float out[8]) {
  words4 a;
  __builtin_memcpy(&a, p, 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    out[2 * j] = bf16_lo(a[j]);
    out[2 * j + 1] = bf16_hi(a[j]);
  }
}

__device__ __forceinline__ void store8u(float* p, const float v[8]) {
  words4 a, b;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a[j] = __float_as_uint(v[j]);
    b[j] = __float_as_uint(v[4 + j]);
  }
  __builtin_memcpy(p, &a, 16);
  __builtin_memcpy(p + 4, &b, 16);
}

__device__ __forceinline__ void store8u(bf16_t* p, const float v[8]) {
  words4 a;
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = Io<bf16_t>::pack2(v[2 * j], v[2 * j + 1]);
  __builtin_memcpy(p, &a, 16);
}

// Elements [t, t + 8) of a row of n; full: t + 8 <= n for the whole wave.
// Elements past the row read as 0 and are not written.
template <typename T>
__device__ __forceinline__ void load_row8(const T* row, int t, int n, bool full, float out[8]) {
  if (full) {
    load8u(row + t, out);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = t + j < n ? Io<T>::load1(row + t + j) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store_row8(T* row, int t, int n, bool full, const float v[8]) {
  if (full) {
    store8u(row + t, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (t + j < n) Io<T>::store1(row + t + j, v[j]);
  }
}

// N (1 or 4) elements.
template <int N>
__device__ __forceinline__ void load_n(const float* p, float* out) {
  __builtin_memcpy(out, p, 4 * N);
}

template <int N>
__device__ __forceinline__ void load_n(const bf16_t* p, float* out) {
  if constexpr (N == 1) {
    out[0] = Io<bf16_t>::load1(p);
  } else {
    words2 w;
    __builtin_memcpy(&w, p, 8);
    out[0] = bf16_lo(w.x);
    out[1] = bf16_hi(w.x);
    out[2] = bf16_lo(w.y);
    out[3] = bf16_hi(w.y);
  }
}

template <int N>
__device__ __forceinline__ void store_n(float* p, const float* v) {
  __builtin_memcpy(p, v, 4 * N);
}

template <int N>
__device__ __forceinline__ void store_n(bf16_t* p, const float* v) {
  if constexpr (N == 1) {
    Io<bf16_t>::store1(p, v[0]);
  } else {
    words2 w;
    w.x = Io<bf16_t>::pack2(v[0], v[1]);
    w.y = Io<bf16_t>::pack2(v[2], v[3]);
    __builtin_memcpy(p, &w, 8);
  }
}

}  // namespace
