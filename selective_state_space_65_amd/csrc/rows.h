// rows.h -- loads and stores of consecutive elements of a row whose start need
// only be element-aligned (rows of an odd length start anywhere).  The target
// takes vector accesses at any element alignment, so a whole piece is one
// 16-byte access (two for 8 fp32 values) whatever the row's length.  A piece
// that ends past the row is read as the row's last 8 elements, shifted into
// place, so that no lane reads past the row and none takes a loop of its own.
// Internal: not part of the C ABI.
#pragma once

#include "device_common.h"

namespace {

typedef uint32_t words2 __attribute__((ext_vector_type(2)));
typedef uint32_t words4 __attribute__((ext_vector_type(4)));
typedef words4 words4_any __attribute__((aligned(2), may_alias));

// 8 bytes at any address.
__device__ __forceinline__ void load_bytes8(const uint8_t* p, uint32_t* lo, uint32_t* hi) {
  words2 w;
  __builtin_memcpy(&w, p, 8);
  *lo = w.x;
  *hi = w.y;
}

// One 16-byte access at any element address.  kStream: the line is read or
// written once and not wanted again soon (non-temporal), so that it does not
// push out what other waves still read.
template <bool kStream>
__device__ __forceinline__ words4 load16(const void* p) {
  if constexpr (kStream) return __builtin_nontemporal_load(static_cast<const words4_any*>(p));
  return *static_cast<const words4_any*>(p);
}

template <bool kStream>
__device__ __forceinline__ void store16(void* p, words4 v) {
  if constexpr (kStream)
    __builtin_nontemporal_store(v, static_cast<words4_any*>(p));
  else
    *static_cast<words4_any*>(p) = v;
}

// 8 consecutive elements as they are in memory: loaded ahead of their use in
// half the registers that 8 fp32 values take when the elements are bf16.
template <typename T>
struct Raw8;

template <>
struct Raw8<float> {
  words4 lo, hi;
  template <bool kStream>
  __device__ __forceinline__ void load(const float* p) {
    lo = load16<kStream>(p);
    hi = load16<kStream>(p + 4);
  }
  __device__ __forceinline__ void load_part(const float* row, int t, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) (j < 4 ? lo : hi)[j & 3] = t + j < n ? __float_as_uint(row[t + j]) : 0u;
  }
  __device__ __forceinline__ void clear() { lo = hi = words4{0, 0, 0, 0}; }
  // Elements s.. move to the front, zeros follow.
  __device__ __forceinline__ void drop(int s) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = lo[j], v[4 + j] = hi[j];
    shift_words<4>(v, s & 4);
    shift_words<2>(v, s & 2);
    shift_words<1>(v, s & 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = s < 8 ? v[j] : 0u;
      hi[j] = s < 8 ? v[4 + j] : 0u;
    }
  }
  template <int n>
  static __device__ __forceinline__ void shift_words(uint32_t v[8], int on) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = on ? (j + n < 8 ? v[j + n] : 0u) : v[j];
  }
  __device__ __forceinline__ void get(float out[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[j] = __uint_as_float(lo[j]);
      out[4 + j] = __uint_as_float(hi[j]);
    }
  }
};

template <>
struct Raw8<bf16_t> {
  words4 w;
  template <bool kStream>
  __device__ __forceinline__ void load(const bf16_t* p) {
    w = load16<kStream>(p);
  }
  __device__ __forceinline__ void load_part(const bf16_t* row, int t, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = t + 2 * j < n ? row[t + 2 * j] : 0u;
      const uint32_t hi = t + 2 * j + 1 < n ? row[t + 2 * j + 1] : 0u;
      w[j] = lo | hi << 16;
    }
  }
  __device__ __forceinline__ void clear() { w = words4{0, 0, 0, 0}; }
  // Elements s.. move to the front, zeros follow.
  __device__ __forceinline__ void drop(int s) {
    uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    if (s & 4) a = c, b = d, c = 0, d = 0;
    if (s & 2) a = b, b = c, c = d, d = 0;
    if (s & 1) a = a >> 16 | b << 16, b = b >> 16 | c << 16, c = c >> 16 | d << 16, d >>= 16;
    w = s < 8 ? words4{a, b, c, d} : words4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void get(float out[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[2 * j] = bf16_lo(w[j]);
      out[2 * j + 1] = bf16_hi(w[j]);
    }
  }
};

template <bool kStream>
__device__ __forceinline__ void store8u(float* p, const float v[8]) {
  words4 a, b;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a[j] = __float_as_uint(v[j]);
    b[j] = __float_as_uint(v[4 + j]);
  }
  store16<kStream>(p, a);
  store16<kStream>(p + 4, b);
}

template <bool kStream>
__device__ __forceinline__ void store8u(bf16_t* p, const float v[8]) {
  words4 a;
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = Io<bf16_t>::pack2(v[2 * j], v[2 * j + 1]);
  store16<kStream>(p, a);
}

// Elements [t0 + l, t0 + l + 8) of a row of n, t0 the same in every lane of the
// row and l >= 0, in two steps, so that several pieces can be in flight before
// the first is touched: request8 loads the piece, or the row's last 8 elements
// where the piece ends past the row; finish8, needed where some lane's piece
// does, shifts those into place.  Elements past the row read as 0.  The loads
// are unconditional: a branch here would have its loads waited for where the
// branches join.  kShort: n may be below 8, and such a row is read element by
// element.
struct Place {
  int base;      // of the lanes' row
  uint32_t off;  // of the lane, so that a scalar base and a 32-bit offset address it
};

__device__ __forceinline__ Place place8(int t0, int l, int n) {
  Place p;
  p.base = min(t0, n - 8);
  p.off = (uint32_t)min(l, n - 8 - p.base);
  return p;
}

template <bool kShort, bool kStream = false, typename T>
__device__ __forceinline__ Raw8<T> request8(const T* row, int t0, int l, int n) {
  Raw8<T> r;
  if (kShort && n < 8) {
    r.load_part(row, t0 + l, n);
  } else {
    const Place p = place8(t0, l, n);
    r.template load<kStream>(row + p.base + p.off);
  }
  return r;
}

template <bool kShort, typename T>
__device__ __forceinline__ void finish8(Raw8<T>& r, int t0, int l, int n) {
  if (kShort && n < 8) return;
  const Place p = place8(t0, l, n);
  const int s = t0 - p.base + l - (int)p.off;
  if (n % 8)
    r.drop(s);
  else if (s)  // pieces are whole or empty
    r.clear();
}

// Elements past the row are not written; full: no lane has any.
template <bool kStream = false, typename T>
__device__ __forceinline__ void store_row8(T* row, int t, int n, bool full, const float v[8]) {
  if (full || t + 8 <= n) {
    store8u<kStream>(row + t, v);
  } else if (t < n) {
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
