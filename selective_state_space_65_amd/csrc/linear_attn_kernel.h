// linear_attn_kernel.h -- the chunked linear-attention kernel, instantiated for
// one io type by each translation unit that includes it.  Internal.
//
// With g_t = log2 a_t and G its running sum, a chunk of C tokens takes
//   out_t   = sI e(G_t) q_t . S  +  sU sI sum_{s <= t} e(G_t - G_s) (q_t . k_s) v_s
//   S      <- e(G_C) S + sU sum_s e(G_C - G_s) k_s v_s^T,            e(x) = 2^x
// and a reverse pass (s >= t, chunks from the last to the first)
//   out_t   = sI e(G_C - G_t) q_t . S + sU sI sum_{s >= t} e(G_s - G_t) (q_t . k_s) v_s
//   S      <- e(G_C) S + sU sum_s e(G_s) k_s v_s^T.
// Every exponent is a difference that is <= 0, taken from sums in 64 bits, so no
// factor overflows and a large step does not blur the small ones behind it; and the
// whole part of an exponent is never rounded with the rest, so no factor is off by more
// than a few 2^-24 of itself.
//
// A block owns one (batch, head), one segment of the tokens and a tile of v's
// columns; each of its waves owns 32 columns, with their whole state (k.d rows)
// in its accumulators.  All four products run on MFMA tiles:
//   scores      k q^T, 16 x 16 tiles of the chunk by turns; scaled, stored to LDS
//   S^T q^T     S as it lies in the accumulators: the rows of the update's left
//               operand are permuted so that a lane's 8 consecutive accumulators
//               are 8 consecutive rows of S, which is an MFMA operand
//   v^T scores^T  on the same accumulators: a lane has one token's outputs
//   the update, whose v are scaled in registers.
// The last three are 32 x 32 tiles: an operand read from LDS feeds twice the
// products of a 16 x 16 one, which the LDS could not keep up with.
// q, k and v tiles are stored as they come (rows of a token); operands that run
// along the tokens are read with the transposing LDS loads (bf16) or by
// single words (fp32).  16-byte units of a tile's rows are permuted by the row so
// that neither kind of read has bank conflicts.
//
// What bounds it (4 x 4096 tokens x 32 heads of 128 x 128, bf16; 182 us for the pass
// with outputs, 77 for the states of 3 of 4 segments, 18 for their join).  The two waves
// a SIMD has, which the state's registers and the tiles' LDS allow, do not hide each
// other: of a wave's time 24% is issue of vector instructions (1306 per wave and chunk, 124 of
// them products, which keep the matrix units busy for 29%), 23% is waiting to issue and
// 42% waiting for LDS, barriers and memory; bytes move at 62% of a copy's rate.  Chunks
// of 64 (32 in fp32): the scores' work per token grows with the chunk, scaling
// the state and the barriers shrink with it, and one of 128 would leave one block a CU.
// 32 columns a wave: with 16 the LDS was the bound (344 us, all passes together, where
// 32 took 243, the scores and the state in one part each).
//
// Roundings (bf16 io).  What is computed and multiplied again -- the scaled v of the
// update, the scores, and the state as an operand -- is split in three bf16 parts (24
// bits), so states and outputs are sums in 32 bits of products exact to 2^-24, and
// only what is written in bf16 is rounded to it.  One part each for the scores and the state
// would leave outputs off by 2.6e-3 of their size, more than the 1.7e-3 of their own rounding,
// and two by 2e-4; the layer above takes 244, 254 and 265 us with one, two and three.
//
// What a zero factor multiplies is dropped, whatever its value, and a NaN or an
// infinity of a token reaches no token that it should not: products on the
// matrix units cannot promise that (0 * inf), so a wave whose outputs of a chunk are
// not all finite leaves its state as it was, and the block does the chunk again for
// it as chunks of one token, in which no other token is there to meet.
#pragma once

#include "device_common.h"
#include "linear_attn.h"
#include "rows.h"

namespace {

using linattn::Args;
using linattn::Exponent;
using linattn::pow2;
using linattn::Role;
using linattn::Side;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 8 values of one row (or column) of an MFMA operand, consecutive along the
// contracted dimension.
template <typename T>
struct Frag;

template <>
struct Frag<bf16_t> {
  bf16x8 v;
};

template <>
struct Frag<float> {
  float v[8];
};

// acc[row][col] += sum over 32 values; lane has values 8 (lane / 16) .. + 7 of row
// (col) lane % 16.  acc element i of a lane: column lane % 16, row 4 (lane / 16) + i.
// 32 x 32 tiles, 16 values: values 8 (lane / 32) .. + 7 of row (col) lane % 32; element i
// is column lane % 32, row 8 (i / 4) + 4 (lane / 32) + i % 4.
__device__ __forceinline__ void mma(f32x4& acc, const Frag<bf16_t>& a, const Frag<bf16_t>& b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
}

__device__ __forceinline__ void mma(f32x4& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], acc, 0, 0, 0);
}

__device__ __forceinline__ void mma(f32x16& acc, const Frag<bf16_t>& a, const Frag<bf16_t>& b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}

__device__ __forceinline__ void mma(f32x16& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], acc, 0, 0, 0);
}

// The upper halves of two words, side by side.
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302);
}

// 8 floats as operands: three in bf16, each the upper half of what the ones before left
// over, so that they hold every bit (an infinity's later ones are NaN).
__device__ __forceinline__ void split(Frag<bf16_t> f[3], const float x[8]) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    words4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = upper_halves(__float_as_uint(r[2 * j]), __float_as_uint(r[2 * j + 1]));
    f[p].v = __builtin_bit_cast(bf16x8, w);
    if (p < 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] -= __uint_as_float(__float_as_uint(r[j]) & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void split(Frag<float> f[1], const float x[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[0].v[j] = x[j];
}

template <typename T>
struct Traits;

template <>
struct Traits<bf16_t> {
  static constexpr int chunk = 64, parts = 3;  // parts: bf16 operands that hold 24 bits
};

template <>
struct Traits<float> {
  static constexpr int chunk = 32, parts = 1;
};

// A tile of rows of COLS elements in LDS.  Unit u (16 bytes) of row r lies at
// u ^ key(r).  The key puts the 16 rows of one unit, which a row read takes at
// once, on different banks; and of a column read the 4 rows x 4 units of 32 lanes
// (bf16), or the two rows 8 apart (fp32).  It is linear in the bits of r % 16, so a
// lane needs one place (a byte offset) for all its reads of a kind: columns x further
// on are place ^ x sizeof(T), rows 16 further on place + 16 kPitch, and rows j < 8
// of 8 further on (place ^ 16 key(j)) + j kPitch, x and j constants.
template <typename T, int COLS>
struct Tile {
  static constexpr unsigned kUnits = COLS * sizeof(T) / 16;
  static constexpr unsigned kPerUnit = 16 / sizeof(T);
  static constexpr unsigned kPitch = COLS * sizeof(T);
  static constexpr __host__ __device__ unsigned key(unsigned r) {
    if (kUnits >= 16 && sizeof(T) == 2) return (r & 3) << 2 | (r >> 2 & 3);
    if (kUnits >= 16) return r & 15;
    if (kUnits == 8) return (r >> 1 & 1) << 2 | (r >> 2 & 3);
    return r >> 2 & 3;
  }
  static __device__ __forceinline__ unsigned at(unsigned r, unsigned c) {  // element offset
    return (r * kUnits + (c / kPerUnit ^ key(r))) * kPerUnit + c % kPerUnit;
  }
  static __device__ __forceinline__ unsigned place(unsigned r, unsigned c) { return at(r, c) * sizeof(T); }
  template <typename V>
  static __device__ __forceinline__ V get(const T* p, unsigned place) {
    return *reinterpret_cast<const V*>(reinterpret_cast<const char*>(p) + place);
  }
  // The 8 values of a row from place(row, column) on; the column is a multiple of 8.
  static __device__ __forceinline__ Frag<T> row(const T* p, unsigned place, unsigned x, unsigned rows) {
    Frag<T> f;
    const unsigned at = (place ^ (unsigned)(x * sizeof(T))) + rows * kPitch;
    if constexpr (sizeof(T) == 2) {
      f.v = get<bf16x8>(p, at);
    } else {
      const float4 lo = get<float4>(p, at);
      const float4 hi = get<float4>(p, (place ^ (unsigned)(x * sizeof(T) + 16)) + rows * kPitch);
      f.v[0] = lo.x; f.v[1] = lo.y; f.v[2] = lo.z; f.v[3] = lo.w;
      f.v[4] = hi.x; f.v[5] = hi.y; f.v[6] = hi.z; f.v[7] = hi.w;
    }
    return f;
  }
  // Place of a column read: rows 8 (lane / 32) .. + 7 of the lane's column, c + lane % 32,
  // or with swap that number with bits 2 and 3 exchanged; c is a multiple of 32.
  static __device__ __forceinline__ unsigned column_place(bool swap, unsigned c, unsigned lane) {
    if constexpr (sizeof(T) == 2) {
      // Lane 4 j + i of 16 gives the address of row j's columns 4 i .. 4 i + 3 and
      // gets column 4 j + i of the four rows (the load transposes).
      const unsigned i = lane & 3, q = swap ? (i & 1) << 1 | i >> 1 : i;
      return place(8 * (lane >> 5) + (lane >> 2 & 3), c + (lane & 16) + 4 * q);
    } else {
      const unsigned i = lane & 31, q = swap ? (i & 19) | (i & 4) << 1 | (i & 8) >> 1 : i;
      return place(8 * (lane >> 5), c + q);
    }
  }
  static __device__ __forceinline__ Frag<T> column(const T* p, unsigned place, unsigned x, unsigned rows) {
    Frag<T> f;
    const auto at = [&](unsigned j) { return (place ^ (unsigned)(x * sizeof(T) ^ key(j) << 4)) + (rows + j) * kPitch; };
    if constexpr (sizeof(T) == 2) {
      typedef __attribute__((address_space(3))) i16x4* lds_ptr;
      const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(reinterpret_cast<const char*>(p) + at(0)));
      const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(reinterpret_cast<const char*>(p) + at(4)));
      f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
#pragma unroll
      for (unsigned j = 0; j < 8; ++j) f.v[j] = get<float>(p, at(j));
    }
    return f;
  }
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16_t x) { return __uint_as_float((uint32_t)x << 16); }

__device__ __forceinline__ void get8(const Frag<bf16_t>& f, float out[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = (float)f.v[j];
}

__device__ __forceinline__ void get8(const Frag<float>& f, float out[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = f.v[j];
}

// What a chunk's decays give.
template <int C>
struct Decays {
  Exponent sum[C];   // G (reverse: -G)
  float in[C];       // factor of q_t . S
  float up[C];       // factor of k_s v_s^T in the update
  float each[C];     // a_t, 0 where the state is dropped
  float total;       // factor of S
  int slow;          // a decay is not a number: token by token
  int zeros;         // some up is 0
  int pad;
};

__device__ __forceinline__ double scan64(double v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// By one wave, a token to a lane.
template <int C>
__device__ __forceinline__ void chunk_decays(Decays<C>* d, float rate, float step, int reset, bool constant, int len,
                                             int lane, const Role& p) {
  double g = reset ? linattn::kDrop : linattn::log2_decay(rate, step);
  const bool bad = !(__builtin_fabs(g) < 1e300);
  double sum;
  if (constant) {
    sum = g * (double)(min(lane, len - 1) + 1);
  } else {
    if (lane >= len) g = 0.0;
    sum = scan64(g, lane);
  }
  const double end = __shfl(sum, 63);
  const float from_start = pow2(sum), to_end = pow2(end - sum);
  const float up = p.s_up * (p.reverse ? from_start : to_end);
  const bool slow = __any(bad && lane < len);
  const bool zeros = __any(up == 0.0f && lane < len);
  if (lane < C) {
    d->sum[lane] = linattn::exponent(p.reverse ? -sum : sum);
    d->in[lane] = p.s_in * (p.reverse ? to_end : from_start);
    d->up[lane] = up;
    d->each[lane] = pow2(g);
  }
  if (lane == 0) {
    d->total = pow2(end);
    d->slow = slow;
    d->zeros = zeros;
  }
}

// a b, and 0 where a factor is 0 whatever the other is.
extern "C" __device__ float ssmi_mul_legacy(float a, float b) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float drop_mul(float a, float b) { return ssmi_mul_legacy(a, b); }

// A condition that hardly ever holds: registers are not spilled elsewhere for
// what it guards.
__device__ __forceinline__ bool rare(bool c) { return __builtin_expect(c, 0); }

// v, unknown to the compiler: what is computed from it stays where it is used.
// Else every LDS address of the chunk loop is computed before it and kept, in
// registers that the products need.
template <typename N>
__device__ __forceinline__ N opaque(N v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ int opaque_scalar(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

constexpr int kWaitVmcnt0 = 0x0F70;  // s_waitcnt vmcnt(0) expcnt(7) lgkmcnt(15): vector memory only

// Rows of one operand of a chunk on their way from memory to LDS: straight there
// (dma), a chunk ahead, where rows are whole 16-byte units; else in pieces of 8
// elements through registers.
template <typename T, int COLS, int C, int kThreads>
struct Stage {
  using Lds = Tile<T, COLS>;
  static constexpr unsigned kPieces = C * COLS / 8;
  // base: the chunk's first row; n elements of each row are there, len rows.  A
  // piece that ends behind its row is read as the row's last 8 elements, shifted.
  static __device__ __forceinline__ void pieces(T* tile, const T* base, uint32_t stride, int n, int len, unsigned tid) {
    if (n < 8) {
      elements(tile, base, stride, n, len);
      return;
    }
    constexpr int kAhead = 4;  // in flight at once
#pragma unroll 1
    for (unsigned p0 = tid; p0 < kPieces; p0 += kAhead * kThreads) {
      Raw8<T> r[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const unsigned p = min(p0 + i * kThreads, kPieces - 1), row = p / (COLS / 8), c = p % (COLS / 8) * 8;
        r[i].template load<false>(base + (min((int)row, len - 1) * stride + (uint32_t)min((int)c, n - 8)));
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const unsigned p = p0 + i * kThreads, row = p / (COLS / 8), c = p % (COLS / 8) * 8;
        if (p >= kPieces) break;
        if (n % 8) finish8<false>(r[i], (int)c, 0, n);
        if ((int)row >= len || (int)c >= n) r[i].clear();
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<words4*>(tile + Lds::at(row, c)) = r[i].w;
        } else {
          *reinterpret_cast<words4*>(tile + Lds::at(row, c)) = r[i].lo;
          *reinterpret_cast<words4*>(tile + Lds::at(row, c + 4)) = r[i].hi;
        }
      }
    }
  }
  // Straight to LDS: an instruction fills 64 units of the tile, lane by lane, so a
  // lane requests the unit that its place holds.  Units behind the row's end and
  // rows behind the last are not requested: the caller keeps those 0.
  static constexpr int kFills = C * (int)Lds::kUnits / 64, kWaves = kThreads / 64;
  static constexpr int kEach = (kFills + kWaves - 1) / kWaves;
  static constexpr uint32_t kNone = ~0u;
  // Bytes from a chunk's first row to what a lane requests, kNone behind the row's end.
  static __device__ __forceinline__ void offsets(uint32_t from[kEach], uint32_t stride, int n, int wave, unsigned lane) {
    const unsigned place = wave * 64 + lane;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const unsigned r = place / Lds::kUnits + i * (kWaves * 64 / Lds::kUnits), u = place % Lds::kUnits ^ Lds::key(r);
      from[i] = (int)(u * Lds::kPerUnit) < n ? (r * stride + u * Lds::kPerUnit) * (uint32_t)sizeof(T) : kNone;
    }
  }
  static __device__ __forceinline__ void dma(T* tile, const T* base, const uint32_t from[kEach], int n, int len, int wave,
                                             unsigned lane) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) T*)tile + wave * 1024);
    if (!rare(len < C || n < COLS)) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (kFills % kWaves && wave + i * kWaves >= kFills) break;
        fill(to + i * kWaves * 1024, base, from[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (kFills % kWaves && wave + i * kWaves >= kFills) break;
        const int r = ((wave + i * kWaves) * 64 + lane) / Lds::kUnits;
        if (r < len && from[i] != kNone) fill(to + i * kWaves * 1024, base, from[i]);
      }
    }
  }
  // The compiler does not see this load, so it waits for none of them before LDS
  // reads of other tiles; the chunk loop waits for all of them itself.  Nor does it see
  // its scalar registers read: m0, the place in LDS, may be one wait state old, and base, which
  // the vector unit may have read back from a lane, five.
  static __device__ __forceinline__ void fill(uint32_t to, const T* base, uint32_t from) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(from), "s"(base), "{m0}"(to) : "memory");
  }
  // Zeros in rows from first on.
  static __device__ __forceinline__ void clear(T* tile, int first, unsigned tid) {
#pragma unroll 1
    for (unsigned i = first * Lds::kUnits + tid; i < C * Lds::kUnits; i += kThreads)
      reinterpret_cast<words4*>(tile)[i] = words4{0, 0, 0, 0};
  }
  // The same, one element at a time and not requested before.
  static __device__ __forceinline__ void elements(T* tile, const T* base, uint32_t stride, int n, int len) {
#pragma unroll 1
    for (unsigned i = threadIdx.x; i < C * COLS; i += kThreads) {
      const unsigned row = i / COLS, c = i % COLS;
      tile[Lds::at(row, c)] = (int)row < len && (int)c < n ? base[row * stride + c] : T(0);
    }
  }
};

// First row of a side for this batch row and head.
template <typename T>
__device__ __forceinline__ const T* side_rows(const Side& s, int64_t batch_tokens, int head) {
  return static_cast<const T*>(s.p) + (batch_tokens * s.heads + head / s.share) * s.d;
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  const float v[4] = {a, b, c, d};
  store_n<4>(p, v);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t round2(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

__device__ __forceinline__ void store4(bf16_t* p, float a, float b, float c, float d) {
  const words2 w = {round2(a, b), round2(c, d)};
  __builtin_memcpy(p, &w, 8);
}

// A row's columns c + 8 g .. c + 8 g + 3, g = 0 .. 3: written from, and dotted with,
// a lane's elements of a 32 x 32 accumulator.  Columns from n on are not there.
// (heads of a row are limited so that byte offsets of a chunk's rows have 32 bits.)
template <bool kWhole, typename T>
__device__ __forceinline__ void store_columns(T* base, uint32_t row, int c, int n, const f32x16& v) {
  T* const at = reinterpret_cast<T*>(reinterpret_cast<char*>(base) + (row + c) * (uint32_t)sizeof(T));
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (kWhole || c + 8 * g + 4 <= n) {
      store4(at + 8 * g, v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (c + 8 * g + j < n) Io<T>::store1(at + 8 * g + j, v[4 * g + j]);
    }
  }
}

template <typename T>
__device__ __forceinline__ float dot_columns(const T* row, int c, int n, const f32x16& v) {
  float t = 0.0f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int at = c + 8 * g;
    if (!rare(at + 4 > n)) {
      float x[4];
      load_n<4>(row + at, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) t = __builtin_fmaf(x[j], v[4 * g + j], t);
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (at + j < n) t = __builtin_fmaf(Io<T>::load1(row + at + j), v[4 * g + j], t);
    }
  }
  return t;
}

template <typename T, int NK, int NW, bool kOut>
struct Layout {
  static constexpr int C = Traits<T>::chunk, DK = 32 * NK, TV = 32 * NW;
  static constexpr int q_bytes = kOut ? C * DK * (int)sizeof(T) : 0;
  static constexpr int k_bytes = C * DK * (int)sizeof(T), v_bytes = C * TV * (int)sizeof(T);
  static constexpr int s_bytes = kOut ? Traits<T>::parts * C * C * (int)sizeof(T) : 0;
  // q's and v's tiles are free for the next chunk's once every wave has its scores and
  // its operands of v; k's is read to the chunk's end and needs a second one for
  // that (so does v's where there are no scores), if the LDS holds two blocks with it
  // or would not without; but three blocks of two waves rather than two of them: 4 x
  // 4096 x 32 heads of 64 x 64 in bf16 214 us with two and 153 with one, 8 x 2048 x 12
  // heads of 64 x 128 in fp32 trained in 694 and 607.
  static constexpr int v_tiles = kOut ? 1 : 2;
  static constexpr int rest = q_bytes + v_tiles * v_bytes + s_bytes + 3 * (int)sizeof(Decays<C>) + 16;
  static constexpr int blocks(int tiles) { return 160 * 1024 / (rest + tiles * k_bytes); }
  static constexpr int k_tiles = NW == 2 && kOut && blocks(2) == 2 && blocks(1) == 3 ? 1
                                 : blocks(2) >= 2 || blocks(1) < 2                    ? 2
                                                                                      : 1;
  static constexpr int bytes = rest + k_tiles * k_bytes;
  // Waves that a SIMD has at once, for the registers' sake.
  static constexpr int waves = NK <= 4 && blocks(k_tiles) * NW > 4 ? 2 : 1;
};

// kOut: false computes the states alone (a segment's own, and its decay).
template <typename T, int NK, int NW, bool kOut>
__global__ __launch_bounds__(64 * NW, (Layout<T, NK, NW, kOut>::waves)) void linear_attn_kernel(const Args a) {
  using L = Layout<T, NK, NW, kOut>;
  constexpr int C = L::C, DK = L::DK, TV = L::TV, RT = C / 32, kThreads = 64 * NW;
  constexpr int kParts = Traits<T>::parts;
  using TileK = Tile<T, DK>;
  using TileV = Tile<T, TV>;
  using TileS = Tile<T, C>;
  __shared__ __align__(16) unsigned char lds[L::bytes];
  T* const qs = reinterpret_cast<T*>(lds);
  T* const k_base = reinterpret_cast<T*>(lds + L::q_bytes);
  T* const v_base = reinterpret_cast<T*>(lds + L::q_bytes + L::k_tiles * L::k_bytes);
  T* const ss = reinterpret_cast<T*>(lds + L::q_bytes + L::k_tiles * L::k_bytes + L::v_tiles * L::v_bytes);
  Decays<C>* const decays =
      reinterpret_cast<Decays<C>*>(lds + L::q_bytes + L::k_tiles * L::k_bytes + L::v_tiles * L::v_bytes + L::s_bytes);
  int* const again = reinterpret_cast<int*>(decays + 3);  // of chunk c in [c & 3]: some wave's outputs are not finite
  const int thread = threadIdx.x, tid = thread, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // ---- which rows, segment and columns this block has
  int r = 0;
  while (r + 1 < a.roles && (int)blockIdx.x >= a.role[r + 1].first_block) ++r;
  const Role& p = a.role[r];
  // State passes leave out the segment that no other starts behind.
  const int parts = kOut ? a.segments : a.segments - 1;
  const int index = (int)blockIdx.x - p.first_block;
  const int tile = index % p.tiles, part = index / p.tiles % parts, row = index / p.tiles / parts;
  const int segment = part + (!kOut && p.reverse ? 1 : 0);
  const int head = row % a.heads;
  const int64_t batch_tokens = row / a.heads * a.seqlen;
  const bool reverse = p.reverse;
  const int dk = p.k.d, dv = p.v.d;
  const int v0 = tile * TV, vc = v0 + wave * 32 + col;  // the lane's column
  const int64_t t_lo = segment * a.segment_len;
  const int64_t t_hi = t_lo + a.segment_len < a.seqlen ? t_lo + a.segment_len : a.seqlen;
  const int chunks = (int)((t_hi - t_lo + C - 1) / C);
  const float rate = a.rate[head];
  const bool constant = !a.step && !a.reset;
  // A chunk's rows are addressed by 32-bit offsets from its first (heads are limited so).
  const uint32_t k_stride = p.k.heads * dk, v_stride = p.v.heads * dv;  // q's rows lie as k's do

  // ---- the state: acc[b][i] is row 32 b + 16 (i / 8) + 8 half + i % 8, column vc
  f32x16 acc[NK];
  const int64_t state_size = (int64_t)dk * dv;
  {
    const int64_t slot = min(segment * p.start_step + p.start_first, p.start_slots - 1);
    const float* from = kOut && p.start ? p.start + ((int64_t)row * p.start_slots + slot) * state_size : nullptr;
    const int64_t k_step = p.transposed ? 1 : dv, at = p.transposed ? (int64_t)vc * dk : vc;
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = 32 * b + 16 * (i >> 3) + (i & 7) + 8 * half;
        acc[b][i] = from && k < dk && vc < dv ? from[at + k * k_step] : 0.0f;
      }
  }
  const auto store_state = [&](float* to) {  // states that are written are never transposed
    const int first = opaque(8 * half);
    if (vc >= dv) return;
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = 32 * b + 16 * (i >> 3) + (i & 7) + first;
        if (k < dk) to[k * dv + vc] = acc[b][i];
      }
  };

  // <meet, state> at a border, this wave's columns of it.
  const auto meet_state = [&](int64_t border) {
    const int first = opaque(8 * half);
    const float* from = p.meet + ((int64_t)row * p.slots + border) * state_size;
    double sum = 0.0;
    uint32_t at = first * dv + vc;
    if (vc < dv) {
#pragma unroll
      for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          __builtin_amdgcn_sched_barrier(0);  // 8 loads at a time: no registers for more
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = from[min(at + (uint32_t)(i * dv), (uint32_t)(dk * dv - 1))];
          at = opaque(at + 16 * dv);
          float some = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            some = 32 * b + 16 * h + i + first < dk ? __builtin_fmaf(x[i], acc[b][8 * h + i], some) : some;
          sum += (double)some;
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    const int part = tile * NW + wave, parts = (dv + 31) / 32;
    if (lane == 0 && part < parts) p.cross[((int64_t)row * p.slots + border) * parts + part] = sum;
  };

  // ---- tiles, requested a chunk ahead; decays, computed a chunk ahead
  using StageK = Stage<T, DK, C, kThreads>;
  using StageV = Stage<T, TV, C, kThreads>;
  const auto k_tile = [&](int i) { return k_base + (i & (L::k_tiles - 1)) * (L::k_bytes / (int)sizeof(T)); };
  const auto v_tile = [&](int i) { return v_base + (i & (L::v_tiles - 1)) * (L::v_bytes / (int)sizeof(T)); };
  const auto chunk_at = [&](int i) { return t_lo + (int64_t)(reverse ? chunks - 1 - i : i) * C; };
  const auto chunk_len = [&](int64_t t0) { return (int)(t_hi - t0 < C ? t_hi - t0 : C); };
  const bool dma = p.dma;
  uint32_t k_from[StageK::kEach], v_from[StageV::kEach];  // q's rows lie as k's do
  StageK::offsets(k_from, k_stride, dk, wave, lane);
  StageV::offsets(v_from, v_stride, dv - v0, wave, lane);
  // First row of what is requested next; chunks are requested in their order.
  const int64_t t_first = chunk_at(0);
  const T* q_next = kOut ? side_rows<T>(p.q, batch_tokens, head) + t_first * (int64_t)k_stride : nullptr;
  const T* k_next = side_rows<T>(p.k, batch_tokens, head) + t_first * (int64_t)k_stride;
  const T* v_next = side_rows<T>(p.v, batch_tokens, head) + t_first * (int64_t)v_stride + v0;
  const int k_move = reverse ? -C * (int)k_stride : C * (int)k_stride;
  const int v_move = reverse ? -C * (int)v_stride : C * (int)v_stride;
  const int last_len = (int)(t_hi - t_lo) - (chunks - 1) * C;  // tokens of the chunk at the segment's end
  const auto len_of = [&](int i) { return i == (reverse ? 0 : chunks - 1) ? last_len : C; };
  const auto request_k = [&](int i) {
    const int len = len_of(i), id = opaque(tid);
    StageK::dma(k_tile(i), k_next, k_from, dk, len, wave, id & 63);
    k_next += k_move;
    if (rare(len < C)) StageK::clear(k_tile(i), len, id);
  };
  const auto request_qv = [&](int i) {
    const int len = len_of(i), id = opaque(tid);
    if constexpr (kOut) {
      StageK::dma(qs, q_next, k_from, dk, len, wave, id & 63);
      q_next += k_move;
    }
    StageV::dma(v_tile(i), v_next, v_from, dv - v0, len, wave, id & 63);
    v_next += v_move;
    if (rare(len < C)) {
      if constexpr (kOut) StageK::clear(qs, len, id);
      StageV::clear(v_tile(i), len, id);
    }
  };
  float next_step = 1.0f;
  int next_reset = 0;
  const auto request_step = [&](int i) {  // of the wave that computes the decays
    const int64_t t0 = chunk_at(i);
    const int64_t at = batch_tokens + t0 + min(lane, chunk_len(t0) - 1);
    if (a.step) next_step = widen(static_cast<const T*>(a.step)[at * a.heads + head]);
    if (a.reset) next_reset = a.reset[at];
  };
  const bool decay_wave = wave == NW - 1;
  // Places of this lane's reads and writes in the tiles.
  const unsigned row16 = TileK::place(lane & 15, 8 * (lane >> 4)), row32 = TileK::place(col, 8 * half);
  const unsigned scores_at = TileS::place(lane & 15, 4 * (lane >> 4)), scores_row = TileS::place(col, 8 * half);
  const unsigned k_column = TileK::column_place(true, 0, lane), v_column = TileV::column_place(false, wave * 32, lane);
  float carried = 1.0f;  // decay of the whole segment
  if (dma) {
    if (dk < DK || dv - v0 < TV) {  // units behind the rows' ends stay 0
      if constexpr (kOut) StageK::clear(qs, 0, tid);
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        StageK::clear(k_tile(i), 0, tid);
        StageV::clear(v_tile(i), 0, tid);
      }
      lds_barrier();
    }
    if (L::k_tiles == 2) request_k(0);
    request_qv(0);
  }
  if (decay_wave) {
    request_step(0);
    chunk_decays<C>(&decays[0], rate, next_step, next_reset, constant, chunk_len(chunk_at(0)), lane, p);
    if (chunks > 1) request_step(1);
  }
  if (tid < 4) again[tid] = 0;
  if constexpr (kOut) {  // scores that no token sees: half of the tiles beside the diagonal's are read
    for (int i = tid; i < kParts * C * C; i += kThreads) ss[i] = 0;
  }

  int c = 0;
  int single = -1;       // chunks of one token: which of chunk c's is in turn
  bool pending = false;  // this wave's state still lacks them
  const auto land = [&] {
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    lds_barrier();  // the next chunk's tiles have landed, the last one's are no longer read; decays and marks are there
  };
  land();
  // The loop has one exit, at its end: with one at its head the state is copied
  // from registers to registers in every turn.
  do {
    const int tid = opaque(thread), lane = tid & 63, col = lane & 31, half = lane >> 5;
    const unsigned k_other = (c & (L::k_tiles - 1)) * L::k_bytes;
    const bool whole = single < 0;
    const int64_t t0 = chunk_at(c) + (whole ? 0 : reverse ? chunk_len(chunk_at(c)) - 1 - single : single);
    const int len = whole ? chunk_len(t0) : 1;
    const Decays<C>& d = whole ? decays[c & 1] : decays[2];
    T* const ks = k_tile(c);
    T* const vs = v_tile(c);
    // This chunk's first rows, found anew where they are wanted: kept, they take
    // scalar registers that the chunks in their common course lack.
    const auto q_at = [&] { const Role& o = a.role[opaque_scalar(r)]; return side_rows<T>(o.q, batch_tokens + t0, head); };
    const auto k_at = [&] { const Role& o = a.role[opaque_scalar(r)]; return side_rows<T>(o.k, batch_tokens + t0, head); };
    const auto v_at = [&] { const Role& o = a.role[opaque_scalar(r)]; return side_rows<T>(o.v, batch_tokens + t0, head) + v0; };
    if (!rare(!whole)) {
      if constexpr (kOut) {  // a border of blocks lies in front of this chunk
        const bool border = reverse ? (t0 + C) % linattn::kBlock == 0 || t0 + C >= a.seqlen : t0 % linattn::kBlock == 0;
        if (rare(border)) {
          if (p.save) store_state(p.save + ((int64_t)row * p.slots + t0 / linattn::kBlock) * state_size);
          if (p.meet) meet_state(t0 / linattn::kBlock + 1);
        }
      }
      if (L::k_tiles == 1 && dma) {
        request_k(c);
        land();
      }
      if (rare(!dma)) {
        if constexpr (kOut) StageK::pieces(qs, q_at(), k_stride, dk, len, tid);
        StageK::pieces(ks, k_at(), k_stride, dk, len, tid);
        StageV::pieces(vs, v_at(), v_stride, dv - v0, len, tid);
        lds_barrier();
      }
    } else {
      // The token in row 0, zeros in the others.
      if constexpr (kOut) StageK::elements(qs, q_at(), k_stride, dk, 1);
      StageK::elements(ks, k_at(), k_stride, dk, 1);
      StageV::elements(vs, v_at(), v_stride, dv - v0, 1);
      if (tid < C) {
        const float each = decays[c & 1].each[t0 - chunk_at(c)];
        Decays<C>& one = decays[2];
        // A decay that is NaN makes the state NaN, what is 0 of it too: here what is
        // read of it, below what is kept.
        one.sum[tid] = Exponent{0, tid == 0 && !reverse && each != each ? each : 0.0f};
        one.in[tid] = tid ? 0.0f : p.s_in * (reverse ? 1.0f : each);
        one.up[tid] = tid ? 0.0f : p.s_up * (reverse || each != each ? each : 1.0f);
        if (tid == 0) {
          one.total = each;
          one.zeros = one.up[0] == 0.0f;
        }
      }
      lds_barrier();
    }
    if (whole) {
      if (tid == 0) again[(c + 1) & 3] = 0;  // last read before this chunk's barrier
      if (dma && c + 1 < chunks) {
        if (L::k_tiles == 2) request_k(c + 1);
        if (!kOut) request_qv(c + 1);
      }
    }

    if constexpr (!kOut) {
      // A row whose factor is 0 is dropped: its k are made 0 (its v below).
      if (whole && rare(d.zeros)) {
#pragma unroll 1
        for (int i = tid; i < C * DK; i += kThreads)
          if (d.up[i / DK] == 0.0f) ks[TileK::at(i / DK, i % DK)] = 0;
        lds_barrier();
      }
    }

    f32x16 out[RT];
    if constexpr (kOut) {
      // ---- scores, a 16 x 16 tile at a time: rows s, columns t
      constexpr int kTiles = C / 16;
      const int quad = lane >> 4, c16 = lane & 15;
      const unsigned k_place = opaque(row16) + k_other, q_place = opaque(row16), s_place = opaque(scores_at);
      for (int n = wave; n < kTiles * (kTiles + 1) / 2; n += NW) {
        const int hi = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3, lo = n - hi * (hi + 1) / 2;
        const int ti = reverse ? lo : hi, si = reverse ? hi : lo;
        f32x4 x = {};
#pragma unroll
        for (int m = 0; m < NK; ++m)
          mma(x, TileK::row(k_base, k_place + 16 * si * TileK::kPitch, 32 * m, 0),
              TileK::row(qs, q_place + 16 * ti * TileK::kPitch, 32 * m, 0));
        const int t = 16 * ti + c16, s0 = 16 * si + 4 * quad;
        const Exponent gt = d.sum[t];
        const float s_both = p.s_in * p.s_up;
        const int late = reverse ? t - s0 : s0 - t;  // seen: not after t
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = pow2(gt, d.sum[s0 + j]);
          y[j] = late <= (reverse ? j : -j) ? x[j] * (e * s_both) : 0.0f;
        }
        const unsigned s_at = (s_place ^ 16 * si * (unsigned)sizeof(T)) + 16 * ti * TileS::kPitch;
        unsigned char* const to = reinterpret_cast<unsigned char*>(ss) + s_at;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const words2 w = {round2(y[0], y[1]), round2(y[2], y[3])};
            *reinterpret_cast<words2*>(to + part * C * C * sizeof(T)) = w;
            y[0] -= bf16_lo(w.x);
            y[1] -= bf16_hi(w.x);
            y[2] -= bf16_lo(w.y);
            y[3] -= bf16_hi(w.y);
          }
        } else {
          *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
      // ---- S^T q^T
#pragma unroll
      for (int ti = 0; ti < RT; ++ti) out[ti] = f32x16{};
#pragma unroll
      for (int f = 0; f < DK / 16; ++f) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = acc[f >> 1][8 * (f & 1) + j];
        Frag<T> s[kParts];
        split(s, x);
        Frag<T> q[RT];
#pragma unroll
        for (int ti = 0; ti < RT; ++ti) q[ti] = TileK::row(qs, row32, 16 * f, 32 * ti);
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int ti = 0; ti < RT; ++ti) mma(out[ti], s[part], q[ti]);
      }
#pragma unroll
      for (int ti = 0; ti < RT; ++ti) {
        const float in = d.in[32 * ti + col];
#pragma unroll
        for (int i = 0; i < 16; ++i) out[ti][i] = drop_mul(in, out[ti][i]);
      }
    }
    if (whole && decay_wave && c + 1 < chunks) {
      chunk_decays<C>(&decays[(c + 1) & 1], rate, next_step, next_reset, constant, chunk_len(chunk_at(c + 1)), lane, p);
      if (c + 2 < chunks) request_step(c + 2);
    }
    Frag<T> v[C / 16];
#pragma unroll
    for (int f = 0; f < C / 16; ++f) v[f] = TileV::column(vs, v_column, 0, 16 * f);
    bool skip = !whole && !pending;
    if (whole) pending = d.slow;
    if constexpr (kOut) {
      lds_barrier();
      if (whole && dma && c + 1 < chunks) request_qv(c + 1);
      // ---- v^T scores^T
      const unsigned s_row = opaque(scores_row);
      const auto seen = [&](int ti, int f) {
#pragma unroll
        for (int part = 0; part < kParts; ++part)
          mma(out[ti], v[f], TileS::row(ss + part * C * C, s_row, 16 * f, 32 * ti));
      };
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int ti = 0; ti < RT; ++ti) seen(ti, 2 * ti + f);
      if constexpr (RT == 2) {
        if (reverse) {
          seen(0, 2);
          seen(0, 3);
        } else {
          seen(1, 0);
          seen(1, 1);
        }
      }
      float nan = 0.0f;  // stays 0 while every output is finite
#pragma unroll
      for (int ti = 0; ti < RT; ++ti)
#pragma unroll
        for (int i = 0; i < 16; ++i) nan = __builtin_fmaf(out[ti][i], 0.0f, nan);
      if (whole && __any(!(nan == 0.0f))) pending = true;
    }
    if (!(whole && d.slow)) carried = drop_mul(d.total, carried);
    if (whole) {
      if (rare(pending)) {
        if (lane == 0) again[c & 3] = 1;
        skip = true;
      }
    }

    if (!rare(skip)) {
      if constexpr (kOut) {
        // ---- outputs: a lane has columns 8 i + 4 half .. + 3 (i < 4) of token 32 ti + col
        const int first = v0 + wave * 32 + 4 * half;
        const uint32_t out_stride = a.heads * dv;
        const int64_t out_first = ((batch_tokens + t0) * a.heads + head) * dv;
        if (!rare(p.out_f32 || len < C || v0 + TV > dv)) {
#pragma unroll
          for (int ti = 0; ti < RT; ++ti)
            store_columns<true>(static_cast<T*>(p.out) + out_first, (32 * ti + col) * out_stride, first, dv, out[ti]);
        } else {
#pragma unroll
          for (int ti = 0; ti < RT; ++ti) {
            if (32 * ti + col >= len) continue;
            if (p.out_f32)
              store_columns<false>(static_cast<float*>(p.out) + out_first, (32 * ti + col) * out_stride, first, dv, out[ti]);
            else
              store_columns<false>(static_cast<T*>(p.out) + out_first, (32 * ti + col) * out_stride, first, dv, out[ti]);
          }
        }
        if (p.with.p) {
#pragma unroll
          for (int ti = 0; ti < RT; ++ti) {
            const int t = 32 * ti + col;
            const bool live = t < len;
            float dot = 0.0f;
            if (live) {
              const T* with = side_rows<T>(p.with, batch_tokens, head) + (t0 + t) * p.with.heads * dv;
              dot = dot_columns(with, first, dv, out[ti]);
            }
            dot += __shfl_xor(dot, 32);
            const int part = tile * NW + wave;
            if (half == 0 && live && part * 32 < dv)
              p.dots[((int64_t)part * a.batch * a.heads + row) * a.seqlen + t0 + t] = dot;
          }
        }
      }
      // ---- the update
      const float total = d.total;
#pragma unroll
      for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] = drop_mul(total, acc[b][i]);
      if (!rare(!whole && d.zeros)) {
        const unsigned k_col = opaque(k_column) + k_other;
#pragma unroll
        for (int f = 0; f < C / 16; ++f) {
          float x[8];
          get8(v[f], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = drop_mul(d.up[16 * f + 8 * half + j], x[j]);
          Frag<T> w[kParts];
          split(w, x);
          constexpr int kPair = NK < 2 ? 1 : 2;
#pragma unroll
          for (int b = 0; b < NK; b += kPair) {
            Frag<T> k[kPair];
#pragma unroll
            for (int u = 0; u < kPair; ++u) k[u] = TileK::column(k_base, k_col, 32 * (b + u), 16 * f);
#pragma unroll
            for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
              for (int u = 0; u < kPair; ++u) mma(acc[b + u], k[u], w[part]);
          }
        }
      }
    }
    land();
    if (whole) {
      if (rare(again[c & 3]))
        single = 0;
      else
        ++c;
    } else if (++single == chunk_len(chunk_at(c))) {
      single = -1;
      pending = false;
      if (++c < chunks && dma && kOut) {  // the next chunk's, which the single tokens wrote over
        q_next -= k_move;
        v_next -= v_move;
        request_qv(c);
        land();
      }
    }
  } while (c < chunks);

  // ---- the segment's end
  if constexpr (kOut) {
    const bool final_segment = reverse ? segment == 0 : segment == a.segments - 1;
    if (final_segment) {
      if (p.last) store_state(p.last + row * state_size);
      if (p.save) store_state(p.save + ((int64_t)row * p.slots + p.slots - 1) * state_size);
      if (p.meet) meet_state(0);
    }
  } else {
    store_state(p.part + ((int64_t)row * a.segments + segment) * state_size);
    if (tile == 0 && tid == 0) p.total[row * a.segments + segment] = carried;
  }
}

template <typename T, int NK, int NW>
hipError_t launch_one(const Args& a, int64_t blocks, bool state_only, hipStream_t st) {
  const dim3 grid((unsigned)blocks), threads(64 * NW);
  if (state_only)
    hipLaunchKernelGGL((linear_attn_kernel<T, NK, NW, false>), grid, threads, 0, st, a);
  else
    hipLaunchKernelGGL((linear_attn_kernel<T, NK, NW, true>), grid, threads, 0, st, a);
  return hipGetLastError();
}

template <typename T, int NW>
hipError_t launch_width(const Args& a, int64_t blocks, bool state_only, hipStream_t st) {
  const int parts = (a.role[0].k.d + 31) / 32;
  if (parts <= 1) return launch_one<T, 1, NW>(a, blocks, state_only, st);
  if (parts <= 2) return launch_one<T, 2, NW>(a, blocks, state_only, st);
  if (parts <= 4) return launch_one<T, 4, NW>(a, blocks, state_only, st);
  return launch_one<T, 8, NW>(a, blocks, state_only, st);
}

template <typename T>
hipError_t launch(const Args& a, int64_t blocks, bool state_only, hipStream_t st) {
  return linattn::tile_width(a.role[0].v.d) == 64 ? launch_width<T, 2>(a, blocks, state_only, st)
                                                  : launch_width<T, 4>(a, blocks, state_only, st);
}

}  // namespace
