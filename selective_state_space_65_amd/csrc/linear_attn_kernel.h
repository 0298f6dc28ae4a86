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
// factor overflows and a large step does not blur the small ones behind it.
//
// A block owns one (batch, head), one segment of the tokens and a tile of v's
// columns; each of its waves owns 32 columns, with their whole state (k.d rows)
// in its accumulators.  All four products run on 32 x 32 MFMA tiles:
//   scores  k q^T, quarters of the chunk by turns; scaled, stored to LDS
//   q . S   S as it lies in the accumulators: the rows of the update's left
//           operand are permuted so that a lane's 8 consecutive accumulators
//           are 8 consecutive rows of S, which is an MFMA operand
//   scores . v
//   the update, whose v are scaled in registers.
// q, k and v tiles are stored as they come (rows of a token); operands that run
// along the tokens are read with the transposing LDS loads (bf16) or by
// single words (fp32).  16-byte units of a tile's rows are permuted by the row so
// that neither kind of read has bank conflicts.
//
// Roundings (bf16 io).  The scaled v of the update are split in three bf16 parts
// (24 bits): states are sums in 32 bits of products exact to 2^-24.  Scores and
// the state as an operand are rounded to bf16 once, half a step each like the
// output itself; kParts = 3 splits them in three (2^-24), for gradients whose dot
// products with the inputs are summed up over the tokens (the decays').
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
using linattn::Role;
using linattn::Side;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
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

// acc[row][col] += sum over 16 values; lanes 0-31 hold values 0-7 of row (col)
// lane, lanes 32-63 values 8-15.  acc element i of a lane: column lane % 32, row
// 8 (i / 4) + 4 (lane / 32) + i % 4.
__device__ __forceinline__ void mma(f32x16& acc, const Frag<bf16_t>& a, const Frag<bf16_t>& b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}

__device__ __forceinline__ void mma(f32x16& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], acc, 0, 0, 0);
}

// 8 floats as kParts operands that sum to them (fp32: one, exact).
template <int kParts>
__device__ __forceinline__ void split(Frag<bf16_t>* f, const float x[8]) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[p].v[j] = (__bf16)r[j];
      if (p + 1 < kParts) r[j] -= (float)f[p].v[j];
    }
  }
}

template <int kParts>
__device__ __forceinline__ void split(Frag<float>* f, const float x[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[0].v[j] = x[j];
}

template <typename T>
struct Traits;

template <>
struct Traits<bf16_t> {
  static constexpr int chunk = 64, update_parts = 3;
};

template <>
struct Traits<float> {
  static constexpr int chunk = 32, update_parts = 1;
};

// A tile of rows of COLS elements in LDS.  Unit u (16 bytes) of row r lies at
// u ^ key(r): the 16 rows of a row read's pass, and the 4 rows x 4 units of a
// transposing read's, then fall on different banks.
template <typename T, int COLS>
struct Tile {
  static constexpr int kUnits = COLS * (int)sizeof(T) / 16;
  static constexpr int kPerUnit = 16 / (int)sizeof(T);
  static __device__ __forceinline__ int key(int r) {
    if constexpr (kUnits >= 16) return (r & 3) << 2 | (r >> 2 & 3);
    if constexpr (kUnits == 8) return (r >> 1 & 1) << 2 | (r >> 2 & 3);
    return r >> 2 & 3;
  }
  static __device__ __forceinline__ int at(int r, int c) {  // element offset
    return (r * kUnits + (c / kPerUnit ^ key(r))) * kPerUnit + c % kPerUnit;
  }
  // Values c .. c + 7 of row r; c is a multiple of 8.
  static __device__ __forceinline__ Frag<T> row(const T* p, int r, int c) {
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      f.v = *reinterpret_cast<const bf16x8*>(p + at(r, c));
    } else {
      const float4 lo = *reinterpret_cast<const float4*>(p + at(r, c));
      const float4 hi = *reinterpret_cast<const float4*>(p + at(r, c + 4));
      f.v[0] = lo.x; f.v[1] = lo.y; f.v[2] = lo.z; f.v[3] = lo.w;
      f.v[4] = hi.x; f.v[5] = hi.y; f.v[6] = hi.z; f.v[7] = hi.w;
    }
    return f;
  }
  // Rows r .. r + 7 (r differs between the wave's halves) of the lane's column:
  // c + lane % 32, or with kSwap that number with bits 2 and 3 exchanged.
  template <bool kSwap>
  static __device__ __forceinline__ Frag<T> column(const T* p, int r, int c, int lane) {
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      // Lane 4 j + i of 16 gives the address of row j's columns 4 i .. 4 i + 3 and
      // gets column 4 i + j of the four rows.
      const int i = lane & 3, q = kSwap ? (i & 1) << 1 | i >> 1 : i;
      const int col = c + (lane & 16) + 4 * q, row0 = r + (lane >> 2 & 3);
      typedef __attribute__((address_space(3))) i16x4* lds_ptr;
      const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + at(row0, col)));
      const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + at(row0 + 4, col)));
      f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int i = lane & 31, q = kSwap ? (i & 19) | (i & 4) << 1 | (i & 8) >> 1 : i;
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] = p[at(r + j, c + q)];
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
  double sum[C];     // G
  float in[C];       // factor of q_t . S
  float up[C];       // factor of k_s v_s^T in the update
  float each[C];     // a_t, 0 where the state is dropped
  float total;       // factor of S
  int slow;          // a decay is not a number: token by token
  int zeros;         // some up is 0
  int pad;
};

constexpr double kDrop = -4096.0;  // a log2 decay at which every factor is 0 (2^-4096)

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
  double g = -(double)rate * (double)step * 1.4426950408889634;
  if (g < kDrop) g = kDrop;  // a NaN stays
  if (reset) g = kDrop;
  const bool bad = !(__builtin_fabs(g) < 1e300);
  double sum;
  if (constant) {
    sum = g * (double)(min(lane, len - 1) + 1);
  } else {
    if (lane >= len) g = 0.0;
    sum = scan64(g, lane);
  }
  const double end = __shfl(sum, 63);
  const float from_start = exp2_hw((float)sum), to_end = exp2_hw((float)(end - sum));
  const float up = p.s_up * (p.reverse ? from_start : to_end);
  const bool slow = __any(bad && lane < len);
  const bool zeros = __any(up == 0.0f && lane < len);
  if (lane < C) {
    d->sum[lane] = sum;
    d->in[lane] = p.s_in * (p.reverse ? to_end : from_start);
    d->up[lane] = up;
    d->each[lane] = exp2_hw((float)g);
  }
  if (lane == 0) {
    d->total = exp2_hw((float)end);
    d->slow = slow;
    d->zeros = zeros;
  }
}

// A wave's LDS writes before it are seen by its own reads after it.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Rows of one operand of a chunk on their way from memory to LDS: pieces of 8
// elements, requested a chunk ahead.
template <typename T, int COLS, int C, int kThreads>
struct Stage {
  using Lds = Tile<T, COLS>;
  static constexpr int kPieces = C * COLS / 8;
  static constexpr int kEach = (kPieces + kThreads - 1) / kThreads;
  Raw8<T> r[kEach];
  // base: the chunk's first row; n elements of each row are there, len rows.
  // Rows of less than 8 are left to elements().
  __device__ __forceinline__ void request(const T* base, uint32_t stride, int n, int len, int tid) {
    if (n < 8) return;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int p = min(tid + i * kThreads, kPieces - 1);
      const uint32_t row = min(p / (COLS / 8), len - 1) * stride;
      r[i].template load<false>(base + (row + (uint32_t)min(p % (COLS / 8) * 8, n - 8)));
    }
  }
  __device__ __forceinline__ void store(T* tile, const T* base, uint32_t stride, int n, int len, int tid) {
    if (n < 8) {
      elements(tile, base, stride, n, len);
      return;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int p = tid + i * kThreads;
      const int row = p / (COLS / 8), c = p % (COLS / 8) * 8;
      if (kPieces % kThreads == 0 || p < kPieces) {
        if (row < len)
          finish8<false>(r[i], c, 0, n);
        else
          r[i].clear();
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<words4*>(tile + Lds::at(row, c)) = r[i].w;
        } else {
          *reinterpret_cast<words4*>(tile + Lds::at(row, c)) = r[i].lo;
          *reinterpret_cast<words4*>(tile + Lds::at(row, c + 4)) = r[i].hi;
        }
      }
    }
  }
  // The same, one element at a time and not requested before.
  static __device__ __forceinline__ void elements(T* tile, const T* base, uint32_t stride, int n, int len) {
#pragma unroll 1
    for (int i = threadIdx.x; i < C * COLS; i += kThreads) {
      const int row = i / COLS, c = i % COLS;
      tile[Lds::at(row, c)] = row < len && c < n ? base[row * stride + c] : T(0);
    }
  }
};

// v, unknown to the compiler: what is computed from it stays where it is used.
// Else every LDS address of the chunk loop is computed before it and kept, in
// registers that the products need.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// First row of a side for this batch row and head.
template <typename T>
__device__ __forceinline__ const T* side_rows(const Side& s, int64_t batch_tokens, int head) {
  return static_cast<const T*>(s.p) + (batch_tokens * s.heads + head / s.share) * s.d;
}

template <typename T, int NK, int NW, int kParts, bool kOut>
struct Layout {
  static constexpr int C = Traits<T>::chunk, DK = 32 * NK, TV = 32 * NW;
  static constexpr int q_bytes = !kOut ? 0 : C * DK * (int)sizeof(T) > NW * 4096 ? C * DK * (int)sizeof(T) : NW * 4096;
  static constexpr int k_bytes = C * DK * (int)sizeof(T), v_bytes = C * TV * (int)sizeof(T);
  static constexpr int s_bytes = kOut ? kParts * C * C * (int)sizeof(T) : 0;
  static constexpr int bytes = q_bytes + k_bytes + v_bytes + s_bytes + 3 * (int)sizeof(Decays<C>) + 8;
};

// kOut: false computes the states alone (a segment's own, and its decay).
template <typename T, int NK, int NW, int kParts, bool kOut>
__global__ __launch_bounds__(64 * NW, NK <= 4 ? 2 : 1) void linear_attn_kernel(const Args a) {
  using L = Layout<T, NK, NW, kParts, kOut>;
  constexpr int C = L::C, DK = L::DK, TV = L::TV, RT = C / 32, kThreads = 64 * NW;
  constexpr int kUp = Traits<T>::update_parts;
  using TileK = Tile<T, DK>;
  using TileV = Tile<T, TV>;
  using TileS = Tile<T, C>;
  using TileO = Tile<float, 32>;
  __shared__ __align__(16) unsigned char lds[L::bytes];
  T* const qs = reinterpret_cast<T*>(lds);
  T* const ks = reinterpret_cast<T*>(lds + L::q_bytes);
  T* const vs = reinterpret_cast<T*>(lds + L::q_bytes + L::k_bytes);
  T* const ss = reinterpret_cast<T*>(lds + L::q_bytes + L::k_bytes + L::v_bytes);
  Decays<C>* const decays =
      reinterpret_cast<Decays<C>*>(lds + L::q_bytes + L::k_bytes + L::v_bytes + L::s_bytes);
  int* const again = reinterpret_cast<int*>(decays + 3);  // of chunk c in [c & 1]: some wave's outputs are not finite
  const int thread = threadIdx.x, tid = thread, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  float* const out_tile = reinterpret_cast<float*>(lds) + wave * 1024;  // q's space, when q is no longer read

  // ---- which rows, segment and columns this block has
  int r = 0;
  while (r + 1 < a.roles && (int64_t)blockIdx.x >= a.role[r + 1].first_block) ++r;
  const Role& p = a.role[r];
  const int64_t index = (int64_t)blockIdx.x - p.first_block;
  const int tile = (int)(index % p.tiles);
  const int64_t rest = index / p.tiles;
  const int segment = (int)(rest % a.segments);
  const int64_t row = rest / a.segments;  // (batch, head)
  const int head = (int)(row % a.heads);
  const int64_t batch_tokens = row / a.heads * a.seqlen;
  const bool reverse = p.reverse;
  const int dk = p.k.d, dv = p.v.d;
  const int v0 = tile * TV, vc = v0 + wave * 32 + col;  // the lane's column
  const int64_t t_lo = segment * a.segment_len;
  const int64_t t_hi = t_lo + a.segment_len < a.seqlen ? t_lo + a.segment_len : a.seqlen;
  const int chunks = (int)((t_hi - t_lo + C - 1) / C);
  const float rate = a.rate[head];
  const bool constant = !a.step && !a.reset;
  const T* const q_rows = kOut ? side_rows<T>(p.q, batch_tokens, head) : nullptr;
  const T* const k_rows = side_rows<T>(p.k, batch_tokens, head);
  const T* const v_rows = side_rows<T>(p.v, batch_tokens, head) + v0;
  // A chunk's rows are addressed by 32-bit offsets from its first (heads are limited so).
  const uint32_t q_stride = kOut ? p.q.heads * dk : 0, k_stride = p.k.heads * dk, v_stride = p.v.heads * dv;

  // ---- the state: acc[b][i] is row 32 b + 16 (i / 8) + 8 half + i % 8, column vc
  f32x16 acc[NK];
  const int64_t state_size = (int64_t)dk * dv;
  const auto state_row = [&](int b, int i) { return 32 * b + 16 * (i >> 3) + 8 * half + (i & 7); };
  {
    const float* from = kOut && p.start ? p.start + (row * p.start_slots + segment * p.start_step) * state_size : nullptr;
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = state_row(b, i);
        float x = 0.0f;
        if (from && k < dk && vc < dv) x = from[p.transposed ? (int64_t)vc * dk + k : (int64_t)k * dv + vc];
        acc[b][i] = x;
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

  // ---- requests, a chunk ahead; decays, computed a chunk ahead of their use
  Stage<T, DK, C, kThreads> q_in, k_in;
  Stage<T, TV, C, kThreads> v_in;
  const auto chunk_at = [&](int i) { return t_lo + (int64_t)(reverse ? chunks - 1 - i : i) * C; };
  const auto chunk_len = [&](int64_t t0) { return (int)(t_hi - t0 < C ? t_hi - t0 : C); };
  const auto request = [&](int i) {
    const int64_t t0 = chunk_at(i);
    const int len = chunk_len(t0), id = opaque(tid);
    if constexpr (kOut) q_in.request(q_rows + t0 * (int64_t)q_stride, q_stride, dk, len, id);
    k_in.request(k_rows + t0 * (int64_t)k_stride, k_stride, dk, len, id);
    v_in.request(v_rows + t0 * (int64_t)v_stride, v_stride, dv - v0, len, id);
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
  float carried = 1.0f;  // decay of the whole segment
  request(0);
  if (decay_wave) {
    request_step(0);
    chunk_decays<C>(&decays[0], rate, next_step, next_reset, constant, chunk_len(chunk_at(0)), lane, p);
    if (chunks > 1) request_step(1);
  }
  if (tid == 0) again[0] = again[1] = 0;

  int c = 0;
  int single = -1;       // chunks of one token: which of chunk c's is in turn
  bool pending = false;  // this wave's state still lacks them
  for (;; ) {
    lds_barrier();  // the last tiles are no longer read; decays and marks are there
    if (single >= 0) {
      if (++single == chunk_len(chunk_at(c))) {
        single = -1;
        pending = false;
        ++c;
      }
    } else if (c > 0 && again[(c - 1) & 1]) {
      --c;
      single = 0;
    }
    if (c == chunks) break;
    const int tid = opaque(thread), lane = tid & 63, col = lane & 31, half = lane >> 5;
    const bool whole = single < 0;
    const int64_t t0 = chunk_at(c) + (whole ? 0 : reverse ? chunk_len(chunk_at(c)) - 1 - single : single);
    const int len = whole ? chunk_len(t0) : 1;
    const Decays<C>& d = whole ? decays[c & 1] : decays[2];
    const T* const q_at = kOut ? q_rows + t0 * (int64_t)q_stride : nullptr;
    const T* const k_at = k_rows + t0 * (int64_t)k_stride;
    const T* const v_at = v_rows + t0 * (int64_t)v_stride;
    if (whole) {
      if (kOut && p.save) {
        // Forward: the state before a block; reverse: the state behind it.
        const bool border = reverse ? (t0 + C) % linattn::kBlock == 0 || t0 + C >= a.seqlen : t0 % linattn::kBlock == 0;
        if (border) store_state(p.save + (row * p.save_slots + t0 / linattn::kBlock) * state_size);
      }
      if constexpr (kOut) q_in.store(qs, q_at, q_stride, dk, len, tid);
      k_in.store(ks, k_at, k_stride, dk, len, tid);
      v_in.store(vs, v_at, v_stride, dv - v0, len, tid);
    } else {
      // The token in row 0, zeros in the others.
      if constexpr (kOut) Stage<T, DK, C, kThreads>::elements(qs, q_at, q_stride, dk, 1);
      Stage<T, DK, C, kThreads>::elements(ks, k_at, k_stride, dk, 1);
      Stage<T, TV, C, kThreads>::elements(vs, v_at, v_stride, dv - v0, 1);
      if (tid < C) {
        const float each = decays[c & 1].each[t0 - chunk_at(c)];
        Decays<C>& one = decays[2];
        one.sum[tid] = 0.0;
        one.in[tid] = tid ? 0.0f : p.s_in * (reverse ? 1.0f : each);
        one.up[tid] = tid ? 0.0f : p.s_up * (reverse ? each : 1.0f);
        if (tid == 0) {
          one.total = each;
          one.zeros = one.up[0] == 0.0f;
        }
      }
    }
    lds_barrier();
    if (whole && c + 1 < chunks) request(c + 1);
    if (whole && tid == 0) again[(c + 1) & 1] = 0;

    if constexpr (!kOut) {
      // A row whose factor is 0 is dropped: its k are made 0 (its v below).
      if (whole && d.zeros) {
#pragma unroll 1
        for (int i = tid; i < C * DK; i += kThreads)
          if (d.up[i / DK] == 0.0f) ks[TileK::at(i / DK, i % DK)] = 0;
        lds_barrier();
      }
    }

    f32x16 out[RT];
    if constexpr (kOut) {
      // ---- scores, a 32 x 32 quarter at a time: rows s, columns t
      constexpr int kQuarters = RT == 2 ? 3 : 1;
      for (int n = wave; n < kQuarters; n += NW) {
        const int ti = reverse ? n >> 1 : (n + 1) >> 1;
        const int si = reverse ? (n + 1) >> 1 : n >> 1;
        f32x16 x = {};
#pragma unroll
        for (int f = 0; f < DK / 16; ++f)
          mma(x, TileK::row(ks, 32 * si + col, 16 * f + 8 * half), TileK::row(qs, 32 * ti + col, 16 * f + 8 * half));
        const int t = 32 * ti + col;
        const double gt = d.sum[t];
        const float s_both = p.s_in * p.s_up;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int s0 = 32 * si + 2 * i + 4 * half;
          float y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double diff = reverse ? d.sum[s0 + j] - gt : gt - d.sum[s0 + j];
            const float e = exp2_hw((float)diff);
            const bool seen = reverse ? s0 + j >= t : s0 + j <= t;
            y[j] = seen && e != 0.0f ? x[i + j] * (e * s_both) : 0.0f;
          }
          if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
              words2 w;
              w.x = Io<bf16_t>::pack2(y[0], y[1]);
              w.y = Io<bf16_t>::pack2(y[2], y[3]);
              *reinterpret_cast<words2*>(ss + part * C * C + TileS::at(t, s0)) = w;
              y[0] -= bf16_lo(w.x);
              y[1] -= bf16_hi(w.x);
              y[2] -= bf16_lo(w.y);
              y[3] -= bf16_hi(w.y);
            }
          } else {
            *reinterpret_cast<float4*>(ss + TileS::at(t, s0)) = make_float4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      // ---- q . S
#pragma unroll
      for (int ti = 0; ti < RT; ++ti) out[ti] = f32x16{};
#pragma unroll
      for (int f = 0; f < DK / 16; ++f) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = acc[f >> 1][8 * (f & 1) + j];
        Frag<T> s[kParts];
        split<kParts>(s, x);
#pragma unroll
        for (int ti = 0; ti < RT; ++ti) {
          const Frag<T> q = TileK::row(qs, 32 * ti + col, 16 * f + 8 * half);
#pragma unroll
          for (int part = 0; part < kParts; ++part) mma(out[ti], q, s[part]);
        }
      }
#pragma unroll
      for (int ti = 0; ti < RT; ++ti)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float f = d.in[32 * ti + 8 * (i >> 2) + 4 * half + (i & 3)];
          out[ti][i] = f == 0.0f ? 0.0f : out[ti][i] * f;
        }
    }
    if (whole && decay_wave && c + 1 < chunks) {
      chunk_decays<C>(&decays[(c + 1) & 1], rate, next_step, next_reset, constant, chunk_len(chunk_at(c + 1)), lane, p);
      if (c + 2 < chunks) request_step(c + 2);
    }
    Frag<T> v[C / 16];
#pragma unroll
    for (int f = 0; f < C / 16; ++f)
      v[f] = TileV::template column<false>(vs, 16 * f + 8 * half, wave * 32, lane);
    bool skip = !whole && !pending;
    if (whole) pending = d.slow;
    if constexpr (kOut) {
      lds_barrier();
      // ---- scores . v
#pragma unroll
      for (int ti = 0; ti < RT; ++ti) {
#pragma unroll
        for (int f = 0; f < C / 16; ++f) {
          if (RT == 2 && (ti == 0 ? f >= 2 && !reverse : f < 2 && reverse)) continue;
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            mma(out[ti], TileS::row(ss + part * C * C, 32 * ti + col, 16 * f + 8 * half), v[f]);
        }
      }
      float nan = 0.0f;  // stays 0 while every output is finite
#pragma unroll
      for (int ti = 0; ti < RT; ++ti)
#pragma unroll
        for (int i = 0; i < 16; ++i) nan = __builtin_fmaf(out[ti][i], 0.0f, nan);
      if (whole && __any(!(nan == 0.0f))) pending = true;
    }
    if (whole) {
      if (pending) {
        if (lane == 0) again[c & 1] = 1;
        skip = true;
      }
      carried *= d.total;
    }

    if (!skip) {
      // ---- the update
      const float total = d.total;
#pragma unroll
      for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] = total == 0.0f ? 0.0f : acc[b][i] * total;
      if (whole || !d.zeros) {
#pragma unroll
        for (int f = 0; f < C / 16; ++f) {
          float x[8];
          get8(v[f], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float up = d.up[16 * f + 8 * half + j];
            x[j] = up == 0.0f ? 0.0f : x[j] * up;
          }
          Frag<T> w[kUp];
          split<kUp>(w, x);
#pragma unroll
          for (int b = 0; b < NK; ++b) {
            const Frag<T> k = TileK::template column<true>(ks, 16 * f + 8 * half, 32 * b, lane);
#pragma unroll
            for (int part = kUp - 1; part >= 0; --part) mma(acc[b], k, w[part]);
          }
        }
      }
      if constexpr (kOut) {
        // ---- outputs: through the wave's own LDS tile, so that a lane has 8 of a row
#pragma unroll
        for (int ti = 0; ti < RT; ++ti) {
          wave_lds_fence();
#pragma unroll
          for (int i = 0; i < 16; ++i) out_tile[TileO::at(8 * (i >> 2) + 4 * half + (i & 3), col)] = out[ti][i];
          wave_lds_fence();
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int piece = lane + 64 * u, rr = piece >> 2, c8 = (piece & 3) * 8;
            const int t = 32 * ti + rr, vcol = v0 + wave * 32 + c8;
            const bool live = t < len && vcol < dv;
            const Frag<float> y = TileO::row(out_tile, rr, c8);
            const int64_t token = batch_tokens + t0 + t;
            if (live) {
              const int64_t at = (token * a.heads + head) * dv;
              if (p.out_f32)
                store_row8(static_cast<float*>(p.out) + at, vcol, dv, false, y.v);
              else
                store_row8(static_cast<T*>(p.out) + at, vcol, dv, false, y.v);
            }
            if (p.with.p) {
              float dot = 0.0f;
              if (live) {
                const T* with = static_cast<const T*>(p.with.p) + (token * p.with.heads + head / p.with.share) * dv;
                Raw8<T> raw = request8<true>(with, vcol, 0, dv);
                finish8<true>(raw, vcol, 0, dv);
                float x[8];
                raw.get(x);
#pragma unroll
                for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(x[j], vcol + j < dv ? y.v[j] : 0.0f, dot);
              }
              dot += __shfl_xor(dot, 1);
              dot += __shfl_xor(dot, 2);
              const int part = tile * NW + wave;
              if ((lane & 3) == 0 && t < len && part * 32 < dv)
                p.dots[((int64_t)part * a.batch * a.heads + row) * a.seqlen + t0 + t] = dot;
            }
          }
        }
      }
    }
    if (whole) ++c;
  }

  // ---- the segment's end
  if constexpr (kOut) {
    const bool final_segment = reverse ? segment == 0 : segment == a.segments - 1;
    if (final_segment) {
      if (p.last) store_state(p.last + row * state_size);
      if (p.save && !reverse) store_state(p.save + (row * p.save_slots + p.save_slots - 1) * state_size);
    }
  } else {
    store_state(p.part + (row * a.segments + segment) * state_size);
    if (tile == 0 && tid == 0) p.total[row * a.segments + segment] = carried;
  }
}

template <typename T, int NK, int NW, int kParts, bool kOut>
hipError_t launch_one(const Args& a, int64_t blocks, hipStream_t st) {
  hipLaunchKernelGGL((linear_attn_kernel<T, NK, NW, kParts, kOut>), dim3((unsigned)blocks), dim3(64 * NW), 0, st, a);
  return hipGetLastError();
}

template <typename T, int NK, int NW>
hipError_t launch_kind(const Args& a, int64_t blocks, bool state_only, bool exact, hipStream_t st) {
  if (state_only) return launch_one<T, NK, NW, 1, false>(a, blocks, st);
  if constexpr (sizeof(T) == 2) {
    if (exact) return launch_one<T, NK, NW, 3, true>(a, blocks, st);
  }
  return launch_one<T, NK, NW, 1, true>(a, blocks, st);
}

template <typename T, int NW>
hipError_t launch_width(const Args& a, int64_t blocks, bool state_only, bool exact, hipStream_t st) {
  const int parts = (a.role[0].k.d + 31) / 32;
  if (parts <= 1) return launch_kind<T, 1, NW>(a, blocks, state_only, exact, st);
  if (parts <= 2) return launch_kind<T, 2, NW>(a, blocks, state_only, exact, st);
  if (parts <= 4) return launch_kind<T, 4, NW>(a, blocks, state_only, exact, st);
  return launch_kind<T, 8, NW>(a, blocks, state_only, exact, st);
}

template <typename T>
hipError_t launch(const Args& a, int64_t blocks, bool state_only, bool exact, hipStream_t st) {
  return linattn::tile_width(a.role[0].v.d) == 64 ? launch_width<T, 2>(a, blocks, state_only, exact, st)
                                                  : launch_width<T, 4>(a, blocks, state_only, exact, st);
}

}  // namespace
