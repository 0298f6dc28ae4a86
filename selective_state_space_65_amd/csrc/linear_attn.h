// linear_attn.h -- arguments of the chunked linear-attention kernels, shared by
// the translation units that build them (one per io type) and the one that
// plans and launches the calls.  Internal: not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.h"

namespace linattn {

constexpr int kBlock = 512;  // tokens between saved states
constexpr int kMaxDim = 256;

// Rows of one operand, [batch, seqlen, heads, d]; head h of the call reads
// head h / share of the operand.
struct Side {
  const void* p;
  int heads, share, d;
};

// One pass  out_t = sU sI sum_s D(t, s) (q_t . k_s) v_s + sI D(t, border) q_t . state,
// s <= t, or s >= t where reverse; the state is q.d = k.d rows by v.d columns.
struct Role {
  Side q, k, v;
  void* out;             // [batch, seqlen, heads, v.d], io or fp32
  int out_f32;
  int reverse;
  int transposed;        // states in memory are [v.d][k.d]
  float s_in, s_up;      // sI, sU
  const float* start;    // state a segment starts from (null: zero): slot segment * start_step + start_first,
  int64_t start_slots;   // or the last one, of start_slots slots for each (batch, head)
  int64_t start_step, start_first;
  float* save;           // forward: state in front of every block of kBlock tokens, and behind the last; may be null
  const float* meet;     // reverse: states as save has them, that this pass's are multiplied with
  double* cross;         // there: <meet, state> in parts, [batch, heads, border][v.d / 32 rounded up]
  int64_t slots;         // of save, meet and cross for each (batch, head)
  float* last;           // state after the last (reverse: before the first) token, may be null
  Side with;             // rows that the outputs are dotted with (p may be null)
  float* dots;           // [v.d / 32 rounded up][batch, heads, seqlen]
  float* part;           // state passes: a segment's own state, [batch, heads, segments][k.d][v.d]
  float* total;          // and its decay, [batch, heads, segments]
  int dma;               // rows are whole 16-byte units at 16-byte addresses
  int tiles;             // blocks side by side along v.d
  int first_block;       // of the launch that is this role's
};

struct Args {
  Role role[3];
  int roles;
  int batch, heads;
  int64_t seqlen;
  const float* rate;
  const void* step;      // may be null
  const uint8_t* reset;  // may be null
  int segments;
  int64_t segment_len;   // a multiple of 64
};

// Columns of one block: 64, or 128 where v.d is above 64.
inline int tile_width(int dv) { return dv > 64 ? 128 : 64; }

// Launches the roles, whose contracted dimensions (k.d) have the same number
// of 32-wide parts (rounded up to 1, 2, 4 or 8) and whose tile widths are the
// same.
hipError_t launch_bf16(const Args& a, int64_t blocks, bool state_only, hipStream_t st);
hipError_t launch_f32(const Args& a, int64_t blocks, bool state_only, hipStream_t st);

// ---- decays, in device code ----------------------------------------------------

constexpr double kDrop = -4096.0;  // a log2 decay at which every factor is 0 (2^-4096)

// log2 of a token's decay; a NaN stays.
__device__ __forceinline__ double log2_decay(float rate, float step) {
  const double g = -(double)rate * (double)step * 1.4426950408889634;
  return g < kDrop ? kDrop : g;
}

// An exponent as a whole number and what is left, within 1/2: rounded to 32 bits, that
// is off by 2^-26 at most whatever the exponent's size, where the exponent in one
// float would be by 2^-18 at 2^-100.  Factors down to e^-80 are off by at most 1.3 x
// 2^-24 of themselves so (47 x 2^-24 with the exponent in one float), states that seven
// chunks were carried over by 5 x 2^-24.
struct Exponent {
  int n;
  float f;
};

__device__ __forceinline__ Exponent exponent(double x) {
  const double n = __builtin_rint(x);
  return Exponent{(int)n, (float)(x - n)};
}

// 2^(a - b); 0 below the smallest normal float.
__device__ __forceinline__ float pow2(Exponent a, Exponent b) {
  const float e = __builtin_ldexpf(exp2_hw(a.f - b.f), a.n - b.n);
  return e < 0x1p-126f ? 0.0f : e;
}

__device__ __forceinline__ float pow2(double x) { return pow2(exponent(x), Exponent{0, 0.0f}); }

}  // namespace linattn
