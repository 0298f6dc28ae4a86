// host_common.h -- host-side helpers shared by the translation units that
// implement the C ABI: the calling thread's HIP error, size products, pointer
// alignment, and the overlap of buffers.  Internal: not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ssm_scan.h"

// The HIP error behind the calling thread's last SSM_ERR_HIP (what
// ssm_last_hip_error reports); defined in ssm_scan.hip.
int& ssmi_last_hip_error();

namespace {

inline ssm_status_t hip_fail(hipError_t e) {
  ssmi_last_hip_error() = (int)e;
  return SSM_ERR_HIP;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

inline size_t io_size(ssm_dtype_t io) { return io == SSM_BF16 ? 2 : 4; }

inline bool aligned(const void* p, size_t k) { return (reinterpret_cast<uintptr_t>(p) % k) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range span(const void* p, int64_t bytes) {
  uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// A launch's lanes are counted in 32 bits.
inline bool launch_ok(int64_t blocks, int64_t threads) { return blocks < ((int64_t)1 << 32) / threads; }

// One buffer of a call, for check_buffers; p may be null (not given).
struct Buf {
  const void* p;
  int64_t bytes;
  size_t align;
};

// Element alignment of every buffer, and no output overlapping an input or
// another output.
inline ssm_status_t check_buffers(const Buf* ins, int n_in, const Buf* outs, int n_out) {
  for (int i = 0; i < n_in; ++i)
    if (ins[i].p && !aligned(ins[i].p, ins[i].align)) return SSM_ERR_ALIGN;
  for (int o = 0; o < n_out; ++o)
    if (outs[o].p && !aligned(outs[o].p, outs[o].align)) return SSM_ERR_ALIGN;
  for (int o = 0; o < n_out; ++o) {
    if (!outs[o].p) continue;
    const Range r = span(outs[o].p, outs[o].bytes);
    for (int i = 0; i < n_in; ++i)
      if (ins[i].p && overlap(r, span(ins[i].p, ins[i].bytes))) return SSM_ERR_ALIAS;
    for (int q = o + 1; q < n_out; ++q)
      if (outs[q].p && overlap(r, span(outs[q].p, outs[q].bytes))) return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

}  // namespace
