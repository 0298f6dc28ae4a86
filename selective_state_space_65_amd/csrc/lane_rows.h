// lane_rows.h -- rows held by groups of G lanes (8 to 64) in pieces of 8
// consecutive numbers: sums over a group's lanes, and its pieces' loads.
// Internal: not part of the C ABI.
#pragma once

#include "rows.h"

namespace {

constexpr int kPiece = 8;  // numbers per lane and piece

template <int ctrl, int row_mask = 0xf>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, row_mask, 0xf, true));
}

// Sum over the G lanes of a group, in all of them.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v = dpp_add<0xb1>(v);  // quad_perm 1,0,3,2
  v = dpp_add<0x4e>(v);  // quad_perm 2,3,0,1
  v = dpp_add<0x141>(v);  // row_half_mirror: the other quad of 8
  if constexpr (G >= 16) v = dpp_add<0x128>(v);  // row_ror 8: the other half of 16
  if constexpr (G == 32) v += __shfl_xor(v, 16);
  if constexpr (G == 64) {
    const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
    const float b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
    const float c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
    const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
    v = (a + b) + (c + d);
  }
  return v;
}

// Whether the piece at column c is whole in every lane of the group.
template <int G>
__device__ __forceinline__ bool whole(int c, int gl, int dim) {
  return c - gl * kPiece + G * kPiece <= dim;
}

// request8 and finish8 for the group's piece of which the lane has column c.
template <int G, typename T>
__device__ __forceinline__ Raw8<T> request_piece(const T* row, int c, int gl, int dim) {
  return request8<G == 8>(row, c - gl * kPiece, gl * kPiece, dim);
}

template <int G, typename T>
__device__ __forceinline__ void finish_piece(Raw8<T>& r, int c, int gl, int dim) {
  if (whole<G>(c, gl, dim)) return;
  if (c - gl * kPiece >= dim)
    r.clear();
  else
    finish8<G == 8>(r, c - gl * kPiece, gl * kPiece, dim);
}

}  // namespace
