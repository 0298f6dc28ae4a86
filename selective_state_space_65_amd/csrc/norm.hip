// norm.hip -- layer and RMS norm with the residual add in front of it: forward
// and backward.  C ABI: include/ssm_scan.h.
//
// A row is held in registers from its one read to its write: G lanes (8 to 64,
// or W waves of 64) take a row, each lane K pieces of 8 consecutive numbers,
// piece k of the row's lanes next to each other so that every access is
// contiguous.  The mean, then the sum of squares about it, are reduced over
// the lanes by DPP and over a row's waves through LDS: every number is read
// once and written once.
//
// The backward gives each group of lanes many rows.  Besides the two sums of
// a row (g and g n) each lane keeps its own columns' sums of dy n and dy in
// registers over all its rows; at the end a block adds its groups' sums in
// LDS and writes one partial row, and a second kernel adds the partial rows,
// all in a fixed order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device_common.h"
#include "host_common.h"
#include "rows.h"
#include "ssm_scan.h"

namespace {

constexpr int kPiece = 8;           // numbers per lane and piece
constexpr int kMaxDim = 32768;      // 16 waves x 64 lanes x 4 pieces x 8
constexpr int kMaxRowWaves = 16;

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

// Sum over a row: its lanes, then its waves (slots: one LDS row per use, so
// that one barrier separates the writes from the reads).
template <int G>
__device__ __forceinline__ float row_sum(float v, float* slots, int lane, int row_wave, int row_waves) {
  v = group_sum<G>(v);
  if (G == 64 && row_waves > 1) {
    if (lane == 0) slots[row_wave] = v;
    lds_barrier();
    v = slots[0];
    for (int w = 1; w < row_waves; ++w) v += slots[w];
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

// ---- the forward -------------------------------------------------------------

struct NormFwdArgs {
  const void* x;
  const void* residual;
  const float* weight;  // may be null
  const float* bias;    // may be null
  void* y;
  void* s;      // may be null
  float* mean;  // may be null
  float* rstd;  // may be null
  int64_t rows;
  int dim;
  int row_waves;
  float eps;
};

// x + residual rounded to the residual's type, as it is stored.
template <typename ResT>
__device__ __forceinline__ float add_res(float x, float r) {
  return round_io<ResT>(x + r);
}

// G lanes a row, K pieces a lane; kRes: a residual is added.
template <typename IoT, typename ResT, int G, int K, bool kRms, bool kRes>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormFwdArgs p) {
  __shared__ float slots[2][kMaxRowWaves];
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int W = G == 64 ? p.row_waves : 1;  // 1 or all of the block's waves
  const int row_wave = W > 1 ? wave : 0;
  const int64_t row = W > 1 ? (int64_t)blockIdx.x : ((int64_t)blockIdx.x * waves + wave) * (64 / G) + lane / G;
  const bool live = row < p.rows;
  const int64_t base = (live ? row : p.rows - 1) * p.dim;
  const IoT* xr = static_cast<const IoT*>(p.x) + base;
  const ResT* rr = static_cast<const ResT*>(p.residual) + (kRes ? base : 0);
  const int dim = p.dim;
  const float count = (float)dim;  // sums are divided by it: a constant row has exactly its mean

  float v[K][kPiece];
  Raw8<IoT> px[K];
  Raw8<ResT> pr[K];
  Raw8<float> pw[K], pb[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = ((k * W + row_wave) * G + gl) * kPiece;
    px[k] = request_piece<G>(xr, c, gl, dim);
    if constexpr (kRes) pr[k] = request_piece<G>(rr, c, gl, dim);
  }
  if constexpr (K == 1) {  // in flight during the sums, where the registers allow
    if (p.weight) pw[0] = request_piece<G>(p.weight, (row_wave * G + gl) * kPiece, gl, dim);
    if (p.bias) pb[0] = request_piece<G>(p.bias, (row_wave * G + gl) * kPiece, gl, dim);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = ((k * W + row_wave) * G + gl) * kPiece;
    finish_piece<G>(px[k], c, gl, dim);
    if constexpr (kRes) finish_piece<G>(pr[k], c, gl, dim);
    px[k].get(v[k]);
    if constexpr (kRes) {
      float r[kPiece];
      pr[k].get(r);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) v[k][j] = add_res<ResT>(v[k][j], r[j]);
    }
  }
  float mean = 0.0f;
  if constexpr (!kRms) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < kPiece; ++j) t += v[k][j];
    mean = row_sum<G>(t, slots[0], lane, row_wave, W) / count;
  }
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = ((k * W + row_wave) * G + gl) * kPiece;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const float d = c + j < dim ? v[k][j] - mean : 0.0f;
      q = __builtin_fmaf(d, d, q);
    }
  }
  const float var = row_sum<G>(q, slots[1], lane, row_wave, W) / count;
  const float rstd = 1.0f / __builtin_sqrtf(var + p.eps);
  if (!live) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = ((k * W + row_wave) * G + gl) * kPiece;
    const bool full = whole<G>(c, gl, dim);
    if constexpr (kRes) {
      if (p.s) store_row8(static_cast<ResT*>(p.s) + base, c, dim, full, v[k]);
    }
    float w[kPiece], b[kPiece], o[kPiece];
    if constexpr (K > 1) {
      if (p.weight) pw[k] = request_piece<G>(p.weight, c, gl, dim);
      if (p.bias) pb[k] = request_piece<G>(p.bias, c, gl, dim);
    }
    if (p.weight) {
      finish_piece<G>(pw[k], c, gl, dim);
      pw[k].get(w);
    }
    if (p.bias) {
      finish_piece<G>(pb[k], c, gl, dim);
      pb[k].get(b);
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      o[j] = (v[k][j] - mean) * rstd;
      if (p.weight) o[j] *= w[j];
      if (p.bias) o[j] += b[j];
    }
    store_row8(static_cast<IoT*>(p.y) + base, c, dim, full, o);
  }
  if (gl == 0 && row_wave == 0) {
    if (!kRms && p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// ---- the backward ------------------------------------------------------------

struct NormBwdArgs {
  const void* dy;
  const void* s;
  const float* weight;  // may be null
  const float* mean;    // layer only
  const float* rstd;
  const void* ds_out;  // may be null
  void* dx;
  void* dres;      // may be null
  float* part;     // [blocks][2][dim], or null without dweight and dbias
  int64_t rows;
  int dim;
  int row_waves;
};

constexpr int kBwdWaves = 8;  // per block

// A block's waves form kBwdWaves / W row groups (times 64 / G for short rows);
// every group takes the rows group, group + groups, ...
template <typename IoT, typename ResT, int G, int K, bool kRms, int kThreads>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormBwdArgs p) {
  __shared__ float slots[2][2][kMaxRowWaves];
  extern __shared__ __align__(16) float cols[];  // [wave groups][2][width] column sums
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int W = G == 64 ? p.row_waves : 1;
  const int row_wave = wave % W, wave_group = wave / W, wave_groups = waves / W;
  const int group = wave_group * (64 / G) + lane / G, groups = wave_groups * (64 / G);
  const int dim = p.dim;
  const float inv = 1.0f / (float)dim;
  float w[K][kPiece], aw[K][kPiece], ab[K][kPiece];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = ((k * W + row_wave) * G + gl) * kPiece;
    if (p.weight) {
      Raw8<float> r = request_piece<G>(p.weight, c, gl, dim);
      finish_piece<G>(r, c, gl, dim);
      r.get(w[k]);
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      if (!p.weight) w[k][j] = 1.0f;
      aw[k][j] = ab[k][j] = 0.0f;
    }
  }
  const int64_t per_sweep = (int64_t)gridDim.x * groups;
  const int64_t sweeps = (p.rows + per_sweep - 1) / per_sweep;
  const int64_t first = (int64_t)blockIdx.x * groups + group;
  // A row's pieces, requested a row ahead where few waves share a compute unit
  // and the registers allow (4096 x 8000 training step 134.6 -> 128.3 us; at one
  // piece the other waves cover the wait, 183.0 us without and 185.8 with at
  // 32768 x 1024).
  constexpr bool kAhead = K == 2;
  Raw8<ResT> next_s[K], next_past[K];
  Raw8<IoT> next_dy[K];
  float next_mean = 0.0f, next_rstd = 0.0f;
  const auto request = [&](int64_t i) {
    const int64_t at = min(first + i * per_sweep, p.rows - 1), base = at * dim;
    if (!kRms) next_mean = p.mean[at];
    next_rstd = p.rstd[at];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = ((k * W + row_wave) * G + gl) * kPiece;
      next_s[k] = request_piece<G>(static_cast<const ResT*>(p.s) + base, c, gl, dim);
      next_dy[k] = request_piece<G>(static_cast<const IoT*>(p.dy) + base, c, gl, dim);
      if (p.ds_out) next_past[k] = request_piece<G>(static_cast<const ResT*>(p.ds_out) + base, c, gl, dim);
    }
  };
  if (kAhead) request(0);
  int parity = 0;
  for (int64_t i = 0; i < sweeps; ++i, parity ^= 1) {
    const int64_t row = first + i * per_sweep;
    const bool live = row < p.rows;
    const int64_t base = (live ? row : p.rows - 1) * dim;
    if (!kAhead) request(i);
    const float mean = next_mean, rstd = next_rstd;
    float n[K][kPiece], dy[K][kPiece];
    Raw8<ResT> past[K];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = ((k * W + row_wave) * G + gl) * kPiece;
      finish_piece<G>(next_s[k], c, gl, dim);
      finish_piece<G>(next_dy[k], c, gl, dim);
      if (p.ds_out) finish_piece<G>(next_past[k], c, gl, dim);
      next_s[k].get(n[k]);
      next_dy[k].get(dy[k]);
      past[k] = next_past[k];
    }
    if (kAhead && i + 1 < sweeps) request(i + 1);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        n[k][j] = (n[k][j] - mean) * rstd;
        const float g = dy[k][j] * w[k][j];  // 0 past the row, where dy is
        if constexpr (!kRms) c1 += g;
        c2 = __builtin_fmaf(g, n[k][j], c2);
        if (live) {
          aw[k][j] = __builtin_fmaf(dy[k][j], n[k][j], aw[k][j]);
          ab[k][j] += dy[k][j];
        }
      }
    }
    c1 = group_sum<G>(c1);
    c2 = group_sum<G>(c2);
    if (G == 64 && W > 1) {
      float* s1 = slots[parity][0];
      float* s2 = slots[parity][1];
      if (lane == 0) s1[wave] = c1, s2[wave] = c2;
      lds_barrier();
      c1 = c2 = 0.0f;
      for (int v = 0; v < W; ++v) c1 += s1[wave_group * W + v], c2 += s2[wave_group * W + v];
    }
    c1 *= inv;
    c2 *= inv;
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = ((k * W + row_wave) * G + gl) * kPiece;
        const bool full = whole<G>(c, gl, dim);
        float o[kPiece];
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
          float g = dy[k][j] * w[k][j];
          if constexpr (!kRms) g -= c1;
          o[j] = rstd * __builtin_fmaf(-n[k][j], c2, g);
        }
        if (p.ds_out) {
          float r[kPiece];
          past[k].get(r);
#pragma unroll
          for (int j = 0; j < kPiece; ++j) o[j] += r[j];
        }
        store_row8(static_cast<IoT*>(p.dx) + base, c, dim, full, o);
        if (p.dres) store_row8(static_cast<ResT*>(p.dres) + base, c, dim, full, o);
      }
    }
  }
  if (!p.part) return;
  float* part = p.part + (int64_t)blockIdx.x * 2 * dim;
  if (wave_groups == 1) {  // the block is one row group: its sums as they are
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = ((k * W + row_wave) * G + gl) * kPiece;
      const bool full = whole<G>(c, gl, dim);
      store_row8(part, c, dim, full, aw[k]);
      store_row8(part + dim, c, dim, full, ab[k]);
    }
    return;
  }
  // Column sums of the block: the groups of a wave by shuffles, then the wave
  // groups' rows side by side in LDS, added in order.
  const int width = K * W * G * kPiece;
  float* mine = cols + wave_group * 2 * width;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = ((k * W + row_wave) * G + gl) * kPiece;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
#pragma unroll
      for (int d = G; d < 64; d <<= 1) {
        aw[k][j] += __shfl_xor(aw[k][j], d);
        ab[k][j] += __shfl_xor(ab[k][j], d);
      }
    }
    if (lane < G) {
#pragma unroll
      for (int j = 0; j < kPiece; j += 4) {
        *reinterpret_cast<float4*>(mine + c + j) = make_float4(aw[k][j], aw[k][j + 1], aw[k][j + 2], aw[k][j + 3]);
        *reinterpret_cast<float4*>(mine + width + c + j) =
            make_float4(ab[k][j], ab[k][j + 1], ab[k][j + 2], ab[k][j + 3]);
      }
    }
  }
  lds_barrier();
  for (int c = threadIdx.x; c < 2 * dim; c += blockDim.x) {
    const float* at = cols + (c < dim ? c : width + c - dim);
    float t = at[0];
    for (int g = 1; g < wave_groups; ++g) t += at[g * 2 * width];
    part[c] = t;
  }
}

// dweight and dbias: 32 columns a block, 32 slices of the partial rows; a slice
// requests 8 of its rows at once, and rows and slices are added in order.
__global__ __launch_bounds__(1024) void norm_bwd_reduce_kernel(const float* part, float* dweight, float* dbias,
                                                               int blocks, int dim) {
  __shared__ float sums[32][33];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col;
  float t = 0.0f;
  if (c < 2 * dim) {
    const float* at = part + c;
    int b = slice;
    for (; b + 7 * 32 < blocks; b += 8 * 32) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = at[(int64_t)(b + j * 32) * 2 * dim];
#pragma unroll
      for (int j = 0; j < 8; ++j) t += v[j];
    }
    for (; b < blocks; b += 32) t += at[(int64_t)b * 2 * dim];
  }
  sums[slice][col] = t;
  lds_barrier();
  if (slice == 0 && c < 2 * dim) {
#pragma unroll
    for (int i = 1; i < 32; ++i) t += sums[i][col];
    float* out = c < dim ? dweight : dbias;
    if (out) out[c < dim ? c : c - dim] = t;
  }
}

// ---- host side ---------------------------------------------------------------

struct NormPlan {
  int group, pieces, row_waves, threads;
  int64_t blocks;
};

// Lanes, pieces and waves of a row.  The fewest lanes that hold it at one piece
// each, up to 8 waves: many short waves keep more rows' loads in flight than
// few long ones.  Forward with a residual, 4 / 2 / 1 pieces, us for io-residual
// bf16-bf16, bf16-fp32, fp32-fp32: 16384 x 2048 53.2 / 52.8 / 53.8, 80.8 / 79.9 /
// 78.4, 107.4 / 105.3 / 103.3; 8192 x 4096 55.2 / 53.2 / 54.4, 83.4 / 78.2 / 75.9,
// 109.2 / 101.5 / 97.8.  With the backward, 16384 x 2048 bf16-bf16, 2 / 1 pieces
// 114.0 / 102.7.  Then two pieces (4096 x 8000, against one piece and 16 waves:
// 53.7 / 61.2, 77.7 / 81.2, 102.7 / 105.6), then four (2048 x 16384, against two
// and 16 waves: 59.6 / 66.8, 86.7 / 93.2, 114.3 / 121.8), then 16 waves, whose
// backward spills (1024 x 32768 training step 332, 434, 478 us where its bytes take
// 104, 182, 208 at a copy's rate; 2048 x 16384, which spills a few, 129, 216, 246).
//
// one_wave: a row of two waves takes one of two pieces.  For forward bf16 rows
// that end inside a piece, where the wave with the end keeps the other waiting.
// Two waves / one: with a bf16 residual 30000 x 777 48.6 / 44.0, 16384 x 1001 30.6
// / 27.7, 65000 x 1023 128.9 / 115.3, 40000 x 515 50.7 / 49.3; with an fp32 residual
// 62.2 / 61.2, 43.6 / 44.6, 175.1 / 176.5, 58.2 / 56.6.  Rows of whole pieces, and
// fp32, where the loads cover it, gain or lose up to 9% by the width: bf16-bf16 30000 x
// 776 39.0 / 39.9, 40000 x 600 45.0 / 43.2; fp32 16384 x 1001 56.6 / 57.5, 40000 x
// 600 85.0 / 78.7.
NormPlan norm_plan(int64_t dim, bool one_wave) {
  NormPlan p;
  p.group = 8;
  while (p.group < 64 && p.group * kPiece < dim) p.group *= 2;
  p.pieces = p.row_waves = 1;
  const auto holds = [&] { return (int64_t)p.group * kPiece * p.pieces * p.row_waves >= dim; };
  if (!holds() && one_wave && dim <= 2 * 64 * kPiece) p.pieces = 2;
  while (!holds() && p.row_waves < 8) p.row_waves *= 2;
  if (!holds()) p.pieces = 2;
  if (!holds()) p.pieces = 4;
  if (!holds()) p.row_waves = 16;
  p.threads = 256;
  p.blocks = 0;
  return p;
}

NormPlan fwd_plan(int64_t rows, int64_t dim, ssm_dtype_t io) {
  NormPlan p = norm_plan(dim, io == SSM_BF16 && dim % kPiece != 0);
  if (p.row_waves > 1) {
    p.threads = 64 * p.row_waves;
    p.blocks = rows;
  } else {
    const int64_t per_block = 4 * (64 / p.group);
    p.blocks = (rows + per_block - 1) / per_block;
  }
  return p;
}

// Two blocks to a compute unit, each with a partial row of column sums; one
// where a row takes the whole block and the partial rows are long.  Training
// steps with a residual, 256 / 512 blocks, us for io-residual bf16-bf16, bf16-fp32,
// fp32-fp32: 2048 x 16384 129 / 139, 216 / 233, 245 / 262; 4096 x 8000 102 / 113,
// 189 / 195, 215 / 223; 8192 x 4096 119 / 105, 183 / 184, 206 / 211 (in bf16 alone the
// second block's loads count for more); 8191 x 1001, four rows to a block, 44 / 38,
// 60 / 56, 61 / 58; 16384 x 2048, two rows to a block, 113 / 99, 183 / 184, 209 /
// 213.  128 blocks lose everywhere.
NormPlan bwd_plan(int64_t rows, int64_t dim) {
  NormPlan p = norm_plan(dim, false);
  const int waves = std::max(p.row_waves, kBwdWaves);
  p.threads = 64 * waves;
  const int64_t groups = (int64_t)(waves / p.row_waves) * (64 / p.group);
  const int64_t most = p.row_waves < kBwdWaves ? 512 : 256;
  p.blocks = std::min<int64_t>(most, (rows + groups - 1) / groups);
  return p;
}

#define SSM_NORM_GEOMETRY(CALL)                  \
  switch (p.group) {                             \
    case 8: CALL(8, 1); break;                   \
    case 16: CALL(16, 1); break;                 \
    case 32: CALL(32, 1); break;                 \
    default:                                     \
      if (p.pieces == 1) { CALL(64, 1); }        \
      else if (p.pieces == 2) { CALL(64, 2); }   \
      else { CALL(64, 4); }                      \
  }

template <typename IoT, typename ResT, bool kRms, bool kRes>
hipError_t launch_norm_fwd(const NormFwdArgs& a, const NormPlan& p, hipStream_t st) {
#define SSM_NORM_CALL(G, K)                                                                                 \
  hipLaunchKernelGGL((norm_fwd_kernel<IoT, ResT, G, K, kRms, kRes>), dim3((unsigned)p.blocks),              \
                     dim3(p.threads), 0, st, a)
  SSM_NORM_GEOMETRY(SSM_NORM_CALL)
#undef SSM_NORM_CALL
  return hipGetLastError();
}

template <typename IoT, typename ResT>
hipError_t launch_norm_fwd(const NormFwdArgs& a, const NormPlan& p, bool rms, hipStream_t st) {
  if (a.residual)
    return rms ? launch_norm_fwd<IoT, ResT, true, true>(a, p, st) : launch_norm_fwd<IoT, ResT, false, true>(a, p, st);
  if constexpr (sizeof(IoT) == sizeof(ResT))  // without a residual its type is the io type
    return rms ? launch_norm_fwd<IoT, ResT, true, false>(a, p, st) : launch_norm_fwd<IoT, ResT, false, false>(a, p, st);
  return hipErrorInvalidValue;
}

template <typename IoT, typename ResT, bool kRms>
hipError_t launch_norm_bwd(const NormBwdArgs& a, const NormPlan& p, hipStream_t st) {
  // Blocks of several row groups join their column sums: kBwdWaves waves of
  // 2 x lanes x 8 floats, at most 32 KB (such rows have one piece).
  const bool join = a.part && p.threads > 64 * p.row_waves;
  const size_t lds = join ? (size_t)(p.threads / 64) * 2 * p.pieces * p.group * kPiece * 4 : 0;
#define SSM_NORM_CALL(G, K)                                                                                     \
  hipLaunchKernelGGL((norm_bwd_kernel<IoT, ResT, G, K, kRms, 64 * kBwdWaves>), dim3((unsigned)p.blocks),        \
                     dim3(p.threads), lds, st, a)
  if (p.threads > 64 * kBwdWaves)
    hipLaunchKernelGGL((norm_bwd_kernel<IoT, ResT, 64, 4, kRms, 64 * kMaxRowWaves>), dim3((unsigned)p.blocks),
                       dim3(p.threads), lds, st, a);
  else
    SSM_NORM_GEOMETRY(SSM_NORM_CALL)
#undef SSM_NORM_CALL
  return hipGetLastError();
}

template <typename IoT, typename ResT>
hipError_t launch_norm_bwd(const NormBwdArgs& a, const NormPlan& p, bool rms, hipStream_t st) {
  return rms ? launch_norm_bwd<IoT, ResT, true>(a, p, st) : launch_norm_bwd<IoT, ResT, false>(a, p, st);
}

ssm_status_t norm_shape(int64_t rows, int64_t dim, ssm_dtype_t io, ssm_dtype_t res_io, int64_t* n) {
  if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_DTYPE;
  if (res_io != io && res_io != SSM_F32) return SSM_ERR_DTYPE;
  if (rows < 1 || dim < 1) return SSM_ERR_SHAPE;
  int64_t bytes;
  if (!mul_ok(rows, dim, n) || !mul_ok(*n, 8, &bytes)) return SSM_ERR_SHAPE;
  if (dim > kMaxDim || rows >= ((int64_t)1 << 31)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

bool norm_kind_ok(ssm_norm_t kind) { return kind == SSM_NORM_LAYER || kind == SSM_NORM_RMS; }

}  // namespace

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------

extern "C" {

ssm_status_t ssm_norm_fwd(int64_t rows, int64_t dim, ssm_dtype_t io, ssm_dtype_t res_io, ssm_norm_t kind,
                          const void* x, const void* residual, const float* weight, const float* bias, float eps,
                          void* y, void* s, float* mean, float* rstd, struct ihipStream_t* stream) {
  int64_t n;
  ssm_status_t st = norm_shape(rows, dim, io, res_io, &n);
  if (st != SSM_OK) return st;
  const NormPlan p = fwd_plan(rows, dim, io);
  if (!norm_kind_ok(kind) || !launch_ok(p.blocks, p.threads)) return SSM_ERR_UNSUPPORTED;
  if (!residual && res_io != io) return SSM_ERR_DTYPE;
  if (!x || !y || (s && !residual)) return SSM_ERR_NULL;
  if (kind == SSM_NORM_RMS) mean = nullptr;
  const size_t es = io_size(io), rs = io_size(res_io);
  const bool in_place = residual && s == residual;
  const Buf ins[] = {{x, n * (int64_t)es, es}, {in_place ? nullptr : residual, n * (int64_t)rs, rs},
                     {weight, dim * 4, 4}, {bias, dim * 4, 4}};
  const Buf outs[] = {{y, n * (int64_t)es, es}, {s, n * (int64_t)rs, rs}, {mean, rows * 4, 4}, {rstd, rows * 4, 4}};
  st = check_buffers(ins, 4, outs, 4);
  if (st != SSM_OK) return st;
  NormFwdArgs a;
  a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.y = y; a.s = s; a.mean = mean; a.rstd = rstd;
  a.rows = rows; a.dim = (int)dim; a.row_waves = p.row_waves; a.eps = eps;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  const bool rms = kind == SSM_NORM_RMS;
  hipError_t e;
  if (io == SSM_F32)
    e = launch_norm_fwd<float, float>(a, p, rms, hs);
  else if (res_io == SSM_BF16)
    e = launch_norm_fwd<bf16_t, bf16_t>(a, p, rms, hs);
  else
    e = launch_norm_fwd<bf16_t, float>(a, p, rms, hs);
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

ssm_status_t ssm_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, ssm_dtype_t io, ssm_dtype_t res_io,
                                          int64_t* bytes) {
  int64_t n;
  ssm_status_t st = norm_shape(rows, dim, io, res_io, &n);
  if (st == SSM_OK && bytes) *bytes = bwd_plan(rows, dim).blocks * 2 * dim * 4;
  return st;
}

ssm_status_t ssm_norm_bwd(int64_t rows, int64_t dim, ssm_dtype_t io, ssm_dtype_t res_io, ssm_norm_t kind,
                          const void* dy, const void* s, const float* weight, const float* mean, const float* rstd,
                          const void* ds_out, void* dx, void* dresidual, float* dweight, float* dbias,
                          void* workspace, int64_t workspace_bytes, struct ihipStream_t* stream) {
  int64_t n;
  ssm_status_t st = norm_shape(rows, dim, io, res_io, &n);
  if (st != SSM_OK) return st;
  if (!norm_kind_ok(kind)) return SSM_ERR_UNSUPPORTED;
  if (!dy || !s || !rstd || !dx || (kind == SSM_NORM_LAYER && !mean)) return SSM_ERR_NULL;
  if (kind == SSM_NORM_RMS) mean = nullptr;
  const NormPlan p = bwd_plan(rows, dim);
  const bool sums = dweight || dbias;
  const int64_t need = sums ? p.blocks * 2 * dim * 4 : 0;
  if (workspace_bytes < need) return SSM_ERR_WORKSPACE;
  if (need && !workspace) return SSM_ERR_NULL;
  if (!need) workspace = nullptr;
  const size_t es = io_size(io), rs = io_size(res_io);
  const Buf ins[] = {{dy, n * (int64_t)es, es}, {s, n * (int64_t)rs, rs}, {weight, dim * 4, 4}, {mean, rows * 4, 4},
                     {rstd, rows * 4, 4}, {ds_out, n * (int64_t)rs, rs}};
  const Buf outs[] = {{dx, n * (int64_t)es, es}, {dresidual, n * (int64_t)rs, rs}, {dweight, dim * 4, 4},
                      {dbias, dim * 4, 4}, {workspace, need, 4}};
  st = check_buffers(ins, 6, outs, 5);
  if (st != SSM_OK) return st;
  NormBwdArgs a;
  a.dy = dy; a.s = s; a.weight = weight; a.mean = mean; a.rstd = rstd; a.ds_out = ds_out; a.dx = dx;
  a.dres = dresidual; a.part = static_cast<float*>(workspace); a.rows = rows; a.dim = (int)dim;
  a.row_waves = p.row_waves;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  const bool rms = kind == SSM_NORM_RMS;
  hipError_t e;
  if (io == SSM_F32)
    e = launch_norm_bwd<float, float>(a, p, rms, hs);
  else if (res_io == SSM_BF16)
    e = launch_norm_bwd<bf16_t, bf16_t>(a, p, rms, hs);
  else
    e = launch_norm_bwd<bf16_t, float>(a, p, rms, hs);
  if (e == hipSuccess && sums) {
    hipLaunchKernelGGL(norm_bwd_reduce_kernel, dim3((unsigned)((2 * dim + 31) / 32)), dim3(1024), 0, hs, a.part,
                       dweight, dbias, (int)p.blocks, (int)dim);
    e = hipGetLastError();
  }
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

}  // extern "C"
