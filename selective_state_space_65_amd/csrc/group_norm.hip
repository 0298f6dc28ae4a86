// group_norm.hip -- group norm over channels-last arrays, with an activation
// and an output gate behind it: forward and backward.  C ABI:
// include/ssm_scan.h.
//
// Two layouts of a group's numbers.
//
// One position (length 1, the norm behind attention's heads): a group is one
// contiguous run of d = channels / groups numbers, held in registers by G lanes
// (8 to 64, up to 4 pieces of 8 a lane) from its one read to its write.  The
// backward gives a group of lanes many batch rows of the same channels, whose
// sums it keeps in registers.  Bound by memory: 16384 x 16 groups of 128 bf16 with a
// gate 45 us forward and 67 + 5 us backward, where a copy of the bytes takes 39 and
// 65.
//
// A map (length above 1, or d above what a wave holds): a block takes a run of
// positions with all their channels, a thread 8 channels and every TY-th of the
// positions, so that all reads are contiguous; channels are joined into groups
// at the end of the run, runs by a small second kernel, and a last kernel reads
// the numbers again and writes.  The variance is joined, from a thread's few numbers
// in flight up to the whole group, from means and sums of squares about them,
//   M = m1 + (m2 - m1) c2 / (c1 + c2),   Q = q1 + q2 + (m2 - m1)^2 c1 c2 / (c1 + c2),
// so that a number far off the others does not blur them; and each run of a channel
// is taken less its first number, so that a large mean does not.  8 x 4096 x 512 bf16
// with an activation: statistics 12 us and output 16 forward, sums 17 and dx 20
// backward, 4 us for each of the three small kernels between (a copy of one array's
// bytes takes 13); the last two move bytes at a copy's rate, the first two are as
// much the time of a block's one or two trips to memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device_common.h"
#include "host_common.h"
#include "lane_rows.h"
#include "ssm_scan.h"

namespace {

constexpr int kMostRun = 64 * kPiece * 4;  // numbers a wave holds
constexpr int kThreads = 256;

struct Args {
  const void* x;
  const void* z;        // may be null
  const float* weight;  // may be null
  const float* bias;    // may be null
  void* y;              // forward
  float* mean;          // [batch, groups]; may be null
  float* rstd;          // [batch, groups]; may be null in the forward
  const void* dy;       // backward from here
  void* dx;
  void* dz;             // may be null
  float* part;          // partial sums, may be null
  float* sums;          // [2][batch, groups]
  int64_t batch, length, channels;
  int groups, d;        // d channels in a group
  int rms, silu;
  float eps;
  int runs;             // maps: blocks along the positions
  int64_t run;          // maps: positions of a block
  int64_t stride;       // one position, backward: batch rows between two of a lane's
};

__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_hw(1.0f + exp2_hw(-x * kLog2e)); }

// f = p or silu(p), and its slope.
__device__ __forceinline__ float activate(float p, bool silu, float* slope) {
  if (!silu) {
    *slope = 1.0f;
    return p;
  }
  const float s = sigmoid_f32(p);
  *slope = s * __builtin_fmaf(p, 1.0f - s, 1.0f);
  return p * s;
}

// y of one number.
__device__ __forceinline__ float output(float n, float w, float b, float z, bool silu, bool gated) {
  float slope;
  const float f = activate(__builtin_fmaf(n, w, b), silu, &slope);
  return gated ? f * silu_f32(z) : f;
}

// dL/dp of one number, p the activation's input, and dL/dz.
__device__ __forceinline__ float inner(float n, float w, float b, float z, float dy, bool silu, bool gated, float* dz) {
  float slope;
  const float f = activate(__builtin_fmaf(n, w, b), silu, &slope);
  *dz = 0.0f;
  if (gated) {
    float gate_slope;
    const float gate = activate(z, true, &gate_slope);
    *dz = dy * f * gate_slope;
    dy *= gate;
  }
  return dy * slope;
}

__device__ __forceinline__ void fill(float v[kPiece], float x) {
#pragma unroll
  for (int j = 0; j < kPiece; ++j) v[j] = x;
}

// ---- one position -------------------------------------------------------------

template <int G, typename T>
__device__ __forceinline__ void piece(const T* row, int c, int gl, int d, float out[kPiece]) {
  Raw8<T> r = request_piece<G>(row, c, gl, d);
  finish_piece<G>(r, c, gl, d);
  r.get(out);
}

// Groups that G lanes have in flight: more bytes, and half the blocks.
constexpr int rows_ahead(int K) { return K == 1 ? 2 : 1; }

template <typename T, int G, int K, bool kGated>
__global__ __launch_bounds__(kThreads) void group_norm_row_fwd_kernel(const Args p) {
  constexpr int U = rows_ahead(K);
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t rows = p.batch * p.groups;
  const int64_t row0 = ((int64_t)blockIdx.x * (kThreads / 64) + wave) * (64 / G) * U + lane / G;
  const int d = p.d;
  const float count = (float)d;
  int64_t at[U];
  Raw8<T> px[U][K], pz[U][K];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = min(row0 + u * (64 / G), rows - 1) * d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      px[u][k] = request_piece<G>(static_cast<const T*>(p.x) + at[u], (k * G + gl) * kPiece, gl, d);
      if constexpr (kGated)
        pz[u][k] = request_piece<G>(static_cast<const T*>(p.z) + at[u], (k * G + gl) * kPiece, gl, d);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * (64 / G);
    const int first = (int)(min(row, rows - 1) % p.groups) * d;
    float v[K][kPiece], t = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      finish_piece<G>(px[u][k], (k * G + gl) * kPiece, gl, d);
      px[u][k].get(v[k]);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) t += v[k][j];
    }
    const float mean = p.rms ? 0.0f : group_sum<G>(t) / count;
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        const float e = (k * G + gl) * kPiece + j < d ? v[k][j] - mean : 0.0f;
        q = __builtin_fmaf(e, e, q);
      }
    const float rstd = 1.0f / __builtin_sqrtf(group_sum<G>(q) / count + p.eps);
    if (row >= rows) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + gl) * kPiece;
      float w[kPiece], b[kPiece], z[kPiece], o[kPiece];
      fill(w, 1.0f);
      fill(b, 0.0f);
      fill(z, 0.0f);
      if (p.weight) piece<G>(p.weight + first, c, gl, d, w);
      if (p.bias) piece<G>(p.bias + first, c, gl, d, b);
      if constexpr (kGated) {
        finish_piece<G>(pz[u][k], c, gl, d);
        pz[u][k].get(z);
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) o[j] = output((v[k][j] - mean) * rstd, w[j], b[j], z[j], p.silu, kGated);
      store_row8(static_cast<T*>(p.y) + at[u], c, d, whole<G>(c, gl, d), o);
    }
    if (gl == 0) {
      if (!p.rms && p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

// A group of lanes has one group of channels and every stride-th batch row.
template <typename T, int G, int K, bool kGated>
__global__ __launch_bounds__(kThreads) void group_norm_row_bwd_kernel(const Args p) {
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = ((int64_t)blockIdx.x * (kThreads / 64) + wave) * (64 / G) + lane / G;
  const int d = p.d, group = (int)(id % p.groups);
  const int64_t b0 = id / p.groups;
  const int64_t sweeps = (p.batch + p.stride - 1) / p.stride;
  float w[K][kPiece], b[K][kPiece], aw[K][kPiece], ab[K][kPiece];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * G + gl) * kPiece;
    fill(w[k], 1.0f);
    fill(b[k], 0.0f);
    fill(aw[k], 0.0f);
    fill(ab[k], 0.0f);
    if (p.weight) piece<G>(p.weight + (int64_t)group * d, c, gl, d, w[k]);
    if (p.bias) piece<G>(p.bias + (int64_t)group * d, c, gl, d, b[k]);
  }
  const float inv = 1.0f / (float)d;
  for (int64_t i = 0; i < sweeps; ++i) {
    const int64_t at_b = b0 + i * p.stride;
    const bool live = b0 < p.stride && at_b < p.batch;
    const int64_t row = (live ? at_b : 0) * p.groups + group, at = row * d;
    const float mean = p.rms ? 0.0f : p.mean[row], rstd = p.rstd[row];
    float n[K][kPiece], g[K][kPiece], dz[K][kPiece];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + gl) * kPiece;
      float z[kPiece];
      piece<G>(static_cast<const T*>(p.x) + at, c, gl, d, n[k]);
      piece<G>(static_cast<const T*>(p.dy) + at, c, gl, d, g[k]);  // 0 past the run: so is all that follows
      fill(z, 0.0f);
      if constexpr (kGated) piece<G>(static_cast<const T*>(p.z) + at, c, gl, d, z);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        n[k][j] = (n[k][j] - mean) * rstd;
        const float dp = inner(n[k][j], w[k][j], b[k][j], z[j], g[k][j], p.silu, kGated, &dz[k][j]);
        if (live) {
          aw[k][j] = __builtin_fmaf(dp, n[k][j], aw[k][j]);
          ab[k][j] += dp;
        }
        g[k][j] = dp * w[k][j];
        c1 += g[k][j];
        c2 = __builtin_fmaf(g[k][j], n[k][j], c2);
      }
    }
    c1 = p.rms ? 0.0f : group_sum<G>(c1) * inv;
    c2 = group_sum<G>(c2) * inv;
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * G + gl) * kPiece;
      float o[kPiece];
#pragma unroll
      for (int j = 0; j < kPiece; ++j) o[j] = rstd * __builtin_fmaf(-n[k][j], c2, g[k][j] - c1);
      store_row8(static_cast<T*>(p.dx) + at, c, d, whole<G>(c, gl, d), o);
      if (kGated && p.dz) store_row8(static_cast<T*>(p.dz) + at, c, d, whole<G>(c, gl, d), dz[k]);
    }
  }
  if (!p.part || b0 >= p.stride) return;
  float* part = p.part + b0 * 2 * p.channels + (int64_t)group * d;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * G + gl) * kPiece;
    store_row8(part, c, d, whole<G>(c, gl, d), aw[k]);
    store_row8(part + p.channels, c, d, whole<G>(c, gl, d), ab[k]);
  }
}

// dweight and dbias from partial rows of 2 x channels: 32 columns a block, 32
// slices of the rows, added in order and in 64 bits.
__global__ __launch_bounds__(1024) void group_norm_columns_kernel(const float* part, float* dweight, float* dbias,
                                                                  int64_t rows, int64_t channels) {
  __shared__ double sums[32][33];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + col;
  double t = 0.0;
  if (c < 2 * channels) {
    int64_t r = slice;
    for (; r + 7 * 32 < rows; r += 8 * 32) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = part[(r + j * 32) * 2 * channels + c];
#pragma unroll
      for (int j = 0; j < 8; ++j) t += (double)v[j];
    }
    for (; r < rows; r += 32) t += (double)part[r * 2 * channels + c];
  }
  sums[slice][col] = t;
  __syncthreads();
  if (slice == 0 && c < 2 * channels) {
#pragma unroll
    for (int i = 1; i < 32; ++i) t += sums[i][col];
    float* out = c < channels ? dweight : dbias;
    if (out) out[c < channels ? c : c - channels] = (float)t;
  }
}

// ---- maps ----------------------------------------------------------------------

// A block's threads: TX along the channels (8 each), TY along the positions; wide
// maps take several columns of TX.
struct Plane {
  int tx, ty, x, y;
  int half;  // the largest power of 2 below ty, 0 for one row: where sums over the rows start to be joined
};

__device__ __forceinline__ Plane plane(int64_t channels) {
  const int pieces = (int)((channels + kPiece - 1) / kPiece);
  Plane t;
  t.tx = min(pieces, kThreads);
  t.ty = kThreads / t.tx;
  t.x = threadIdx.x % t.tx;
  t.y = threadIdx.x / t.tx;
  t.half = t.ty > 1 ? 1 << (31 - __builtin_clz(t.ty - 1)) : 0;
  return t;
}

// kShort: fewer than 8 channels.  A kernel of its own: the branch it takes to a
// load would have each load waited for.
template <bool kShort, typename T>
__device__ __forceinline__ Raw8<T> request_at(const T* row, int c, int n) {
  return request8<kShort>(row, c, 0, n);
}

template <bool kShort, typename T>
__device__ __forceinline__ void finish_at(Raw8<T>& r, int c, int n, float out[kPiece]) {
  finish8<kShort>(r, c, 0, n);
  r.get(out);
}

// Positions that a thread has in flight: 128 bytes of one to three arrays.
template <typename T, int kArrays>
constexpr int kAhead = kArrays == 1 ? 16 / sizeof(T) : kArrays == 2 ? 8 / sizeof(T) : 2;

// Mean and squares about it of the groups that columns [c0, c1) have, from their
// columns' means and squares; G lanes a group.  A group that began in an earlier
// column is joined with what is there.
template <int G>
__device__ __forceinline__ void join_columns(const Args& p, const float* means, const float* squares, int c0, int c1,
                                             float count, float* out) {
  const int gl = threadIdx.x & (G - 1);
  for (int g = c0 / p.d + threadIdx.x / G; g <= (c1 - 1) / p.d; g += kThreads / G) {
    const int lo = max(g * p.d, c0) - c0, hi = min((g + 1) * p.d, c1) - c0;
    const float here = (float)(hi - lo);
    float m = 0.0f, q = 0.0f;
    for (int i = lo + gl; i < hi; i += G) m += means[i];
    m = group_sum<G>(m) / here;
    for (int i = lo + gl; i < hi; i += G) {
      const float e = means[i] - m;
      q += __builtin_fmaf(count * e, e, squares[i]);
    }
    q = group_sum<G>(q);
    if (gl) continue;
    if (g * p.d < c0) {
      const float before = (float)(c0 - g * p.d), m0 = out[g], all = before + here, e = m - m0;
      m = m0 + e * (here / all);
      q += out[p.groups + g] + count * e * e * (before * here / all);
    }
    out[g] = m;
    out[p.groups + g] = q;
  }
}

// part[batch][run][2][groups]: each run's means, and sums of squares about them.
template <typename T, bool kShort>
__global__ __launch_bounds__(kThreads) void group_norm_map_stats_kernel(const Args p) {
  __shared__ float cols[2][kThreads * kPiece], counts[kThreads];
  const Plane t = plane(p.channels);
  const int64_t batch = blockIdx.x / p.runs;
  const int run = (int)(blockIdx.x % p.runs);
  const int64_t l0 = run * p.run, l1 = min(l0 + p.run, p.length);
  const float count = (float)(l1 - l0);
  const int n = (int)p.channels;
  const T* x = static_cast<const T*>(p.x) + batch * p.length * n;
  float* out = p.part + (batch * p.runs + run) * 2 * p.groups;
  for (int c0 = 0; c0 < n; c0 += t.tx * kPiece) {
    const int c = c0 + t.x * kPiece;
    const bool live = t.y < t.ty && c < n;
    // Of the thread's own positions, less the run's first number.
    float pivot[kPiece], mean[kPiece], squares[kPiece], seen = 0.0f;
    fill(mean, 0.0f);
    fill(squares, 0.0f);
    if (live) {
      Raw8<T> first = request_at<kShort>(x + l0 * n, c, n);
      for (int64_t l = l0 + t.y; l < l1; l += kAhead<T, 1> * t.ty) {
        Raw8<T> r[kAhead<T, 1>];
        float v[kAhead<T, 1>][kPiece];
#pragma unroll
        for (int u = 0; u < kAhead<T, 1>; ++u) r[u] = request_at<kShort>(x + min(l + u * t.ty, l1 - 1) * n, c, n);
        if (l == l0 + t.y) {
          finish_at<kShort>(first, c, n, pivot);
          if (p.rms) fill(pivot, 0.0f);
        }
        float more = 0.0f;
#pragma unroll
        for (int u = 0; u < kAhead<T, 1>; ++u) {
          finish_at<kShort>(r[u], c, n, v[u]);
          more += l + u * t.ty < l1 ? 1.0f : 0.0f;
        }
        const float one = 1.0f / more, share = more / (seen + more), both = seen * share;
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
          float m = 0.0f, q = 0.0f;
#pragma unroll
          for (int u = 0; u < kAhead<T, 1>; ++u) {
            v[u][j] -= pivot[j];
            m += l + u * t.ty < l1 ? v[u][j] : 0.0f;
          }
          m = p.rms ? 0.0f : m * one;
#pragma unroll
          for (int u = 0; u < kAhead<T, 1>; ++u) {
            const float e = l + u * t.ty < l1 ? v[u][j] - m : 0.0f;
            q = __builtin_fmaf(e, e, q);
          }
          const float e = m - mean[j];
          mean[j] = __builtin_fmaf(e, share, mean[j]);
          squares[j] += __builtin_fmaf(e * both, e, q);
        }
        seen += more;
      }
    }
    // Over the block's rows of threads, by halves; a thread's place in cols is, in row 0,
    // that of its channels.
    float* const means = &cols[0][threadIdx.x * kPiece];
    float* const sums = &cols[1][threadIdx.x * kPiece];
    const auto keep = [&](bool whole) {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        means[j] = whole && !p.rms ? pivot[j] + mean[j] : mean[j];
        sums[j] = squares[j];
      }
      counts[threadIdx.x] = seen;
    };
    __syncthreads();
    if (live) keep(t.half == 0);
    for (int step = t.half; step > 0; step /= 2) {
      __syncthreads();
      if (!live || t.y >= step || t.y + step >= t.ty) continue;
      const int other = step * t.tx;
      const float more = counts[threadIdx.x + other];
      if (more > 0.0f) {
        const float share = more / (seen + more), both = seen * share;
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
          const float e = means[other * kPiece + j] - mean[j];
          mean[j] = __builtin_fmaf(e, share, mean[j]);
          squares[j] += __builtin_fmaf(e * both, e, sums[other * kPiece + j]);
        }
        seen += more;
      }
      keep(step == 1);
    }
    __syncthreads();
    const int c1 = min(n, c0 + t.tx * kPiece);
    if (p.d <= 8)
      join_columns<8>(p, cols[0], cols[1], c0, c1, count, out);
    else if (p.d <= 32)
      join_columns<16>(p, cols[0], cols[1], c0, c1, count, out);
    else
      join_columns<64>(p, cols[0], cols[1], c0, c1, count, out);
  }
}

// Runs joined: mean and rstd of a (batch, group), a wave each.
__global__ __launch_bounds__(kThreads) void group_norm_map_join_kernel(const Args p) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= p.batch * p.groups) return;
  const int64_t batch = row / p.groups;
  const int g = (int)(row % p.groups);
  const float* part = p.part + batch * p.runs * 2 * p.groups + g;
  // Means and squares about the first run's mean.
  const double all = (double)p.length, m0 = (double)part[0];
  double m = 0.0, q = 0.0;
  for (int r = lane; r < p.runs; r += 64) {
    const double count = (double)(min(r * p.run + p.run, p.length) - r * p.run);
    const double e = (double)part[(int64_t)r * 2 * p.groups] - m0;
    m += count * e;
    q += (double)part[((int64_t)r * 2 + 1) * p.groups] + count * (double)p.d * e * e;
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    m += __shfl_xor(m, s);
    q += __shfl_xor(q, s);
  }
  if (lane == 0) {
    q -= m * m / all * (double)p.d;
    if (p.mean) p.mean[row] = (float)(m0 + m / all);
    p.rstd[row] = (float)(1.0 / __builtin_sqrt(q / (all * p.d) + (double)p.eps));
  }
}

// What a thread's 8 channels have in common over the positions.
struct Columns {
  float w[kPiece], b[kPiece], mean[kPiece], rstd[kPiece];
};

// f(j, group of channel c + j), with one division.
template <typename F>
__device__ __forceinline__ void each_group(const Args& p, int c, int n, F f) {
  int g = c / p.d, left = p.d - (c - g * p.d);
#pragma unroll
  for (int j = 0; j < kPiece; ++j) {
    f(j, g);
    if (--left == 0 && c + j + 1 < n) ++g, left = p.d;
  }
}

template <bool kShort>
__device__ __forceinline__ void load_columns(const Args& p, int64_t batch, int c, int n, Columns* k) {
  fill(k->w, 1.0f);
  fill(k->b, 0.0f);
  if (p.weight) {
    Raw8<float> r = request_at<kShort>(p.weight, c, n);
    finish_at<kShort>(r, c, n, k->w);
  }
  if (p.bias) {
    Raw8<float> r = request_at<kShort>(p.bias, c, n);
    finish_at<kShort>(r, c, n, k->b);
  }
  each_group(p, c, n, [&](int j, int g) {
    const int64_t row = batch * p.groups + g;
    k->mean[j] = p.rms ? 0.0f : p.mean[row];
    k->rstd[j] = p.rstd[row];
  });
}

template <typename T, bool kGated, bool kShort>
__global__ __launch_bounds__(kThreads) void group_norm_map_fwd_kernel(const Args p) {
  const Plane t = plane(p.channels);
  const int64_t batch = blockIdx.x / p.runs;
  const int run = (int)(blockIdx.x % p.runs);
  const int64_t l0 = run * p.run, l1 = min(l0 + p.run, p.length);
  const int n = (int)p.channels;
  const int64_t base = batch * p.length * n;
  if (t.y >= t.ty) return;
  for (int c = t.x * kPiece; c < n; c += t.tx * kPiece) {
    Columns k;
    load_columns<kShort>(p, batch, c, n, &k);
    for (int64_t l = l0 + t.y; l < l1; l += kAhead<T, kGated ? 2 : 1> * t.ty) {
      Raw8<T> rx[kAhead<T, kGated ? 2 : 1>], rz[kAhead<T, kGated ? 2 : 1>];
#pragma unroll
      for (int u = 0; u < kAhead<T, kGated ? 2 : 1>; ++u) {
        const int64_t at = base + min(l + u * t.ty, l1 - 1) * n;
        rx[u] = request_at<kShort>(static_cast<const T*>(p.x) + at, c, n);
        if constexpr (kGated) rz[u] = request_at<kShort>(static_cast<const T*>(p.z) + at, c, n);
      }
#pragma unroll
      for (int u = 0; u < kAhead<T, kGated ? 2 : 1>; ++u) {
        if (l + u * t.ty >= l1) break;
        float v[kPiece], z[kPiece];
        finish_at<kShort>(rx[u], c, n, v);
        fill(z, 0.0f);
        if constexpr (kGated) finish_at<kShort>(rz[u], c, n, z);
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
          v[j] = output((v[j] - k.mean[j]) * k.rstd[j], k.w[j], k.b[j], z[j], p.silu, kGated);
        store_row8(static_cast<T*>(p.y) + base + (l + u * t.ty) * n, c, n, c + kPiece <= n, v);
      }
    }
  }
}

// part[batch][run][2][channels]: sums of dp n and of dp.
template <typename T, bool kGated, bool kShort>
__global__ __launch_bounds__(kThreads) void group_norm_map_sums_kernel(const Args p) {
  __shared__ float cols[2][kThreads * kPiece];
  const Plane t = plane(p.channels);
  const int64_t batch = blockIdx.x / p.runs;
  const int run = (int)(blockIdx.x % p.runs);
  const int64_t l0 = run * p.run, l1 = min(l0 + p.run, p.length);
  const int n = (int)p.channels;
  const int64_t base = batch * p.length * n;
  float* out = p.part + (batch * p.runs + run) * 2 * n;
  for (int c0 = 0; c0 < n; c0 += t.tx * kPiece) {
    const int c = c0 + t.x * kPiece;
    const bool live = t.y < t.ty && c < n;
    float aw[kPiece], ab[kPiece];
    fill(aw, 0.0f);
    fill(ab, 0.0f);
    if (live) {
      Columns k;
      load_columns<kShort>(p, batch, c, n, &k);
      for (int64_t l = l0 + t.y; l < l1; l += kAhead<T, kGated ? 3 : 2> * t.ty) {
        Raw8<T> rx[kAhead<T, kGated ? 3 : 2>], rd[kAhead<T, kGated ? 3 : 2>], rz[kAhead<T, kGated ? 3 : 2>];
#pragma unroll
        for (int u = 0; u < kAhead<T, kGated ? 3 : 2>; ++u) {
          const int64_t at = base + min(l + u * t.ty, l1 - 1) * n;
          rx[u] = request_at<kShort>(static_cast<const T*>(p.x) + at, c, n);
          rd[u] = request_at<kShort>(static_cast<const T*>(p.dy) + at, c, n);
          if constexpr (kGated) rz[u] = request_at<kShort>(static_cast<const T*>(p.z) + at, c, n);
        }
#pragma unroll
        for (int u = 0; u < kAhead<T, kGated ? 3 : 2>; ++u) {
          if (l + u * t.ty >= l1) break;
          float v[kPiece], d[kPiece], z[kPiece];
          finish_at<kShort>(rx[u], c, n, v);
          finish_at<kShort>(rd[u], c, n, d);
          fill(z, 0.0f);
          if constexpr (kGated) finish_at<kShort>(rz[u], c, n, z);
#pragma unroll
          for (int j = 0; j < kPiece; ++j) {
            float dz;
            const float m = (v[j] - k.mean[j]) * k.rstd[j];
            const float dp = inner(m, k.w[j], k.b[j], z[j], d[j], p.silu, kGated, &dz);
            aw[j] = __builtin_fmaf(dp, m, aw[j]);
            ab[j] += dp;
          }
        }
      }
    }
    float* const own_w = &cols[0][threadIdx.x * kPiece];
    float* const own_b = &cols[1][threadIdx.x * kPiece];
    const auto keep = [&] {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) own_w[j] = aw[j], own_b[j] = ab[j];
    };
    __syncthreads();
    if (live) keep();
    for (int step = t.half; step > 0; step /= 2) {
      __syncthreads();
      if (!live || t.y >= step || t.y + step >= t.ty) continue;
      const int other = step * t.tx * kPiece;
#pragma unroll
      for (int j = 0; j < kPiece; ++j) aw[j] += own_w[other + j], ab[j] += own_b[other + j];
      keep();
    }
    if (live && t.y == 0) {
      store_row8(out, c, n, c + kPiece <= n, aw);
      store_row8(out + n, c, n, c + kPiece <= n, ab);
    }
  }
}

// A batch row's runs of sums added into its first run's place, in 64 bits (there may
// be many): 32 columns of the 2 x channels a block, 16 slices of the runs, each added in order.
__global__ __launch_bounds__(512) void group_norm_map_columns_kernel(const Args p, int64_t tiles) {
  __shared__ double sums[16][33];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t batch = blockIdx.x / tiles, n = 2 * p.channels, c = blockIdx.x % tiles * 32 + col;
  float* part = p.part + batch * p.runs * n;
  double t = 0.0;
  if (c < n) {
    constexpr int kRows = 8;
    for (int r = slice; r < p.runs; r += kRows * 16) {
      float v[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) v[j] = part[min(r + j * 16, p.runs - 1) * n + c];
#pragma unroll
      for (int j = 0; j < kRows; ++j) t += r + j * 16 < p.runs ? (double)v[j] : 0.0;
    }
  }
  sums[slice][col] = t;
  __syncthreads();
  if (slice == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 16; ++i) t += sums[i][col];
    part[c] = (float)t;
  }
}

// sums[0 / 1][batch, group]: mean over the group of g n and of g (g = dp weight),
// a wave each; in the blocks behind those, dweight and dbias: 32 columns a block, 8
// slices of the batch rows, each added in order.  All in 64 bits: a group may have as many
// channels, and a call as many batch rows, as a sum in 32 bits loses its last bits over.
__global__ __launch_bounds__(kThreads) void group_norm_map_reduce_kernel(const Args p, int64_t group_blocks,
                                                                         float* dweight, float* dbias) {
  const int64_t n = p.channels, rows = p.batch * p.groups, pitch = p.runs * 2 * n;
  if (blockIdx.x >= group_blocks) {
    constexpr int kSlices = kThreads / 32, kRows = 8;  // rows in flight
    __shared__ double sums[kSlices][33];
    const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (blockIdx.x - group_blocks) * 32 + col;
    double t = 0.0;
    if (c < 2 * n) {
      for (int64_t b = slice; b < p.batch; b += kRows * kSlices) {
        float v[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) v[j] = p.part[min(b + j * kSlices, p.batch - 1) * pitch + c];
#pragma unroll
        for (int j = 0; j < kRows; ++j) t += b + j * kSlices < p.batch ? (double)v[j] : 0.0;
      }
    }
    sums[slice][col] = t;
    __syncthreads();
    float* out = c < n ? dweight : dbias;
    if (slice == 0 && c < 2 * n && out) {
#pragma unroll
      for (int i = 1; i < kSlices; ++i) t += sums[i][col];
      out[c < n ? c : c - n] = (float)t;
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t first = row % p.groups * p.d;
  const float* at = p.part + row / p.groups * pitch + first;
  double c1 = 0.0, c2 = 0.0;
  for (int i = lane; i < p.d; i += 64) {
    const double w = p.weight ? (double)p.weight[first + i] : 1.0;
    c2 = __builtin_fma((double)at[i], w, c2);
    c1 = __builtin_fma((double)at[n + i], w, c1);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    c1 += __shfl_xor(c1, m);
    c2 += __shfl_xor(c2, m);
  }
  if (lane == 0) {
    const double count = (double)p.length * (double)p.d;
    p.sums[row] = (float)(c2 / count);
    p.sums[rows + row] = (float)(c1 / count);
  }
}

template <typename T, bool kGated, bool kShort>
__global__ __launch_bounds__(kThreads) void group_norm_map_bwd_kernel(const Args p) {
  const Plane t = plane(p.channels);
  const int64_t batch = blockIdx.x / p.runs;
  const int run = (int)(blockIdx.x % p.runs);
  const int64_t l0 = run * p.run, l1 = min(l0 + p.run, p.length);
  const int n = (int)p.channels;
  const int64_t base = batch * p.length * n, rows = p.batch * p.groups;
  if (t.y >= t.ty) return;
  for (int c = t.x * kPiece; c < n; c += t.tx * kPiece) {
    Columns k;
    load_columns<kShort>(p, batch, c, n, &k);
    float c1[kPiece], c2[kPiece];
    each_group(p, c, n, [&](int j, int g) {
      const int64_t row = batch * p.groups + g;
      c2[j] = p.sums[row];
      c1[j] = p.rms ? 0.0f : p.sums[rows + row];
    });
    for (int64_t l = l0 + t.y; l < l1; l += kAhead<T, kGated ? 3 : 2> * t.ty) {
      Raw8<T> rx[kAhead<T, kGated ? 3 : 2>], rd[kAhead<T, kGated ? 3 : 2>], rz[kAhead<T, kGated ? 3 : 2>];
#pragma unroll
      for (int u = 0; u < kAhead<T, kGated ? 3 : 2>; ++u) {
        const int64_t at = base + min(l + u * t.ty, l1 - 1) * n;
        rx[u] = request_at<kShort>(static_cast<const T*>(p.x) + at, c, n);
        rd[u] = request_at<kShort>(static_cast<const T*>(p.dy) + at, c, n);
        if constexpr (kGated) rz[u] = request_at<kShort>(static_cast<const T*>(p.z) + at, c, n);
      }
#pragma unroll
      for (int u = 0; u < kAhead<T, kGated ? 3 : 2>; ++u) {
        if (l + u * t.ty >= l1) break;
        float v[kPiece], d[kPiece], z[kPiece], dz[kPiece];
        finish_at<kShort>(rx[u], c, n, v);
        finish_at<kShort>(rd[u], c, n, d);
        fill(z, 0.0f);
        if constexpr (kGated) finish_at<kShort>(rz[u], c, n, z);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
          const float m = (v[j] - k.mean[j]) * k.rstd[j];
          const float g = inner(m, k.w[j], k.b[j], z[j], d[j], p.silu, kGated, &dz[j]) * k.w[j];
          v[j] = k.rstd[j] * __builtin_fmaf(-m, c2[j], g - c1[j]);
        }
        const int64_t at = base + (l + u * t.ty) * n;
        store_row8(static_cast<T*>(p.dx) + at, c, n, c + kPiece <= n, v);
        if (kGated && p.dz) store_row8(static_cast<T*>(p.dz) + at, c, n, c + kPiece <= n, dz);
      }
    }
  }
}

// ---- host side ---------------------------------------------------------------

struct Plan {
  bool map;
  int lanes, pieces;    // one position: of a run of channels
  int64_t row_blocks;   // forward
  int64_t stride, bwd_blocks;
  int64_t runs, run;    // maps
};

Plan make_plan(int64_t batch, int64_t length, int64_t channels, int64_t groups) {
  Plan p = {};
  const int64_t d = channels / groups;
  p.map = length > 1 || d > kMostRun;
  if (!p.map) {
    p.lanes = 8;
    while (p.lanes < 64 && p.lanes * kPiece < d) p.lanes *= 2;
    p.pieces = 1;
    while ((int64_t)p.lanes * kPiece * p.pieces < d) p.pieces *= 2;
    const int64_t per_block = kThreads / p.lanes;
    const int64_t fwd_rows = per_block * rows_ahead(p.pieces);
    p.row_blocks = (batch * groups + fwd_rows - 1) / fwd_rows;
    // Batch rows side by side: 2048 blocks, but no more partial rows than 512, or than 2048
    // where those are not yet 512 blocks; and at most 256 batch rows to a lane: no sum gets long.
    const int64_t most = std::max<int64_t>(512, std::min<int64_t>(2048, 512 * per_block / groups));
    const int64_t least = (batch + 255) / 256;
    p.stride = std::min<int64_t>(batch, std::max<int64_t>(least, std::min<int64_t>(most, 2048 * per_block / groups)));
    p.bwd_blocks = (p.stride * groups + per_block - 1) / per_block;
  } else {
    const int64_t pieces = (channels + kPiece - 1) / kPiece;
    const int64_t ty = kThreads / std::min<int64_t>(pieces, kThreads);
    // Blocks for the whole chip, and at most 128 positions to a thread: no sum gets long.
    const int64_t wanted = std::max((1024 + batch - 1) / batch, (length + 128 * ty - 1) / (128 * ty));
    // Positions that a block's threads have in flight; but one where they go over several columns.
    const int64_t least = pieces > kThreads ? 1 : ty * 4;
    p.runs = std::max<int64_t>(1, std::min(wanted, (length + least - 1) / least));
    p.run = (length + p.runs - 1) / p.runs;
    p.runs = (length + p.run - 1) / p.run;
  }
  return p;
}

ssm_status_t check_shape(int64_t batch, int64_t length, int64_t channels, int64_t groups, ssm_dtype_t io, int64_t* n) {
  if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_DTYPE;
  if (batch < 1 || length < 1 || channels < 1 || groups < 1 || channels % groups) return SSM_ERR_SHAPE;
  int64_t bytes;
  if (!mul_ok(batch, length, n) || !mul_ok(*n, channels, n) || !mul_ok(*n, 64, &bytes)) return SSM_ERR_SHAPE;
  if (channels > 65536) return SSM_ERR_UNSUPPORTED;
  const Plan p = make_plan(batch, length, channels, groups);
  // A wave a (batch, group) and 512 threads for 32 sums of a batch row, between a map's passes.
  if (p.map && (!launch_ok(batch * groups, 64) || !launch_ok(batch * ((2 * channels + 31) / 32) + channels, 512)))
    return SSM_ERR_UNSUPPORTED;
  if (!launch_ok(p.map ? batch * p.runs : p.row_blocks, kThreads)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Workspace of the forward: maps' partial sums, and mean and rstd where they are not asked for.
int64_t fwd_bytes(const Plan& p, int64_t batch, int64_t groups) {
  return p.map ? (batch * p.runs * 2 * groups + 2 * batch * groups) * 4 : 0;
}

int64_t bwd_bytes(const Plan& p, int64_t batch, int64_t channels, int64_t groups, bool sums) {
  if (p.map) return (batch * p.runs * 2 * channels + 2 * batch * groups) * 4;
  return sums ? p.stride * 2 * channels * 4 : 0;
}

#define SSM_GROUP_NORM_GEOMETRY(CALL)                \
  switch (p.lanes) {                                 \
    case 8: CALL(8, 1); break;                       \
    case 16: CALL(16, 1); break;                     \
    case 32: CALL(32, 1); break;                     \
    default:                                         \
      if (p.pieces == 1) { CALL(64, 1); }            \
      else if (p.pieces == 2) { CALL(64, 2); }       \
      else { CALL(64, 4); }                          \
  }

template <typename T, bool kGated>
hipError_t launch_fwd(const Args& a, const Plan& p, hipStream_t st) {
  const dim3 threads(kThreads);
  if (!p.map) {
#define SSM_GROUP_NORM_CALL(G, K)                                                                              \
  hipLaunchKernelGGL((group_norm_row_fwd_kernel<T, G, K, kGated>), dim3((unsigned)p.row_blocks), threads, 0, st, a)
    SSM_GROUP_NORM_GEOMETRY(SSM_GROUP_NORM_CALL)
#undef SSM_GROUP_NORM_CALL
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(a.batch * p.runs));
  if (a.channels < kPiece)
    hipLaunchKernelGGL((group_norm_map_stats_kernel<T, true>), grid, threads, 0, st, a);
  else
    hipLaunchKernelGGL((group_norm_map_stats_kernel<T, false>), grid, threads, 0, st, a);
  const int64_t per_block = kThreads / 64;
  hipLaunchKernelGGL(group_norm_map_join_kernel, dim3((unsigned)((a.batch * a.groups + per_block - 1) / per_block)),
                     threads, 0, st, a);
  if (a.channels < kPiece)
    hipLaunchKernelGGL((group_norm_map_fwd_kernel<T, kGated, true>), grid, threads, 0, st, a);
  else
    hipLaunchKernelGGL((group_norm_map_fwd_kernel<T, kGated, false>), grid, threads, 0, st, a);
  return hipGetLastError();
}

template <typename T, bool kGated>
hipError_t launch_bwd(const Args& a, const Plan& p, float* dweight, float* dbias, hipStream_t st) {
  const dim3 threads(kThreads);
  if (!p.map) {
#define SSM_GROUP_NORM_CALL(G, K)                                                                              \
  hipLaunchKernelGGL((group_norm_row_bwd_kernel<T, G, K, kGated>), dim3((unsigned)p.bwd_blocks), threads, 0, st, a)
    SSM_GROUP_NORM_GEOMETRY(SSM_GROUP_NORM_CALL)
#undef SSM_GROUP_NORM_CALL
    if (a.part)
      hipLaunchKernelGGL(group_norm_columns_kernel, dim3((unsigned)((2 * a.channels + 31) / 32)), dim3(1024), 0, st,
                         a.part, dweight, dbias, p.stride, a.channels);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(a.batch * p.runs));
  const bool narrow = a.channels < kPiece;
  if (narrow)
    hipLaunchKernelGGL((group_norm_map_sums_kernel<T, kGated, true>), grid, threads, 0, st, a);
  else
    hipLaunchKernelGGL((group_norm_map_sums_kernel<T, kGated, false>), grid, threads, 0, st, a);
  const int64_t tiles = (2 * a.channels + 31) / 32, per_block = kThreads / 64;
  const int64_t group_blocks = (a.batch * a.groups + per_block - 1) / per_block;
  const int64_t column_blocks = dweight || dbias ? (2 * a.channels + 31) / 32 : 0;
  if (p.runs > 1)
    hipLaunchKernelGGL(group_norm_map_columns_kernel, dim3((unsigned)(a.batch * tiles)), dim3(512), 0, st, a, tiles);
  hipLaunchKernelGGL(group_norm_map_reduce_kernel, dim3((unsigned)(group_blocks + column_blocks)), threads, 0, st, a,
                     group_blocks, dweight, dbias);
  if (narrow)
    hipLaunchKernelGGL((group_norm_map_bwd_kernel<T, kGated, true>), grid, threads, 0, st, a);
  else
    hipLaunchKernelGGL((group_norm_map_bwd_kernel<T, kGated, false>), grid, threads, 0, st, a);
  return hipGetLastError();
}

Args make_args(int64_t batch, int64_t length, int64_t channels, int64_t groups, const Plan& p, ssm_norm_t kind,
               ssm_act_t act) {
  Args a = {};
  a.batch = batch;
  a.length = length;
  a.channels = channels;
  a.groups = (int)groups;
  a.d = (int)(channels / groups);
  a.rms = kind == SSM_NORM_RMS;
  a.silu = act == SSM_ACT_SILU;
  a.runs = (int)p.runs;
  a.run = p.run;
  a.stride = p.stride;
  return a;
}

bool options_ok(ssm_norm_t kind, ssm_act_t act) {
  return (kind == SSM_NORM_LAYER || kind == SSM_NORM_RMS) && (act == SSM_ACT_NONE || act == SSM_ACT_SILU);
}

}  // namespace

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------

extern "C" {

ssm_status_t ssm_group_norm_fwd_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int64_t groups,
                                                ssm_dtype_t io, int64_t* bytes) {
  int64_t n;
  const ssm_status_t st = check_shape(batch, length, channels, groups, io, &n);
  if (st == SSM_OK && bytes) *bytes = fwd_bytes(make_plan(batch, length, channels, groups), batch, groups);
  return st;
}

ssm_status_t ssm_group_norm_fwd(int64_t batch, int64_t length, int64_t channels, int64_t groups, ssm_dtype_t io,
                                ssm_norm_t kind, ssm_act_t act, const void* x, const void* z, const float* weight,
                                const float* bias, float eps, void* y, float* mean, float* rstd, void* workspace,
                                int64_t workspace_bytes, struct ihipStream_t* stream) {
  int64_t n;
  ssm_status_t st = check_shape(batch, length, channels, groups, io, &n);
  if (st != SSM_OK) return st;
  if (!options_ok(kind, act)) return SSM_ERR_UNSUPPORTED;
  if (!x || !y) return SSM_ERR_NULL;
  if (kind == SSM_NORM_RMS) mean = nullptr;
  const Plan p = make_plan(batch, length, channels, groups);
  const int64_t need = fwd_bytes(p, batch, groups), rows = batch * groups;
  if (workspace_bytes < need) return SSM_ERR_WORKSPACE;
  if (need && !workspace) return SSM_ERR_NULL;
  if (!need) workspace = nullptr;
  const size_t es = io_size(io);
  const Buf ins[] = {{x, n * (int64_t)es, es}, {z, n * (int64_t)es, es}, {weight, channels * 4, 4}, {bias, channels * 4, 4}};
  const Buf outs[] = {{y, n * (int64_t)es, es}, {mean, rows * 4, 4}, {rstd, rows * 4, 4}, {workspace, need, 4}};
  st = check_buffers(ins, 4, outs, 4);
  if (st != SSM_OK) return st;
  Args a = make_args(batch, length, channels, groups, p, kind, act);
  a.x = x; a.z = z; a.weight = weight; a.bias = bias; a.eps = eps; a.y = y;
  a.mean = mean; a.rstd = rstd;
  a.part = static_cast<float*>(workspace);
  if (p.map) {
    float* stats = a.part + batch * p.runs * 2 * groups;
    if (!a.mean) a.mean = stats;
    if (!a.rstd) a.rstd = stats + rows;
  }
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  hipError_t e;
  if (io == SSM_F32)
    e = z ? launch_fwd<float, true>(a, p, hs) : launch_fwd<float, false>(a, p, hs);
  else
    e = z ? launch_fwd<bf16_t, true>(a, p, hs) : launch_fwd<bf16_t, false>(a, p, hs);
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

ssm_status_t ssm_group_norm_bwd_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int64_t groups,
                                                ssm_dtype_t io, int64_t* bytes) {
  int64_t n;
  const ssm_status_t st = check_shape(batch, length, channels, groups, io, &n);
  if (st == SSM_OK && bytes) *bytes = bwd_bytes(make_plan(batch, length, channels, groups), batch, channels, groups, true);
  return st;
}

ssm_status_t ssm_group_norm_bwd(int64_t batch, int64_t length, int64_t channels, int64_t groups, ssm_dtype_t io,
                                ssm_norm_t kind, ssm_act_t act, const void* dy, const void* x, const void* z,
                                const float* weight, const float* bias, const float* mean, const float* rstd, void* dx,
                                void* dz, float* dweight, float* dbias, void* workspace, int64_t workspace_bytes,
                                struct ihipStream_t* stream) {
  int64_t n;
  ssm_status_t st = check_shape(batch, length, channels, groups, io, &n);
  if (st != SSM_OK) return st;
  if (!options_ok(kind, act)) return SSM_ERR_UNSUPPORTED;
  if (!dy || !x || !rstd || !dx || (kind == SSM_NORM_LAYER && !mean)) return SSM_ERR_NULL;
  if (kind == SSM_NORM_RMS) mean = nullptr;
  if (!z) dz = nullptr;
  const Plan p = make_plan(batch, length, channels, groups);
  const int64_t need = bwd_bytes(p, batch, channels, groups, dweight || dbias), rows = batch * groups;
  if (workspace_bytes < need) return SSM_ERR_WORKSPACE;
  if (need && !workspace) return SSM_ERR_NULL;
  if (!need) workspace = nullptr;
  const size_t es = io_size(io);
  const int64_t bytes = n * (int64_t)es;
  const Buf ins[] = {{dy, bytes, es}, {x, bytes, es}, {z, bytes, es}, {weight, channels * 4, 4}, {bias, channels * 4, 4},
                     {mean, rows * 4, 4}, {rstd, rows * 4, 4}};
  const Buf outs[] = {{dx, bytes, es}, {dz, bytes, es}, {dweight, channels * 4, 4}, {dbias, channels * 4, 4},
                      {workspace, need, 4}};
  st = check_buffers(ins, 7, outs, 5);
  if (st != SSM_OK) return st;
  Args a = make_args(batch, length, channels, groups, p, kind, act);
  a.dy = dy; a.x = x; a.z = z; a.weight = weight; a.bias = bias;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.dx = dx; a.dz = dz;
  a.part = static_cast<float*>(workspace);
  a.sums = p.map ? a.part + batch * p.runs * 2 * channels : nullptr;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  hipError_t e;
  if (io == SSM_F32)
    e = z ? launch_bwd<float, true>(a, p, dweight, dbias, hs) : launch_bwd<float, false>(a, p, dweight, dbias, hs);
  else
    e = z ? launch_bwd<bf16_t, true>(a, p, dweight, dbias, hs) : launch_bwd<bf16_t, false>(a, p, dweight, dbias, hs);
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

}  // extern "C"
