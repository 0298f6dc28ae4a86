// linear_attn.hip -- linear attention with a decay for each head: planning and
// launching the chunked passes, the small kernels between them, and the decode
// step.  C ABI: include/ssm_scan.h.
//
// With few (batch, head) pairs the tokens are cut into segments: a state pass
// gives every segment's own state, a join turns them into the states the
// segments start from, and the main pass runs all segments at once.  The
// backward takes the forward's states from its checkpoints where dq's segments are
// whole blocks of them, and else from a state pass of its own.
//
// The backward is the same pass three times over,
//   dq = pass(dy, v, k), state S^T;   dv = reverse pass(k, q, dy), state R;
//   dk = reverse pass(v, dy, q), state R^T,        R_t = dL/dS_t,
// S from the forward's checkpoints.  The decays' gradient is
//   dL/dg_t = <a_t S_{t-1}, R_t>
//           = sum over u >= t in the block of (q_u . dq_u - k_u . dk_u) + <S, R> behind the block
//           = <S, R> in front of the block - sum over u < t in it of the same
// since all that is written and read behind t cancels in the sum; blocks are
// kBlock tokens, so that no longer sum loses what it cancels to, and the two say how far
// the sums' roundings have come.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device_common.h"
#include "host_common.h"
#include "linear_attn.h"
#include "rows.h"
#include "ssm_scan.h"

namespace {

using linattn::Args;
using linattn::kBlock;
using linattn::Role;
using linattn::Side;

// ---- between the passes ------------------------------------------------------

// States of the segments' own tokens become the states the segments start from.
// A thread has one element of the state and walks the segments, 8 requested at
// once (in slots that it alone reads and writes).
struct Join {
  float* part;
  const float* total;
  const float* first;  // may be null (0)
  int64_t first_step;  // from row to row of first
  int reverse;
};

__global__ __launch_bounds__(256) void linear_attn_join_kernel(const Join one, const Join other, int64_t n, int segments) {
  const Join& p = blockIdx.z ? other : one;
  float* const part = p.part;
  const float* const total = p.total;
  const float* const first = p.first;
  const int reverse = p.reverse;
  const int64_t row = blockIdx.y;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float* at = part + row * segments * n + i;
  const float* decay = total + row * segments;
  float s = first ? first[row * p.first_step + i] : 0.0f;
  for (int j0 = 0; j0 < segments; j0 += 8) {
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = min(j0 + u, segments - 2);  // the last segment's own state is not wanted
      x[u] = at[(reverse ? segments - 1 - j : j) * n];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (j0 + u >= segments) break;
      const int j = reverse ? segments - 1 - (j0 + u) : j0 + u;
      at[j * n] = s;
      if (j0 + u == segments - 1) break;
      const float d = decay[j];
      s = (d == 0.0f ? 0.0f : s * d) + x[u];
    }
  }
}

// dq and dk of a group (blockIdx.y): its heads' parts, added in order.
template <typename T>
__global__ __launch_bounds__(256) void linear_attn_group_kernel(const float* part_q, const float* part_k, T* dq, T* dk,
                                                                int64_t n, int share, int d) {
  const float* const part = blockIdx.y ? part_k : part_q;
  T* const out = blockIdx.y ? dk : dq;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {  // [token][group][d]
    const int64_t tg = i / d;
    const float* at = part + tg * share * d + i % d;
    float t = at[0];
    for (int h = 1; h < share; ++h) t += at[(int64_t)h * d];
    Io<T>::store1(out + i, t);
  }
}

struct DecayArgs {
  const double* cross;   // <S, R> in parts, [rows][blocks + 1][parts_v], in front of each block and behind the last
  const float* dots_q;   // [parts_qk][rows][seqlen]
  const float* dots_k;   // the same
  const float* rate;
  const void* step;      // may be null
  const uint8_t* reset;  // may be null
  void* dstep;           // may be null
  double* drate;         // [rows][blocks]
  int64_t rows, seqlen;
  int heads, blocks, parts_qk, parts_v;
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// One block of kBlock tokens of one (batch, head), a token to a thread.  Nothing is
// carried over a reset or what is a decay of 0 to the passes, so the sums run
// between such tokens (or the block's ends) and from either side: what is carried
// into a run, 0 or <S, R> in front of the block, is known as well as what is carried
// out of it.  The roundings between the two ends are spread over the run's tokens
// as a walk between two fixed ends would be; and where a token of the run is not
// finite, the side that it does not lie on holds.
template <typename T>
__global__ __launch_bounds__(kBlock) void linear_attn_decay_kernel(const DecayArgs p) {
  constexpr int kWaves = kBlock / 64;
  __shared__ uint64_t cuts[kWaves];
  __shared__ double heads[kWaves], tails[kWaves], sums[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int block = (int)(blockIdx.x % p.blocks);
  const int64_t row = blockIdx.x / p.blocks;
  const int head = (int)(row % p.heads);
  const int64_t t = (int64_t)block * kBlock + tid;
  const int count = (int)min((int64_t)kBlock, p.seqlen - (int64_t)block * kBlock);
  const int64_t at = row / p.heads * p.seqlen + t;
  const float rate = p.rate[head];
  float step = 1.0f;
  const double* borders = p.cross + (row * (p.blocks + 1) + block) * p.parts_v;
  double carried_in = 0.0, carried_out = 0.0;
  for (int i = 0; i < p.parts_v; ++i) {
    carried_in += borders[i];
    carried_out += borders[p.parts_v + i];
  }
  double w = 0.0;
  bool dropped = false;
  if (tid < count) {
    for (int i = 0; i < p.parts_qk; ++i) {
      const int64_t dot = (i * p.rows + row) * p.seqlen + t;
      w += (double)p.dots_q[dot] - (double)p.dots_k[dot];
    }
    if (p.step) step = Io<T>::load1(static_cast<const T*>(p.step) + at * p.heads + head);
    dropped = (p.reset && p.reset[at]) || linattn::pow2(linattn::log2_decay(rate, step)) == 0.0f;
  }
  const uint64_t here = __ballot(dropped);
  if (lane == 0) cuts[wave] = here;
  __syncthreads();
  // The token's run, [first, next).
  int first = -1, next = -1;
  for (int v = wave; v >= 0 && first < 0; --v) {
    const uint64_t m = v == wave ? here & (~0ull >> (63 - lane)) : cuts[v];
    if (m) first = v * 64 + 63 - __builtin_clzll(m);
  }
  for (int v = wave; v < kWaves && next < 0; ++v) {
    const uint64_t m = v == wave ? here & ~(~0ull >> (63 - lane)) : cuts[v];
    if (m) next = v * 64 + __builtin_ctzll(m);
  }
  if (first >= 0) carried_in = 0.0;
  if (next >= 0) carried_out = 0.0;
  first = max(first, 0);
  if (next < 0) next = count;
  double behind = w, before = w;  // over the run's tokens of this wave from this one on, and up to it
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double b = __shfl_down(behind, m), f = __shfl_up(before, m);
    if (lane + m < 64 && tid + m < next) behind += b;
    if (lane >= m && tid - m >= first) before += f;
  }
  if (lane == 0) heads[wave] = behind;
  if (lane == 63) tails[wave] = before;
  before = __shfl_up(before, 1);  // up to the one in front of it
  if (lane == 0 || tid == first) before = 0.0;
  __syncthreads();
  for (int v = wave + 1; v < kWaves && v * 64 < next; ++v) behind += heads[v];
  for (int v = wave - 1; v >= 0 && v * 64 + 63 >= first; --v) before += tails[v];
  const double from_end = carried_out + behind, from_start = carried_in - before;
  const bool end_ok = __builtin_fabs(from_end) < 1e300, start_ok = __builtin_fabs(from_start) < 1e300;
  double g = end_ok ? from_end : from_start;
  if (end_ok && start_ok) g += (from_start - from_end) * (double)(next - tid) / (double)(next - first);
  if (dropped) g = 0.0;
  double sum = 0.0;
  if (tid < count) {
    if (!dropped) sum = g * (double)step;
    if (p.dstep) Io<T>::store1(static_cast<T*>(p.dstep) + at * p.heads + head, dropped ? 0.0f : (float)(-g * (double)rate));
  }
  sum = wave_sum(sum);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    double all = sums[0];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) all += sums[v];
    p.drate[row * p.blocks + block] = all;
  }
}

// drate[h] = -sum over the batch rows and blocks, in a fixed order.
__global__ __launch_bounds__(256) void linear_attn_drate_kernel(const double* part, float* drate, int64_t batch,
                                                                int heads, int blocks) {
  __shared__ double slots[4];
  const int head = blockIdx.x, tid = threadIdx.x;
  double t = 0.0;
  for (int64_t i = tid; i < batch * blocks; i += 256)
    t += part[(i / blocks * heads + head) * blocks + i % blocks];
  t = wave_sum(t);
  if ((tid & 63) == 0) slots[tid >> 6] = t;
  __syncthreads();
  if (tid == 0) drate[head] = -(float)((slots[0] + slots[1]) + (slots[2] + slots[3]));
}

// ---- the decode step ---------------------------------------------------------

struct StepArgs {
  float* state;
  const void* q;
  const void* k;
  const void* v;
  const float* rate;
  const void* step;  // may be null
  void* y;
  float scale;
  int heads, groups, dk, dv, width;  // width: lanes along a row of the state
};

// A block has `width` x kVec columns of one (batch, head)'s state; its lanes take
// every 256 / width-th row, kAhead of them in flight.  Memory's: 256 x 40 heads of
// 128 x 128 in bf16 move 1.35 GB in 263 us, what a copy of them takes; one stream of 20
// heads of 64 x 128 takes 4.1 us.
template <typename T, int kVec>
__global__ __launch_bounds__(256) void linear_attn_step_kernel(const StepArgs p) {
  constexpr int kAhead = 8;
  __shared__ float sums[256 * kVec];
  __shared__ float keys[2][256];
  const int tid = threadIdx.x, x = tid & (p.width - 1), rows = 256 / p.width, y0 = tid / p.width;
  const int64_t row = blockIdx.x;
  const int head = (int)(row % p.heads);
  const int64_t batch = row / p.heads;
  const int c = (blockIdx.y * p.width + x) * kVec;
  const bool live = c < p.dv;
  const int64_t side = (batch * p.groups + head / (p.heads / p.groups)) * p.dk;
  const int cc = live ? c : 0;
  float* state = p.state + row * p.dk * p.dv + cc;
  float s[kAhead][kVec];
  const auto request = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load_n<kVec>(state + (int64_t)min(k0 + u * rows, p.dk - 1) * p.dv, s[u]);
  };
  request(y0);
  if (tid < p.dk) {
    keys[0][tid] = Io<T>::load1(static_cast<const T*>(p.q) + side + tid);
    keys[1][tid] = Io<T>::load1(static_cast<const T*>(p.k) + side + tid);
  }
  float v[kVec], out[kVec];
  load_n<kVec>(static_cast<const T*>(p.v) + row * p.dv + cc, v);
  const float step = p.step ? Io<T>::load1(static_cast<const T*>(p.step) + row) : 1.0f;
  const float a = linattn::pow2(linattn::log2_decay(p.rate[head], step));
#pragma unroll
  for (int j = 0; j < kVec; ++j) out[j] = 0.0f;
  lds_barrier();
  for (int k0 = y0; k0 < p.dk; k0 += kAhead * rows) {
    if (k0 != y0) request(k0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u * rows;
      if (k >= p.dk) break;
      const float kk = keys[1][k], qq = keys[0][k];
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        s[u][j] = __builtin_fmaf(kk, v[j], a == 0.0f ? 0.0f : s[u][j] * a);
        out[j] = __builtin_fmaf(qq, s[u][j], out[j]);
      }
      if (live) store_n<kVec>(state + (int64_t)k * p.dv, s[u]);
    }
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) sums[(y0 * p.width + x) * kVec + j] = out[j];
  lds_barrier();
  const int n = p.width * kVec, column = blockIdx.y * n + tid;
  if (tid < n && column < p.dv) {
    float t = sums[tid];
    for (int i = 1; i < rows; ++i) t += sums[i * n + tid];
    Io<T>::store1(static_cast<T*>(p.y) + row * p.dv + column, t * p.scale);
  }
}

// ---- host side ---------------------------------------------------------------

struct Sizes {
  int64_t batch, seqlen, heads, groups, dk, dv;
  ssm_dtype_t io;
  int64_t rows() const { return batch * heads; }
  int64_t state() const { return dk * dv; }
  int64_t blocks() const { return (seqlen + kBlock - 1) / kBlock; }
};

ssm_status_t check_sizes(const Sizes& s) {
  if (s.io != SSM_F32 && s.io != SSM_BF16) return SSM_ERR_DTYPE;
  if (s.batch < 1 || s.seqlen < 1 || s.heads < 1 || s.groups < 1 || s.dk < 1 || s.dv < 1) return SSM_ERR_SHAPE;
  if (s.heads % s.groups) return SSM_ERR_SHAPE;
  int64_t n, m;
  if (!mul_ok(s.batch, s.seqlen, &n) || !mul_ok(n, s.heads, &n)) return SSM_ERR_SHAPE;
  if (!mul_ok(n, s.dk, &m) || !mul_ok(m, 64, &m) || !mul_ok(n, s.dv, &m) || !mul_ok(m, 64, &m)) return SSM_ERR_SHAPE;
  if (!mul_ok(s.batch, s.heads, &n) || !mul_ok(n, s.dk, &n) || !mul_ok(n, s.dv, &n) ||
      !mul_ok(n, s.seqlen / kBlock + 3, &n) || !mul_ok(n, 16, &n))
    return SSM_ERR_SHAPE;
  if (s.dk > linattn::kMaxDim || s.dv > linattn::kMaxDim) return SSM_ERR_UNSUPPORTED;
  if (s.heads > 16384 || s.batch > ((int64_t)1 << 30)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

int64_t tiles(int64_t dv) { return (dv + linattn::tile_width((int)dv) - 1) / linattn::tile_width((int)dv); }

constexpr int64_t kUnit = 64;  // tokens; a segment is so many of them, a multiple of either chunk

struct Split {
  int64_t per, count;  // units of a segment, segments
  bool blocks() const { return per * kUnit % kBlock == 0 || count == 1; }
};

// Blocks of a pass that the chip holds at once: as the LDS and registers of its
// kernel allow (in bf16 three parts of the scores take more LDS: 8 x 2048 x 20 heads of
// 64 x 128 trained in 663 us so, 685 counting three blocks a compute unit; 4 x 4096 x 32
// of 128 x 64 in 962, and 1038).
int64_t resident(int64_t dk, int64_t dv, ssm_dtype_t io) {
  const bool two = io == SSM_BF16 ? dk > 64 || dv > 64 : dk > 64 && dv > 64;
  return 256 * (dk > 128 ? 1 : two ? 2 : 3);
}

// Segments: as many as are resident at once, of two units or more.
Split split_tokens(const Sizes& s, int64_t most) {
  const int64_t units = (s.seqlen + kUnit - 1) / kUnit;
  Split p{units, 1};
  const int64_t wanted = std::max<int64_t>(1, most);
  p.per = std::max<int64_t>(std::min<int64_t>(2, units), (units + wanted - 1) / wanted);
  p.count = (units + p.per - 1) / p.per;
  return p;
}

Split fwd_split(const Sizes& s) { return split_tokens(s, resident(s.dk, s.dv, s.io) / (s.rows() * tiles(s.dv))); }

// What the pass with the fewest blocks asks for; dq's and dk's may be coarser.
Split bwd_split(const Sizes& s) {
  const int64_t to_v = resident(s.dk, s.dv, s.io) / (s.rows() * tiles(s.dv));
  const int64_t to_qk = resident(s.dv, s.dk, s.io) / (s.rows() * 2 * tiles(s.dk));
  Split p = split_tokens(s, std::max(to_v, to_qk));
  const int64_t block = kBlock / kUnit;
  if (p.per >= block) {  // whole blocks: the forward's states are checkpoints
    p.per = p.per / block * block;
    p.count = ((s.seqlen + kUnit - 1) / kUnit + p.per - 1) / p.per;
  }
  return p;
}

// dq's and dk's passes: where the segments are parts of a block, whole blocks, which
// start from checkpoints and from every so many-th of dv's states, if their blocks
// still fill the chip: 8 x 2048 x 12 heads of 64 x 128 fp32 train in 614 us so, in 672
// with one split and a pass for the forward's states.
Split qk_split(const Sizes& s, const Split& p) {
  const int64_t block = kBlock / kUnit;
  if (p.blocks() || block % p.per || 2 * s.rows() * tiles(s.dk) * s.blocks() < resident(s.dv, s.dk, s.io)) return p;
  return Split{block, s.blocks()};
}

// Segments' states and decays.
int64_t segment_bytes(const Sizes& s, const Split& p) { return p.count > 1 ? s.rows() * p.count * (s.state() + 1) * 4 : 0; }

struct BwdSpace {
  int64_t states, segments, cross, dots_q, dots_k, drate, dq, dk, bytes;  // offsets
};

BwdSpace bwd_space(const Sizes& s, bool decays) {
  BwdSpace w;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 15) / 16 * 16;
    return here;
  };
  w.drate = take(decays ? s.rows() * s.blocks() * 8 : 0);
  const Split p = bwd_split(s);
  w.segments = take(segment_bytes(s, p));
  w.states = take(qk_split(s, p).blocks() ? 0 : segment_bytes(s, p));
  w.cross = take(decays ? s.rows() * (s.blocks() + 1) * ((s.dv + 31) / 32) * 8 : 0);
  w.dots_q = take(decays ? (s.dk + 31) / 32 * s.rows() * s.seqlen * 4 : 0);
  w.dots_k = take(decays ? (s.dk + 31) / 32 * s.rows() * s.seqlen * 4 : 0);
  const bool shared = s.groups != s.heads;
  w.dq = take(shared ? s.rows() * s.seqlen * s.dk * 4 : 0);
  w.dk = take(shared ? s.rows() * s.seqlen * s.dk * 4 : 0);
  w.bytes = at;
  return w;
}

bool whole_units(const Side& s, size_t es) { return s.d * es % 16 == 0 && aligned(s.p, 16); }

hipError_t launch_pass(Args a, int64_t blocks, bool state_only, ssm_dtype_t io, hipStream_t st) {
  const size_t es = io_size(io);
  for (int i = 0; i < a.roles; ++i) {
    Role& r = a.role[i];
    r.dma = whole_units(r.q, es) && whole_units(r.k, es) && whole_units(r.v, es);
  }
  return io == SSM_BF16 ? linattn::launch_bf16(a, blocks, state_only, st)
                        : linattn::launch_f32(a, blocks, state_only, st);
}

Args pass_args(const Sizes& s, const Split& p, const float* rate, const void* step, const uint8_t* reset) {
  Args a = {};
  a.batch = (int)s.batch;
  a.heads = (int)s.heads;
  a.seqlen = s.seqlen;
  a.rate = rate;
  a.step = step;
  a.reset = reset;
  a.segments = (int)p.count;
  a.segment_len = p.per * kUnit;
  return a;
}

// The states that the segments start from: of one or two roles, `first` in front of
// all tokens (behind them, reverse), into their spaces (segment_bytes each).
struct Front {
  const float* state;  // may be null
  int64_t step;        // from (batch, head) to (batch, head)
};

hipError_t segment_states(Args a, const Role* roles, const Front* first, void* const* space, int count, const Sizes& s,
                          hipStream_t st) {
  Join join[2] = {};
  a.roles = count;
  int64_t blocks = 0;
  for (int i = 0; i < count; ++i) {
    Role& r = a.role[i] = roles[i];
    r.part = static_cast<float*>(space[i]);
    r.total = r.part + s.rows() * a.segments * s.state();
    r.tiles = (int)tiles(s.dv);
    r.first_block = (int)blocks;
    blocks += s.rows() * r.tiles * (a.segments - 1);
    join[i] = Join{r.part, r.total, first[i].state, first[i].step, r.reverse};
  }
  const hipError_t e = launch_pass(a, blocks, true, s.io, st);
  if (e != hipSuccess) return e;
  const int64_t n = s.state();
  hipLaunchKernelGGL(linear_attn_join_kernel, dim3((unsigned)((n + 255) / 256), (unsigned)s.rows(), (unsigned)count),
                     dim3(256), 0, st, join[0], join[1], n, a.segments);
  return hipGetLastError();
}

bool passes_ok(const Sizes& s, const Split& p, int64_t blocks_each) {
  return s.rows() < 65536 * (int64_t)16 && launch_ok(s.rows() * p.count * blocks_each, 256);
}

}  // namespace

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------

extern "C" {

ssm_status_t ssm_linear_attn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads, int64_t groups,
                                                 int64_t dk, int64_t dv, ssm_dtype_t io, int64_t* bytes) {
  const Sizes s{batch, seqlen, heads, groups, dk, dv, io};
  const ssm_status_t st = check_sizes(s);
  if (st == SSM_OK && bytes) *bytes = segment_bytes(s, fwd_split(s));
  return st;
}

ssm_status_t ssm_linear_attn_fwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t groups, int64_t dk, int64_t dv,
                                 ssm_dtype_t io, const void* q, const void* k, const void* v, const float* rate,
                                 const void* step, const uint8_t* reset, const float* h0, float scale, void* y,
                                 float* last_state, float* ckpt, void* workspace, int64_t workspace_bytes,
                                 struct ihipStream_t* stream) {
  const Sizes s{batch, seqlen, heads, groups, dk, dv, io};
  ssm_status_t st = check_sizes(s);
  if (st != SSM_OK) return st;
  const Split p = fwd_split(s);
  if (!passes_ok(s, p, tiles(dv))) return SSM_ERR_UNSUPPORTED;
  if (!q || !k || !v || !rate || !y) return SSM_ERR_NULL;
  const int64_t need = segment_bytes(s, p);
  if (workspace_bytes < need) return SSM_ERR_WORKSPACE;
  if (need && !workspace) return SSM_ERR_NULL;
  if (!need) workspace = nullptr;
  const size_t es = io_size(io);
  const int64_t tokens = batch * seqlen, state = s.rows() * s.state() * 4;
  const bool in_place = h0 && last_state == h0;
  const Buf ins[] = {{q, tokens * groups * dk * (int64_t)es, es}, {k, tokens * groups * dk * (int64_t)es, es},
                     {v, tokens * heads * dv * (int64_t)es, es}, {rate, heads * 4, 4},
                     {step, tokens * heads * (int64_t)es, es}, {reset, tokens, 1}, {in_place ? nullptr : h0, state, 4}};
  const Buf outs[] = {{y, tokens * heads * dv * (int64_t)es, es}, {last_state, state, 4},
                      {ckpt, state * (s.blocks() + 1), 4}, {workspace, need, 8}};
  st = check_buffers(ins, 7, outs, 4);
  if (st != SSM_OK) return st;
  if (in_place && !aligned(h0, 4)) return SSM_ERR_ALIGN;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  Args a = pass_args(s, p, rate, step, reset);
  const int share = (int)(heads / groups);
  Role r = {};
  r.q = Side{q, (int)groups, share, (int)dk};
  r.k = Side{k, (int)groups, share, (int)dk};
  r.v = Side{v, (int)heads, 1, (int)dv};
  r.s_in = scale;
  r.s_up = 1.0f;
  r.start = h0;
  r.start_slots = 1;
  hipError_t e = hipSuccess;
  if (p.count > 1) {
    const Front first{h0, s.state()};
    e = segment_states(a, &r, &first, &workspace, 1, s, hs);
    r.start = static_cast<const float*>(workspace);
    r.start_slots = p.count;
    r.start_step = 1;
  }
  if (e == hipSuccess) {
    r.out = y;
    r.save = ckpt;
    r.slots = s.blocks() + 1;
    r.last = last_state;
    r.tiles = (int)tiles(dv);
    a.role[0] = r;
    a.roles = 1;
    e = launch_pass(a, s.rows() * r.tiles * p.count, false, io, hs);
  }
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

ssm_status_t ssm_linear_attn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads, int64_t groups,
                                                 int64_t dk, int64_t dv, ssm_dtype_t io, int decays, int64_t* bytes) {
  const Sizes s{batch, seqlen, heads, groups, dk, dv, io};
  const ssm_status_t st = check_sizes(s);
  if (st == SSM_OK && bytes) *bytes = bwd_space(s, decays != 0).bytes;
  return st;
}

ssm_status_t ssm_linear_attn_bwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t groups, int64_t dk, int64_t dv,
                                 ssm_dtype_t io, const void* q, const void* k, const void* v, const float* rate,
                                 const void* step, const uint8_t* reset, const float* ckpt, float scale,
                                 const void* dy, const float* dlast, void* dq, void* dk_out, void* dv_out,
                                 float* drate, void* dstep, float* dh0, void* workspace, int64_t workspace_bytes,
                                 struct ihipStream_t* stream) {
  const Sizes s{batch, seqlen, heads, groups, dk, dv, io};
  ssm_status_t st = check_sizes(s);
  if (st != SSM_OK) return st;
  const Split p = bwd_split(s), qk = qk_split(s, p);
  if (!passes_ok(s, p, 2 * tiles(dk) + tiles(dv)) || !launch_ok(s.rows() * s.blocks(), kBlock)) return SSM_ERR_UNSUPPORTED;
  if (!q || !k || !v || !rate || !ckpt || !dy || !dq || !dk_out || !dv_out) return SSM_ERR_NULL;
  if (!step) dstep = nullptr;
  const bool decays = drate || dstep;
  const BwdSpace w = bwd_space(s, decays);
  if (workspace_bytes < w.bytes) return SSM_ERR_WORKSPACE;
  if (w.bytes && !workspace) return SSM_ERR_NULL;
  if (!w.bytes) workspace = nullptr;
  const size_t es = io_size(io);
  const int64_t tokens = batch * seqlen, state = s.rows() * s.state() * 4;
  const int64_t qk_bytes = tokens * groups * dk * (int64_t)es, v_bytes = tokens * heads * dv * (int64_t)es;
  const int64_t step_bytes = tokens * heads * (int64_t)es;
  const Buf ins[] = {{q, qk_bytes, es}, {k, qk_bytes, es}, {v, v_bytes, es}, {rate, heads * 4, 4},
                     {step, step_bytes, es}, {reset, tokens, 1}, {ckpt, state * (s.blocks() + 1), 4},
                     {dy, v_bytes, es}, {dlast, state, 4}};
  const Buf outs[] = {{dq, qk_bytes, es}, {dk_out, qk_bytes, es}, {dv_out, v_bytes, es}, {drate, heads * 4, 4},
                      {dstep, step_bytes, es}, {dh0, state, 4}, {workspace, w.bytes, 8}};
  st = check_buffers(ins, 9, outs, 7);
  if (st != SSM_OK) return st;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  char* const space = static_cast<char*>(workspace);
  const auto at = [&](int64_t offset) { return reinterpret_cast<float*>(space + offset); };
  Args a = pass_args(s, p, rate, step, reset);
  const int share = (int)(heads / groups);
  const Side qs{q, (int)groups, share, (int)dk}, ks{k, (int)groups, share, (int)dk};
  const Side vs{v, (int)heads, 1, (int)dv}, ys{dy, (int)heads, 1, (int)dv};
  Role to_q = {}, to_k = {}, to_v = {};
  to_v.q = ks; to_v.k = qs; to_v.v = ys;
  to_v.reverse = 1;
  to_v.s_in = 1.0f;
  to_v.s_up = scale;
  to_v.start = dlast;
  to_v.start_slots = 1;
  to_q.start = ckpt;
  to_q.start_slots = s.blocks() + 1;
  to_q.start_step = qk.per * kUnit / kBlock;
  hipError_t e = hipSuccess;
  if (p.count > 1) {
    Role forward = {};  // S again, from the states in front of all tokens
    forward.q = qs; forward.k = ks; forward.v = vs;
    forward.s_in = forward.s_up = 1.0f;
    const Role roles[2] = {to_v, forward};
    const Front first[2] = {{dlast, s.state()}, {ckpt, (s.blocks() + 1) * s.state()}};
    void* const spaces[2] = {at(w.segments), at(w.states)};
    e = segment_states(a, roles, first, spaces, qk.blocks() ? 1 : 2, s, hs);
    if (e != hipSuccess) return hip_fail(e);
    to_v.start = at(w.segments);
    to_v.start_slots = p.count;
    to_v.start_step = 1;
    if (!qk.blocks()) {
      to_q.start = at(w.states);
      to_q.start_slots = p.count;
      to_q.start_step = 1;
    }
  }
  to_v.out = dv_out;
  to_v.last = dh0;
  to_v.tiles = (int)tiles(dv);
  if (decays) {
    to_v.meet = ckpt;
    to_v.cross = reinterpret_cast<double*>(space + w.cross);
    to_v.slots = s.blocks() + 1;
  }
  to_k = to_v;
  to_k.q = vs; to_k.k = ys; to_k.v = qs;
  to_k.transposed = 1;
  to_k.last = nullptr;
  to_k.meet = nullptr;
  to_k.tiles = (int)tiles(dk);
  if (p.count > 1) {  // the state behind each segment of qk is that behind its last one of p
    to_k.start_step = qk.per / p.per;
    to_k.start_first = to_k.start_step - 1;
  }
  to_q.q = ys; to_q.k = vs; to_q.v = ks;
  to_q.transposed = 1;
  to_q.s_in = scale;
  to_q.s_up = 1.0f;
  to_q.tiles = to_k.tiles;
  const bool shared = groups != heads;
  to_q.out = shared ? at(w.dq) : dq;
  to_k.out = shared ? at(w.dk) : dk_out;
  to_q.out_f32 = to_k.out_f32 = shared;
  if (decays) {
    to_q.with = qs;
    to_q.dots = at(w.dots_q);
    to_k.with = ks;
    to_k.dots = at(w.dots_k);
  }
  // dq's and dk's passes contract v's columns, dv's contracts q's.
  const int64_t q_blocks = s.rows() * to_q.tiles * qk.count, v_blocks = s.rows() * to_v.tiles * p.count;
  to_k.first_block = (int)q_blocks;
  a.role[0] = to_q;
  a.role[1] = to_k;
  a.roles = 2;
  a.segments = (int)qk.count;
  a.segment_len = qk.per * kUnit;
  e = launch_pass(a, 2 * q_blocks, false, io, hs);
  if (e != hipSuccess) return hip_fail(e);
  a.role[0] = to_v;
  a.roles = 1;
  a.segments = (int)p.count;
  a.segment_len = p.per * kUnit;
  e = launch_pass(a, v_blocks, false, io, hs);
  if (e != hipSuccess) return hip_fail(e);
  if (shared) {
    const int64_t n = tokens * groups * dk;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 65536);
    if (io == SSM_BF16)
      hipLaunchKernelGGL(linear_attn_group_kernel<bf16_t>, dim3(blocks, 2), dim3(256), 0, hs, at(w.dq), at(w.dk),
                         static_cast<bf16_t*>(dq), static_cast<bf16_t*>(dk_out), n, share, (int)dk);
    else
      hipLaunchKernelGGL(linear_attn_group_kernel<float>, dim3(blocks, 2), dim3(256), 0, hs, at(w.dq), at(w.dk),
                         static_cast<float*>(dq), static_cast<float*>(dk_out), n, share, (int)dk);
    e = hipGetLastError();
    if (e != hipSuccess) return hip_fail(e);
  }
  if (decays) {
    DecayArgs d = {};
    d.cross = to_v.cross;
    d.dots_q = at(w.dots_q);
    d.dots_k = at(w.dots_k);
    d.rate = rate;
    d.step = step;
    d.reset = reset;
    d.dstep = dstep;
    d.drate = reinterpret_cast<double*>(space + w.drate);
    d.rows = s.rows();
    d.seqlen = seqlen;
    d.heads = (int)heads;
    d.blocks = (int)s.blocks();
    d.parts_qk = (int)((dk + 31) / 32);
    d.parts_v = (int)((dv + 31) / 32);
    const unsigned blocks = (unsigned)(s.rows() * s.blocks());
    if (io == SSM_BF16)
      hipLaunchKernelGGL(linear_attn_decay_kernel<bf16_t>, dim3(blocks), dim3(kBlock), 0, hs, d);
    else
      hipLaunchKernelGGL(linear_attn_decay_kernel<float>, dim3(blocks), dim3(kBlock), 0, hs, d);
    if (drate)
      hipLaunchKernelGGL(linear_attn_drate_kernel, dim3((unsigned)heads), dim3(256), 0, hs, d.drate, drate, batch,
                         (int)heads, d.blocks);
    e = hipGetLastError();
  }
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

ssm_status_t ssm_linear_attn_state_update(int64_t batch, int64_t heads, int64_t groups, int64_t dk, int64_t dv,
                                          ssm_dtype_t io, float* state, const void* q, const void* k, const void* v,
                                          const float* rate, const void* step, float scale, void* y,
                                          struct ihipStream_t* stream) {
  const Sizes s{batch, 1, heads, groups, dk, dv, io};
  ssm_status_t st = check_sizes(s);
  if (st != SSM_OK) return st;
  if (!launch_ok(s.rows(), 256)) return SSM_ERR_UNSUPPORTED;
  if (!state || !q || !k || !v || !rate || !y) return SSM_ERR_NULL;
  const size_t es = io_size(io);
  const int64_t rows = s.rows(), qk_bytes = batch * groups * dk * (int64_t)es;
  const Buf ins[] = {{q, qk_bytes, es}, {k, qk_bytes, es}, {v, rows * dv * (int64_t)es, es}, {rate, heads * 4, 4},
                     {step, rows * (int64_t)es, es}};
  const Buf outs[] = {{state, rows * s.state() * 4, 4}, {y, rows * dv * (int64_t)es, es}};
  st = check_buffers(ins, 5, outs, 2);
  if (st != SSM_OK) return st;
  StepArgs a;
  a.state = state; a.q = q; a.k = k; a.v = v; a.rate = rate; a.step = step; a.y = y; a.scale = scale;
  a.heads = (int)heads; a.groups = (int)groups; a.dk = (int)dk; a.dv = (int)dv;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  const int vec = dv % 4 ? 1 : 4;
  const int64_t units = (dv + vec - 1) / vec;
  a.width = 64;
  while (a.width > 8 && (a.width / 2 >= units || rows * ((units + a.width - 1) / a.width) < 512)) a.width /= 2;
  const dim3 grid((unsigned)rows, (unsigned)((units + a.width - 1) / a.width));
  if (io == SSM_BF16) {
    if (vec == 4)
      hipLaunchKernelGGL((linear_attn_step_kernel<bf16_t, 4>), grid, dim3(256), 0, hs, a);
    else
      hipLaunchKernelGGL((linear_attn_step_kernel<bf16_t, 1>), grid, dim3(256), 0, hs, a);
  } else {
    if (vec == 4)
      hipLaunchKernelGGL((linear_attn_step_kernel<float, 4>), grid, dim3(256), 0, hs, a);
    else
      hipLaunchKernelGGL((linear_attn_step_kernel<float, 1>), grid, dim3(256), 0, hs, a);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

}  // extern "C"
