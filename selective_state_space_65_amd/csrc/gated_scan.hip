// gated_scan.hip -- gated linear recurrence (one state per channel, a gate per
// token): prefill, backward and decode step.  C ABI: include/ssm_scan.h.
//
//   h_l = a_l h_{l-1} + w_l x_l,   a from the gate, w from a (see the header)
//
// Each token is an affine map of the state, and maps compose:
// (a2, b2) after (a1, b1) = (a1 a2, a2 b1 + b2).  A lane takes 8 consecutive
// tokens of one channel (16 bytes of bf16, 32 of fp32) and reduces them to one
// map; a group of G lanes covers a tile of 8 G tokens and scans its lanes'
// maps by DPP; the state after the tile is the carry into the next.  From the
// state before its chunk each lane then runs its 8 tokens again and stores y.
// Every stream is read once and written once.
//
// The backward walks the tiles from the last to the first.  In a tile it
// recomputes the states from the forward's checkpoint before it (the forward
// writes one every 128 tokens, the tiles of 512 read every fourth) and runs the
// adjoint lambda_l = q_l + a_{l+1} lambda_{l+1}, which is the same
// kind of recurrence in the other direction: mu_l = a_l lambda_l is carried
// from lane to lane by maps mu -> A mu + B and a suffix scan.
//
// A token with a = 0 (a reset, or a gate that underflows) drops the state
// whatever its value, so 0 * Inf must not appear: a tile in which any lane of
// the wave has such a token runs the selecting form of each step (kDrop), and
// every other tile the plain one.  Products of many a's are kept at 2^-149, the
// smallest float, or above so that they cannot reach 0 by underflow and be
// taken for a drop.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device_common.h"
#include "host_common.h"
#include "rows.h"
#include "ssm_scan.h"

namespace {

constexpr int kTok = 8;          // tokens per lane
constexpr int kCkptStep = 128;   // tokens between checkpoints, as the header has it
constexpr int kMaxWaves = 16;    // waves that share one channel
constexpr int kMaxBwdWaves = 8;  // ... in the backward, which takes more registers

// bf16 rows go past the caches: an access of a wave covers whole lines, each
// touched once (forward at 4 x 4096 x 4096 116.8 -> 112.9 us, with its backward
// 317.7 -> 303.2 us, interleaved).  An fp32 piece is two accesses to the same
// line, and its second half would miss (8 x 1536 x 2048 219 -> 231 us).  With an
// operator behind it that reads y, or every gradient, the difference stays
// where the tensors are larger than the caches (4 x 4096 x 4096, forward and a
// product 172 -> 163 us, training step and two products 422 -> 378) and turns
// where they are not (1 x 4096 x 4096 training step and products 102 -> 106 us, 8
// x 1024 x 1024 62 -> 65).
template <typename IoT>
constexpr bool streamed = sizeof(IoT) == 2;

struct GatedArgs {
  const void* x;
  const void* gate;
  const float* gate_bias;  // may be null
  const float* rate;       // read by the kRate kernels only
  const void* z;           // may be null
  const uint8_t* reset;    // may be null
  const float* h0;         // may be null
  void* y;
  float* last;  // may be null
  float* ckpt;  // may be null in the forward
  // backward only
  const void* dy;
  const float* dlast;  // may be null
  void* dx;
  void* dgate;
  void* dz;      // may be null
  float* dbias;  // may be null: per-row sums [batch][dim], or [dim] where a block has every batch row
  float* drate;  // likewise
  float* dh0;    // may be null
  int64_t channels;  // batch * dim
  int64_t dim;
  int seqlen;
  int ckpts;  // checkpoints per channel
  int waves;  // waves of a row (64-lane groups only)
  int join;   // backward: batch rows of a channel that a block has, all of them, or 1
};

// ---- affine maps h -> a h + b ------------------------------------------------

struct Map {
  float a, b;
};

// A product of a's kept off 0, at the smallest subnormal: a state of size H then
// shows at most H 2^-149 (5e-7 for the largest H) where its product with the
// gates is gone, which is what rounding the product to a subnormal costs
// anyway.  The factors are not negative, so their bits order as unsigned
// integers and a NaN, above them all, stays.
__device__ __forceinline__ float off_zero(float a) { return __uint_as_float(max(__float_as_uint(a), 1u)); }

template <bool kDrop>
__device__ __forceinline__ float apply(Map m, float h) {
  const float r = __builtin_fmaf(m.a, h, m.b);
  if constexpr (kDrop) return m.a == 0.0f ? m.b : r;
  return r;
}

// `late` after `early`.
template <bool kDrop>
__device__ __forceinline__ Map compose(Map late, Map early) {
  Map r;
  r.b = apply<kDrop>(late, early.b);
  r.a = off_zero(late.a * early.a);
  if constexpr (kDrop) r.a = (late.a == 0.0f || early.a == 0.0f) ? 0.0f : r.a;
  return r;
}

// DPP move: lanes without a source lane, or in a row that row_mask leaves out, keep `keep`.
template <int ctrl, int row_mask = 0xf>
__device__ __forceinline__ float dpp(float keep, float src) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(keep), __float_as_int(src), ctrl, row_mask, 0xf, false));
}

template <int ctrl, int row_mask = 0xf>
__device__ __forceinline__ Map dpp(Map m) {
  return Map{dpp<ctrl, row_mask>(1.0f, m.a), dpp<ctrl, row_mask>(0.0f, m.b)};
}

__device__ __forceinline__ float lane_of(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

constexpr int kRowShl = 0x100, kRowShr = 0x110, kWaveShl1 = 0x130, kWaveShr1 = 0x138, kRowBcast15 = 0x142,
              kRowBcast31 = 0x143, kRowNewBcast = 0x150;

// One step of the in-row scan, for groups of G lanes: the map `s` lanes below
// (up: above), the identity where that lane belongs to another group.
template <int G, int s, bool kUp>
__device__ __forceinline__ Map neighbour(Map m, int gl) {
  Map e = dpp<(kUp ? kRowShl : kRowShr) + s>(m);
  if constexpr (G < 16) {
    const bool inside = kUp ? gl + s < G : gl >= s;
    e.a = inside ? e.a : 1.0f;
    e.b = inside ? e.b : 0.0f;
  }
  return e;
}

// Inclusive prefix over the group (tokens run with the lanes).
template <int G, bool kDrop>
__device__ __forceinline__ Map prefix(Map m, int gl) {
  if constexpr (G >= 2) m = compose<kDrop>(m, neighbour<G, 1, false>(m, gl));
  if constexpr (G >= 4) m = compose<kDrop>(m, neighbour<G, 2, false>(m, gl));
  if constexpr (G >= 8) m = compose<kDrop>(m, neighbour<G, 4, false>(m, gl));
  if constexpr (G >= 16) m = compose<kDrop>(m, neighbour<G, 8, false>(m, gl));
  if constexpr (G >= 32) m = compose<kDrop>(m, dpp<kRowBcast15, 0xa>(m));
  if constexpr (G == 64) m = compose<kDrop>(m, dpp<kRowBcast31, 0xc>(m));
  return m;
}

// Inclusive suffix over the group (the adjoint runs against the lanes).  Rows
// of 16 lanes by DPP; across the four rows of a wave the row totals (in each
// row's first lane) are read into scalars.
template <int G, bool kDrop>
__device__ __forceinline__ Map suffix(Map m, int gl) {
  if constexpr (G >= 2) m = compose<kDrop>(m, neighbour<G, 1, true>(m, gl));
  if constexpr (G >= 4) m = compose<kDrop>(m, neighbour<G, 2, true>(m, gl));
  if constexpr (G >= 8) m = compose<kDrop>(m, neighbour<G, 4, true>(m, gl));
  if constexpr (G >= 16) m = compose<kDrop>(m, neighbour<G, 8, true>(m, gl));
  if constexpr (G == 32) {  // the odd row's total into the even row before it
    const bool even = gl < 16;
    const bool low = (threadIdx.x & 32) == 0;
    Map e;
    e.a = !even ? 1.0f : low ? lane_of(m.a, 16) : lane_of(m.a, 48);
    e.b = !even ? 0.0f : low ? lane_of(m.b, 16) : lane_of(m.b, 48);
    m = compose<kDrop>(m, e);
  }
  if constexpr (G == 64) {
    const Map r1{lane_of(m.a, 16), lane_of(m.b, 16)};
    const Map r2{lane_of(m.a, 32), lane_of(m.b, 32)};
    const Map r3{lane_of(m.a, 48), lane_of(m.b, 48)};
    const Map r23 = compose<kDrop>(r2, r3);
    const Map r123 = compose<kDrop>(r1, r23);
    const int row = gl >> 4;
    Map e;
    e.a = row == 0 ? r123.a : row == 1 ? r23.a : row == 2 ? r3.a : 1.0f;
    e.b = row == 0 ? r123.b : row == 1 ? r23.b : row == 2 ? r3.b : 0.0f;
    m = compose<kDrop>(m, e);
  }
  return m;
}

// The value of the lane before (after) in the group; `edge` in its first (last) lane.
template <int G>
__device__ __forceinline__ float lane_before(float v, float edge, int gl) {
  if constexpr (G == 1) return edge;
  if constexpr (G == 64) return dpp<kWaveShr1>(edge, v);
  const float r = G == 32 ? dpp<kWaveShr1>(edge, v) : dpp<kRowShr + 1>(edge, v);
  return G != 16 && gl == 0 ? edge : r;
}

template <int G>
__device__ __forceinline__ float lane_after(float v, float edge, int gl) {
  if constexpr (G == 1) return edge;
  if constexpr (G == 64) return dpp<kWaveShl1>(edge, v);
  const float r = G == 32 ? dpp<kWaveShl1>(edge, v) : dpp<kRowShl + 1>(edge, v);
  return G != 16 && gl == G - 1 ? edge : r;
}

// The value of the group's last (first) lane, in all its lanes.
template <int G>
__device__ __forceinline__ float last_lane(float v, int lane) {
  if constexpr (G == 1) return v;
  if constexpr (G == 64) return lane_of(v, 63);
  if constexpr (G == 32) return lane < 32 ? lane_of(v, 31) : lane_of(v, 63);
  if constexpr (G == 16) return dpp<kRowNewBcast + 15>(v, v);
  return __shfl(v, lane | (G - 1));
}

template <int G>
__device__ __forceinline__ float first_lane(float v, int lane) {
  if constexpr (G == 1) return v;
  if constexpr (G == 64) return lane_of(v, 0);
  if constexpr (G == 32) return lane < 32 ? lane_of(v, 0) : lane_of(v, 32);
  if constexpr (G == 16) return dpp<kRowNewBcast>(v, v);
  return __shfl(v, lane & ~(G - 1));
}

// ---- the gate ----------------------------------------------------------------

// Per-channel constants of the gate.  e^-(g + bias) is eb * 2^(nb - g log2 e)
// with nb the whole number next to -bias log2 e and eb = e^(-bias - nb ln 2), the
// rest, from ln 2 in two parts (the reduction of Cody and Waite).  Rounding
// bias * log2 e instead would shift every token of a channel the same way, which
// a long memory adds up; the whole of e^-bias in eb would let the other factor
// overflow, or vanish, before the product does.  A bias beyond 2^14 closes or
// opens its gate, or meets a g whose own rounding is as large: it goes into the
// exponent as it is, infinities too.
struct GateParams {
  float eb, nb, rate, nr;
};

constexpr float kLn2Low = -1.9046542e-9f;  // ln 2 - kLn2

template <bool kRate>
__device__ __forceinline__ GateParams gate_params(const float* gate_bias, const float* rate, int64_t d) {
  GateParams p;
  const float bias = gate_bias ? gate_bias[d] : 0.0f;
  const bool split = __builtin_fabsf(bias) <= 16384.0f;
  const float n = __builtin_rintf(-bias * kLog2e);
  const float r = __builtin_fmaf(-n, kLn2Low, __builtin_fmaf(-n, kLn2, -bias));
  p.eb = split ? expf(r) : 1.0f;
  p.nb = split ? n : -bias * kLog2e;
  p.rate = kRate ? rate[d] : 0.0f;
  p.nr = -p.rate * kLog2e;
  return p;
}

// s = sigmoid(v), t = 1 - s, the decay a and om = 1 - a.  Whichever of the two
// is small comes from its own formula and the other is 1 minus it, one
// rounding: a long memory (a near 1) multiplies any bias of a by 1 / (1 - a).
struct Gate {
  float s, t, a, om;
};

// kSlow: the rate is below 1/4, so every token takes the series.
template <bool kRate, bool kSlow = false>
__device__ __forceinline__ Gate gate_of(float g, const GateParams& p) {
  Gate r;
  const float e = p.eb * exp2_hw(__builtin_fmaf(g, -kLog2e, p.nb));
  const float q = rcp_hw(1.0f + e);
  const bool open = e < 1.0f;
  r.t = open ? e * q : 1.0f - q;
  r.s = open ? 1.0f - e * q : q;
  if constexpr (kRate) {
    // 1 - e^-c: below 1/4 by its series (to c^6, within c^6/5040 < 5e-8 of it)
    const float c = p.rate * r.s;
    float m = __builtin_fmaf(c, -1.0f / 720.0f, 1.0f / 120.0f);
    m = __builtin_fmaf(c, m, -1.0f / 24.0f);
    m = __builtin_fmaf(c, m, 1.0f / 6.0f);
    m = __builtin_fmaf(c, m, -0.5f);
    m = __builtin_fmaf(c, m, 1.0f);
    r.om = c * m;
    r.a = __builtin_fmaf(-c, m, 1.0f);
    if constexpr (!kSlow) {
      const float e = exp2_hw(p.nr * r.s);
      const bool near = c < 0.25f;
      r.om = near ? r.om : 1.0f - e;
      r.a = near ? r.a : e;
    }
  } else {
    r.a = r.s;
    r.om = r.t;
  }
  return r;
}

// The gates of a lane's tokens.  slow: every lane's rate is below 1/4 (models
// with a long memory keep it there), which saves the exponential of each token
// (4 x 4096 x 4096 bf16, whose vector units were 95% busy: forward 121 -> 100
// us, training step 311 -> 287).
template <bool kRate>
__device__ __forceinline__ void gates_of(const float g[kTok], const GateParams& p, bool slow, Gate out[kTok]) {
  if (kRate && slow) {
#pragma unroll
    for (int j = 0; j < kTok; ++j) out[j] = gate_of<kRate, true>(g[j], p);
  } else {
#pragma unroll
    for (int j = 0; j < kTok; ++j) out[j] = gate_of<kRate>(g[j], p);
  }
}

template <int kMode>
__device__ __forceinline__ float input_weight(float a, float om) {
  if constexpr (kMode == SSM_GATED_PLAIN) return 1.0f;
  if constexpr (kMode == SSM_GATED_CONVEX) return om;
  return __builtin_amdgcn_sqrtf(om * (1.0f + a));
}

__device__ __forceinline__ float sigmoid_f32(float z) { return rcp_hw(1.0f + exp2_hw(-z * kLog2e)); }

// Bit j set where token t + j starts a sequence.
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* row, int t, int seqlen, bool full) {
  uint32_t lo = 0, hi = 0;
  if (full || t + 8 <= seqlen) {
    load_bytes8(row + t, &lo, &hi);
  } else if (t < seqlen) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (t + j < seqlen) lo |= (uint32_t)row[t + j] << (8 * j);
      if (t + 4 + j < seqlen) hi |= (uint32_t)row[t + 4 + j] << (8 * j);
    }
  }
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    bits |= ((lo >> (8 * j)) & 0xffu) ? 1u << j : 0u;
    bits |= ((hi >> (8 * j)) & 0xffu) ? 16u << j : 0u;
  }
  return bits;
}

// Bits where the state is dropped: resets and gates that are exactly 0.
__device__ __forceinline__ uint32_t drop_bits(const float a[kTok], uint32_t resets) {
  float m = a[0];
#pragma unroll
  for (int j = 1; j < kTok; ++j) m = __builtin_fminf(m, a[j]);
  if (__builtin_expect(__ballot(m == 0.0f) != 0, 0)) {
#pragma unroll
    for (int j = 0; j < kTok; ++j) resets |= a[j] == 0.0f ? 1u << j : 0u;
  }
  return resets;
}

// A lane's tokens as one map.
template <bool kDrop>
__device__ __forceinline__ Map chunk_map(const float a[kTok], const float b[kTok], uint32_t drop) {
  Map m{a[0], b[0]};
#pragma unroll
  for (int j = 1; j < kTok; ++j) {
    const float h = __builtin_fmaf(a[j], m.b, b[j]);
    m.b = kDrop && (drop >> j & 1) ? b[j] : h;
    m.a *= a[j];
  }
  m.a = off_zero(m.a);
  if constexpr (kDrop) m.a = drop ? 0.0f : m.a;
  return m;
}

template <bool kDrop>
__device__ __forceinline__ float next_state(float a, float b, float h, uint32_t drop, int j) {
  const float r = __builtin_fmaf(a, h, b);
  return kDrop && (drop >> j & 1) ? b : r;
}

// ---- the forward -------------------------------------------------------------

// The scan of one tile: `before` is the state before the lane's chunk, h[j] the
// states of its tokens, and carry moves on to the state after the tile.
template <int G, bool kDrop>
__device__ __forceinline__ void scan_tile(const float a[kTok], const float b[kTok], uint32_t drop, int lane, int gl,
                                          int wave, int waves, Map* totals, float& carry, float h[kTok],
                                          float& before) {
  const Map m = prefix<G, kDrop>(chunk_map<kDrop>(a, b, drop), gl);
  float in = carry;
  if (G == 64 && waves > 1) {
    // Each wave's total through LDS; every wave folds all of them, taking its
    // own carry-in on the way.
    if (lane == 63) totals[wave] = m;
    lds_barrier();
    float c = carry;
    for (int w = 0; w < waves; ++w) {
      if (w == wave) in = c;
      c = apply<true>(totals[w], c);
    }
    carry = c;
  } else {
    carry = last_lane<G>(apply<kDrop>(m, in), lane);
  }
  before = lane_before<G>(apply<kDrop>(m, in), in, gl);
  float s = before;
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    s = next_state<kDrop>(a[j], b[j], s, drop, j);
    h[j] = s;
  }
}

// G lanes per channel.  G < 64: rows of one tile, 64 / G channels a wave.
// G = 64: a block owns one channel and its waves take consecutive tiles of 512
// tokens, joined through LDS.
template <typename IoT, int G, int kMode, bool kRate>
__global__ __launch_bounds__(G == 64 ? 64 * kMaxWaves : 256) void gated_fwd_kernel(GatedArgs p) {
  __shared__ Map totals[2][G == 64 ? kMaxWaves : 1];
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  int64_t ch = G == 64 ? (int64_t)blockIdx.x : ((int64_t)blockIdx.x * waves + wave) * (64 / G) + lane / G;
  const bool live = ch < p.channels;
  ch = live ? ch : p.channels - 1;
  const int64_t bt = ch / p.dim, d = ch - bt * p.dim;
  const int L = p.seqlen;
  const IoT* xr = static_cast<const IoT*>(p.x) + ch * L;
  const IoT* gr = static_cast<const IoT*>(p.gate) + ch * L;
  const IoT* zr = static_cast<const IoT*>(p.z) + (p.z ? ch * L : 0);
  IoT* yr = static_cast<IoT*>(p.y) + ch * L;
  const uint8_t* rr = p.reset + (p.reset ? bt * L : 0);
  float* ck = p.ckpt + (p.ckpt ? ch * p.ckpts : 0);
  constexpr bool kStream = streamed<IoT>;
  const GateParams gp = gate_params<kRate>(p.gate_bias, p.rate, d);
  const bool slow = kRate && __ballot(!(gp.rate < 0.25f)) == 0;
  float carry = p.h0 ? p.h0[ch] : 0.0f;
  // last_state may be h0: every wave has its value before any wave can end.
  if (G == 64 && waves > 1) __syncthreads();

  constexpr int kTile = G * kTok;
  const int step = G == 64 ? kTile * waves : kTile;
  // The next tile's pieces are requested before this one is worked on.
  Raw8<IoT> nx, ng, nz;
  const auto request = [&](int base) {
    const int t0 = G == 64 ? base + wave * kTile : base;
    nx = request8<G == 1, kStream>(xr, t0, gl * kTok, L);
    ng = request8<G == 1, kStream>(gr, t0, gl * kTok, L);
    if (p.z) nz = request8<G == 1, kStream>(zr, t0, gl * kTok, L);
  };
  request(0);
  int parity = 0;
  for (int base = 0; base < L; base += step, parity ^= 1) {
    const int t0 = G == 64 ? base + wave * kTile : base;
    const int t = t0 + gl * kTok;
    const bool full = t0 + kTile <= L;  // uniform over the wave
    float xv[kTok], gv[kTok], a[kTok], b[kTok], h[kTok];
    if (!full) {
      finish8<G == 1>(nx, t0, gl * kTok, L);
      finish8<G == 1>(ng, t0, gl * kTok, L);
      if (p.z) finish8<G == 1>(nz, t0, gl * kTok, L);
    }
    nx.get(xv);
    ng.get(gv);
    const Raw8<IoT> zc = nz;
    uint32_t drop = p.reset ? reset_bits(rr, t, L, full) : 0;
    if (G == 64 && base + step < L) request(base + step);
    Gate g[kTok];
    gates_of<kRate>(gv, gp, slow, g);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      a[j] = g[j].a;
      b[j] = input_weight<kMode>(g[j].a, g[j].om) * xv[j];
    }
    if (!full) {  // tokens past the end leave the state as it is
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        a[j] = t + j < L ? a[j] : 1.0f;
        b[j] = t + j < L ? b[j] : 0.0f;
      }
    }
    drop = drop_bits(a, drop);
    float before;
    if (__ballot(drop != 0))
      scan_tile<G, true>(a, b, drop, lane, gl, wave, waves, totals[parity], carry, h, before);
    else
      scan_tile<G, false>(a, b, drop, lane, gl, wave, waves, totals[parity], carry, h, before);
    if (p.ckpt && (t & (kCkptStep - 1)) == 0 && t < L && live) ck[t / kCkptStep] = before;
    if (p.z) {
      float zv[kTok];
      zc.get(zv);
#pragma unroll
      for (int j = 0; j < kTok; ++j) h[j] *= silu_f32(zv[j]);
    }
    if (live) store_row8<kStream>(yr, t, L, full, h);
    if constexpr (G < 64) break;  // such a row is one tile
  }
  if (p.last && live && gl == 0 && (G < 64 || wave == 0)) p.last[ch] = carry;
}

// ---- the backward ------------------------------------------------------------

// One tile of the backward.  ds holds dy silu'(z) and becomes dz; with a rate,
// dg comes back without its factor.
template <int G, int kMode, bool kRate, bool kDrop>
__device__ __forceinline__ void bwd_tile(const float x[kTok], const Gate g[kTok], const float q[kTok], float h_in,
                                         uint32_t drop, int valid, int lane, int gl, int wave, int waves, Map* totals,
                                         float& mu, float ds[kTok], float dx[kTok], float dg[kTok], float& sum_r) {
  float a[kTok], b[kTok], w[kTok], hp[kTok];  // hp: the state before each token
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    a[j] = g[j].a;
    w[j] = input_weight<kMode>(g[j].a, g[j].om);
    b[j] = w[j] * x[j];
  }
  // The states, from the state before the tile.
  const Map f = prefix<G, kDrop>(chunk_map<kDrop>(a, b, drop), gl);
  float s = lane_before<G>(apply<kDrop>(f, h_in), h_in, gl);
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    hp[j] = s;
    s = next_state<kDrop>(a[j], b[j], s, drop, j);
    ds[j] *= s;
  }
  if (valid < kTok) {  // tokens past the end: no gradient, whatever the state
#pragma unroll
    for (int j = 0; j < kTok; ++j) hp[j] = j < valid ? hp[j] : 0.0f;
  }
  // The adjoint: mu_j = a_j lambda_j, lambda_j = q_j + mu_{j+1}, as the lane's
  // map of the mu that enters from the right.
  Map r{1.0f, 0.0f};
#pragma unroll
  for (int j = kTok - 1; j >= 0; --j) {
    const float lam = r.b + q[j];
    r.b = kDrop && (drop >> j & 1) ? 0.0f : a[j] * lam;
    r.a *= a[j];
  }
  r.a = off_zero(r.a);
  if constexpr (kDrop) r.a = drop ? 0.0f : r.a;
  r = suffix<G, kDrop>(r, gl);
  float in = mu;
  if (G == 64 && waves > 1) {
    if (lane == 0) totals[wave] = r;
    lds_barrier();
    float c = mu;
    for (int v = waves - 1; v >= 0; --v) {
      if (v == wave) in = c;
      c = apply<true>(totals[v], c);
    }
    mu = c;
  } else {
    mu = first_lane<G>(apply<kDrop>(r, in), lane);
  }
  float m = lane_after<G>(apply<kDrop>(r, in), in, gl);
  float tr = 0.0f;
#pragma unroll
  for (int j = kTok - 1; j >= 0; --j) {
    const bool dropped = kDrop && (drop >> j & 1);
    const float lam = q[j] + m;
    dx[j] = lam * w[j];
    float da = dropped ? 0.0f : hp[j];  // dL/da over lambda
    if constexpr (kMode == SSM_GATED_CONVEX) da -= x[j];
    if constexpr (kMode == SSM_GATED_NORM) {
      // dw/da = -a / w; da/dv vanishes faster than w, so 0 where w underflows
      const float slope = w[j] > 0.0f ? a[j] * rcp_hw(w[j]) : 0.0f;
      da = __builtin_fmaf(-slope, x[j], da);
    }
    da *= lam;
    const float st = g[j].s * g[j].t;
    if constexpr (kRate) {
      // da/dv = -rate a s t (the caller has the rate), da/drate = -a s
      const float na = -da * a[j];
      dg[j] = na * st;
      tr = __builtin_fmaf(na, g[j].s, tr);
    } else {
      dg[j] = da * st;
    }
    m = dropped ? 0.0f : a[j] * lam;
  }
  sum_r += tr;
}

// Four waves on a SIMD in bf16 (128 registers; 4 x 4096 x 4096 training step 285
// us, 296 at three); fp32 would spill there (4 x 4096 x 1024 145.2 us, 142.2 at
// three).
//
// Where p.join is the batch, a block has every batch row of its channels and
// writes their sums itself: with G < 64 in groups next to each other, with
// G = 64 in rows of p.waves waves.
template <typename IoT, int G, int kMode, bool kRate>
__global__ __launch_bounds__(G == 64 ? 64 * kMaxBwdWaves : 256, sizeof(IoT) == 2 ? 4 : 3) void gated_bwd_kernel(
    GatedArgs p) {
  constexpr int kSlots = G == 64 ? kMaxWaves : 256 / G;  // waves or groups of a block
  __shared__ Map totals[2][G == 64 ? kMaxWaves : 1];
  __shared__ Map sums[kSlots];
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  const int block_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block_waves = blockDim.x >> 6;
  const int waves = G == 64 ? p.waves : block_waves;  // of a row
  const int wave = G == 64 ? block_wave % waves : block_wave, first = block_wave - wave;
  const int slot = G == 64 ? block_wave / waves : block_wave * (64 / G) + lane / G;
  const int own = (G == 64 ? block_waves / waves : kSlots) / p.join;  // channels of the block
  int64_t ch = (int64_t)blockIdx.x * own;
  bool live = true;
  if (p.join > 1) {
    const int64_t c = ch + slot / p.join;
    live = slot < own * p.join && c < p.dim;
    ch = slot % p.join * p.dim + c;
  } else {
    ch += slot;
    live = ch < p.channels;
  }
  ch = live ? ch : p.channels - 1;
  const int64_t bt = ch / p.dim, d = ch - bt * p.dim;
  const int L = p.seqlen;
  const IoT* xr = static_cast<const IoT*>(p.x) + ch * L;
  const IoT* gr = static_cast<const IoT*>(p.gate) + ch * L;
  const IoT* zr = static_cast<const IoT*>(p.z) + (p.z ? ch * L : 0);
  const IoT* dyr = static_cast<const IoT*>(p.dy) + ch * L;
  IoT* dxr = static_cast<IoT*>(p.dx) + ch * L;
  IoT* dgr = static_cast<IoT*>(p.dgate) + ch * L;
  IoT* dzr = static_cast<IoT*>(p.dz) + (p.dz ? ch * L : 0);
  const uint8_t* rr = p.reset + (p.reset ? bt * L : 0);
  const float* ck = p.ckpt + ch * p.ckpts;
  constexpr bool kStream = streamed<IoT>;
  const GateParams gp = gate_params<kRate>(p.gate_bias, p.rate, d);
  const bool slow = kRate && __ballot(!(gp.rate < 0.25f)) == 0;
  float mu = p.dlast ? p.dlast[ch] : 0.0f;
  float sum_b = 0.0f, sum_r = 0.0f;

  constexpr int kTile = G * kTok;
  const int step = G == 64 ? kTile * waves : kTile;
  // The tile before (in time) is requested before this one is worked on (4 x
  // 4096 x 4096 bf16 training step 318 -> 312 us, 1 x 512 x 32768 85 -> 78).
  Raw8<IoT> nx, ng, nz, nq;
  float nh;
  const auto request = [&](int base) {
    const int t0 = G == 64 ? base + wave * kTile : base;
    nx = request8<G == 1, kStream>(xr, t0, gl * kTok, L);
    ng = request8<G == 1, kStream>(gr, t0, gl * kTok, L);
    nq = request8<G == 1, kStream>(dyr, t0, gl * kTok, L);
    if (p.z) nz = request8<G == 1, kStream>(zr, t0, gl * kTok, L);
    nh = t0 < L ? ck[t0 / kCkptStep] : 0.0f;
  };
  request((L - 1) / step * step);
  int parity = 0;
  for (int base = (L - 1) / step * step; base >= 0; base -= step, parity ^= 1) {
    const int t0 = G == 64 ? base + wave * kTile : base;
    const int t = t0 + gl * kTok;
    const bool full = t0 + kTile <= L;
    const int valid = L - t;
    float x[kTok], gv[kTok], q[kTok], ds[kTok], dx[kTok], dg[kTok];
    Gate g[kTok];
    if (!full) {
      finish8<G == 1>(nx, t0, gl * kTok, L);
      finish8<G == 1>(ng, t0, gl * kTok, L);
      finish8<G == 1>(nq, t0, gl * kTok, L);
      if (p.z) finish8<G == 1>(nz, t0, gl * kTok, L);
    }
    nx.get(x);
    ng.get(gv);
    nq.get(q);
    const Raw8<IoT> zc = nz;
    const float h_in = nh;
    if (G == 64 && base >= step) request(base - step);
    uint32_t drop = p.reset ? reset_bits(rr, t, L, full) : 0;
    gates_of<kRate>(gv, gp, slow, g);
    if (!full) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (t + j >= L) g[j].a = 1.0f, g[j].om = 0.0f, g[j].t = 0.0f, g[j].s = 0.0f, x[j] = 0.0f, q[j] = 0.0f;
      }
    }
    if (p.z) {
      float zv[kTok];
      zc.get(zv);
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const float sg = sigmoid_f32(zv[j]);
        const float sz = zv[j] * sg;
        ds[j] = q[j] * __builtin_fmaf(sz, 1.0f - sg, sg);  // dy silu'(z)
        q[j] *= sz;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kTok; ++j) ds[j] = 0.0f;
    }
    {
      float a[kTok];
#pragma unroll
      for (int j = 0; j < kTok; ++j) a[j] = g[j].a;
      drop = drop_bits(a, drop);
    }
    if (__ballot(drop != 0))
      bwd_tile<G, kMode, kRate, true>(x, g, q, h_in, drop, valid, lane, gl, wave, waves, totals[parity] + first, mu,
                                      ds, dx, dg, sum_r);
    else
      bwd_tile<G, kMode, kRate, false>(x, g, q, h_in, drop, valid, lane, gl, wave, waves, totals[parity] + first, mu,
                                       ds, dx, dg, sum_r);
    float tb = 0.0f;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if constexpr (kRate) dg[j] *= gp.rate;
      tb += dg[j];
    }
    sum_b += tb;
    if (live) {
      store_row8<kStream>(dxr, t, L, full, dx);
      store_row8<kStream>(dgr, t, L, full, dg);
      if (p.dz) store_row8<kStream>(dzr, t, L, full, ds);
    }
    if constexpr (G < 64) break;
  }
  // Row sums: over the group's lanes, then over the block's waves.
#pragma unroll
  for (int s = 1; s < G; s <<= 1) {
    sum_b += __shfl_xor(sum_b, s);
    if constexpr (kRate) sum_r += __shfl_xor(sum_r, s);
  }
  if (p.dh0 && live && gl == 0 && (G < 64 || wave == 0)) p.dh0[ch] = mu;
  int64_t out = ch;
  bool writes = live && gl == 0;
  const int parts = G == 64 ? block_waves : p.join;  // sums that make one output
  if (parts > 1) {
    if (gl == 0) sums[G == 64 ? block_wave : slot] = Map{sum_b, sum_r};
    lds_barrier();
    const int c = G == 64 ? 0 : threadIdx.x;  // of the block's channels
    if (G < 64) out = (int64_t)blockIdx.x * own + c;
    if (G == 64 && p.join > 1) out = d;
    writes = G == 64 ? threadIdx.x == 0 : c < own && out < p.dim;
    if (writes) {
      sum_b = sum_r = 0.0f;
      for (int i = c * parts; i < (c + 1) * parts; ++i) {
        sum_b += sums[i].a;
        sum_r += sums[i].b;
      }
    }
  }
  if (writes) {
    if (p.dbias) p.dbias[out] = sum_b;
    if (kRate && p.drate) p.drate[out] = sum_r;
  }
}

// out[d] = the sum over the batch rows: 32 channels a block, blockDim / 32
// slices of the rows.  A slice requests 8 of its rows at once; rows and slices
// are added in order, in 64 bits, since a batch of many short rows is a long
// sum (65536 rows of one token, one chain of 32 bits: off by 7e-4 of the sum).
constexpr int kReduceSlices = 32;

__global__ __launch_bounds__(32 * kReduceSlices) void gated_bwd_reduce_kernel(const float* bias_part,
                                                                             const float* rate_part, float* dbias,
                                                                             float* drate, int64_t batch,
                                                                             int64_t dim) {
  __shared__ double sums[2][kReduceSlices][33];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5, slices = blockDim.x >> 5;
  const int64_t d = (int64_t)blockIdx.x * 32 + col;
  double sb = 0.0, sr = 0.0;
  if (d < dim) {
    int64_t b = slice;
    for (; b + 7 * slices < batch; b += 8 * slices) {
      float vb[8], vr[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        vb[j] = dbias ? bias_part[(b + j * slices) * dim + d] : 0.0f;
        vr[j] = drate ? rate_part[(b + j * slices) * dim + d] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sb += vb[j], sr += vr[j];
    }
    for (; b < batch; b += slices) {
      if (dbias) sb += bias_part[b * dim + d];
      if (drate) sr += rate_part[b * dim + d];
    }
  }
  sums[0][slice][col] = sb;
  sums[1][slice][col] = sr;
  lds_barrier();
  if (slice == 0 && d < dim) {
    for (int i = 1; i < slices; ++i) sb += sums[0][i][col], sr += sums[1][i][col];
    if (dbias) dbias[d] = (float)sb;
    if (drate) drate[d] = (float)sr;
  }
}

// ---- the decode step ---------------------------------------------------------

struct StepArgs {
  float* state;
  const void* x;
  const void* gate;
  const float* gate_bias;
  const float* rate;
  const void* z;
  void* y;
  int64_t dim;
  int blocks_per_row;
};

// V channels per thread (4: dim a multiple of 4, so they are of one batch row
// and whole; 1: any dim).
template <typename IoT, int V, int kMode, bool kRate>
__global__ __launch_bounds__(256) void gated_step_kernel(StepArgs p) {
  const int row = blockIdx.x / p.blocks_per_row;
  const int64_t d = ((int64_t)(blockIdx.x - row * p.blocks_per_row) * blockDim.x + threadIdx.x) * V;
  if (d >= p.dim) return;
  const int64_t i = row * p.dim + d;
  float x[V], g[V], z[V], h[V], y[V];
  load_n<V>(static_cast<const IoT*>(p.x) + i, x);
  load_n<V>(static_cast<const IoT*>(p.gate) + i, g);
  load_n<V>(p.state + i, h);
  if (p.z) load_n<V>(static_cast<const IoT*>(p.z) + i, z);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const GateParams gp = gate_params<kRate>(p.gate_bias, p.rate, d + j);
    const Gate gt = gate_of<kRate>(g[j], gp);
    const float b = input_weight<kMode>(gt.a, gt.om) * x[j];
    h[j] = gt.a == 0.0f ? b : __builtin_fmaf(gt.a, h[j], b);
    y[j] = p.z ? h[j] * silu_f32(z[j]) : h[j];
  }
  store_n<V>(p.state + i, h);
  store_n<V>(static_cast<IoT*>(p.y) + i, y);
}

// ---- host side ---------------------------------------------------------------

constexpr int64_t kMaxSeqlen = (int64_t)1 << 30;  // token offsets in a row fit an int

struct GatedShape {
  int64_t bd, bdl, ckpts, row_bytes;
};

ssm_status_t gated_shape(int64_t batch, int64_t dim, int64_t seqlen, ssm_dtype_t io, GatedShape* s) {
  if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_DTYPE;
  if (batch < 1 || dim < 1 || seqlen < 1) return SSM_ERR_SHAPE;
  int64_t bytes;
  if (!mul_ok(batch, dim, &s->bd) || !mul_ok(s->bd, seqlen, &s->bdl) || !mul_ok(s->bdl, 8, &bytes) ||
      !mul_ok(s->bd, 64, &bytes) || !mul_ok(batch, seqlen, &bytes))
    return SSM_ERR_SHAPE;
  if (seqlen >= kMaxSeqlen || s->bd >= ((int64_t)1 << 31)) return SSM_ERR_UNSUPPORTED;
  s->ckpts = (seqlen + kCkptStep - 1) / kCkptStep;
  s->row_bytes = s->bdl * (int64_t)io_size(io);
  return SSM_OK;
}

bool gated_mode_ok(ssm_gated_mode_t mode) {
  return mode == SSM_GATED_PLAIN || mode == SSM_GATED_CONVEX || mode == SSM_GATED_NORM;
}

struct GatedPlan {
  int group;  // lanes per channel
  int waves;  // of a row, 64-lane groups
  int threads;
  int64_t blocks;
  int join;  // backward: batch rows of a channel in one block, all of them or 1
};

// Waves that share a row of `tiles` 512-token tiles.  More waves fill the chip
// (up to 12 for each of the 1024 SIMDs, resident or queued; past `enough` a
// row gets no more), but the row is walked in steps of that many tiles, and a
// last step that is mostly empty costs a whole one; 16 waves that walk it in a
// single step have nothing to load ahead and one block to a compute unit.  1, 2,
// 3, 4, 8 and 16 are the counts whose blocks fill a compute unit's registers.
// Measured (us, bf16 unless said, waves in brackets): forward 3 x 1001 x 8001
// 47.9 [8] 56.4 [16] 52.8 [6]; 4 x 1024 x 4160 30.3 [3] 33.9 [5] 41.9 [8]; 2 x
// 5120 x 1500 29.5 [3] 35.6 [4] 36.1 [2]; fp32 1 x 2560 x 131072 750 [16] 774
// [8] 798 [10], 8 x 1536 x 2048 72.7 [4] 78.9 [2], 1 x 2560 x 8192 65.1 [8]
// 70.5 [16]; training step 4 x 1024 x 4160 86.8 [3] 102.5 [4] 124 [5]; 8 x 512
// x 8200 160 [4] 188 [6] 207 [5]; 8 x 1536 x 2048 fp32 220.5 [2] 228.8 [1].
//
// `enough` ends the larger counts above 12288 channels.  Measured past that edge,
// the larger count is still the better one by up to 8% (4 x 3500 x 2048 fp32:
// forward 87.5 [2, as planned] 80.8 [4], training step 256.9 [1, as planned] 242.1
// [2] 238.4 [4]; 8 x 2560 x 4096: forward 117.4 [2, as planned] 111.2 [4], training
// step 340.4 [1, as planned] 322.4 [4]); in bf16 at 2048 tokens 2 waves are the
// best on both sides (8 x 1600 training step 107.7 [1, as planned] 104.2 [2] 108.4
// [4]).  So the edge costs time above it and is no optimum.
constexpr int64_t kFewWaves = 12288;
constexpr int64_t kEnoughFwd = 49152;
constexpr int64_t kEnoughBwd = 24576;

int64_t row_waves(int64_t channels, int64_t tiles, int64_t most, int64_t enough) {
  if (channels * most < kFewWaves) {  // few rows: all the waves, balanced over the steps
    const int64_t steps = (tiles + most - 1) / most;
    return (tiles + steps - 1) / steps;
  }
  int64_t best = 1;
  double least = 0.0;
  for (int64_t w : {1, 2, 3, 4, 8, 16}) {
    if (w > most || w > tiles || (w > 1 && channels * w > enough && channels * best >= kFewWaves)) break;
    const int64_t steps = (tiles + w - 1) / w;
    double cost = (double)(steps * w) / (double)tiles;
    if (steps == 1 && w == 16) cost *= 1.1;
    if (channels * w < kFewWaves) cost += (double)kFewWaves / (double)(channels * w);
    if (w == 1 || cost <= least) best = w, least = cost;
  }
  return best;
}

// Rows of at most 256 tokens take the fewest lanes that hold them in one tile
// (1, 8, 16 or 32), several channels to a wave.  Longer rows take whole waves:
// groups of 16 lanes walking a long row lost to them even where they fill the
// chip (4 x 4096 x 4096 bf16 forward 123.2 us at 16 lanes, 112.5 at 64).
//
// In the backward a block takes all batch rows of its channels where they fit
// (8 waves, or 256 lanes), so that their sums need no second launch: while the
// launches are what the call waits for (bf16 training steps, two launches -> one:
// 3 x 1000 x 777 35.6 -> 31.4 us, 4 x 1024 x 1024 35.3 -> 31.2, 8 x 1024 x 512
// 35.4 -> 31.3, 4 x 4096 x 256 35.0 -> 31.1; in fp32 35.3 -> 33.8, 41.6 -> 44.5,
// 42.7 -> 41.9, 39.9 -> 41.1).  Larger rows of a batch lie far apart, often a
// power of two, and read together they meet in the same memory channels (bf16
// 4 x 4096 x 1024 72 -> 76 us, 32 x 2400 x 60 36 -> 43, 4 x 4096 x 4096 296 -> 357;
// fp32 4 x 2048 x 600 55 -> 63); small ones can lose to it too (32 x 2048 x 60
// 35.0 -> 37.2, fp32 43.5 -> 51.0).
constexpr int64_t kJoinTokens = (int64_t)1 << 22;

GatedPlan gated_plan(int64_t batch, int64_t dim, int64_t seqlen, bool backward) {
  const int64_t channels = batch * dim;
  GatedPlan p;
  p.waves = p.join = 1;
  const bool small = backward && channels * seqlen <= kJoinTokens;
  if (seqlen <= 32 * kTok) {
    p.group = 1;
    while (p.group * kTok < seqlen) p.group = p.group == 1 ? 8 : 2 * p.group;
    p.threads = 256;
    const int64_t slots = 256 / p.group;
    if (small && batch <= slots) p.join = (int)batch;
    const int64_t per_block = p.join > 1 ? slots / p.join : slots;
    p.blocks = ((p.join > 1 ? dim : channels) + per_block - 1) / per_block;
  } else {
    const int64_t tiles = (seqlen + 64 * kTok - 1) / (64 * kTok);
    const int64_t waves = backward ? row_waves(channels, tiles, kMaxBwdWaves, kEnoughBwd)
                                   : row_waves(channels, tiles, kMaxWaves, kEnoughFwd);
    p.group = 64;
    p.waves = (int)waves;
    if (small && batch * waves <= kMaxBwdWaves) p.join = (int)batch;
    p.threads = (int)(64 * waves * p.join);
    p.blocks = channels / p.join;
  }
  return p;
}

template <typename IoT, int kMode, bool kRate, bool kBwd>
hipError_t launch_gated(const GatedArgs& a, const GatedPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.blocks), block(p.threads);
#define SSM_GATED_LAUNCH(G)                                                                          \
  if constexpr (kBwd)                                                                                \
    hipLaunchKernelGGL((gated_bwd_kernel<IoT, G, kMode, kRate>), grid, block, 0, st, a);             \
  else                                                                                               \
    hipLaunchKernelGGL((gated_fwd_kernel<IoT, G, kMode, kRate>), grid, block, 0, st, a);             \
  break
  switch (p.group) {
    case 1: SSM_GATED_LAUNCH(1);
    case 8: SSM_GATED_LAUNCH(8);
    case 16: SSM_GATED_LAUNCH(16);
    case 32: SSM_GATED_LAUNCH(32);
    default: SSM_GATED_LAUNCH(64);
  }
#undef SSM_GATED_LAUNCH
  return hipGetLastError();
}

template <typename IoT, bool kBwd>
hipError_t launch_gated(const GatedArgs& a, const GatedPlan& p, ssm_gated_mode_t mode, hipStream_t st) {
  switch (mode) {
    case SSM_GATED_PLAIN:
      return a.rate ? launch_gated<IoT, SSM_GATED_PLAIN, true, kBwd>(a, p, st)
                    : launch_gated<IoT, SSM_GATED_PLAIN, false, kBwd>(a, p, st);
    case SSM_GATED_CONVEX:
      return a.rate ? launch_gated<IoT, SSM_GATED_CONVEX, true, kBwd>(a, p, st)
                    : launch_gated<IoT, SSM_GATED_CONVEX, false, kBwd>(a, p, st);
    default:
      return a.rate ? launch_gated<IoT, SSM_GATED_NORM, true, kBwd>(a, p, st)
                    : launch_gated<IoT, SSM_GATED_NORM, false, kBwd>(a, p, st);
  }
}

template <typename IoT, int V>
hipError_t launch_step(const StepArgs& a, ssm_gated_mode_t mode, unsigned blocks, int threads, hipStream_t st) {
#define SSM_GATED_STEP(M)                                                                                  \
  if (a.rate)                                                                                              \
    hipLaunchKernelGGL((gated_step_kernel<IoT, V, M, true>), dim3(blocks), dim3(threads), 0, st, a);       \
  else                                                                                                     \
    hipLaunchKernelGGL((gated_step_kernel<IoT, V, M, false>), dim3(blocks), dim3(threads), 0, st, a);      \
  break
  switch (mode) {
    case SSM_GATED_PLAIN: SSM_GATED_STEP(SSM_GATED_PLAIN);
    case SSM_GATED_CONVEX: SSM_GATED_STEP(SSM_GATED_CONVEX);
    default: SSM_GATED_STEP(SSM_GATED_NORM);
  }
#undef SSM_GATED_STEP
  return hipGetLastError();
}

GatedArgs gated_args(const GatedShape& s, int64_t dim, int64_t seqlen, const void* x, const void* gate,
                     const float* gate_bias, const float* rate, const void* z, const uint8_t* reset) {
  GatedArgs a{};
  a.x = x; a.gate = gate; a.gate_bias = gate_bias; a.rate = rate; a.z = z; a.reset = reset;
  a.channels = s.bd; a.dim = dim; a.seqlen = (int)seqlen; a.ckpts = (int)s.ckpts;
  return a;
}

// Workspace of the backward: dgate_bias and drate sums per batch row, where no
// block has them all.
int64_t bwd_workspace(const GatedShape& s, const GatedPlan& p, int64_t batch) {
  return p.join == batch ? 0 : 2 * s.bd * 4;
}

}  // namespace

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------

extern "C" {

ssm_status_t ssm_gated_scan_fwd(int64_t batch, int64_t dim, int64_t seqlen, ssm_dtype_t io, ssm_gated_mode_t mode,
                                const void* x, const void* gate, const float* gate_bias, const float* rate,
                                const void* z, const uint8_t* reset, const float* h0, void* y, float* last_state,
                                float* ckpt, struct ihipStream_t* stream) {
  GatedShape s;
  ssm_status_t st = gated_shape(batch, dim, seqlen, io, &s);
  if (st != SSM_OK) return st;
  const GatedPlan p = gated_plan(batch, dim, seqlen, false);
  if (!gated_mode_ok(mode) || !launch_ok(p.blocks, p.threads)) return SSM_ERR_UNSUPPORTED;
  if (!x || !gate || !y) return SSM_ERR_NULL;
  const size_t es = io_size(io);
  const bool in_place = h0 && h0 == last_state;
  const Buf ins[] = {{x, s.row_bytes, es}, {gate, s.row_bytes, es}, {z, s.row_bytes, es}, {gate_bias, dim * 4, 4},
                     {rate, dim * 4, 4}, {reset, batch * seqlen, 1}, {in_place ? nullptr : h0, s.bd * 4, 4}};
  const Buf outs[] = {{y, s.row_bytes, es}, {last_state, s.bd * 4, 4}, {ckpt, s.bd * s.ckpts * 4, 4}};
  st = check_buffers(ins, 7, outs, 3);
  if (st != SSM_OK) return st;
  GatedArgs a = gated_args(s, dim, seqlen, x, gate, gate_bias, rate, z, reset);
  a.h0 = h0; a.y = y; a.last = last_state; a.ckpt = ckpt;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  hipError_t e =
      io == SSM_BF16 ? launch_gated<bf16_t, false>(a, p, mode, hs) : launch_gated<float, false>(a, p, mode, hs);
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

ssm_status_t ssm_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t seqlen, ssm_dtype_t io,
                                                int64_t* bytes) {
  GatedShape s;
  ssm_status_t st = gated_shape(batch, dim, seqlen, io, &s);
  if (st == SSM_OK && bytes) *bytes = bwd_workspace(s, gated_plan(batch, dim, seqlen, true), batch);
  return st;
}

ssm_status_t ssm_gated_scan_bwd(int64_t batch, int64_t dim, int64_t seqlen, ssm_dtype_t io, ssm_gated_mode_t mode,
                                const void* x, const void* gate, const float* gate_bias, const float* rate,
                                const void* z, const uint8_t* reset, const float* ckpt, const void* dy,
                                const float* dlast, void* dx, void* dgate, float* dgate_bias, float* drate, void* dz,
                                float* dh0, void* workspace, int64_t workspace_bytes, struct ihipStream_t* stream) {
  GatedShape s;
  ssm_status_t st = gated_shape(batch, dim, seqlen, io, &s);
  if (st != SSM_OK) return st;
  const GatedPlan p = gated_plan(batch, dim, seqlen, true);
  if (!gated_mode_ok(mode) || !launch_ok(p.blocks, p.threads)) return SSM_ERR_UNSUPPORTED;
  if (!x || !gate || !ckpt || !dy || !dx || !dgate) return SSM_ERR_NULL;
  if (!rate) drate = nullptr;
  if (!z) dz = nullptr;
  const int64_t need = bwd_workspace(s, p, batch);
  if (workspace_bytes < need) return SSM_ERR_WORKSPACE;
  if (need && !workspace) return SSM_ERR_NULL;
  if (!need) workspace = nullptr;
  const size_t es = io_size(io);
  const Buf ins[] = {{x, s.row_bytes, es}, {gate, s.row_bytes, es}, {z, s.row_bytes, es}, {gate_bias, dim * 4, 4},
                     {rate, dim * 4, 4}, {reset, batch * seqlen, 1}, {ckpt, s.bd * s.ckpts * 4, 4},
                     {dy, s.row_bytes, es}, {dlast, s.bd * 4, 4}};
  const Buf outs[] = {{dx, s.row_bytes, es}, {dgate, s.row_bytes, es}, {dz, s.row_bytes, es},
                      {dgate_bias, dim * 4, 4}, {drate, dim * 4, 4}, {dh0, s.bd * 4, 4}, {workspace, need, 4}};
  st = check_buffers(ins, 9, outs, 7);
  if (st != SSM_OK) return st;
  GatedArgs a = gated_args(s, dim, seqlen, x, gate, gate_bias, rate, z, reset);
  a.ckpt = const_cast<float*>(ckpt);
  a.dy = dy; a.dlast = dlast; a.dx = dx; a.dgate = dgate; a.dz = dz; a.dh0 = dh0;
  float* part = static_cast<float*>(workspace);
  a.waves = p.waves;
  a.join = p.join;
  a.dbias = dgate_bias ? (part ? part : dgate_bias) : nullptr;
  a.drate = drate ? (part ? part + s.bd : drate) : nullptr;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  hipError_t e =
      io == SSM_BF16 ? launch_gated<bf16_t, true>(a, p, mode, hs) : launch_gated<float, true>(a, p, mode, hs);
  if (e == hipSuccess && part && (dgate_bias || drate)) {
    int slices = 2;  // 8 rows each where the batch has them
    while (slices < kReduceSlices && 8 * slices < batch) slices *= 2;
    hipLaunchKernelGGL(gated_bwd_reduce_kernel, dim3((unsigned)((dim + 31) / 32)), dim3(32 * slices), 0, hs, part,
                       part + s.bd, dgate_bias, drate, batch, dim);
    e = hipGetLastError();
  }
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

ssm_status_t ssm_gated_state_update(int64_t batch, int64_t dim, ssm_dtype_t io, ssm_gated_mode_t mode, float* state,
                                    const void* x, const void* gate, const float* gate_bias, const float* rate,
                                    const void* z, void* y, struct ihipStream_t* stream) {
  GatedShape s;
  ssm_status_t st = gated_shape(batch, dim, 1, io, &s);
  if (st != SSM_OK) return st;
  const int vec = dim % 4 == 0 ? 4 : 1;
  const int64_t lanes = dim / vec;
  const int threads = (int)std::min<int64_t>(256, (lanes + 63) / 64 * 64);
  const int64_t per_row = (lanes + threads - 1) / threads;
  if (!gated_mode_ok(mode) || !launch_ok(batch * per_row, threads)) return SSM_ERR_UNSUPPORTED;
  if (!state || !x || !gate || !y) return SSM_ERR_NULL;
  const size_t es = io_size(io);
  const Buf ins[] = {{x, s.row_bytes, es}, {gate, s.row_bytes, es}, {z, s.row_bytes, es}, {gate_bias, dim * 4, 4},
                     {rate, dim * 4, 4}};
  const Buf outs[] = {{y, s.row_bytes, es}, {state, s.bd * 4, 4}};
  st = check_buffers(ins, 5, outs, 2);
  if (st != SSM_OK) return st;
  StepArgs a;
  a.state = state; a.x = x; a.gate = gate; a.gate_bias = gate_bias; a.rate = rate; a.z = z; a.y = y;
  a.dim = dim; a.blocks_per_row = (int)per_row;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  const unsigned blocks = (unsigned)(batch * per_row);
  hipError_t e;
  if (io == SSM_BF16)
    e = vec == 4 ? launch_step<bf16_t, 4>(a, mode, blocks, threads, hs)
                 : launch_step<bf16_t, 1>(a, mode, blocks, threads, hs);
  else
    e = vec == 4 ? launch_step<float, 4>(a, mode, blocks, threads, hs)
                 : launch_step<float, 1>(a, mode, blocks, threads, hs);
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

}  // extern "C"
