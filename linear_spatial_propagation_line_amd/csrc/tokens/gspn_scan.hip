// Selective scan of a state space block, forward and backward.
//
//   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t x_t B_t[n]
//   y_t    = sum_n C_t[n] h_t[n] + D x_t,     out_t = y_t silu(z_t)
//
// and backwards, with gy_t = grad_out_t silu(z_t) and g_t = dL/dh_t:
//
//   g_t      = C_t gy_t + exp(d_{t+1} A) g_{t+1}
//   dC_t[n]  = sum over channels of gy_t h_t[n]
//   dB_t[n]  = sum over channels of d_t x_t g_t[n]
//   dx_t     = D gy_t + d_t sum_n g_t B_t
//   dd_t     = x_t sum_n g_t B_t + sum_n A[n] m_t[n],   m_t = g_t exp(d_t A) h_{t-1}
//   dA[n]    = sum over entries and tokens of d_t m_t[n]
//
// Bound by the vector ALU: per token, channel and state one exponential
// (8.3 cycles per wavefront on this chip), two products and two multiply-adds
// (4.1 each), against 8 bytes moved per token and channel. So a lane owns one
// channel, 64 adjacent channels per workgroup, and states stay in registers;
// every row of x, dt, z is one coalesced access; B_t and C_t are the same for
// a whole wavefront and are read by scalar loads into scalar registers, where
// they cost the vector ALU nothing, from an fp32 copy (pack_kernel).
//
// The four wavefronts of a workgroup share the channels and split the states.
// That gives four times the wavefronts of one lane holding all states, and the
// work that is per token and channel rather than per state (softplus, gate,
// conversions) is split as well: for 16 tokens at a time each wavefront
// prepares four tokens into LDS, runs its own states over all 16, and finishes
// four tokens from the four partial results.
//
// Few channels still do not fill the chip: the token axis is then cut into
// segments. A first pass finds each segment's state from zero and its sum of
// d (the product of its decays is exp(A sum d): one exponential), and the full
// pass folds the segments before its own into the state that it starts from.
// The full pass reads the initial state from a copy that the first pass leaves:
// its last segment may store the end state over it before others have begun.
//
// Measured, bf16, 16 states, 2304 channels, a call among calls: 8192 tokens 173
// us, of which the states' own operations need 48; 8 x 2048 training step 985 us.
// The profiler, whose launches do not overlap, gives the kernels 192 us together
// (first pass 72, full pass 115, B and C 5) and 1055 (forward 118 + 190, adjoint
// first pass 130, backward 582, sums of dB and dC 21, of the parameters 6, B and C
// twice 5). Waits for LDS and memory are a third of the wavefronts' cycles.
#include <cmath>

#include "gspn_mfma.hpp"
#include "gspn_tokens.hpp"

namespace gspn {

namespace {

// up to this many tokens: the single-token kernel (64 x 2304 channels, 16
// states, through it and through the chunks: 4 tokens 13.4 us, 28.7; 16 tokens 37, 29)
constexpr int kStepMax = 4;
constexpr int kW = 4;                   // wavefronts of a workgroup
constexpr int kS = kScanSave;           // tokens prepared together
constexpr int kOwn = kS / kW;           // of which each wavefront prepares these
constexpr int kThreads = 64 * kW;

template <typename T> struct ScanP {
  const T *x, *dt, *z, *gy;
  int64_t xb, xr, db, dr, zb, zr, gb, gr;
  const float *A, *D, *bias, *state, *gstate;
  const int32_t* lens;
  const T *Bm, *Cm;
  int64_t bb, br, bh, cb, cr, ch;
  T* out;
  float* state_out;
  float* saved;        // [B][chunks][NP][C]
  float* pack;         // [B][G][kW][Lp][2][NS]
  float* sum_d;        // [B][segs][C]
  float* carry;        // [B][segs][NP][C]: the segments' local results (forward: of the last
                       // segment, which has none, a copy of the initial state)
  // backward
  T *dx, *ddt, *dz;
  float* partA;        // [B * segs][C][N]
  float* partD;        // [B * segs][C], then the same for dt_bias
  float* partBC;       // [B][G][tiles][Lp][kW][2][NS]
  float* dstate;
  int64_t B, L, Lp, C, G, Cg, chunks;   // Lp: L rounded up to whole chunks
  int N, tiles, segs, segChunks, softplus;
  uint32_t block0;        // first workgroup of this launch
  bool whole, whole_bc;   // single tokens: states, B and C in whole aligned pieces of four
};

// ---- B and C as fp32, zeros past N states and past the entry's tokens --------
template <typename T, int NS>
__global__ __launch_bounds__(256) void pack_kernel(ScanP<T> a) {
  int64_t i = (static_cast<int64_t>(a.block0) + blockIdx.x) * 256 + threadIdx.x;
  const int n = static_cast<int>(i % (2 * NS));
  i /= 2 * NS;
  const int w = static_cast<int>(i % kW);     // reads of a token's states stay adjacent
  i /= kW;
  const int64_t t = i % a.Lp;
  i /= a.Lp;
  const int64_t g = i % a.G, b = i / a.G;
  if (b >= a.B) return;
  const int k = w * NS + n % NS;
  float v = 0.0f;
  if (k < a.N && t < seq_len(a.lens, b, a.L))
    v = n < NS ? ld1(a.Bm + b * a.bb + t * a.br + g * a.bh + k)
               : ld1(a.Cm + b * a.cb + t * a.cr + g * a.ch + k);
  a.pack[(((b * a.G + g) * kW + w) * a.Lp + t) * (2 * NS) + n] = v;
}

// The per-token operands of kB tokens: B and C of this wavefront's states,
// uniform over the wavefront, by scalar loads, and values of the lane's channel
// from LDS. Both count in one counter that a scalar load lets be waited for
// only as a whole. So a batch is loaded while the one before is computed with,
// and waited for once: wait_lds_scalar(), issue the next, compute.
template <int NS> struct Batch {
  static constexpr int kB = NS == 1 ? 4 : (NS <= 4 ? 2 : 1);   // 16 scalar registers, held twice
  float b[kB][NS], c[kB][NS];
};
__device__ __forceinline__ void wait_lds_scalar() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));   // lgkmcnt(0) alone
  __builtin_amdgcn_sched_barrier(0);
}
// tokens t .. t + kB - 1 (rows are adjacent in pack)
template <int NS> __device__ __forceinline__ void load_batch(const float* pack, int64_t t, Batch<NS>& o) {
  constexpr int kB = Batch<NS>::kB;
  const float* row = pack + t * (2 * NS);
  asm volatile("" : "+s"(row));   // keeps the loads here, and apart from other loads of these rows
  typedef const __attribute__((address_space(4))) float* cptr;
  const cptr q = (cptr)(uintptr_t)row;
#pragma unroll
  for (int k = 0; k < kB; ++k) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      o.b[k][n] = q[k * 2 * NS + n];
      o.c[k][n] = q[k * 2 * NS + NS + n];
    }
  }
}

// Four token rows of a [B, L, C] input, starting at token t and clamped to
// the last one: uniform row addresses, the lane's channel as the offset.
template <typename T>
__device__ __forceinline__ void load_rows(const T* base, int64_t stride, int64_t t, int64_t last,
                                          uint32_t c, T (&r)[kOwn]) {
  const T* row = base + (t < last ? t : last) * stride;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    r[k] = row[c];
    row += t + k < last ? stride : 0;
  }
}

// The kernel's arguments, read again from where the launch put them: keeping
// all of them in scalar registers through the loops would crowd out B and C.
template <typename T> using Args = const __attribute__((address_space(4))) ScanP<T>*;
template <typename T> __device__ __forceinline__ Args<T> args_again() {
  uint64_t k = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(k));
  return reinterpret_cast<Args<T>>(k);
}

// where a workgroup works: entry b, group g, the lane's channel, its segment
template <typename T> struct Place {
  int64_t b, g, seg, t0, t1, end;   // tokens t0 .. t1 - 1, padding t1 .. end - 1
  uint32_t c;
  int tile, lane, w;
  bool live;
};
template <typename T>
__device__ __forceinline__ Place<T> place(const ScanP<T>& a, int segs, int first_seg) {
  Place<T> p;
  p.lane = threadIdx.x & 63;
  p.w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t i = blockIdx.x + a.block0;
  p.tile = static_cast<int>(i % a.tiles);
  i /= a.tiles;
  p.g = i % static_cast<uint32_t>(a.G);
  i /= static_cast<uint32_t>(a.G);
  p.seg = first_seg + i % segs;
  p.b = i / segs;
  const int64_t k = p.tile * int64_t(64) + p.lane;
  p.live = k < a.Cg;
  p.c = static_cast<uint32_t>(p.g * a.Cg + (p.live ? k : a.Cg - 1));   // idle lanes read the last channel
  const int64_t n = seq_len(a.lens, p.b, a.L);
  p.t0 = p.seg * a.segChunks * kS;
  p.end = p.t0 + a.segChunks * kS;
  if (p.end > a.L) p.end = a.L;
  p.t1 = p.end < n ? p.end : n;
  return p;
}

template <typename T> __device__ __forceinline__ float step_size(const ScanP<T>& a, float dt, float bias) {
  const float v = dt + bias;
  return a.softplus ? softplus_f32(v) : v;
}

// this wavefront's states of the lane's channel: A log2(e), zero past N
template <typename T, int NS>
__device__ __forceinline__ void load_A(const ScanP<T>& a, const Place<T>& p, float (&A2)[NS]) {
#pragma unroll
  for (int n = 0; n < NS; ++n)
    A2[n] = p.w * NS + n < a.N ? a.A[p.c * a.N + p.w * NS + n] * kLog2e : 0.0f;
}

// this wavefront's states at the front or back end of the token axis, from
// `from` [B][C][N] (zeros when null)
template <typename T, int NS>
__device__ __forceinline__ void load_state(const ScanP<T>& a, const Place<T>& p, const float* from, float (&h)[NS]) {
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    const int k = p.w * NS + n;
    h[n] = from && k < a.N ? from[(p.b * a.C + p.c) * a.N + k] : 0.0f;
  }
}
// this wavefront's first state of the lane's channel in a segment's part of carry
template <typename T, int NS>
__device__ __forceinline__ int64_t carry_at(const ScanP<T>& a, const Place<T>& p, int64_t seg) {
  return ((p.b * a.segs + seg) * (kW * NS) + p.w * NS) * a.C + p.c;
}

// What the segments before this one (after it: kReverse) hand to it, folded
// in order from their local results and sums of d; before all of them stands
// the initial state, or (kReverse) grad_state.
template <typename T, int NS, bool kReverse>
__device__ __forceinline__ void carried_in(const ScanP<T>& a, const Place<T>& p, const float (&A2)[NS],
                                           float (&h)[NS]) {
  if (kReverse || a.segs == 1) {
    load_state(a, p, kReverse ? a.gstate : a.state, h);
  } else {
    const int64_t at = carry_at<T, NS>(a, p, a.segs - 1);
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = a.state ? a.carry[at + n * a.C] : 0.0f;
  }
  const int count = static_cast<int>(kReverse ? a.segs - 1 - p.seg : p.seg);
  constexpr int kAt = 8;   // segments loaded together
  for (int i = 0; i < count; i += kAt) {
    float local[kAt][NS], sum[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int q = i + j < count ? i + j : count - 1;
      const int64_t seg = kReverse ? a.segs - 1 - q : q, at = carry_at<T, NS>(a, p, seg);
      sum[j] = a.sum_d[(p.b * a.segs + seg) * a.C + p.c];
#pragma unroll
      for (int n = 0; n < NS; ++n) local[j][n] = a.carry[at + n * a.C];
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      if (i + j < count) {
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          // exp(A sum d) as the square of its root, below 2^128: where states
          // grow (d A > 0) it would overflow over a state that is 0 or tiny
          const float half = __builtin_amdgcn_exp2f(fminf(A2[n] * (0.5f * sum[j]), 127.0f));
          h[n] = __builtin_fmaf(half * h[n], half, local[j][n]);
        }
      }
    }
  }
  // have the values here, so that no wait for them is left inside the loops
#pragma unroll
  for (int n = 0; n < NS; ++n) asm volatile("" : "+v"(h[n]));
}

// ---- forward ----------------------------------------------------------------
template <typename T, int NS>
__global__ __launch_bounds__(kThreads) void scan_fwd_kernel(ScanP<T> a) {
  constexpr int kB = Batch<NS>::kB;
  __shared__ float sd[kS][64], sx[kS][64], sy[kW][kS][64];   // d, d x, partial y
  const Place<T> p = place(a, a.segs, 0);
  const int lane = p.lane, w = p.w;
  const float bias = a.bias ? a.bias[p.c] : 0.0f, Dc = a.D ? a.D[p.c] : 0.0f;
  float A2[NS], h[NS];
  load_A(a, p, A2);
  carried_in<T, NS, false>(a, p, A2, h);
  const bool zp = a.z != nullptr, keep = a.saved != nullptr;
  const float* pack = a.pack + ((p.b * a.G + p.g) * kW + w) * a.Lp * (2 * NS);

  T rx[kOwn], rd[kOwn], rz[kOwn];
  auto fetch = [&](int64_t c0) {
    const Args<T> k = args_again<T>();
    load_rows(k->x + p.b * k->xb, k->xr, c0 + w * kOwn, p.t1 - 1, p.c, rx);
    load_rows(k->dt + p.b * k->db, k->dr, c0 + w * kOwn, p.t1 - 1, p.c, rd);
    if (zp) load_rows(k->z + p.b * k->zb, k->zr, c0 + w * kOwn, p.t1 - 1, p.c, rz);
  };
  if (p.t0 < p.t1) fetch(p.t0);
  for (int64_t c0 = p.t0; c0 < p.t1; c0 += kS) {
    const int left = static_cast<int>(p.t1 - c0 < kS ? p.t1 - c0 : kS) - w * kOwn;   // own tokens here
    float x[kOwn], gate[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      // a token past the end has d = 0, which leaves the states as they are
      x[k] = to_f32(rx[k]);
      const float d = k < left ? step_size(a, to_f32(rd[k]), bias) : 0.0f;
      sd[w * kOwn + k][lane] = d;
      sx[w * kOwn + k][lane] = k < left ? d * x[k] : 0.0f;
      gate[k] = 1.0f;
      if (zp) {
        const float z = to_f32(rz[k]);
        gate[k] = z * sigmoid_f32(z);
      }
    }
    if (keep && p.live) {
      const Args<T> k = args_again<T>();
      float* s = k->saved + ((p.b * k->chunks + c0 / kS) * (kW * NS) + w * NS) * k->C;
#pragma unroll
      for (int n = 0; n < NS; ++n) s[n * k->C + p.c] = h[n];
    }
    lds_barrier();
    if (c0 + kS < p.t1) fetch(c0 + kS);
    Batch<NS> bc[2];
    float d[2][kB], dx[2][kB];
    auto issue = [&](int q) {
      load_batch<NS>(pack, c0 + q * kB, bc[q & 1]);
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        d[q & 1][k] = sd[q * kB + k][lane];
        dx[q & 1][k] = sx[q * kB + k][lane];
      }
    };
    issue(0);
#pragma unroll
    for (int q = 0; q < kS / kB; ++q) {
      wait_lds_scalar();
      if (q + 1 < kS / kB) issue(q + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        float y = 0.0f;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const float e = __builtin_amdgcn_exp2f(d[q & 1][k] * A2[n]);
          h[n] = __builtin_fmaf(e, h[n], dx[q & 1][k] * bc[q & 1].b[k][n]);
          y = __builtin_fmaf(bc[q & 1].c[k][n], h[n], y);
        }
        sy[w][q * kB + k][lane] = y;
      }
    }
    lds_barrier();
    const Args<T> again = args_again<T>();
    T* o = again->out + (p.b * again->L + c0 + w * kOwn) * again->C;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      float y = Dc * x[k];
#pragma unroll
      for (int q = 0; q < kW; ++q) y += sy[q][w * kOwn + k][lane];
      if (p.live && k < left) Store<T>::put(o, p.c, y * gate[k]);
      o += again->C;
    }
  }
  if (!p.live) return;
  T* op = a.out + p.b * a.L * a.C;
  for (int64_t t = (p.t1 > p.t0 ? p.t1 : p.t0) + w; t < p.end; t += kW) Store<T>::put(op + t * a.C, p.c, 0.0f);
  if (p.seg == a.segs - 1 && a.state_out) {
#pragma unroll
    for (int n = 0; n < NS; ++n)
      if (w * NS + n < a.N) a.state_out[(p.b * a.C + p.c) * a.N + w * NS + n] = h[n];
  }
}

// First pass over a segment: its end state from zero and its sum of d
// (kReverse false), or, from its last token back, the g that it hands to the
// segment before it, from zero behind it (kReverse true). The segment that
// hands nothing on is left out.
template <typename T, int NS, bool kReverse>
__global__ __launch_bounds__(kThreads) void scan_local_kernel(ScanP<T> a) {
  // d, and d x (forward) or grad_out silu(z) (reverse); two chunks' worth, so
  // that one barrier per chunk is enough
  constexpr int kB = Batch<NS>::kB;
  __shared__ float sd[2][kS][64], sx[2][kS][64];
  __shared__ float sum[kW][64];
  const Place<T> p = place(a, a.segs - 1, kReverse ? 1 : 0);
  const int lane = p.lane, w = p.w;
  const float bias = a.bias ? a.bias[p.c] : 0.0f;
  float A2[NS], h[NS], sum_d = 0.0f;
  load_A(a, p, A2);
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    h[n] = 0.0f;
    asm volatile("" : "+v"(A2[n]));   // loaded before the loop
  }
  const T* dp = a.dt + p.b * a.db;
  const T* xp = kReverse ? a.gy + p.b * a.gb : a.x + p.b * a.xb;
  const int64_t xr = kReverse ? a.gr : a.xr;
  const T* zp = kReverse && a.z ? a.z + p.b * a.zb : nullptr;
  const float* pack = a.pack + ((p.b * a.G + p.g) * kW + w) * a.Lp * (2 * NS);
  T rx[kOwn], rd[kOwn], rz[kOwn];
  auto fetch = [&](int64_t c0) {
    load_rows(xp, xr, c0 + w * kOwn, p.t1 - 1, p.c, rx);
    load_rows(dp, a.dr, c0 + w * kOwn, p.t1 - 1, p.c, rd);
    if (zp) load_rows(zp, a.zr, c0 + w * kOwn, p.t1 - 1, p.c, rz);
  };
  const int64_t chunks = p.t1 > p.t0 ? (p.t1 - p.t0 + kS - 1) / kS : 0;
  auto start = [&](int64_t i) { return p.t0 + (kReverse ? chunks - 1 - i : i) * kS; };
  if (chunks > 0) fetch(start(0));
  for (int64_t i = 0; i < chunks; ++i) {
    const int64_t c0 = start(i);
    const int buf = i & 1;
    const int left = static_cast<int>(p.t1 - c0 < kS ? p.t1 - c0 : kS) - w * kOwn;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const float d = k < left ? step_size(a, to_f32(rd[k]), bias) : 0.0f;
      float v = to_f32(rx[k]);
      if constexpr (kReverse) {
        if (zp) {
          const float z = to_f32(rz[k]);
          v *= z * sigmoid_f32(z);
        }
      } else {
        v *= d;
      }
      sum_d += d;
      sd[buf][w * kOwn + k][lane] = d;
      sx[buf][w * kOwn + k][lane] = k < left ? v : 0.0f;
    }
    lds_barrier();
    if (i + 1 < chunks) fetch(start(i + 1));
    Batch<NS> bc[2];
    float d[2][kB], v[2][kB];
    auto issue = [&](int q) {   // batches in the order of the walk
      const int t = kReverse ? kS - (q + 1) * kB : q * kB;
      load_batch<NS>(pack, c0 + t, bc[q & 1]);
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        d[q & 1][k] = sd[buf][t + k][lane];
        v[q & 1][k] = sx[buf][t + k][lane];
      }
    };
    issue(0);
#pragma unroll
    for (int q = 0; q < kS / kB; ++q) {
      wait_lds_scalar();
      if (q + 1 < kS / kB) issue(q + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const int k = kReverse ? kB - 1 - j : j;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const float e = __builtin_amdgcn_exp2f(d[q & 1][k] * A2[n]);
          if constexpr (kReverse) h[n] = e * __builtin_fmaf(bc[q & 1].c[k][n], v[q & 1][k], h[n]);
          else h[n] = __builtin_fmaf(e, h[n], v[q & 1][k] * bc[q & 1].b[k][n]);
        }
      }
    }
  }
  sum[w][lane] = sum_d;
  __syncthreads();
  if (!p.live) return;
  if (w == 0)
    a.sum_d[(p.b * a.segs + p.seg) * a.C + p.c] = sum[0][lane] + sum[1][lane] + sum[2][lane] + sum[3][lane];
  const int64_t at = carry_at<T, NS>(a, p, p.seg);
#pragma unroll
  for (int n = 0; n < NS; ++n) a.carry[at + n * a.C] = h[n];
  if (!kReverse && p.seg == 0 && a.state) {   // the copy of the initial state
    const int64_t to = carry_at<T, NS>(a, p, a.segs - 1);
    load_state(a, p, a.state, h);
#pragma unroll
    for (int n = 0; n < NS; ++n) a.carry[to + n * a.C] = h[n];
  }
}

// ---- few tokens: the serving step -------------------------------------------
// P lanes per channel with four states each (one 16-byte access of the state
// per lane), so that a small batch still spreads over the chip. Bound by the
// state's bytes, or by launch latency for small batches.
template <typename T, int P>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanP<T> a) {
  constexpr uint32_t per = 256 / P;
  const uint32_t ctiles = (static_cast<uint32_t>(a.C) + per - 1) / per;
  const uint32_t blk = blockIdx.x + a.block0;
  const int64_t b = blk / ctiles;
  const int q = threadIdx.x % P;
  const uint32_t c0 = (blk % ctiles) * per + threadIdx.x / P;
  const bool live = c0 < a.C;
  const int64_t c = live ? c0 : a.C - 1;
  const int64_t g = static_cast<uint32_t>(c) / static_cast<uint32_t>(a.Cg), n0 = 4 * q;
  const int64_t len = seq_len(a.lens, b, a.L);
  const int64_t si = (b * a.C + c) * a.N + n0;
  float A2[4] = {0.0f, 0.0f, 0.0f, 0.0f}, h[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool wide = a.whole;   // rows of four states are whole and aligned
  if (wide) {
    if (n0 < a.N) {
      run_ld<4>(a.A, c * a.N + n0, A2);
      if (a.state) run_ld<4>(a.state, si, h);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (n0 + k < a.N) {
        A2[k] = a.A[c * a.N + n0 + k];
        if (a.state) h[k] = a.state[si + k];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) A2[k] *= kLog2e;
  if (a.saved && live) {   // the state before token 0, padding states (zeros) included
#pragma unroll
    for (int k = 0; k < 4; ++k) a.saved[(b * 4 * P + n0 + k) * a.C + c] = h[k];
  }
  const float bias = a.bias ? a.bias[c] : 0.0f, Dc = a.D ? a.D[c] : 0.0f;
  for (int64_t t = 0; t < a.L; ++t) {
    float y = 0.0f;
    if (t < len) {
      const float x = ld1(a.x + b * a.xb + t * a.xr + c);
      const float d = step_size(a, ld1(a.dt + b * a.db + t * a.dr + c), bias);
      const float dx = d * x;
      const T* Bt = a.Bm + b * a.bb + t * a.br + g * a.bh;
      const T* Ct = a.Cm + b * a.cb + t * a.cr + g * a.ch;
      float Bv[4] = {0.0f, 0.0f, 0.0f, 0.0f}, Cv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (a.whole_bc) {
        if (n0 < a.N) {
          const auto u = V4<T>::load(Bt, n0), v = V4<T>::load(Ct, n0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            Bv[k] = V4<T>::get(u, k);
            Cv[k] = V4<T>::get(v, k);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (n0 + k < a.N) {
            Bv[k] = ld1(Bt + n0 + k);
            Cv[k] = ld1(Ct + n0 + k);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A2[k]), h[k], dx * Bv[k]);
        y = __builtin_fmaf(Cv[k], h[k], y);
      }
#pragma unroll
      for (int m = 1; m < P; m *= 2) y += __shfl_xor(y, m);
      y = __builtin_fmaf(Dc, x, y);
      if (a.z) {
        const float z = ld1(a.z + b * a.zb + t * a.zr + c);
        y *= z * sigmoid_f32(z);
      }
    }
    if (live && q == 0) Store<T>::put(a.out, (b * a.L + t) * a.C + c, y);
  }
  if (live && a.state_out && n0 < a.N) {
    if (wide) {
      run_st<4>(a.state_out, si, h);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n0 + k < a.N) a.state_out[si + k] = h[k];
    }
  }
}

// ---- backward ---------------------------------------------------------------
// Sums each of M values over the wavefront's 64 lanes by halving: while more
// than one value is left, a step joins two values into one register, each
// half of the lanes keeping one of them, so M values take about 2 M + 6
// operations instead of 6 M. Lane l ends with value wave_sum_index<M>(l).
template <int D> __device__ __forceinline__ float partner_add(float a, float b) {
  // a + the value of b in the partner lane, for partners within 16 lanes
  constexpr int ctrl = D == 8 ? 0x128 : (D == 4 ? 0x141 : (D == 2 ? 0x4e : 0xb1));   // ror 8, half mirror, quads
  return a + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(b), ctrl, 0xf, 0xf, true));
}
template <int M, int D> __device__ __forceinline__ void wave_halve(float (&v)[M], int count, int lane) {
  // `count` (a compile-time constant after unrolling) values are left
  if (count > 1) {
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
      if (i < count / 2) {
        const int k = i + count / 2;
        if constexpr (D == 32 || D == 16) {
          const auto r = D == 32 ? __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[k < M ? k : 0]), false, false)
                                 : __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[k < M ? k : 0]), false, false);
          v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        } else {
          const bool hi = lane & D;
          const float o = v[k < M ? k : 0];
          v[i] = partner_add<D>(hi ? o : v[i], hi ? v[i] : o);
        }
      }
    }
  } else if constexpr (D == 32 || D == 16) {
    const auto r = D == 32 ? __builtin_amdgcn_permlane32_swap(__float_as_uint(v[0]), __float_as_uint(v[0]), false, false)
                           : __builtin_amdgcn_permlane16_swap(__float_as_uint(v[0]), __float_as_uint(v[0]), false, false);
    v[0] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    v[0] = partner_add<D>(v[0], v[0]);
  }
}
template <int M> __device__ __forceinline__ float wave_sum(float (&v)[M], int lane) {
  static_assert(M == 2 || M == 4 || M == 8 || M == 16, "");
  wave_halve<M, 32>(v, M, lane);
  wave_halve<M, 16>(v, M / 2, lane);
  wave_halve<M, 8>(v, M / 4, lane);
  wave_halve<M, 4>(v, M / 8, lane);
  wave_halve<M, 2>(v, M / 16, lane);
  wave_halve<M, 1>(v, M / 32, lane);
  return v[0];
}
template <int M> __device__ __forceinline__ int wave_sum_index(int lane) {
  int i = 0, left = M;
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) {
    if (left > 1) {
      left /= 2;
      i += lane & d ? left : 0;
    }
  }
  return i;
}

// The backward pass of one segment, from its last token to its first, given
// g carried in from behind it, 16 tokens at a time: each wavefront prepares
// four tokens, runs its states forward from the saved ones (states and decays
// stay in registers; with eight states per wavefront the decays are computed
// again), walks back over them, and finishes four tokens.
template <typename T, int NS>
__global__ __launch_bounds__(kThreads, 2) void scan_bwd_kernel(ScanP<T> a) {
  constexpr bool kKeep = NS <= 4;    // decays kept: 16 NS registers
  __shared__ float sd[kS][64], sx[kS][64], sg[kS][64];                    // d, d x, gy
  __shared__ float sy[kW][kS][64], su[kW][kS][64], sv[kW][kS][64];        // partial y, sum g B, sum A m
  constexpr int kB = Batch<NS>::kB;
  const Place<T> p = place(a, a.segs, 0);
  const int lane = p.lane, w = p.w;
  const float bias = a.bias ? a.bias[p.c] : 0.0f, Dc = a.D ? a.D[p.c] : 0.0f;
  float A2[NS], g[NS], dA[NS], dD = 0.0f, dbias = 0.0f;
  load_A(a, p, A2);
  carried_in<T, NS, true>(a, p, A2, g);
#pragma unroll
  for (int n = 0; n < NS; ++n) dA[n] = 0.0f;
  const bool zp = a.z != nullptr;
  const float* pack = a.pack + ((p.b * a.G + p.g) * kW + w) * a.Lp * (2 * NS);
  float* part = a.partBC + (((p.b * a.G + p.g) * a.tiles + p.tile) * a.Lp * kW + w) * (2 * NS);
  // kSame lanes end a sum with the same value, so each of them keeps another
  // token's and one store writes kSame tokens
  constexpr int kSame = 32 / NS < kS ? 32 / NS : kS;
  const int slot = wave_sum_index<2 * NS>(lane), turn = lane & (32 / NS - 1);

  for (int64_t t = (p.t1 > p.t0 ? p.t1 : p.t0) + w; t < p.end; t += kW) {
    if (p.live) {
      const int64_t at = (p.b * a.L + t) * a.C + p.c;
      Store<T>::put(a.dx, at, 0.0f);
      Store<T>::put(a.ddt, at, 0.0f);
      if (zp) Store<T>::put(a.dz, at, 0.0f);
    }
  }
  // whole chunks of padding; a chunk that holds a token is written below
  for (int64_t t = p.t1 > p.t0 ? (p.t1 + kS - 1) / kS * kS : p.t0; t < p.end; ++t)
    if (lane < 2 * NS) part[t * (kW * 2 * NS) + lane] = 0.0f;

  T rx[kOwn], rd[kOwn], rz[kOwn], rg[kOwn];
  float rh[NS];
  auto fetch = [&](int64_t c0) {
    const Args<T> k = args_again<T>();
    load_rows(k->x + p.b * k->xb, k->xr, c0 + w * kOwn, p.t1 - 1, p.c, rx);
    load_rows(k->dt + p.b * k->db, k->dr, c0 + w * kOwn, p.t1 - 1, p.c, rd);
    load_rows(k->gy + p.b * k->gb, k->gr, c0 + w * kOwn, p.t1 - 1, p.c, rg);
    if (zp) load_rows(k->z + p.b * k->zb, k->zr, c0 + w * kOwn, p.t1 - 1, p.c, rz);
    const float* s = k->saved + ((p.b * k->chunks + c0 / kS) * (kW * NS) + w * NS) * k->C;
#pragma unroll
    for (int n = 0; n < NS; ++n) rh[n] = s[n * k->C + p.c];
  };
  const int64_t chunks = p.t1 > p.t0 ? (p.t1 - p.t0 + kS - 1) / kS : 0;
  if (chunks > 0) fetch(p.t0 + (chunks - 1) * kS);
  for (int64_t i = chunks - 1; i >= 0; --i) {
    const int64_t c0 = p.t0 + i * kS;
    const int left = static_cast<int>(p.t1 - c0 < kS ? p.t1 - c0 : kS) - w * kOwn;
    float x[kOwn], d[kOwn], slope[kOwn], gz[kOwn], gsl[kOwn];   // gsl: grad_out silu'(z)
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const bool in = k < left;
      const float v = to_f32(rd[k]) + bias;
      x[k] = to_f32(rx[k]);
      slope[k] = 1.0f;
      d[k] = a.softplus ? softplus_f32(v, &slope[k]) : v;
      gz[k] = to_f32(rg[k]);
      gsl[k] = 0.0f;
      if (zp) {
        const float z = to_f32(rz[k]), s = sigmoid_f32(z);
        gsl[k] = gz[k] * (s * __builtin_fmaf(z, 1.0f - s, 1.0f));
        gz[k] *= z * s;
      }
      const int r = w * kOwn + k;
      // idle lanes and tokens past the end add nothing to any sum
      const bool on = in && p.live;
      sd[r][lane] = in ? d[k] : 0.0f;
      sx[r][lane] = on ? d[k] * x[k] : 0.0f;
      sg[r][lane] = on ? gz[k] : 0.0f;
    }
    float h[kS + 1][NS], e[kKeep ? kS : 1][NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) h[0][n] = rh[n];
    lds_barrier();
    Batch<NS> bc[2];
    float bd[2][kB], bx[2][kB], bg[2][kB];
    auto issue = [&](int q, int buf) {   // batch q of the chunk's tokens
      load_batch<NS>(pack, c0 + q * kB, bc[buf]);
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        bd[buf][k] = sd[q * kB + k][lane];
        bx[buf][k] = sx[q * kB + k][lane];
        bg[buf][k] = sg[q * kB + k][lane];
      }
    };
    constexpr int kQ = kS / kB;
    issue(0, 0);
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      wait_lds_scalar();
      // after the last batch the walk back begins, with the same one
      if (q + 1 < kQ) issue(q + 1, (q + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        float y = 0.0f;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const int t = q * kB + k;
          const float f = __builtin_amdgcn_exp2f(bd[q & 1][k] * A2[n]);
          if constexpr (kKeep) e[t][n] = f;
          h[t + 1][n] = __builtin_fmaf(f, h[t][n], bx[q & 1][k] * bc[q & 1].b[k][n]);
          y = __builtin_fmaf(bc[q & 1].c[k][n], h[t + 1][n], y);
        }
        sy[w][q * kB + k][lane] = y;
      }
    }
    float held = 0.0f;
#pragma unroll
    for (int q = kQ - 1; q >= 0; --q) {
      if (q < kQ - 1) wait_lds_scalar();
      // the chunk before: late enough that half of the states are done with
      if (q == kQ / 2 - 1 && i > 0) fetch(c0 - kS);
      if (q > 0) issue(q - 1, (q - 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = kB - 1; k >= 0; --k) {
        const int t = q * kB + k;
        const float dk = bd[q & 1][k], dx = bx[q & 1][k], gk = bg[q & 1][k];
        float du = 0.0f, dd = 0.0f, v[2 * NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          g[n] = __builtin_fmaf(bc[q & 1].c[k][n], gk, g[n]);
          const float back = g[n] * (kKeep ? e[kKeep ? t : 0][n] : __builtin_amdgcn_exp2f(dk * A2[n]));
          const float m = back * h[t][n];
          du = __builtin_fmaf(g[n], bc[q & 1].b[k][n], du);
          dd = __builtin_fmaf(m, A2[n], dd);
          dA[n] = __builtin_fmaf(m, dk, dA[n]);
          v[n] = dx * g[n];
          v[NS + n] = gk * h[t + 1][n];
          g[n] = back;
        }
        su[w][t][lane] = du;
        sv[w][t][lane] = dd;
        const float sum = wave_sum<2 * NS>(v, lane);
        held = turn == t % kSame ? sum : held;
        if (t % kSame == 0 && turn < kSame) part[(c0 + t + turn) * (kW * 2 * NS) + slot] = held;
      }
    }
    lds_barrier();
    const Args<T> again = args_again<T>();
    const int64_t row = (p.b * again->L + c0 + w * kOwn) * again->C;
    T *dxp = again->dx + row, *ddtp = again->ddt + row, *dzp = again->dz + row;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int r = w * kOwn + k;
      float y = Dc * x[k], du = 0.0f, dd = 0.0f;
#pragma unroll
      for (int q = 0; q < kW; ++q) {
        y += sy[q][r][lane];
        du += su[q][r][lane];
        dd += sv[q][r][lane];
      }
      if (k < left) {
        const float ddt = __builtin_fmaf(x[k], du, dd * kLn2) * slope[k];
        dbias += ddt;
        dD = __builtin_fmaf(gz[k], x[k], dD);
        if (p.live) {
          Store<T>::put(dxp, p.c, __builtin_fmaf(Dc, gz[k], d[k] * du));
          Store<T>::put(ddtp, p.c, ddt);
          if (zp) Store<T>::put(dzp, p.c, y * gsl[k]);
        }
      }
      dxp += again->C;
      ddtp += again->C;
      dzp += again->C;
    }
  }
  __syncthreads();
  sd[w][lane] = dD;
  sx[w][lane] = dbias;
  __syncthreads();
  if (!p.live) return;
  const int64_t pi = p.b * a.segs + p.seg;
  if (w == 0) {
    a.partD[pi * a.C + p.c] = sd[0][lane] + sd[1][lane] + sd[2][lane] + sd[3][lane];
    a.partD[(a.B * a.segs + pi) * a.C + p.c] = sx[0][lane] + sx[1][lane] + sx[2][lane] + sx[3][lane];
  }
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    const int k = w * NS + n;
    if (k < a.N) {
      a.partA[(pi * a.C + p.c) * a.N + k] = dA[n];
      if (p.seg == 0 && a.dstate) a.dstate[(p.b * a.C + p.c) * a.N + k] = g[n];
    }
  }
}

// dB, dC: the channel tiles' sums added in tile order
template <typename T, int NS>
__global__ __launch_bounds__(256) void reduce_bc_kernel(ScanP<T> a, T* dB, T* dC) {
  int64_t i = (static_cast<int64_t>(a.block0) + blockIdx.x) * 256 + threadIdx.x;
  const int n = static_cast<int>(i % (kW * 2 * NS));
  i /= kW * 2 * NS;
  const int64_t t = i % a.L;
  i /= a.L;   // entry and group
  if (i >= a.B * a.G) return;
  const float* q = a.partBC + (i * a.tiles * a.Lp + t) * (kW * 2 * NS) + n;
  float s = 0.0f;
  for (int k = 0; k < a.tiles; ++k) s += q[k * a.Lp * (kW * 2 * NS)];
  const int64_t b = i / a.G, g = i - b * a.G;
  const int m = n / (2 * NS) * NS + n % NS;
  if (m < a.N) Store<T>::put(n % (2 * NS) < NS ? dB : dC, ((b * a.L + t) * a.G + g) * a.N + m, s);
}

// ---- host -------------------------------------------------------------------
// states per wavefront: 1, 2, 4 or 8
int scan_ns(int64_t N) { return N <= 4 ? 1 : (N <= 8 ? 2 : (N <= 16 ? 4 : 8)); }
int scan_np(int64_t N) { return kW * scan_ns(N); }

constexpr int64_t kMaxSegs = 64;
struct Cut {
  int64_t chunks;
  int tiles, segs, segChunks;
};
// Segments of the token axis. Cutting adds the first pass, so it pays only
// where whole-axis workgroups would leave compute units idle or unevenly
// loaded. For each number of segments the time is estimated as the workgroups
// on the fullest compute unit times a workgroup's tokens times the cycles
// that a token takes (measured on full compute units, with four states per
// wavefront: 190 forward, 127 in a first pass, 647 backward), a quarter more
// where one workgroup has a compute unit to itself, plus what every
// workgroup spends before its first token and on folding the segments before
// its own. With padded entries the work is taken to be half of the tokens
// once there are segments to leave out.
// Both sides of the choice, bf16, 16 states, 2304 channels, us cut and whole:
// 1 x 8192 forward 179, 1612; 16 x 2048 ragged forward 269, 424; 8 x 2048
// training step 985, 1459.
Cut cut_scan(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G, bool ragged, bool bwd) {
  Cut k;
  k.chunks = std::max<int64_t>(1, cdiv(L, kS));
  k.tiles = static_cast<int>(cdiv(C / G, 64));
  const int64_t groups = std::max<int64_t>(1, B * G * k.tiles);
  const double ns = scan_ns(N), full = bwd ? 125 * ns + 147 : 35 * ns + 50, first = 24 * ns + 30;
  double best = 0;
  k.segChunks = static_cast<int>(k.chunks);
  for (int64_t s = 1; s <= std::min<int64_t>(k.chunks, kMaxSegs); ++s) {
    const int64_t each = cdiv(k.chunks, s), segs = cdiv(k.chunks, each);
    const double part = ragged ? 0.5 + 0.5 / segs : 1.0;
    const double per = std::ceil(groups * segs * part / 256), per1 = std::ceil(groups * (segs - 1) * part / 256);
    const double cost = (per + 0.7) * each * kS * full + std::ceil(per / 4) * (4000.0 + 100.0 * segs) +
                        (segs > 1 ? (per1 + 0.7) * each * kS * first + std::ceil(per1 / 4) * 4000.0 + 8000.0 : 0.0);
    if (s == 1 || cost < best) {
      best = cost;
      k.segChunks = static_cast<int>(each);
    }
    if (per >= 16) break;
  }
  k.segs = static_cast<int>(cdiv(k.chunks, k.segChunks));
  return k;
}
// most segments that any call of this shape may use, for its workspace
int64_t most_segs(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G, bool bwd) {
  return std::max(cut_scan(B, L, C, N, G, false, bwd).segs, cut_scan(B, L, C, N, G, true, bwd).segs);
}

struct Space {
  size_t pack, sum_d, carry, saved, partA, partD, partBC, total;
};
Space scan_space(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G, bool bwd) {
  Space s{};
  if (!bwd && L <= kStepMax) return s;
  const Cut k = cut_scan(B, L, C, N, G, false, bwd);
  const int64_t np = scan_np(N), Lp = k.chunks * kS;
  size_t at = 0;
  auto take = [&](int64_t floats) {
    const size_t here = at;
    at += up256(static_cast<size_t>(floats) * sizeof(float));
    return here;
  };
  const int64_t fsegs = most_segs(B, L, C, N, G, false), bsegs = bwd ? most_segs(B, L, C, N, G, true) : 1;
  const int64_t segs = std::max(fsegs, bsegs);
  s.pack = take(B * G * Lp * 2 * np);
  if (segs > 1) {
    s.sum_d = take(B * segs * C);
    s.carry = take(B * segs * np * C);
  }
  if (bwd) {
    s.saved = take(B * k.chunks * np * C);   // used when the caller kept none
    s.partA = take(B * bsegs * C * N);
    s.partD = take(2 * B * bsegs * C);
    s.partBC = take(B * G * k.tiles * Lp * 2 * np);
  }
  s.total = at;
  return s;
}

template <typename T> ScanP<T> scan_params(const gspn_scan_args& a, bool bwd) {
  ScanP<T> p{};
  p.x = static_cast<const T*>(a.x.p); p.xb = a.x.batch; p.xr = a.x.row;
  p.dt = static_cast<const T*>(a.dt.p); p.db = a.dt.batch; p.dr = a.dt.row;
  p.z = static_cast<const T*>(a.z.p); p.zb = a.z.batch; p.zr = a.z.row;
  p.A = a.A; p.D = a.D; p.bias = a.dt_bias; p.state = a.state; p.lens = a.lens;
  p.Bm = static_cast<const T*>(a.Bm.p); p.bb = a.Bm.batch; p.br = a.Bm.row; p.bh = a.Bm.head;
  p.Cm = static_cast<const T*>(a.Cm.p); p.cb = a.Cm.batch; p.cr = a.Cm.row; p.ch = a.Cm.head;
  p.out = static_cast<T*>(a.out);
  p.state_out = a.state_out;
  p.saved = static_cast<float*>(a.saved);
  p.B = a.B; p.L = a.L; p.C = a.C; p.G = a.G; p.Cg = a.C / a.G;
  p.N = static_cast<int>(a.N);
  p.softplus = a.softplus;
  const Cut k = cut_scan(a.B, a.L, a.C, a.N, a.G, a.lens != nullptr, bwd);
  p.chunks = k.chunks; p.tiles = k.tiles; p.segs = k.segs; p.segChunks = k.segChunks;
  p.Lp = k.chunks * kS;
  return p;
}

float* at_bytes(void* ws, size_t off) { return reinterpret_cast<float*>(static_cast<char*>(ws) + off); }

// one kernel of the scan over a grid of workgroups of 256, in order
template <typename T, typename... A>
hipError_t launch(const char* name, void (*kern)(ScanP<T>, A...), int64_t grid, ScanP<T> p, hipStream_t stream,
                  Tracer* tr, A... more) {
  tr->before(stream, name, p.B);
  const hipError_t e = in_parts(grid, [&](int64_t first, unsigned count) {
    p.block0 = static_cast<uint32_t>(first);
    hipLaunchKernelGGL(kern, dim3(count), dim3(256), 0, stream, p, more...);
  });
  tr->after(stream);
  return e;
}

// the forward passes over whole prompts; p.saved set: states are kept
template <typename T, int NS>
hipError_t scan_passes(const ScanP<T>& p, hipStream_t stream, Tracer* tr) {
  const int64_t grid = p.B * p.segs * p.G * p.tiles;
  if (p.segs > 1) {
    const hipError_t e =
        launch("scan_local", scan_local_kernel<T, NS, false>, grid / p.segs * (p.segs - 1), p, stream, tr);
    if (e != hipSuccess) return e;
  }
  return launch("scan_fwd", scan_fwd_kernel<T, NS>, grid, p, stream, tr);
}

template <typename T, int NS> hipError_t run_pack(const ScanP<T>& p, hipStream_t stream, Tracer* tr) {
  return launch("scan_pack", pack_kernel<T, NS>, cdiv(p.B * p.G * p.Lp * kW * 2 * NS, 256), p, stream, tr);
}

template <typename T, int NS>
hipError_t scan_fwd_ns(const gspn_scan_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  ScanP<T> p = scan_params<T>(a, false);
  const Space s = scan_space(a.B, a.L, a.C, a.N, a.G, false);
  p.pack = at_bytes(ws, s.pack);
  p.sum_d = at_bytes(ws, s.sum_d);
  p.carry = at_bytes(ws, s.carry);
  const hipError_t e = run_pack<T, NS>(p, stream, tr);
  return e != hipSuccess ? e : scan_passes<T, NS>(p, stream, tr);
}

template <typename T>
hipError_t scan_fwd_dt(const gspn_scan_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.L <= kStepMax) {
    ScanP<T> p = scan_params<T>(a, false);
    p.whole = a.N % 4 == 0 && wide_ok(a.A, 16, 4, {}) && (!a.state || wide_ok(a.state, 16, 4, {})) &&
              (!a.state_out || wide_ok(a.state_out, 16, 4, {}));
    p.whole_bc = a.N % 4 == 0 &&
                 wide_ok(a.Bm.p, 4 * sizeof(T), sizeof(T), {a.Bm.batch, a.Bm.row, a.Bm.head}) &&
                 wide_ok(a.Cm.p, 4 * sizeof(T), sizeof(T), {a.Cm.batch, a.Cm.row, a.Cm.head});
    const int lanes = scan_np(a.N) / 4;
    const int64_t grid = a.B * cdiv(a.C, 256 / lanes);
    auto kern = lanes == 1 ? scan_step_kernel<T, 1> : lanes == 2 ? scan_step_kernel<T, 2>
              : lanes == 4 ? scan_step_kernel<T, 4> : scan_step_kernel<T, 8>;
    return launch("scan_step", kern, grid, p, stream, tr);
  }
  switch (scan_ns(a.N)) {
    case 1: return scan_fwd_ns<T, 1>(a, ws, stream, tr);
    case 2: return scan_fwd_ns<T, 2>(a, ws, stream, tr);
    case 4: return scan_fwd_ns<T, 4>(a, ws, stream, tr);
    default: return scan_fwd_ns<T, 8>(a, ws, stream, tr);
  }
}

template <typename T, int NS>
hipError_t scan_bwd_ns(const gspn_scan_args& a, const gspn_scan_grads& g, void* ws,
                       hipStream_t stream, Tracer* tr) {
  ScanP<T> p = scan_params<T>(a, true);
  const Space s = scan_space(a.B, a.L, a.C, a.N, a.G, true);
  p.pack = at_bytes(ws, s.pack);
  p.sum_d = at_bytes(ws, s.sum_d);
  p.carry = at_bytes(ws, s.carry);
  p.gy = static_cast<const T*>(g.grad_out.p); p.gb = g.grad_out.batch; p.gr = g.grad_out.row;
  p.gstate = g.grad_state;
  p.partA = at_bytes(ws, s.partA);
  p.partD = at_bytes(ws, s.partD);
  p.partBC = at_bytes(ws, s.partBC);
  p.dx = static_cast<T*>(g.x);
  p.ddt = static_cast<T*>(g.dt);
  p.dz = static_cast<T*>(g.z);
  p.dstate = g.state;
  const int64_t grid = p.B * p.segs * p.G * p.tiles;
  hipError_t e = hipSuccess;
  if (p.B > 0) {
    if (p.L > 0) {
      if ((e = run_pack<T, NS>(p, stream, tr)) != hipSuccess) return e;
      if (!p.saved) {
        // find the states again: the forward passes, their output into dx
        // (written again below)
        ScanP<T> f = p;
        const Cut k = cut_scan(a.B, a.L, a.C, a.N, a.G, a.lens != nullptr, false);
        f.segs = k.segs;
        f.segChunks = k.segChunks;
        f.saved = p.saved = at_bytes(ws, s.saved);
        f.out = p.dx;
        f.z = nullptr;
        f.state_out = nullptr;
        if ((e = scan_passes<T, NS>(f, stream, tr)) != hipSuccess) return e;
      }
      if (p.segs > 1) {
        e = launch("scan_local", scan_local_kernel<T, NS, true>, grid / p.segs * (p.segs - 1), p, stream, tr);
        if (e != hipSuccess) return e;
      }
    }
    if ((e = launch("scan_bwd", scan_bwd_kernel<T, NS>, grid, p, stream, tr)) != hipSuccess) return e;
    if (p.L > 0) {   // zeros where there are no channels
      e = launch("scan_reduce_bc", reduce_bc_kernel<T, NS>, cdiv(p.B * p.G * p.L * kW * 2 * NS, 256), p, stream, tr,
                 static_cast<T*>(g.Bm), static_cast<T*>(g.Cm));
      if (e != hipSuccess) return e;
    }
  }
  const int64_t rows = p.B * p.segs;
  return reduce_rows(RowSums{{p.partA, p.partD, p.partD + rows * p.C}, {g.A, g.D, g.dt_bias},
                             {p.C * p.N, p.C, p.C}, rows}, stream, tr);
}

template <typename T>
hipError_t scan_bwd_dt(const gspn_scan_args& a, const gspn_scan_grads& g, void* ws,
                       hipStream_t stream, Tracer* tr) {
  switch (scan_ns(a.N)) {
    case 1: return scan_bwd_ns<T, 1>(a, g, ws, stream, tr);
    case 2: return scan_bwd_ns<T, 2>(a, g, ws, stream, tr);
    case 4: return scan_bwd_ns<T, 4>(a, g, ws, stream, tr);
    default: return scan_bwd_ns<T, 8>(a, g, ws, stream, tr);
  }
}

}  // namespace

size_t scan_saved_bytes(int64_t B, int64_t L, int64_t C, int64_t N) {
  return static_cast<size_t>(B * std::max<int64_t>(1, cdiv(L, kS)) * scan_np(N) * C) *
         sizeof(float);
}
size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G) {
  return scan_space(B, L, C, N, G, false).total;
}
size_t scan_bwd_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G) {
  return scan_space(B, L, C, N, G, true).total;
}

hipError_t launch_scan(const gspn_scan_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return scan_fwd_dt<float>(a, ws, stream, tr);
  return scan_fwd_dt<bf16_t>(a, ws, stream, tr);
}
hipError_t launch_scan_bwd(const gspn_scan_args& a, const gspn_scan_grads& g, void* ws,
                           hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return scan_bwd_dt<float>(a, g, ws, stream, tr);
  return scan_bwd_dt<bf16_t>(a, g, ws, stream, tr);
}

}  // namespace gspn
