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
// (quarter rate), two products and two multiply-adds, against 8 bytes moved
// per token and channel. So a lane owns one channel with all its N states in
// registers, 64 adjacent channels per wavefront: the states need no exchange
// between lanes, every row of x, dt, z is one coalesced access, and B_t, C_t
// are the same for the whole wavefront. They are read by scalar loads into
// scalar registers, where they cost the vector ALU nothing, from an fp32
// copy padded to NP states (pack_kernel).
//
// Few channels do not fill the chip: the token axis is then cut into
// segments. A first pass finds each segment's state from zero and its sum of
// d (the product of its decays is exp(A sum d): one exponential), a small
// kernel carries states across segments, and the full pass starts every
// segment from its carried state.
#include "gspn_mfma.hpp"
#include "gspn_tokens.hpp"

namespace gspn {

namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(4))) f32x8* cvec8;

constexpr int kStepMax = 4;   // up to this many tokens: the single-token kernel
constexpr int kSub = 8;       // tokens loaded together; divides kScanSave

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
  float* pack;         // [B][G][L][2][NP]
  float* sum_d;        // [B][segs][C]
  float* carry;        // [B][segs][NP][C]: local results, then carried-in values
  // backward
  T *dx, *ddt, *dz;
  float* partA;        // [B * segs][NP][C]
  float* partD;        // [B * segs][C], then the same for dt_bias
  float* partBC;       // [B][G][tiles][L][2][NP]
  float* dstate;
  int64_t B, L, C, G, Cg, chunks;
  int N, tiles, segs, segChunks, softplus;
};

// ---- B and C as fp32 rows of NP states, zeros past N ------------------------
template <typename T, int NP>
__global__ __launch_bounds__(256) void pack_kernel(ScanP<T> a) {
  int64_t i = blockIdx.x * int64_t(256) + threadIdx.x;
  const int n = static_cast<int>(i % (2 * NP));
  i /= 2 * NP;
  const int64_t t = i % a.L;
  i /= a.L;
  const int64_t g = i % a.G, b = i / a.G;
  if (b >= a.B) return;
  const int k = n % NP;
  float v = 0.0f;
  if (k < a.N && t < seq_len(a.lens, b, a.L))
    v = n < NP ? ld1(a.Bm + b * a.bb + t * a.br + g * a.bh + k)
               : ld1(a.Cm + b * a.cb + t * a.cr + g * a.ch + k);
  a.pack[((b * a.G + g) * a.L + t) * (2 * NP) + n] = v;
}

template <int NP> struct BCRow {
  float b[NP], c[NP];
};
// token t's B and C, uniform over the wavefront: scalar loads
template <int NP>
__device__ __forceinline__ void load_bc(const float* pack, int64_t t, float (&b)[NP], float (&c)[NP]) {
  const cvec8 q = (cvec8)(uintptr_t)(pack + t * (2 * NP));
#pragma unroll
  for (int k = 0; k < NP / 8; ++k) {
    const f32x8 u = q[k], v = q[NP / 8 + k];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      b[8 * k + e] = u[e];
      c[8 * k + e] = v[e];
    }
  }
}

// where a wavefront works: entry b, group g, its channel, its segment
template <typename T> struct Place {
  int64_t b, g, seg, c, t0, t1, n;
  int tile;
  bool live;
};
template <typename T> __device__ __forceinline__ Place<T> place(const ScanP<T>& a) {
  Place<T> p;
  int64_t i = blockIdx.x;
  p.tile = static_cast<int>(i % a.tiles);
  i /= a.tiles;
  p.g = i % a.G;
  i /= a.G;
  p.seg = i % a.segs;
  p.b = i / a.segs;
  const int64_t k = p.tile * int64_t(64) + threadIdx.x;
  p.live = k < a.Cg;
  p.c = p.g * a.Cg + (p.live ? k : a.Cg - 1);   // idle lanes read the last channel
  p.n = seq_len(a.lens, p.b, a.L);
  p.t0 = p.seg * a.segChunks * kScanSave;
  p.t1 = p.t0 + a.segChunks * kScanSave;
  if (p.t1 > p.n) p.t1 = p.n;
  return p;
}

template <typename T> __device__ __forceinline__ float step_size(const ScanP<T>& a, float dt, float bias) {
  const float v = dt + bias;
  return a.softplus ? softplus_f32(v) : v;
}

// ---- forward ----------------------------------------------------------------
// kSummary: only the segment's end state from zero and its sum of d
template <typename T, int NP, bool kSummary>
__global__ __launch_bounds__(64) void scan_fwd_kernel(ScanP<T> a) {
  const Place<T> p = place(a);
  const float bias = a.bias ? a.bias[p.c] : 0.0f, Dc = a.D ? a.D[p.c] : 0.0f;
  float A2[NP], h[NP];
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    A2[n] = n < a.N ? a.A[p.c * a.N + n] * kLog2e : 0.0f;
    h[n] = 0.0f;
  }
  if constexpr (!kSummary) {
    if (a.segs > 1) {
#pragma unroll
      for (int n = 0; n < NP; ++n) h[n] = a.carry[((p.b * a.segs + p.seg) * NP + n) * a.C + p.c];
    } else if (a.state) {
#pragma unroll
      for (int n = 0; n < NP; ++n)
        if (n < a.N) h[n] = a.state[(p.b * a.C + p.c) * a.N + n];
    }
  }
  const T* xp = a.x + p.b * a.xb + p.c;
  const T* dp = a.dt + p.b * a.db + p.c;
  const T* zp = a.z ? a.z + p.b * a.zb + p.c : nullptr;
  const float* pack = a.pack + (p.b * a.G + p.g) * a.L * (2 * NP);
  T* op = a.out + p.b * a.L * a.C + p.c;
  float sum_d = 0.0f;

  T rx[kSub], rd[kSub], rz[kSub];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      const int64_t u = t + k < p.t1 ? t + k : p.t1 - 1;
      rx[k] = xp[u * a.xr];
      rd[k] = dp[u * a.dr];
      if (!kSummary && zp) rz[k] = zp[u * a.zr];
    }
  };
  if (p.t0 < p.t1) fetch(p.t0);
  for (int64_t t = p.t0; t < p.t1; t += kSub) {
    float x[kSub], d[kSub], z[kSub];
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      x[k] = to_f32(rx[k]);
      d[k] = to_f32(rd[k]);
      if (!kSummary && zp) z[k] = to_f32(rz[k]);
    }
    if (t + kSub < p.t1) fetch(t + kSub);
    if constexpr (!kSummary) {
      if (a.saved && t % kScanSave == 0 && p.live) {
        float* s = a.saved + (p.b * a.chunks + t / kScanSave) * NP * a.C + p.c;
#pragma unroll
        for (int n = 0; n < NP; ++n) s[n * a.C] = h[n];
      }
    }
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      if (t + k < p.t1) {
        float Bt[NP], Ct[NP];
        load_bc<NP>(pack, t + k, Bt, Ct);
        const float dk = step_size(a, d[k], bias), dx = dk * x[k];
        float y = Dc * x[k];
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          const float e = __builtin_amdgcn_exp2f(dk * A2[n]);
          h[n] = __builtin_fmaf(e, h[n], dx * Bt[n]);
          if constexpr (!kSummary) y = __builtin_fmaf(Ct[n], h[n], y);
        }
        if constexpr (kSummary) {
          sum_d += dk;
        } else {
          if (zp) y *= z[k] * sigmoid_f32(z[k]);
          if (p.live) Store<T>::put(op, (t + k) * a.C, y);
        }
      }
    }
  }
  if (!p.live) return;
  if constexpr (kSummary) {
    a.sum_d[(p.b * a.segs + p.seg) * a.C + p.c] = sum_d;
#pragma unroll
    for (int n = 0; n < NP; ++n) a.carry[((p.b * a.segs + p.seg) * NP + n) * a.C + p.c] = h[n];
  } else {
    // padding of this segment
    const int64_t end = p.seg + 1 == a.segs ? a.L : (p.seg + 1) * a.segChunks * kScanSave;
    for (int64_t t = p.t1 > p.t0 ? p.t1 : p.t0; t < end; ++t) Store<T>::put(op, t * a.C, 0.0f);
    if (a.segs == 1 && a.state_out) {
#pragma unroll
      for (int n = 0; n < NP; ++n)
        if (n < a.N) a.state_out[(p.b * a.C + p.c) * a.N + n] = h[n];
    }
  }
}

// Carries over the segments of one (entry, state): carry holds the segments'
// local results and receives the value each segment starts from. kReverse
// runs from the last segment to the first (the backward pass's g).
template <typename T, int NP, bool kReverse>
__global__ __launch_bounds__(64) void carry_kernel(ScanP<T> a, const float* from, float* to) {
  int64_t i = blockIdx.x;
  const int64_t ctiles = (a.C + 63) / 64;
  const int64_t c = (i % ctiles) * 64 + threadIdx.x;
  i /= ctiles;
  const int n = static_cast<int>(i % a.N);
  const int64_t b = i / a.N;
  if (c >= a.C) return;
  const float A2 = a.A[c * a.N + n] * kLog2e;
  float h = from ? from[(b * a.C + c) * a.N + n] : 0.0f;
  for (int k = 0; k < a.segs; ++k) {
    const int64_t s = b * a.segs + (kReverse ? a.segs - 1 - k : k);
    float* q = a.carry + (s * NP + n) * a.C + c;
    const float local = *q;
    *q = h;
    h = __builtin_fmaf(__builtin_amdgcn_exp2f(A2 * a.sum_d[s * a.C + c]), h, local);
  }
  if (to) to[(b * a.C + c) * a.N + n] = h;
}

// ---- few tokens: the serving step -------------------------------------------
// P lanes per channel with four states each (one 16-byte access of the state
// per lane), so that a small batch still spreads over the chip. Bound by the
// state's bytes, or by launch latency for small batches.
template <typename T, int P>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanP<T> a) {
  const int64_t per = 256 / P, ctiles = (a.C + per - 1) / per;
  const int64_t b = blockIdx.x / ctiles;
  const int q = threadIdx.x % P;
  const int64_t c0 = (blockIdx.x % ctiles) * per + threadIdx.x / P;
  const bool live = c0 < a.C;
  const int64_t c = live ? c0 : a.C - 1, g = c / a.Cg, n0 = 4 * q;
  const int64_t len = seq_len(a.lens, b, a.L);
  const int64_t si = (b * a.C + c) * a.N + n0;
  const bool vec = a.N % 4 == 0;   // then rows of four states are whole (and 16-byte aligned)
  float A2[4], h[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    A2[k] = n0 + k < a.N ? a.A[c * a.N + n0 + k] * kLog2e : 0.0f;
    if (a.state && !vec && n0 + k < a.N) h[k] = a.state[si + k];
  }
  const bool wide = vec && ((reinterpret_cast<uintptr_t>(a.state) | reinterpret_cast<uintptr_t>(a.state_out)) % 16 == 0);
  if (a.state && vec && n0 < a.N) {
    if (wide) {
      run_ld<4>(a.state, si, h);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = a.state[si + k];
    }
  }
  if (a.saved && live) {   // the state before token 0; the launch covers all padded states
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
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (n0 + k < a.N) {
          h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A2[k]), h[k], dx * ld1(Bt + n0 + k));
          y = __builtin_fmaf(ld1(Ct + n0 + k), h[k], y);
        }
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
// the segment's g from zero behind it, and its sum of d
template <typename T, int NP>
__global__ __launch_bounds__(64) void scan_adj_kernel(ScanP<T> a) {
  const Place<T> p = place(a);
  const float bias = a.bias ? a.bias[p.c] : 0.0f;
  float A2[NP], g[NP];
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    A2[n] = n < a.N ? a.A[p.c * a.N + n] * kLog2e : 0.0f;
    g[n] = 0.0f;
  }
  const T* dp = a.dt + p.b * a.db + p.c;
  const T* zp = a.z ? a.z + p.b * a.zb + p.c : nullptr;
  const T* gp = a.gy + p.b * a.gb + p.c;
  const float* pack = a.pack + (p.b * a.G + p.g) * a.L * (2 * NP);
  float sum_d = 0.0f;
  T rd[kSub], rz[kSub], rg[kSub];
  auto fetch = [&](int64_t t) {   // tokens t, t - 1, ...
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      const int64_t u = t - k > p.t0 ? t - k : p.t0;
      rd[k] = dp[u * a.dr];
      rg[k] = gp[u * a.gr];
      if (zp) rz[k] = zp[u * a.zr];
    }
  };
  if (p.t0 < p.t1) fetch(p.t1 - 1);
  for (int64_t t = p.t1 - 1; t >= p.t0; t -= kSub) {
    float d[kSub], z[kSub], gy[kSub];
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      d[k] = to_f32(rd[k]);
      gy[k] = to_f32(rg[k]);
      if (zp) z[k] = to_f32(rz[k]);
    }
    if (t - kSub >= p.t0) fetch(t - kSub);
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      if (t - k >= p.t0) {
        float Bt[NP], Ct[NP];
        load_bc<NP>(pack, t - k, Bt, Ct);
        const float dk = step_size(a, d[k], bias);
        const float gz = zp ? gy[k] * (z[k] * sigmoid_f32(z[k])) : gy[k];
        sum_d += dk;
#pragma unroll
        for (int n = 0; n < NP; ++n)
          g[n] = __builtin_amdgcn_exp2f(dk * A2[n]) * __builtin_fmaf(Ct[n], gz, g[n]);
      }
    }
  }
  if (!p.live) return;
  a.sum_d[(p.b * a.segs + p.seg) * a.C + p.c] = sum_d;
#pragma unroll
  for (int n = 0; n < NP; ++n) a.carry[((p.b * a.segs + p.seg) * NP + n) * a.C + p.c] = g[n];
}

// Sums each of M values over the wavefront's 64 lanes by halving: a step
// joins two values into one register, each half of the lanes keeping one of
// them, so M values take about 2 M operations instead of 6 M. Lane l ends
// with value wave_sum_index<M>(l).
__device__ __forceinline__ float dpp_add(float a, float b, int which) {
  // a + the value of b in the partner lane
  int m;
  switch (which) {
    case 8: m = __builtin_amdgcn_update_dpp(0, __float_as_int(b), 0x128, 0xf, 0xf, true); break;   // row_ror:8
    case 4: m = __builtin_amdgcn_update_dpp(0, __float_as_int(b), 0x141, 0xf, 0xf, true); break;   // half mirror
    case 2: m = __builtin_amdgcn_update_dpp(0, __float_as_int(b), 0x4e, 0xf, 0xf, true); break;    // quad 2 3 0 1
    default: m = __builtin_amdgcn_update_dpp(0, __float_as_int(b), 0xb1, 0xf, 0xf, true); break;   // quad 1 0 3 2
  }
  return a + __int_as_float(m);
}
template <int M> __device__ __forceinline__ float wave_sum(float (&v)[M], int lane) {
  static_assert(M == 16 || M == 32 || M == 64, "");
#pragma unroll
  for (int i = 0; i < M / 2; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + M / 2]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int i = 0; i < M / 4; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + M / 4]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int i = 0; i < M / 8; ++i) {
    const bool hi = lane & 8;
    v[i] = dpp_add(hi ? v[i + M / 8] : v[i], hi ? v[i] : v[i + M / 8], 8);
  }
#pragma unroll
  for (int i = 0; i < M / 16; ++i) {
    const bool hi = lane & 4;
    v[i] = dpp_add(hi ? v[i + M / 16] : v[i], hi ? v[i] : v[i + M / 16], 4);
  }
  if constexpr (M >= 32) {
#pragma unroll
    for (int i = 0; i < M / 32; ++i) {
      const bool hi = lane & 2;
      v[i] = dpp_add(hi ? v[i + M / 32] : v[i], hi ? v[i] : v[i + M / 32], 2);
    }
  } else {
    v[0] = dpp_add(v[0], v[0], 2);
  }
  if constexpr (M >= 64) {
    const bool hi = lane & 1;
    v[0] = dpp_add(hi ? v[1] : v[0], hi ? v[0] : v[1], 1);
  } else {
    v[0] = dpp_add(v[0], v[0], 1);
  }
  return v[0];
}
template <int M> __device__ __forceinline__ int wave_sum_index(int lane) {
  int i = (lane & 32 ? M / 2 : 0) + (lane & 16 ? M / 4 : 0) + (lane & 8 ? M / 8 : 0) +
          (lane & 4 ? M / 16 : 0);
  if (M >= 32) i += lane & 2 ? M / 32 : 0;
  if (M >= 64) i += lane & 1;
  return i;
}

// The backward pass of one segment, from its last token to its first, given
// g carried in from behind it. Chunks of kScanSave tokens start from their
// saved state: a walk forward leaves the state before each block of TS
// tokens in LDS, then the blocks are taken in reverse, each recomputing its
// states into registers before walking back over them.
template <typename T, int NP, int TS>
__global__ __launch_bounds__(64) void scan_bwd_kernel(ScanP<T> a) {
  constexpr int kBlocks = kScanSave / TS;
  __shared__ float mid[kBlocks - 1][NP][64];
  const Place<T> p = place(a);
  const int lane = threadIdx.x;
  const float bias = a.bias ? a.bias[p.c] : 0.0f, Dc = a.D ? a.D[p.c] : 0.0f;
  float A2[NP], g[NP], dA[NP], dD = 0.0f, dbias = 0.0f;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    A2[n] = n < a.N ? a.A[p.c * a.N + n] * kLog2e : 0.0f;
    dA[n] = 0.0f;
    g[n] = 0.0f;
  }
  if (a.segs > 1) {
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (n < a.N) g[n] = a.carry[((p.b * a.segs + p.seg) * NP + n) * a.C + p.c];
  } else if (a.gstate) {
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (n < a.N) g[n] = a.gstate[(p.b * a.C + p.c) * a.N + n];
  }
  const T* xp = a.x + p.b * a.xb + p.c;
  const T* dp = a.dt + p.b * a.db + p.c;
  const T* zp = a.z ? a.z + p.b * a.zb + p.c : nullptr;
  const T* gp = a.gy + p.b * a.gb + p.c;
  const int64_t row0 = p.b * a.L * a.C + p.c;
  const float* pack = a.pack + (p.b * a.G + p.g) * a.L * (2 * NP);
  float* part = a.partBC + ((p.b * a.G + p.g) * a.tiles + p.tile) * a.L * (2 * NP);
  const int slot = wave_sum_index<2 * NP>(lane);
  const bool writer = (lane & (NP == 8 ? 3 : NP == 16 ? 1 : 0)) == 0;

  // padding of this segment
  {
    const int64_t end = p.seg + 1 == a.segs ? a.L : (p.seg + 1) * a.segChunks * kScanSave;
    for (int64_t t = p.t1 > p.t0 ? p.t1 : p.t0; t < end; ++t) {
      if (p.live) {
        Store<T>::put(a.dx, row0 + t * a.C, 0.0f);
        Store<T>::put(a.ddt, row0 + t * a.C, 0.0f);
        if (a.dz) Store<T>::put(a.dz, row0 + t * a.C, 0.0f);
      }
      if (lane < 2 * NP) part[t * (2 * NP) + lane] = 0.0f;
    }
  }

  const int64_t last = p.t1 > p.t0 ? (p.t1 - 1) / kScanSave : -1, first = p.t0 / kScanSave;
  for (int64_t ck = last; ck >= first; --ck) {
    const int64_t c0 = ck * kScanSave, c1 = c0 + kScanSave < p.t1 ? c0 + kScanSave : p.t1;
    const int nb = static_cast<int>((c1 - c0 + TS - 1) / TS);   // blocks of this chunk
    float h0[NP];
    {
      const float* s = a.saved + (p.b * a.chunks + ck) * NP * a.C + p.c;
#pragma unroll
      for (int n = 0; n < NP; ++n) h0[n] = s[n * a.C];
    }
    for (int blk = 0; blk + 1 < nb; ++blk) {
      const int64_t t = c0 + blk * TS;
#pragma unroll
      for (int n = 0; n < NP; ++n) mid[blk][n][lane] = h0[n];
      float x[TS], d[TS];
#pragma unroll
      for (int k = 0; k < TS; ++k) {
        x[k] = to_f32(xp[(t + k) * a.xr]);
        d[k] = to_f32(dp[(t + k) * a.dr]);
      }
#pragma unroll
      for (int k = 0; k < TS; ++k) {
        float Bt[NP], Ct[NP];
        load_bc<NP>(pack, t + k, Bt, Ct);
        const float dk = step_size(a, d[k], bias), dx = dk * x[k];
#pragma unroll
        for (int n = 0; n < NP; ++n)
          h0[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(dk * A2[n]), h0[n], dx * Bt[n]);
      }
    }
    for (int blk = nb - 1; blk >= 0; --blk) {
      const int64_t t = c0 + blk * TS;
      if (blk + 1 < nb) {
#pragma unroll
        for (int n = 0; n < NP; ++n) h0[n] = mid[blk][n][lane];
      }
      float x[TS], raw[TS], d[TS], z[TS], gy[TS], y[TS], h[TS + 1][NP];
#pragma unroll
      for (int k = 0; k < TS; ++k) {
        const int64_t u = t + k < c1 ? t + k : c1 - 1;
        x[k] = to_f32(xp[u * a.xr]);
        raw[k] = to_f32(dp[u * a.dr]) + bias;
        gy[k] = to_f32(gp[u * a.gr]);
        z[k] = zp ? to_f32(zp[u * a.zr]) : 0.0f;
        y[k] = Dc * x[k];
      }
#pragma unroll
      for (int n = 0; n < NP; ++n) h[0][n] = h0[n];
#pragma unroll
      for (int k = 0; k < TS; ++k) {
        d[k] = a.softplus ? softplus_f32(raw[k]) : raw[k];
        if (t + k < c1) {
          float Bt[NP], Ct[NP];
          load_bc<NP>(pack, t + k, Bt, Ct);
          const float dx = d[k] * x[k];
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            h[k + 1][n] = __builtin_fmaf(__builtin_amdgcn_exp2f(d[k] * A2[n]), h[k][n], dx * Bt[n]);
            y[k] = __builtin_fmaf(Ct[n], h[k + 1][n], y[k]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NP; ++n) h[k + 1][n] = h[k][n];
        }
      }
#pragma unroll
      for (int k = TS - 1; k >= 0; --k) {
        if (t + k < c1) {
          float Bt[NP], Ct[NP];
          load_bc<NP>(pack, t + k, Bt, Ct);
          float gz = gy[k];
          if (zp) {
            const float sg = sigmoid_f32(z[k]);
            gz = gy[k] * (z[k] * sg);
            if (p.live)
              Store<T>::put(a.dz, row0 + (t + k) * a.C,
                            gy[k] * y[k] * (sg * __builtin_fmaf(z[k], 1.0f - sg, 1.0f)));
          }
          const float dx = d[k] * x[k];
          float du = 0.0f, dd = 0.0f, bc[2 * NP];
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            g[n] = __builtin_fmaf(Ct[n], gz, g[n]);
            const float back = g[n] * __builtin_amdgcn_exp2f(d[k] * A2[n]);
            const float m = back * h[k][n];
            du = __builtin_fmaf(g[n], Bt[n], du);
            dd = __builtin_fmaf(m, A2[n], dd);
            dA[n] = __builtin_fmaf(m, d[k], dA[n]);
            bc[n] = p.live ? dx * g[n] : 0.0f;
            bc[NP + n] = p.live ? gz * h[k + 1][n] : 0.0f;
            g[n] = back;
          }
          float ddt = __builtin_fmaf(x[k], du, dd * kLn2);
          if (a.softplus) ddt *= sigmoid_f32(raw[k]);
          dbias += ddt;
          dD = __builtin_fmaf(gz, x[k], dD);
          if (p.live) {
            Store<T>::put(a.dx, row0 + (t + k) * a.C, __builtin_fmaf(Dc, gz, d[k] * du));
            Store<T>::put(a.ddt, row0 + (t + k) * a.C, ddt);
          }
          const float s = wave_sum<2 * NP>(bc, lane);
          if (writer) part[(t + k) * (2 * NP) + slot] = s;
        }
      }
    }
  }
  if (!p.live) return;
  const int64_t pi = p.b * a.segs + p.seg;
#pragma unroll
  for (int n = 0; n < NP; ++n)
    if (n < a.N) a.partA[(pi * a.C + p.c) * a.N + n] = dA[n];
  a.partD[pi * a.C + p.c] = dD;
  a.partD[(a.B * a.segs + pi) * a.C + p.c] = dbias;
  if (a.segs == 1 && a.dstate) {
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (n < a.N) a.dstate[(p.b * a.C + p.c) * a.N + n] = g[n];
  }
}

// dB, dC: the channel tiles' sums added in tile order
template <typename T, int NP>
__global__ __launch_bounds__(256) void reduce_bc_kernel(ScanP<T> a, T* dB, T* dC) {
  int64_t i = blockIdx.x * int64_t(256) + threadIdx.x;
  const int n = static_cast<int>(i % (2 * NP));
  i /= 2 * NP;
  const int64_t t = i % a.L;
  i /= a.L;   // entry and group
  if (i >= a.B * a.G) return;
  const float* q = a.partBC + (i * a.tiles * a.L + t) * (2 * NP) + n;
  float s = 0.0f;
  for (int k = 0; k < a.tiles; ++k) s += q[k * a.L * (2 * NP)];
  const int64_t b = i / a.G, g = i - b * a.G;
  const int m = n % NP;
  if (m < a.N) Store<T>::put(n < NP ? dB : dC, ((b * a.L + t) * a.G + g) * a.N + m, s);
}

// ---- host -------------------------------------------------------------------
int scan_np(int64_t N) { return N <= 8 ? 8 : (N <= 16 ? 16 : 32); }

struct Cut {
  int64_t chunks;
  int tiles, segs, segChunks;
};
// Segments of the token axis. Cutting doubles the work (the first pass), so
// it pays when the whole-axis wavefronts would leave more than half of the
// chip's 4 SIMDs per compute unit idle; then as many segments as give two
// wavefronts per SIMD, of at least one chunk.
Cut cut_scan(int64_t B, int64_t L, int64_t C, int64_t G) {
  Cut k;
  k.chunks = std::max<int64_t>(1, cdiv(L, kScanSave));
  k.tiles = static_cast<int>(cdiv(C / G, 64));
  const int64_t waves = std::max<int64_t>(1, B * G * k.tiles), simds = 1024;
  k.segChunks = static_cast<int>(k.chunks);
  if (waves < simds / 2) {
    const int64_t want = std::min<int64_t>(k.chunks, cdiv(2 * simds, waves));
    k.segChunks = static_cast<int>(cdiv(k.chunks, want));
  }
  k.segs = static_cast<int>(cdiv(k.chunks, k.segChunks));
  return k;
}

struct Space {
  size_t pack, sum_d, carry, saved, partA, partD, partBC, total;
};
Space scan_space(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G, bool bwd) {
  Space s{};
  if (!bwd && L <= kStepMax) return s;
  const Cut k = cut_scan(B, L, C, G);
  const int64_t np = scan_np(N);
  size_t at = 0;
  auto take = [&](int64_t floats) {
    const size_t here = at;
    at += up256(static_cast<size_t>(floats) * sizeof(float));
    return here;
  };
  s.pack = take(B * G * L * 2 * np);
  if (k.segs > 1) {
    s.sum_d = take(B * k.segs * C);
    s.carry = take(B * k.segs * np * C);
  }
  if (bwd) {
    s.saved = take(B * k.chunks * np * C);   // used when the caller kept none
    s.partA = take(B * k.segs * C * N);
    s.partD = take(2 * B * k.segs * C);
    s.partBC = take(B * G * k.tiles * L * 2 * np);
  }
  s.total = at;
  return s;
}

template <typename T> ScanP<T> scan_params(const gspn_scan_args& a) {
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
  const Cut k = cut_scan(a.B, a.L, a.C, a.G);
  p.chunks = k.chunks; p.tiles = k.tiles; p.segs = k.segs; p.segChunks = k.segChunks;
  return p;
}

float* at_bytes(void* ws, size_t off) { return reinterpret_cast<float*>(static_cast<char*>(ws) + off); }

#define GSPN_LAUNCH(name, units, kern, grid, block, ...)                                     \
  do {                                                                                       \
    tr->before(stream, name, units);                                                         \
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(block), 0, stream,      \
                       __VA_ARGS__);                                                         \
    tr->after(stream);                                                                       \
    const hipError_t e_ = hipGetLastError();                                                 \
    if (e_ != hipSuccess) return e_;                                                         \
  } while (0)

// the forward passes over whole prompts; p.saved set: states are kept
template <typename T, int NP>
hipError_t scan_passes(const ScanP<T>& p, hipStream_t stream, Tracer* tr) {
  const int64_t grid = p.B * p.segs * p.G * p.tiles;
  if (p.segs > 1) {
    GSPN_LAUNCH("scan_summary", p.B, (scan_fwd_kernel<T, NP, true>), grid, 64, p);
    GSPN_LAUNCH("scan_carry", p.B, (carry_kernel<T, NP, false>), p.B * p.N * cdiv(p.C, 64), 64, p,
                p.state, p.state_out);
  }
  GSPN_LAUNCH("scan_fwd", p.B, (scan_fwd_kernel<T, NP, false>), grid, 64, p);
  return hipSuccess;
}

template <typename T, int NP>
hipError_t scan_fwd_np(const gspn_scan_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  ScanP<T> p = scan_params<T>(a);
  const Space s = scan_space(a.B, a.L, a.C, a.N, a.G, false);
  p.pack = at_bytes(ws, s.pack);
  p.sum_d = at_bytes(ws, s.sum_d);
  p.carry = at_bytes(ws, s.carry);
  GSPN_LAUNCH("scan_pack", p.B, (pack_kernel<T, NP>), cdiv(p.B * p.G * p.L * 2 * NP, 256), 256, p);
  return scan_passes<T, NP>(p, stream, tr);
}

template <typename T>
hipError_t scan_fwd_dt(const gspn_scan_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.L <= kStepMax) {
    const ScanP<T> p = scan_params<T>(a);
    const int lanes = a.N <= 4 && !a.saved ? 1 : scan_np(a.N) / 4;
    const int64_t grid = a.B * cdiv(a.C, 256 / lanes);
    switch (lanes) {
      case 1: GSPN_LAUNCH("scan_step", a.B, (scan_step_kernel<T, 1>), grid, 256, p); break;
      case 2: GSPN_LAUNCH("scan_step", a.B, (scan_step_kernel<T, 2>), grid, 256, p); break;
      case 4: GSPN_LAUNCH("scan_step", a.B, (scan_step_kernel<T, 4>), grid, 256, p); break;
      default: GSPN_LAUNCH("scan_step", a.B, (scan_step_kernel<T, 8>), grid, 256, p); break;
    }
    return hipSuccess;
  }
  switch (scan_np(a.N)) {
    case 8: return scan_fwd_np<T, 8>(a, ws, stream, tr);
    case 16: return scan_fwd_np<T, 16>(a, ws, stream, tr);
    default: return scan_fwd_np<T, 32>(a, ws, stream, tr);
  }
}

template <typename T, int NP>
hipError_t scan_bwd_np(const gspn_scan_args& a, const gspn_scan_grads& g, void* ws,
                       hipStream_t stream, Tracer* tr) {
  ScanP<T> p = scan_params<T>(a);
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
  const bool any = p.B > 0 && p.L > 0;
  const int64_t grid = p.B * p.segs * p.G * p.tiles;
  if (any) {
    GSPN_LAUNCH("scan_pack", p.B, (pack_kernel<T, NP>), cdiv(p.B * p.G * p.L * 2 * NP, 256), 256, p);
    if (!p.saved) {
      // find the states again: the forward passes, their output into dx
      // (written again below)
      ScanP<T> f = p;
      f.saved = p.saved = at_bytes(ws, s.saved);
      f.out = p.dx;
      f.z = nullptr;
      f.state_out = nullptr;
      const hipError_t e = scan_passes<T, NP>(f, stream, tr);
      if (e != hipSuccess) return e;
    }
    if (p.segs > 1) {
      GSPN_LAUNCH("scan_adjoint", p.B, (scan_adj_kernel<T, NP>), grid, 64, p);
      GSPN_LAUNCH("scan_carry", p.B, (carry_kernel<T, NP, true>), p.B * p.N * cdiv(p.C, 64), 64, p,
                  p.gstate, p.dstate);
    }
  }
  if (p.B > 0)
    GSPN_LAUNCH("scan_bwd", p.B, (scan_bwd_kernel<T, NP, NP == 32 ? 4 : 8>), grid, 64, p);
  if (any)
    GSPN_LAUNCH("scan_reduce_bc", p.B, (reduce_bc_kernel<T, NP>),
                cdiv(p.B * p.G * p.L * 2 * NP, 256), 256, p, static_cast<T*>(g.Bm),
                static_cast<T*>(g.Cm));
  const int64_t rows = p.B * p.segs;
  hipError_t e = reduce_rows<float>(p.partA, rows, p.C * p.N, g.A, stream, tr);
  if (e == hipSuccess && g.D) e = reduce_rows<float>(p.partD, rows, p.C, g.D, stream, tr);
  if (e == hipSuccess && g.dt_bias)
    e = reduce_rows<float>(p.partD + rows * p.C, rows, p.C, g.dt_bias, stream, tr);
  return e;
}

template <typename T>
hipError_t scan_bwd_dt(const gspn_scan_args& a, const gspn_scan_grads& g, void* ws,
                       hipStream_t stream, Tracer* tr) {
  switch (scan_np(a.N)) {
    case 8: return scan_bwd_np<T, 8>(a, g, ws, stream, tr);
    case 16: return scan_bwd_np<T, 16>(a, g, ws, stream, tr);
    default: return scan_bwd_np<T, 32>(a, g, ws, stream, tr);
  }
}

}  // namespace

size_t scan_saved_bytes(int64_t B, int64_t L, int64_t C, int64_t N) {
  return static_cast<size_t>(B * std::max<int64_t>(1, cdiv(L, kScanSave)) * scan_np(N) * C) *
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
