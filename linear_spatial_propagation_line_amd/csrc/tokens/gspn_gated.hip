// Gated linear recurrence over tokens, forward and backward.
//
//   s = sigmoid(r),  log a = A s,  u = sigmoid(i) x,  beta = sqrt(1 - a^2),
//   h_t = a_t h_{t-1} + beta_t u_t,  out = h
// and from the end, with g_t = dL/dh_t = grad_out_t + a_{t+1} g_{t+1},
//   k = dL/dlog a = g (a h_{t-1} - (a^2 / beta) u),
//   dr = k A s (1 - s),  dA = sum k s,
//   dx = g beta sigmoid(i),  di = g beta x sigmoid(i) (1 - sigmoid(i)).
//
// a and e = a - 1 each have their own digits: 1 - a^2 = -e (2 + e) where a is close to
// 1, and products of small a, which e has lost (1 + e is off by 2^-25 whatever a is: by
// 17 % at exp(-16)). What hangs on a times a state, the gradients of r, A and the
// state among it, keeps them at every A <= 0.
//
// Bound by memory, with five or six transcendentals a value close behind
// (four values moved forward, eight backward): so each value is read once and
// its gates are computed once. A workgroup owns a chunk of tokens of
// 64 V channels and keeps it in registers; its wavefronts own runs of tokens.
// A chunk's effect on the state is h -> P h + H. Chunks of a chain (the chunks
// of one entry's channels) hand the state on through memory: each publishes
// (P, H) as soon as it has them, and the state behind it when it knows the
// one before. A chunk waits until some chunk of the kWindow before it has
// published its state and all between have published (P, H), and folds
// forward from there, which gives the same bits whichever it was.
//
// Every wait ends: a workgroup takes the next chunk of its chain from a
// counter, so all that it waits for were taken before by workgroups that
// are running, the first of which waits for nothing. What is handed on is one
// word that cannot be torn (4 or 8 bytes, written and read by relaxed
// device-scope atomics) and says itself whether it is there: the workspace is
// filled with a pattern that no published value has.
//
// 8 x 2048 x 2304 bf16: forward 72 us (4.2 TB/s), backward 131 to 137 (3.9 TB/s); one entry of
// 32768 tokens forward 139 (4.3 TB/s). A large copy: 5.1 TB/s.
#include "gspn_mfma.hpp"
#include "gspn_tokens.hpp"

namespace gspn {

namespace {

constexpr int kChunkF = 128;   // tokens of a chunk, forward (32768 x 2304 143 us, with 64 157)
constexpr int kChunkB = 64;    // backward: also what the saved states are apart
constexpr int kWindow = 4;     // chunks that one looks back
constexpr int kRunF = 16;      // tokens of a wavefront's run, forward
constexpr int kRunB = 8;       // backward, which keeps twice the values of a token

// Up to how many tokens a lane walks all of them, by the number of lanes (of V channels):
// chunks cost by the rounds in which their workgroups run, a walk by its length. us by
// lanes and by chunks, bf16, pairs: 1152 lanes 12 tokens 6.0 and 6.3, 16 7.2 and 6.4;
// 73728 lanes 28 tokens 16.9 and 17.4, 32 18.7 and 17.2; 92160 lanes 32 tokens 18.9 and 20.1,
// 48 26.6 and 22.2; 589824 lanes 32 tokens 67 and 102. Single channels, whose chunks hold half as
// much: 80080 lanes 24 tokens 10.8 and 11.5, 28 13.4 and 12.4; 96096 28 tokens 14.8 and 14.6, 32 16.6
// and 15.5 (the worse of both, by 7 %); 128128 32 tokens 17.2 and 18.2, 48 24.2 and 20.8.
template <int V> constexpr int64_t short_tokens(int64_t lanes) {
  return lanes < 65536 ? 12 : (lanes < 90112 ? 20 + 4 * V : 32);
}
constexpr uint32_t kAbsent = 0xffffffffu;

template <typename T> struct GatedP {
  const T* x; int64_t xb, xr;
  const T* r; int64_t rb, rr;
  const T* i; int64_t ib, ir;
  const T* gy; int64_t gb, gr;
  const float* A; const float* state; const int32_t* lens;
  T* out; float* state_out; float* saved;
  T* dx; T* dr; T* di; float* dstate; const float* gstate; float* part;
  uint64_t* total;     // [chains][chunks][64 V]: P (low word) and H of a chunk
  uint32_t* behind;    // [chains][chunks][64 V]: the state behind a chunk
  uint32_t* counter;   // [chains], 16 words apart
  int64_t L, C, B;
  int64_t chunks, ctiles;
  int64_t saves;   // saved states of an entry
  int64_t block0;
};

// 1 / (1 + exp(-v)); the exponential may be infinite, the result is then 0
__device__ __forceinline__ float gate_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
}
// The same and 1 - it, each to its own digits; the exponential is kept finite, so
// far below zero the gate is 2^-126.
__device__ __forceinline__ void gate_both(float v, float& open, float& shut) {
  const float t = __builtin_amdgcn_exp2f(fminf(v * -kLog2e, 126.0f));
  open = __builtin_amdgcn_rcpf(1.0f + t);
  shut = t * open;
}
// a = exp(v) and e = a - 1, v <= 0
struct Decay {
  float a, e;
};
__device__ __forceinline__ Decay decay_f32(float v) {
  const float x = __builtin_amdgcn_exp2f(v * kLog2e), p = expm1_series(v);
  const bool near = fabsf(v) < kExpm1Series;
  return Decay{near ? 1.0f + p : x, near ? p : x - 1.0f};
}
// Both in one word: a, or -|e| where a is above exp(-1/4); a sign says which
__device__ __forceinline__ float decay_word(const Decay& d) { return d.a > 0.75f ? copysignf(d.e, -1.0f) : d.a; }
__device__ __forceinline__ Decay word_decay(float w) {
  const float one = __int_as_float((__float_as_int(w) >> 31) & 0x3f800000);
  return Decay{w + one, w + (one - 1.0f)};
}
// What was derived from the words so far is not kept in registers but derived again
// (kept, the backward pass in bf16 takes 128 and spills 19; this way 120, and 8 x 2048 x
// 2304 135 us; with 1 + e, six spilled, 143)
template <int N, int V> __device__ __forceinline__ void forget(float (&w)[N][V]) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) asm("" : "+v"(w[k][v]));
}
// 1 - a^2 from e = a - 1 <= 0
__device__ __forceinline__ float left_f32(float e) { return -e * (2.0f + e); }

// N rows of a [L, C] tensor's tile from row t on, clamped to the last of n > 0:
// the row's address is uniform, the lane's place in it `off` bytes
template <int N, typename T, int V>
__device__ __forceinline__ void load_rows(const T* tile, int64_t stride, int64_t t, int64_t n, uint32_t off,
                                          Raw<T, V> (&r)[N]) {
  const char* p = reinterpret_cast<const char*>(tile + t * stride);
  const int64_t step = stride * static_cast<int64_t>(sizeof(T));
  if (t + N <= n) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      r[k].load(reinterpret_cast<const T*>(p + off));
      p += step;
    }
  } else {
    const int some = static_cast<int>(n - t);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      r[k].load(reinterpret_cast<const T*>(p + off));
      if (k + 1 < some) p += step;
    }
  }
}
template <int V, typename T> __device__ __forceinline__ void put_row(T* row, uint32_t off, const float (&y)[V]) {
  stream_stv<V>(reinterpret_cast<T*>(reinterpret_cast<char*>(row) + off), y);
}

// zeros in `rows` rows of V values
template <int V, typename T> __device__ __forceinline__ void zero_rows(T* p, int64_t stride, int rows, uint32_t off) {
  const float zero[V] = {};
  for (int k = 0; k < rows; ++k) put_row<V>(p + k * stride, off, zero);
}

// the published forms
__device__ __forceinline__ uint32_t present(float v) {
  const uint32_t w = __float_as_uint(v);
  return w == kAbsent ? 0x7fc00000u : w;   // that NaN as another
}
__device__ __forceinline__ void publish_total(uint64_t* p, float P, float H) {
  __hip_atomic_store(p, static_cast<uint64_t>(__float_as_uint(H)) << 32 | present(P), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(uint32_t* p, float h) {
  __hip_atomic_store(p, present(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The value before place q >= 1 of a chain; place k of it lies at
// [k * stride]. Folds forward from the latest published state within the
// window; comes back when there is one. The place before is asked first, and
// alone: where there are many chains it is mostly there, and asking costs more than
// the answer (8 x 2048 x 2304, backward, when measured: 144 us; a window
// of 4 at once 150, of 8 160, of 16 186).
__device__ __forceinline__ float look_back(const uint64_t* total, const uint32_t* behind, int64_t q, int64_t stride) {
  const uint32_t last = __hip_atomic_load(behind + (q - 1) * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (last != kAbsent) return __uint_as_float(last);
  for (;;) {
    uint64_t t[kWindow];
    uint32_t s[kWindow];
#pragma unroll
    for (int k = 0; k < kWindow; ++k) {
      const int64_t at = (q - 1 - k >= 0 ? q - 1 - k : 0) * stride;
      s[k] = __hip_atomic_load(behind + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      t[k] = __hip_atomic_load(total + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    bool have = false;
    float h = 0.0f;
#pragma unroll
    for (int k = kWindow - 1; k >= 0; --k) {
      const bool there = k < q && s[k] != kAbsent;
      const bool step = have && static_cast<uint32_t>(t[k]) != kAbsent;
      const float next = __builtin_fmaf(__uint_as_float(static_cast<uint32_t>(t[k])), h,
                                        __uint_as_float(static_cast<uint32_t>(t[k] >> 32)));
      h = there ? __uint_as_float(s[k]) : next;
      have = there || step;
    }
    if (have) return h;
    __builtin_amdgcn_s_sleep(2);
  }
}

// A workgroup's chunk. Chains are dealt out by the workgroup's number, their
// chunks in the order in which workgroups ask.
struct Place {
  int64_t b, ct, q, chain;
};
template <typename P> __device__ __forceinline__ Place take_place(const P& a, uint32_t* slot) {
  const int64_t chains = a.B * a.ctiles, g = a.block0 + blockIdx.x;
  Place p;
  p.chain = g % chains;
  p.q = 0;
  if (a.chunks > 1) {
    if (threadIdx.x == 0) *slot = atomicAdd(a.counter + p.chain * 16, 1u);
    __syncthreads();
    p.q = __builtin_amdgcn_readfirstlane(*slot);
  }
  p.b = p.chain / a.ctiles;
  p.ct = p.chain - p.b * a.ctiles;
  return p;
}

template <typename T, int V>
__global__ __launch_bounds__(64 * kChunkF / kRunF, 4) void gated_kernel(GatedP<T> a) {
  constexpr int kWaves = kChunkF / kRunF;
  __shared__ uint32_t slot;
  __shared__ float sp[kWaves][64 * V], sh[kWaves][64 * V], before[64 * V];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = take_place(a, &slot);
  const int64_t n = seq_len(a.lens, at.b, a.L), t0 = at.q * kChunkF + wave * kRunF;
  const int64_t c0 = at.ct * 64 * V, c = c0 + lane * V;
  const bool mine = c < a.C;
  const uint32_t place = mine ? lane * V : 0, off = place * sizeof(T);   // lanes past the channels read the first
  const int rows = static_cast<int>(a.L - t0 < 0 ? 0 : (a.L - t0 < kRunF ? a.L - t0 : kRunF));
  const int live = static_cast<int>(n - t0 < 0 ? 0 : (n - t0 < kRunF ? n - t0 : kRunF));
  T* o = a.out + (at.b * a.L + t0) * a.C + c0;
  // a chunk of padding has nothing to hand on: those behind it are padding too
  if (at.q * kChunkF >= n && at.q > 0) {
    if (a.out && mine) zero_rows<V>(o, a.C, rows, off);
    return;
  }
  float decay[kRunF][V], bu[kRunF][V], P[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    P[v] = 1.0f;
    H[v] = 0.0f;
  }
  if (live > 0) {
    Raw<T, V> x[kRunF], r[kRunF], i[kRunF];
    load_rows(a.r + at.b * a.rb + c0, a.rr, t0, n, off, r);
    load_rows(a.i + at.b * a.ib + c0, a.ir, t0, n, off, i);
    load_rows(a.x + at.b * a.xb + c0, a.xr, t0, n, off, x);
    float A[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = a.A[c0 + place + v];
#pragma unroll
    for (int k = 0; k < kRunF; ++k) {
      float xv[V], rv[V], iv[V];
      x[k].wide(xv);
      r[k].wide(rv);
      i[k].wide(iv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Decay d = decay_f32(A[v] * gate_f32(rv[v]));
        decay[k][v] = d.a;
        bu[k][v] = __builtin_amdgcn_sqrtf(left_f32(d.e)) * gate_f32(iv[v]) * xv[v];
      }
    }
    if (live < kRunF) {   // padding leaves the state
#pragma unroll
      for (int k = 0; k < kRunF; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          decay[k][v] = k < live ? decay[k][v] : 1.0f;
          bu[k][v] = k < live ? bu[k][v] : 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < kRunF; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        H[v] = __builtin_fmaf(decay[k][v], H[v], bu[k][v]);
        P[v] *= decay[k][v];
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sp[wave][lane * V + v] = P[v];
    sh[wave][lane * V + v] = H[v];
  }
  lds_barrier();
  const int64_t stride = 64 * V;
  if (threadIdx.x < 64 * V) {
    // one channel per lane
    const int j = threadIdx.x;
    const int64_t ch = c0 + j, base = at.chain * a.chunks * stride + j;
    float p = 1.0f, h = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      h = __builtin_fmaf(sp[w][j], h, sh[w][j]);
      p *= sp[w][j];
    }
    float first;
    if (at.q == 0) {
      first = a.state && ch < a.C ? a.state[at.b * a.C + ch] : 0.0f;
    } else {
      publish_total(a.total + base + at.q * stride, p, h);
      first = look_back(a.total + base, a.behind + base, at.q, stride);
    }
    const float last = __builtin_fmaf(p, first, h);
    if (a.chunks > 1) publish_state(a.behind + base + at.q * stride, last);
    before[j] = first;
    if (ch < a.C) {
      if (a.saved) {
        // the states that the backward pass begins its chunks with
        float* to = a.saved + (at.b * a.saves + at.q * (kChunkF / kChunkB)) * a.C + ch;
        float hs = first;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          if (w % (kChunkB / kRunF) == 0 && at.q * kChunkF + w * kRunF < n) to[w / (kChunkB / kRunF) * a.C] = hs;
          hs = __builtin_fmaf(sp[w][j], hs, sh[w][j]);
        }
      }
      if (a.state_out && n <= (at.q + 1) * kChunkF) a.state_out[at.b * a.C + ch] = n == 0 ? first : last;
    }
  }
  lds_barrier();
  if (!a.out || !mine) return;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = before[lane * V + v];
    for (int w = 0; w < wave; ++w) h[v] = __builtin_fmaf(sp[w][lane * V + v], h[v], sh[w][lane * V + v]);
  }
  if (live == 0) {
    zero_rows<V>(o, a.C, rows, off);
    return;
  }
#pragma unroll
  for (int k = 0; k < kRunF; ++k) {
    float y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = __builtin_fmaf(decay[k][v], h[v], bu[k][v]);
      y[v] = k < live ? h[v] : 0.0f;
    }
    if (k < rows) put_row<V>(o, off, y);
    o += a.C;
  }
}

// Few tokens: a lane walks all of them. state_out may be state.
template <typename T, int V>
__global__ __launch_bounds__(256) void gated_short_kernel(GatedP<T> a) {
  const int64_t g = (a.block0 + blockIdx.x) * 256 + threadIdx.x, pieces = a.C / V;
  const int64_t b = g / pieces, c = (g - b * pieces) * V;
  if (b >= a.B) return;
  const int64_t n = seq_len(a.lens, b, a.L);
  float h[V], A[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = a.A[c + v];
    h[v] = a.state ? a.state[b * a.C + c + v] : 0.0f;
    if (a.saved) a.saved[b * a.C + c + v] = h[v];
  }
  if (!a.out && !a.state_out) return;
  T* o = a.out + b * a.L * a.C + c;
  for (int64_t t = 0; t < a.L; ++t) {
    float y[V] = {};
    if (t < n) {
      float xv[V], rv[V], iv[V];
      Raw<T, V> x, r, i;
      x.load(a.x + b * a.xb + t * a.xr + c);
      r.load(a.r + b * a.rb + t * a.rr + c);
      i.load(a.i + b * a.ib + t * a.ir + c);
      x.wide(xv);
      r.wide(rv);
      i.wide(iv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Decay d = decay_f32(A[v] * gate_f32(rv[v]));
        h[v] = __builtin_fmaf(d.a, h[v], __builtin_amdgcn_sqrtf(left_f32(d.e)) * gate_f32(iv[v]) * xv[v]);
        y[v] = h[v];
      }
    }
    if (a.out) stv<V>(o + t * a.C, y);
  }
  if (a.state_out)
#pragma unroll
    for (int v = 0; v < V; ++v) a.state_out[b * a.C + c + v] = h[v];
}

// Backward: chunks from the last; what is handed on is a_t g_t, by the same
// rule. The states within the chunk are found again from the one before it.
template <typename T, int V>
__global__ __launch_bounds__(64 * kChunkB / kRunB, sizeof(T) == 2 || V == 1 ? 4 : 2) void gated_bwd_kernel(GatedP<T> a) {
  constexpr int kWaves = kChunkB / kRunB;
  __shared__ uint32_t slot;
  __shared__ float sp[kWaves][64 * V], sh[kWaves][64 * V], sg[kWaves][64 * V], after[64 * V];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = take_place(a, &slot);
  const int64_t q = a.chunks - 1 - at.q;
  const int64_t n = seq_len(a.lens, at.b, a.L), t0 = q * kChunkB + wave * kRunB;
  const int64_t c0 = at.ct * 64 * V, c = c0 + lane * V;
  const bool mine = c < a.C;
  const uint32_t place = mine ? lane * V : 0, off = place * sizeof(T);
  const int rows = static_cast<int>(a.L - t0 < 0 ? 0 : (a.L - t0 < kRunB ? a.L - t0 : kRunB));
  const int live = static_cast<int>(n - t0 < 0 ? 0 : (n - t0 < kRunB ? n - t0 : kRunB));
  const int64_t to = (at.b * a.L + t0) * a.C + c0;
  const int64_t row = (at.b * a.chunks + q) * a.C;
  if (q * kChunkB >= n) {   // padding, nothing is handed on
    if (mine) {
      zero_rows<V>(a.dx + to, a.C, rows, off);
      zero_rows<V>(a.dr + to, a.C, rows, off);
      zero_rows<V>(a.di + to, a.C, rows, off);
    }
    if (threadIdx.x < 64 * V) {
      const int64_t ch = c0 + threadIdx.x;
      if (ch < a.C) {
        a.part[row + ch] = 0.0f;
        if (n == 0 && q == 0 && a.dstate) a.dstate[at.b * a.C + ch] = a.gstate ? a.gstate[at.b * a.C + ch] : 0.0f;
      }
    }
    return;
  }
  // kept of every token: the decay's word, beta sigmoid(i), and the inputs as stored, whose gates are opened
  // again at the end (kept open they would take registers that a second workgroup lives from)
  float aw[kRunB][V], bw[kRunB][V], P[V], H[V], G[V], A[V];
  Raw<T, V> x[kRunB], gy[kRunB], r[kRunB], i[kRunB];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    P[v] = 1.0f;
    H[v] = G[v] = 0.0f;
    A[v] = a.A[c0 + place + v];
  }
  if (live > 0) {
    load_rows(a.r + at.b * a.rb + c0, a.rr, t0, n, off, r);
    load_rows(a.i + at.b * a.ib + c0, a.ir, t0, n, off, i);
    load_rows(a.x + at.b * a.xb + c0, a.xr, t0, n, off, x);
    load_rows(a.gy + at.b * a.gb + c0, a.gr, t0, n, off, gy);
#pragma unroll
    for (int k = 0; k < kRunB; ++k) {
      float rv[V], iv[V];
      r[k].wide(rv);
      i[k].wide(iv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Decay d = decay_f32(A[v] * gate_f32(rv[v]));
        aw[k][v] = decay_word(d);
        bw[k][v] = __builtin_amdgcn_sqrtf(left_f32(d.e)) * gate_f32(iv[v]);
      }
    }
    if (live < kRunB) {
      // padding: no decay, no input, no gradient; its x and grad_out are the last token's
#pragma unroll
      for (int k = 0; k < kRunB; ++k)
        if (k >= live) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            aw[k][v] = -0.0f;
            bw[k][v] = 0.0f;
          }
          gy[k] = Raw<T, V>{};
        }
    }
#pragma unroll
    for (int k = 0; k < kRunB; ++k) {
      float xv[V];
      x[k].wide(xv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float av = word_decay(aw[k][v]).a;
        H[v] = __builtin_fmaf(av, H[v], bw[k][v] * xv[v]);
        P[v] *= av;
      }
    }
#pragma unroll
    for (int k = kRunB - 1; k >= 0; --k) {
      float gv[V];
      gy[k].wide(gv);
#pragma unroll
      for (int v = 0; v < V; ++v) G[v] = word_decay(aw[k][v]).a * (G[v] + gv[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sp[wave][lane * V + v] = P[v];
    sh[wave][lane * V + v] = H[v];
    sg[wave][lane * V + v] = G[v];
  }
  lds_barrier();
  const int64_t stride = 64 * V;
  if (threadIdx.x < 64 * V) {
    const int j = threadIdx.x;
    const int64_t ch = c0 + j, base = at.chain * a.chunks * stride + j;
    float p = 1.0f, g = 0.0f;
#pragma unroll
    for (int k = kWaves - 1; k >= 0; --k) {
      g = __builtin_fmaf(sp[k][j], g, sg[k][j]);
      p *= sp[k][j];
    }
    // chunks of padding come first in the chain and hand nothing on
    const int64_t dead = a.chunks - (n + kChunkB - 1) / kChunkB;
    float first;
    if (at.q == dead) {
      first = a.gstate && ch < a.C ? a.gstate[at.b * a.C + ch] : 0.0f;
    } else {
      publish_total(a.total + base + at.q * stride, p, g);
      first = look_back(a.total + base + dead * stride, a.behind + base + dead * stride, at.q - dead, stride);
    }
    const float last = __builtin_fmaf(p, first, g);
    if (a.chunks > 1) publish_state(a.behind + base + at.q * stride, last);
    after[j] = first;
    if (q == 0 && a.dstate && ch < a.C) a.dstate[at.b * a.C + ch] = last;
  }
  lds_barrier();
  float h[V], g[V], dA[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = lane * V + v;
    h[v] = a.saved[row + c0 + place + v];
    for (int k = 0; k < wave; ++k) h[v] = __builtin_fmaf(sp[k][j], h[v], sh[k][j]);
    g[v] = after[j];
    for (int k = kWaves - 1; k > wave; --k) g[v] = __builtin_fmaf(sp[k][j], g[v], sg[k][j]);
    dA[v] = 0.0f;
  }
  if (live > 0) {
    float hp[kRunB][V];   // the state before each token
#pragma unroll
    for (int k = 0; k < kRunB; ++k) {
      float xv[V];
      x[k].wide(xv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        hp[k][v] = h[v];
        h[v] = __builtin_fmaf(word_decay(aw[k][v]).a, h[v], bw[k][v] * xv[v]);
      }
    }
    forget(aw);
    int64_t o = to + (kRunB - 1) * a.C;
#pragma unroll
    for (int k = kRunB - 1; k >= 0; --k) {
      float xv[V], gv[V], rv[V], iv[V], dx[V], dr[V], di[V];
      x[k].wide(xv);
      gy[k].wide(gv);
      r[k].wide(rv);
      i[k].wide(iv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // (a^2 / beta) u = a^2 (beta u) / (1 - a^2); 0 where a is 1 to within the smallest normal number
        const Decay d = word_decay(aw[k][v]);
        const float av = d.a, left = left_f32(d.e);
        const float inv = left > 1.17549435e-38f ? __builtin_amdgcn_rcpf(left) : 0.0f;
        float s, sshut, w, wshut;
        gate_both(rv[v], s, sshut);
        gate_both(iv[v], w, wshut);
        const float gt = g[v] + gv[v];
        const float ga = gt * av;
        const float ks = ga * __builtin_fmaf(-av * inv, bw[k][v] * xv[v], hp[k][v]) * s;
        dx[v] = gt * bw[k][v];
        di[v] = dx[v] * xv[v] * wshut;
        dr[v] = ks * A[v] * sshut;
        // padding leaves g; its products are no zeros beside an x or a g that is not finite
        if (k < live) dA[v] += ks;
        else dx[v] = dr[v] = di[v] = 0.0f;
        g[v] = ga;
      }
      if (k < rows && mine) {
        put_row<V>(a.dx + o, off, dx);
        put_row<V>(a.dr + o, off, dr);
        put_row<V>(a.di + o, off, di);
      }
      o -= a.C;
    }
  } else if (mine) {
    zero_rows<V>(a.dx + to, a.C, rows, off);
    zero_rows<V>(a.dr + to, a.C, rows, off);
    zero_rows<V>(a.di + to, a.C, rows, off);
  }
  lds_barrier();
#pragma unroll
  for (int v = 0; v < V; ++v) sp[wave][lane * V + v] = dA[v];
  lds_barrier();
  if (threadIdx.x < 64 * V) {
    const int64_t ch = c0 + threadIdx.x;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) sum += sp[k][threadIdx.x];
    if (ch < a.C) a.part[row + ch] = sum;
  }
}

// marks what chunks hand on as absent and clears the counters
__global__ __launch_bounds__(256) void gated_clear_kernel(u32x4* marks, int64_t nmarks, uint32_t* counter, int64_t ncounter) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < nmarks; i += step)
    marks[i] = u32x4{kAbsent, kAbsent, kAbsent, kAbsent};
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < ncounter; i += step) counter[i] = 0;
}

// The workspace of a chain of chunks: totals, states, counters. Sized for whole tiles
// of 128 channels, which tiles of 64 fill as well or less, and counters of tiles of 64.
struct ChainSpace {
  size_t total, behind, counter, bytes;
};
ChainSpace chain_space(int64_t B, int64_t L, int64_t C, int chunk) {
  const int64_t chunks = cdiv(L, chunk);
  ChainSpace s{};
  if (chunks <= 1) return s;
  const size_t n = static_cast<size_t>(B * chunks * cdiv(C, 128) * 128);
  s.total = 0;
  s.behind = n * 8;
  s.counter = s.behind + n * 4;
  s.bytes = up256(s.counter + static_cast<size_t>(B * cdiv(C, 64)) * 64);
  return s;
}

template <typename T> GatedP<T> gated_params(const gspn_gated_args& a) {
  GatedP<T> p{};
  p.x = static_cast<const T*>(a.x.p);
  p.xb = a.x.batch;
  p.xr = a.x.row;
  p.r = static_cast<const T*>(a.r.p);
  p.rb = a.r.batch;
  p.rr = a.r.row;
  p.i = static_cast<const T*>(a.i.p);
  p.ib = a.i.batch;
  p.ir = a.i.row;
  p.A = a.A;
  p.state = a.state;
  p.lens = a.lens;
  p.out = static_cast<T*>(a.out);
  p.state_out = a.state_out;
  p.saved = static_cast<float*>(a.saved);
  p.L = a.L;
  p.C = a.C;
  p.B = a.B;
  p.saves = std::max<int64_t>(1, cdiv(a.L, kChunkB));
  return p;
}

template <typename T, int V>
hipError_t clear_chain(GatedP<T>& p, int chunk, void* ws, hipStream_t stream, Tracer* tr) {
  p.ctiles = cdiv(p.C, 64 * V);
  p.chunks = std::max<int64_t>(1, cdiv(p.L, chunk));
  if (p.chunks <= 1) return hipSuccess;
  const ChainSpace s = chain_space(p.B, p.L, p.C, chunk);
  char* w = static_cast<char*>(ws);
  p.total = reinterpret_cast<uint64_t*>(w + s.total);
  p.behind = reinterpret_cast<uint32_t*>(w + s.behind);
  p.counter = reinterpret_cast<uint32_t*>(w + s.counter);
  const int64_t marks = static_cast<int64_t>(s.counter / 16), counters = p.B * p.ctiles * 16;
  tr->before(stream, "gated_clear", p.B);
  hipLaunchKernelGGL(gated_clear_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(cdiv(marks, 256), 2048))), dim3(256),
                     0, stream, reinterpret_cast<u32x4*>(w), marks, p.counter, counters);
  const hipError_t e = hipGetLastError();
  tr->after(stream);
  return e;
}

template <typename T, int V>
hipError_t gated_fwd(GatedP<T> p, void* ws, hipStream_t stream, Tracer* tr) {
  if (p.L <= short_tokens<V>(p.B * (p.C / V))) {
    tr->before(stream, "gated_short", p.B);
    const hipError_t e = in_parts(cdiv(p.B * (p.C / V), 256), [&](int64_t first, unsigned count) {
      p.block0 = first;
      hipLaunchKernelGGL((gated_short_kernel<T, V>), dim3(count), dim3(256), 0, stream, p);
    });
    tr->after(stream);
    return e;
  }
  hipError_t e = clear_chain<T, V>(p, kChunkF, ws, stream, tr);
  if (e != hipSuccess) return e;
  tr->before(stream, "gated", p.B);
  e = in_parts(p.B * p.ctiles * p.chunks, [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((gated_kernel<T, V>), dim3(count), dim3(64 * kChunkF / kRunF), 0, stream, p);
  });
  tr->after(stream);
  return e;
}

template <typename T, int V>
hipError_t gated_bwd(GatedP<T> p, const gspn_gated_grads& g, void* ws, hipStream_t stream, Tracer* tr) {
  const ChainSpace s = chain_space(p.B, p.L, p.C, kChunkB);   // the larger one
  char* w = static_cast<char*>(ws) + s.bytes;
  hipError_t e = hipSuccess;
  if (p.B > 0) {
    if (!p.saved) {   // the states before the chunks, found again
      p.saved = reinterpret_cast<float*>(w);
      w += up256(gated_saved_bytes(p.B, p.L, p.C));
      GatedP<T> f = p;
      f.out = nullptr;
      f.state_out = nullptr;
      if ((e = gated_fwd<T, V>(f, ws, stream, tr)) != hipSuccess) return e;
    }
    p.part = reinterpret_cast<float*>(w);
    if ((e = clear_chain<T, V>(p, kChunkB, ws, stream, tr)) != hipSuccess) return e;
    tr->before(stream, "gated_bwd", p.B);
    e = in_parts(p.B * p.ctiles * p.chunks, [&](int64_t first, unsigned count) {
      p.block0 = first;
      hipLaunchKernelGGL((gated_bwd_kernel<T, V>), dim3(count), dim3(64 * kChunkB / kRunB), 0, stream, p);
    });
    tr->after(stream);
    if (e != hipSuccess) return e;
  }
  RowSums sums{};
  sums.part[0] = p.part;
  sums.out[0] = g.A;
  sums.cols[0] = p.C;
  sums.rows = p.B * p.saves;
  return reduce_rows(sums, stream, tr);
}

template <typename T>
hipError_t gated_dt(const gspn_gated_args& a, const gspn_gated_grads* g, void* ws, hipStream_t stream, Tracer* tr) {
  GatedP<T> p = gated_params<T>(a);
  const size_t es = sizeof(T), two = 2 * es;
  bool pair = a.C % 2 == 0 && (a.B * a.L == 0 || (wide_ok(a.x.p, two, es, {a.x.batch, a.x.row}) &&
              wide_ok(a.r.p, two, es, {a.r.batch, a.r.row}) && wide_ok(a.i.p, two, es, {a.i.batch, a.i.row})));
  if (!g) {
    pair = pair && wide_ok(a.out, two, es, {});
    return pair ? gated_fwd<T, 2>(p, ws, stream, tr) : gated_fwd<T, 1>(p, ws, stream, tr);
  }
  p.out = nullptr;
  p.state_out = nullptr;
  p.gy = static_cast<const T*>(g->grad_out.p);
  p.gb = g->grad_out.batch;
  p.gr = g->grad_out.row;
  p.dx = static_cast<T*>(g->x);
  p.dr = static_cast<T*>(g->r);
  p.di = static_cast<T*>(g->i);
  p.dstate = g->state;
  p.gstate = g->grad_state;
  pair = pair && (a.B * a.L == 0 || wide_ok(p.gy, two, es, {p.gb, p.gr})) && wide_ok(p.dx, two, es, {}) &&
         wide_ok(p.dr, two, es, {}) && wide_ok(p.di, two, es, {});
  return pair ? gated_bwd<T, 2>(p, *g, ws, stream, tr) : gated_bwd<T, 1>(p, *g, ws, stream, tr);
}

}  // namespace

size_t gated_saved_bytes(int64_t B, int64_t L, int64_t C) {
  return static_cast<size_t>(B * std::max<int64_t>(1, cdiv(L, kChunkB)) * C) * 4;
}
size_t gated_workspace_bytes(int64_t B, int64_t L, int64_t C) {
  return chain_space(B, L, C, kChunkB).bytes;   // as the backward pass's chunks need it
}
size_t gated_bwd_workspace_bytes(int64_t B, int64_t L, int64_t C) {
  return chain_space(B, L, C, kChunkB).bytes + 2 * up256(gated_saved_bytes(B, L, C));
}

hipError_t launch_gated(const gspn_gated_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return gated_dt<float>(a, nullptr, ws, stream, tr);
  return gated_dt<bf16_t>(a, nullptr, ws, stream, tr);
}
hipError_t launch_gated_bwd(const gspn_gated_args& a, const gspn_gated_grads& g, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return gated_dt<float>(a, &g, ws, stream, tr);
  return gated_dt<bf16_t>(a, &g, ws, stream, tr);
}

}  // namespace gspn
