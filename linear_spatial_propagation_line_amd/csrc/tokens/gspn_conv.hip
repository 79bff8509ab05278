// Short causal convolution over tokens, forward and backward.
//
//   pre[t] = bias + sum_{j<K} w[j] xx[t + j],  xx = state ++ x,  out = silu(pre)
//   dpre   = grad_out * silu'(pre)
//   dxx[s] = sum_j w[j] dpre[s - j] (+ grad_state where state_out holds the row),
//   dw[j] = sum_t dpre[t] xx[t + j],  db = sum_t dpre[t]
//
// Bound by memory: 2 K + 5 operations against 2 elements moved per value
// (forward), so the work is to move each row once in wide accesses. A lane
// owns V adjacent channels (16 bytes) and walks a run of tokens with the last
// K - 1 rows in registers, so each row is read once per run plus K - 1 rows
// of the run before (from L2); the run's rows are all loaded first, which keeps
// that many 16-byte loads in flight per lane. 8x4096x2304 bf16: 69 us, 4.4 TB/s
// (a large copy reaches 4.9), fp32 119 us, 5.1 TB/s; a training step 187 to 239 us
// by box, fp32 351, where its passes' bytes take 155 and 311 at the copy's rate.
#include "gspn_mfma.hpp"
#include "gspn_tokens.hpp"

namespace gspn {

namespace {

constexpr int kRun = 16;     // tokens one lane walks, all loaded before the first is used
constexpr int kStepBwd = 8;  // backward: tokens loaded together
// Backward: tokens per run. Long runs leave few partial sums and re-read few
// rows; shorter ones where the wavefronts would not fill the chip four times
// (training step, bf16, 8x4096x2304: 64 tokens 187 us, 16 tokens 213;
// 3x1021x1153: 35, 30).
int64_t bwd_run(int64_t B, int64_t L, int64_t C) {
  for (int64_t run = 64; run > 16; run /= 2)
    if (B * cdiv(L, run) * cdiv(C, 256) >= 4096) return run;
  return 16;
}

template <typename T> struct ConvP {
  const T* x; int64_t xb, xr;
  const T* gy; int64_t gb, gr;
  const T* w; const T* bias; const T* state; const int32_t* lens;
  T* out; T* state_out;
  T* dx; T* dstate; const T* gstate; float* part;
  int64_t L, C;
  int64_t run, runs;  // backward: tokens per run; runs per entry (at least 1)
  int64_t ctiles;     // tiles of 64 * V channels
  uint32_t block0;    // first workgroup of this launch
  int silu;
};

// V values at p, widened
template <int V, typename T> __device__ __forceinline__ void ldv(const T* p, float* d) {
  if constexpr (V == 1) {
    d[0] = to_f32(p[0]);
  } else if constexpr (V == 4) {
    const auto q = V4<T>::load(p, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = V4<T>::get(q, e);
  } else {
    run_ld<V>(p, 0, d);
  }
}
template <int V, typename T> __device__ __forceinline__ void stv(T* p, const float* d) {
  if constexpr (V == 1) Store<T>::put(p, 0, d[0]);
  else if constexpr (V == 4) V4<T>::store(p, 0, d);
  else run_st<V>(p, 0, d);
}

// V values as they lie in memory
template <typename T, int V> struct Raw {
  static constexpr int kWords = V * static_cast<int>(sizeof(T)) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  Words q;
  __device__ __forceinline__ void load(const T* p) { q = *reinterpret_cast<const Words*>(p); }
  __device__ __forceinline__ void wide(float* d) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      if constexpr (sizeof(T) == 4) {
        d[k] = __uint_as_float(q[k]);
      } else {
        d[2 * k] = bf16_lo(q[k]);
        d[2 * k + 1] = bf16_hi(q[k]);
      }
    }
  }
};
template <typename T> struct Raw<T, 1> {
  T q;
  __device__ __forceinline__ void load(const T* p) { q = *p; }
  __device__ __forceinline__ void wide(float* d) const { d[0] = to_f32(q); }
};
// rows t .. t + N - 1 of a [B, L, C] tensor's entry, clamped to the last of n
template <int N, typename T, int V>
__device__ __forceinline__ void load_run(const T* base, int64_t stride, int64_t t, int64_t n, Raw<T, V> (&r)[N]) {
  const T* p = base + t * stride;
  if (t + N <= n) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      r[k].load(p);
      p += stride;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      r[k].load(p);
      p += t + k + 1 < n ? stride : 0;
    }
  }
}

// taps and bias of V channels; V > 1: whole pieces, taps of a channel adjacent
template <int K, int V, typename T>
__device__ __forceinline__ void load_taps(const T* w, const T* bias, int64_t c, float (&tap)[K][V], float (&b)[V]) {
  if constexpr (V > 1) {
    Raw<T, V> raw[K + 1];
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].load(w + c * K + k * V);
    if (bias) raw[K].load(bias + c);
    float flat[K * V];
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].wide(flat + k * V);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j < K; ++j) tap[j][e] = flat[e * K + j];
      b[e] = 0.0f;
    }
    if (bias) raw[K].wide(b);
  } else {
#pragma unroll
    for (int j = 0; j < K; ++j) tap[j][0] = ld1(w + c * K + j);
    b[0] = bias ? ld1(bias + c) : 0.0f;
  }
}

// row t of xx without the K - 1 offset: x[t] for 0 <= t < n, the state for
// t < 0 (zeros without one); rows past n are not read
template <int K, int V, typename T>
__device__ __forceinline__ void row_at(const ConvP<T>& a, int64_t b, int64_t c, int64_t t,
                                       int64_t n, float* d) {
  if (t >= 0 && t < n) {
    ldv<V>(a.x + b * a.xb + t * a.xr + c, d);
  } else if (t < 0 && a.state) {
    ldv<V>(a.state + (b * (K - 1) + (t + K - 1)) * a.C + c, d);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) d[e] = 0.0f;
  }
}

template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvP<T> a) {
  // four runs of one channel tile per workgroup, one per wavefront
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t rgroups = static_cast<uint32_t>((a.runs + 3) / 4), ctiles = static_cast<uint32_t>(a.ctiles);
  uint32_t i = blockIdx.x + a.block0;
  const uint32_t ct = i % ctiles;
  i /= ctiles;
  const int64_t rg = i % rgroups, b = i / rgroups;
  const int64_t run = rg * 4 + wave, c = (static_cast<int64_t>(ct) * 64 + lane) * V;
  if (run >= a.runs || c >= a.C) return;
  const int64_t n = seq_len(a.lens, b, a.L);
  const int64_t t0 = run * kRun, t1 = t0 + kRun < a.L ? t0 + kRun : a.L;

  // the run's rows first; a run of padding reads nothing
  const int live = static_cast<int>(n - t0 < 0 ? 0 : (n - t0 < kRun ? n - t0 : kRun));
  Raw<T, V> raw[kRun];
  if (live > 0) load_run(a.x + b * a.xb + c, a.xr, t0, n, raw);
  float w[K][V], bias[V], win[K - 1 > 0 ? K - 1 : 1][V];
  load_taps<K, V>(a.w, a.bias, c, w, bias);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) row_at<K, V>(a, b, c, t0 - (K - 1) + j, n, win[j]);
  // the run that reads the old state also writes the new one (they may be
  // the same memory): rows n - (K - 1) .. n - 1 of state ++ x
  if (run == 0 && a.state_out) {
    float last[K - 1 > 0 ? K - 1 : 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row_at<K, V>(a, b, c, n - (K - 1) + j, n, last[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) stv<V>(a.state_out + (b * (K - 1) + j) * a.C + c, last[j]);
  }
  T* o = a.out + (b * a.L + t0) * a.C + c;
  const int rows = static_cast<int>(t1 - t0);
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    float y[V];
    if (k < live) {
      float r[V];
      raw[k].wide(r);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float s = bias[e];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s = __builtin_fmaf(w[j][e], win[j][e], s);
        s = __builtin_fmaf(w[K - 1][e], r[e], s);
        if (a.silu) s *= sigmoid_f32(s);
        y[e] = s;
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) win[j][e] = win[j + 1][e];
        if (K > 1) win[K > 1 ? K - 2 : 0][e] = r[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = 0.0f;
    }
    if (k < rows) stv<V>(o, y);
    o += a.C;
  }
}

// A run computes dpre for its own tokens and the K - 1 after
// them (which its dx needs too); dw and db take its own tokens only. Rows are
// loaded eight at a time, for the K - 1 too: 24 rows for a run of 16, 72 for one
// of 64 (3x1021x1153 fp32, runs of 16: 66 MB read where x and grad_out are 28). The
// partial sums of the workgroup's four runs are joined in LDS, in run order,
// into row (b, group of runs) of part: [K + 1][C], taps first, then the bias.
// HANDED: there is a grad_state (a look at every row whether it has one costs
// the other calls 4 %: 8x4096x2304, bf16, training step 231 us, 240).
template <typename T, int K, int V, bool HANDED>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvP<T> a) {
  __shared__ float acc[3][(K + 1) * V][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t rgroups = static_cast<uint32_t>((a.runs + 3) / 4), ctiles = static_cast<uint32_t>(a.ctiles);
  uint32_t i = blockIdx.x + a.block0;
  const uint32_t ct = i % ctiles;
  i /= ctiles;
  const int64_t rg = i % rgroups, b = i / rgroups;
  const int64_t run = rg * 4 + wave, c = (static_cast<int64_t>(ct) * 64 + lane) * V;
  const bool live = run < a.runs && c < a.C;

  float w[K][V], bias[V], win[K][V], dp[K][V], dw[K][V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    db[e] = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = dp[j][e] = 0.0f;
  }
  if (live) {
    const int64_t n = seq_len(a.lens, b, a.L);
    const int64_t t0 = run * a.run, t1 = t0 + a.run < a.L ? t0 + a.run : a.L;
    load_taps<K, V>(a.w, a.bias, c, w, bias);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row_at<K, V>(a, b, c, t0 - (K - 1) + j, n, win[j + 1]);
    Raw<T, V> rx[kStepBwd], rg[kStepBwd];
    for (int64_t t = t0; t < t1 + K - 1; t += kStepBwd) {
      // tokens from here on that are no padding; others give dpre = 0
      const int tokens = static_cast<int>(n - t < 0 ? 0 : (n - t < kStepBwd ? n - t : kStepBwd));
      const int rows = static_cast<int>(t1 - t < kStepBwd ? t1 - t : kStepBwd);   // of this run (may be <= 0)
      const int need = static_cast<int>(t1 + K - 1 - t < kStepBwd ? t1 + K - 1 - t : kStepBwd);
      if (tokens > 0) {
        load_run(a.x + b * a.xb + c, a.xr, t, n, rx);
        load_run(a.gy + b * a.gb + c, a.gr, t, n, rg);
      }
#pragma unroll
      for (int k = 0; k < kStepBwd; ++k) {
        if (k < need) {
          float o[V], r[V], gy[V];
          if (k < tokens) {
            rx[k].wide(r);
            rg[k].wide(gy);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
              win[j][e] = win[j + 1][e];
              dp[j][e] = dp[j + 1][e];
            }
            dp[K - 1][e] = 0.0f;
            if (k < tokens) {
              win[K - 1][e] = r[e];
              float s = bias[e];
#pragma unroll
              for (int j = 0; j < K; ++j) s = __builtin_fmaf(w[j][e], win[j][e], s);
              float d = gy[e];
              if (a.silu) {
                const float sg = sigmoid_f32(s);
                d *= sg * __builtin_fmaf(s, 1.0f - sg, 1.0f);
              }
              dp[K - 1][e] = d;
              if (k < rows) {
                db[e] += d;
#pragma unroll
                for (int j = 0; j < K; ++j) dw[j][e] = __builtin_fmaf(d, win[j][e], dw[j][e]);
              }
            }
            // dxx of row s = t + k - (K - 1): w[j] meets dpre[s + K - 1 - j]
            o[e] = 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j) o[e] = __builtin_fmaf(w[j][e], dp[K - 1 - j][e], o[e]);
          }
          const int64_t s = t + k - (K - 1);
          if constexpr (HANDED) {
            if (s >= n - (K - 1) && s < n) {   // one of state_out's rows
              float gs[V];
              ldv<V>(a.gstate + (b * (K - 1) + s - (n - (K - 1))) * a.C + c, gs);
#pragma unroll
              for (int e = 0; e < V; ++e) o[e] += gs[e];
            }
          }
          if (s >= t0) {
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = s < n ? o[e] : 0.0f;
            stv<V>(a.dx + (b * a.L + s) * a.C + c, o);
          } else if (run == 0 && a.dstate) {
            stv<V>(a.dstate + (b * (K - 1) + s + K - 1) * a.C + c, o);
          }
        }
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j < K; ++j) acc[wave - 1][j * V + e][lane] = dw[j][e];
      acc[wave - 1][K * V + e][lane] = db[e];
    }
  }
  __syncthreads();
  if (wave == 0 && c < a.C) {
    float* p = a.part + (b * rgroups + rg) * (K + 1) * a.C + c;
#pragma unroll
    for (int j = 0; j <= K; ++j) {
      float s[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[e] = j < K ? dw[j < K ? j : 0][e] : db[e];
#pragma unroll
        for (int q = 0; q < 3; ++q) s[e] += acc[q][j * V + e][lane];
      }
      // part is fp32 and its rows need not be 16-byte aligned
#pragma unroll
      for (int e = 0; e < V; ++e) p[j * a.C + e] = s[e];
    }
  }
}

// columns of part summed over its rows; the taps' sums go to dw [C][K] and
// the last C columns to db
template <typename T>
__global__ __launch_bounds__(512) void conv_reduce_kernel(const float* part, int64_t rows, int64_t C, int K,
                                                          int64_t block0, T* dw, T* db) {
  __shared__ float acc[8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t cols = (K + 1) * C, i = (blockIdx.x + block0) * 64 + lane;
  float s = 0.0f;
  if (i < cols)
    for (int64_t r = wave; r < rows; r += 8) s += part[r * cols + i];
  acc[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < cols) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += acc[q][lane];
    const int64_t j = i / C, c = i - j * C;
    if (j < K) Store<T>::put(dw, c * K + j, s);
    else if (db) Store<T>::put(db, c, s);
  }
}

__global__ __launch_bounds__(512) void reduce_rows_kernel(RowSums r) {
  __shared__ float acc[8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t blk = blockIdx.x + r.block0;
  int k = 0;   // the table this block works on
  while (k < 2 && blk >= (r.cols[k] + 63) / 64) {
    blk -= (r.cols[k] + 63) / 64;
    ++k;
  }
  const float* part = k == 0 ? r.part[0] : (k == 1 ? r.part[1] : r.part[2]);
  float* out = k == 0 ? r.out[0] : (k == 1 ? r.out[1] : r.out[2]);
  const int64_t cols = k == 0 ? r.cols[0] : (k == 1 ? r.cols[1] : r.cols[2]), i = blk * 64 + lane;
  float s = 0.0f;
  if (i < cols)
    for (int64_t q = wave; q < r.rows; q += 8) s += part[q * cols + i];
  acc[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < cols) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += acc[q][lane];
    out[i] = s;
  }
}

template <typename T> ConvP<T> conv_params(const gspn_conv_args& a) {
  ConvP<T> p{};
  p.x = static_cast<const T*>(a.x.p);
  p.xb = a.x.batch;
  p.xr = a.x.row;
  p.w = static_cast<const T*>(a.weight);
  p.bias = static_cast<const T*>(a.bias);
  p.state = static_cast<const T*>(a.state);
  p.lens = a.lens;
  p.out = static_cast<T*>(a.out);
  p.state_out = static_cast<T*>(a.state_out);
  p.L = a.L;
  p.C = a.C;
  p.runs = std::max<int64_t>(1, cdiv(a.L, kRun));
  p.silu = a.silu;
  return p;
}

template <typename T, int K>
hipError_t conv_dt(const gspn_conv_args& a, const gspn_conv_grads* g, void* ws, hipStream_t stream,
                   Tracer* tr) {
  // backward: four channels per lane, since their sums and windows fill registers
  constexpr int V = 16 / sizeof(T), VB = 4;
  ConvP<T> p = conv_params<T>(a);
  const size_t es = sizeof(T);
  bool wide = a.C % V == 0 && wide_ok(a.x.p, 16, es, {a.x.batch, a.x.row}) &&
              wide_ok(a.weight, 16, es, {}) && (!a.bias || wide_ok(a.bias, 16, es, {})) &&
              (!a.state || wide_ok(a.state, 16, es, {}));
  if (g) {
    p.gy = static_cast<const T*>(g->grad_out.p);
    p.gb = g->grad_out.batch;
    p.gr = g->grad_out.row;
    p.dx = static_cast<T*>(g->x);
    p.dstate = static_cast<T*>(g->state);
    p.gstate = static_cast<const T*>(g->grad_state);
    p.part = static_cast<float*>(ws);
    p.run = bwd_run(a.B, a.L, a.C);
    p.runs = std::max<int64_t>(1, cdiv(a.L, p.run));
    wide = wide && wide_ok(p.gy, 16, es, {p.gb, p.gr}) && wide_ok(p.dx, 16, es, {}) &&
           (!p.dstate || wide_ok(p.dstate, 16, es, {})) && (!p.gstate || wide_ok(p.gstate, 16, es, {}));
  } else {
    wide = wide && wide_ok(p.out, 16, es, {}) && (!p.state_out || wide_ok(p.state_out, 16, es, {}));
  }
  p.ctiles = cdiv(a.C, 64 * (wide ? (g ? VB : V) : 1));
  const int64_t rgroups = cdiv(p.runs, 4);
  constexpr bool kState = K > 1;
  auto kern = !g ? (wide ? conv_fwd_kernel<T, K, V> : conv_fwd_kernel<T, K, 1>)
              : kState && p.gstate ? (wide ? conv_bwd_kernel<T, K, VB, kState> : conv_bwd_kernel<T, K, 1, kState>)
                                   : (wide ? conv_bwd_kernel<T, K, VB, false> : conv_bwd_kernel<T, K, 1, false>);
  tr->before(stream, g ? "conv_bwd" : "conv_fwd", a.B);
  hipError_t e = in_parts(a.B * rgroups * p.ctiles, [&](int64_t first, unsigned count) {
    p.block0 = static_cast<uint32_t>(first);
    hipLaunchKernelGGL(kern, dim3(count), dim3(256), 0, stream, p);
  });
  tr->after(stream);
  if (e != hipSuccess || !g) return e;
  tr->before(stream, "conv_reduce", a.B);
  e = in_parts(cdiv((K + 1) * a.C, 64), [&](int64_t first, unsigned count) {
    hipLaunchKernelGGL(conv_reduce_kernel<T>, dim3(count), dim3(512), 0, stream, p.part, a.B * rgroups, a.C, K, first,
                       static_cast<T*>(g->weight), static_cast<T*>(g->bias));
  });
  tr->after(stream);
  return e;
}

template <typename T>
hipError_t conv_k(const gspn_conv_args& a, const gspn_conv_grads* g, void* ws, hipStream_t stream,
                  Tracer* tr) {
  switch (a.K) {
    case 1: return conv_dt<T, 1>(a, g, ws, stream, tr);
    case 2: return conv_dt<T, 2>(a, g, ws, stream, tr);
    case 3: return conv_dt<T, 3>(a, g, ws, stream, tr);
    default: return conv_dt<T, 4>(a, g, ws, stream, tr);
  }
}

}  // namespace

hipError_t reduce_rows(const RowSums& s, hipStream_t stream, Tracer* tr) {
  RowSums r = s;
  int64_t grid = 0;
  for (int k = 0; k < 3; ++k) {
    if (!r.out[k]) r.cols[k] = 0;
    grid += cdiv(r.cols[k], 64);
  }
  if (grid == 0) return hipSuccess;
  tr->before(stream, "reduce_rows", r.rows);
  const hipError_t e = in_parts(grid, [&](int64_t first, unsigned count) {
    r.block0 = first;
    hipLaunchKernelGGL(reduce_rows_kernel, dim3(count), dim3(512), 0, stream, r);
  });
  tr->after(stream);
  return e;
}

size_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t K) {
  const int64_t rgroups = cdiv(std::max<int64_t>(1, cdiv(L, bwd_run(B, L, C))), 4);
  return static_cast<size_t>(B * rgroups * (K + 1) * C) * sizeof(float);
}

hipError_t launch_conv(const gspn_conv_args& a, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return conv_k<float>(a, nullptr, nullptr, stream, tr);
  return conv_k<bf16_t>(a, nullptr, nullptr, stream, tr);
}

hipError_t launch_conv_bwd(const gspn_conv_args& a, const gspn_conv_grads& g, void* ws,
                           hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return conv_k<float>(a, &g, ws, stream, tr);
  return conv_k<bf16_t>(a, &g, ws, stream, tr);
}

}  // namespace gspn
