// Internal interface and device helpers of the token-sequence operators
// (causal convolution, selective scan, cross attention).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gspn_device.hpp"
#include "gspn_launch.hpp"
#include "gspn_tokens.h"

namespace gspn {

// Validated problems go to the launchers as the ABI's own argument structs.
size_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t K);
hipError_t launch_conv(const gspn_conv_args& a, hipStream_t stream, Tracer* tr);
hipError_t launch_conv_bwd(const gspn_conv_args& a, const gspn_conv_grads& g, void* ws,
                           hipStream_t stream, Tracer* tr);

constexpr int kScanSave = 16;   // tokens between saved states
size_t scan_saved_bytes(int64_t B, int64_t L, int64_t C, int64_t N);
size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G);
hipError_t launch_scan(const gspn_scan_args& a, void* ws, hipStream_t stream, Tracer* tr);
size_t scan_bwd_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G);
hipError_t launch_scan_bwd(const gspn_scan_args& a, const gspn_scan_grads& g, void* ws,
                           hipStream_t stream, Tracer* tr);

size_t attn_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t E);
hipError_t launch_attn(const gspn_attn_args& a, void* ws, hipStream_t stream, Tracer* tr);
size_t attn_bwd_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv,
                                int64_t E);
hipError_t launch_attn_bwd(const gspn_attn_args& a, const gspn_attn_grads& g, void* ws,
                           hipStream_t stream, Tracer* tr);

size_t embed_bwd_workspace_bytes(int64_t B, int64_t L, int64_t V, int64_t D);
hipError_t launch_embed(const gspn_embed_args& a, hipStream_t stream, Tracer* tr);
hipError_t launch_embed_bwd(const gspn_embed_args& a, const gspn_embed_grads& g, void* ws,
                            hipStream_t stream, Tracer* tr);

// Tokens sorted by their row of a table of V rows, in token order within a row:
// row v owns places start[v] .. start[v + 1] - 1 (start [V + 1]); place holds each
// place's token (x) and its row (y). Padding and ids outside the table are left out. ws: token_sort_bytes() bytes (gspn_embed.hip)
struct TokenSort {
  const int32_t* start;
  const int2* place;
};
size_t token_sort_bytes(int64_t tokens, int64_t V);
hipError_t sort_tokens(const void* ids, int ids64, int64_t ids_batch, const int32_t* lens, int64_t B,
                       int64_t L, int64_t V, void* ws, TokenSort* out, hipStream_t stream, Tracer* tr);

// Sums of the rows of sorted tokens, in fp32 and token order, a run's into its row of
// the table ([V, D] in dtype, zeros in rows without a token) or, by_place, into row
// `start` of an fp32 table. weight: a factor of every token, or null. part:
// run_part_bytes() bytes (gspn_embed.hip)
struct RunSum {
  TokenSort sort;
  gspn_dtype dtype;
  const void* x;
  int64_t batch, row, L, tokens;   // token t is row t % L of entry t / L
  const float* weight;
  float scale;
  void* out;
  int by_place;
  float* part;
  int64_t V, D;
};
size_t run_part_bytes(int64_t tokens, int64_t D);
hipError_t run_sums(const RunSum& r, hipStream_t stream, Tracer* tr);

size_t gated_saved_bytes(int64_t B, int64_t L, int64_t C);
size_t gated_workspace_bytes(int64_t B, int64_t L, int64_t C);
hipError_t launch_gated(const gspn_gated_args& a, void* ws, hipStream_t stream, Tracer* tr);
size_t gated_bwd_workspace_bytes(int64_t B, int64_t L, int64_t C);
hipError_t launch_gated_bwd(const gspn_gated_args& a, const gspn_gated_grads& g, void* ws,
                            hipStream_t stream, Tracer* tr);

size_t loss_workspace_bytes(int64_t B, int64_t L, int64_t V, int64_t D, gspn_dtype dt);
hipError_t launch_loss(const gspn_loss_args& a, void* ws, hipStream_t stream, Tracer* tr);
size_t loss_bwd_workspace_bytes(int64_t B, int64_t L, int64_t V, int64_t D, gspn_dtype dt);
hipError_t launch_loss_bwd(const gspn_loss_args& a, const gspn_loss_grads& g, void* ws,
                           hipStream_t stream, Tracer* tr);

// Up to three tables of fp32 partial sums, [rows][cols] each, summed over
// their rows into fp32 results, in row order within each of eight interleaved
// row sets whose sums are then added in order; rows = 0 writes zeros, a table
// without a result is left out (gspn_conv.hip)
struct RowSums {
  const float* part[3];
  float* out[3];
  int64_t cols[3];
  int64_t rows;
  int64_t block0 = 0;   // set by reduce_rows
};
hipError_t reduce_rows(const RowSums& s, hipStream_t stream, Tracer* tr);

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch takes fewer than 2^32 threads; what is above is cut off without an
// error. Where the host checks admit more workgroups than that, they go out in
// parts of at most kMostBlocks (of up to 512 threads): part(first, count), in
// order; the kernel adds `first`.
constexpr int64_t kMostBlocks = int64_t(1) << 22;
template <typename F> hipError_t in_parts(int64_t blocks, F&& part, int64_t most = kMostBlocks) {
  for (int64_t first = 0; first < blocks; first += most) {
    part(first, static_cast<unsigned>(std::min(most, blocks - first)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// a host-side check that a pointer and the strides used with it keep
// `bytes`-wide accesses aligned
inline bool wide_ok(const void* p, size_t bytes, size_t es, std::initializer_list<int64_t> strides) {
  if (reinterpret_cast<uintptr_t>(p) % bytes) return false;
  for (const int64_t s : strides)
    if ((static_cast<uint64_t>(s) * es) % bytes) return false;
  return true;
}

// ---- device helpers ---------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T> __device__ __forceinline__ float ld1(const T* p) { return to_f32(*p); }

// V values at p, widened
template <int V, typename T> __device__ __forceinline__ void ldv(const T* p, float* d) {
  if constexpr (V == 1) {
    d[0] = to_f32(p[0]);
  } else if constexpr (V == 2) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t q = *reinterpret_cast<const uint32_t*>(p);
      d[0] = bf16_lo(q);
      d[1] = bf16_hi(q);
    } else {
      const float2 q = *reinterpret_cast<const float2*>(p);
      d[0] = q.x;
      d[1] = q.y;
    }
  } else if constexpr (V == 4) {
    const auto q = V4<T>::load(p, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = V4<T>::get(q, e);
  } else {
    run_ld<V>(p, 0, d);
  }
}
template <int V, typename T> __device__ __forceinline__ void stv(T* p, const float* d) {
  if constexpr (V == 1) {
    Store<T>::put(p, 0, d[0]);
  } else if constexpr (V == 2) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(d[0], d[1]);
    else *reinterpret_cast<float2*>(p) = make_float2(d[0], d[1]);
  } else if constexpr (V == 4) {
    V4<T>::store(p, 0, d);
  } else {
    run_st<V>(p, 0, d);
  }
}

// The same past the caches, for results that are written once and read by other
// calls (gated recurrence 8 x 2048 x 2304: 72.5 us against 77, backward 137 against 146)
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <int V, typename T> __device__ __forceinline__ void stream_stv(T* p, const float* d) {
  static_assert(V <= 2, "pairs at most");
  if constexpr (V == 1) {   // rows that begin anywhere, in part lines
    stv<V>(p, d);
  } else if constexpr (sizeof(T) == 2) {
    __builtin_nontemporal_store(pack_bf16x2(d[0], d[1]), reinterpret_cast<uint32_t*>(p));
  } else {
    __builtin_nontemporal_store(u32x2{__float_as_uint(d[0]), __float_as_uint(d[1])}, reinterpret_cast<u32x2*>(p));
  }
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

// sigmoid(v) = (v < 0 ? e : 1) / (1 + e), e = exp(-|v|) in [0, 1]: nothing
// overflows, and far below zero it is 0, so that v sigmoid(v) is 0 also at the
// type's lowest value (a capped exponential left about 2^-125 there, and -8
// as the product)
__device__ __forceinline__ float sigmoid_f32(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  return (v < 0.0f ? e : 1.0f) * recip(1.0f + e);
}

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1]. The
// logarithm is 2 atanh(s), s = e / (2 + e) <= 1/3; atanh(s) / s is a
// polynomial in s^2 fitted on [0, 1/9] (relative error 4e-9), which keeps the
// relative precision that log(1 + e) loses for small e. `slope` receives the
// derivative, 1 / (1 + exp(-v)).
__device__ __forceinline__ float softplus_f32(float v, float* slope = nullptr) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
  const float q = s * s;
  float p = __builtin_fmaf(q, 0.140807269f, 0.139821724f);
  p = __builtin_fmaf(q, p, 0.200123257f);
  p = __builtin_fmaf(q, p, 0.333331602f);
  p = __builtin_fmaf(q, p, 1.0f);
  if (slope) *slope = (v < 0.0f ? e : 1.0f) * recip(1.0f + e);
  return __builtin_fmaf(2.0f * s, p, fmaxf(v, 0.0f));
}

// exp(v) - 1. Below 1/4 its series, cut off at 2e-9 of it and rounded by some two steps
// of 2^-24; from there on the difference, whose exponential's rounding counts up to
// four times (5 steps just above 1/4, fewer further on).
constexpr float kExpm1Series = 0.25f;
__device__ __forceinline__ float expm1_series(float v) {
  float p = __builtin_fmaf(v, 1.0f / 5040.0f, 1.0f / 720.0f);
  p = __builtin_fmaf(v, p, 1.0f / 120.0f);
  p = __builtin_fmaf(v, p, 1.0f / 24.0f);
  p = __builtin_fmaf(v, p, 1.0f / 6.0f);
  p = __builtin_fmaf(v, p, 0.5f);
  return __builtin_fmaf(v, p, 1.0f) * v;
}
__device__ __forceinline__ float expm1_f32(float v) {
  const float d = __builtin_amdgcn_exp2f(v * kLog2e) - 1.0f;
  return fabsf(v) < kExpm1Series ? expm1_series(v) : d;
}
// length of entry b: lens[b] clamped to 0 .. L, or L
__device__ __forceinline__ int64_t seq_len(const int32_t* lens, int64_t b, int64_t L) {
  if (!lens) return L;
  const int64_t n = lens[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

// Tokens t, t + apart, ... (a.tokens of them in all, a.L to an entry, ids a.ids with
// entry stride a.ids_batch, a.ids64 for int64): whether each is a token at all and
// no padding, and its id, -1 where it is not in 0 .. a.V - 1. All ids are loaded,
// whatever they are for, so that no load waits for another.
template <int N, typename P>
__device__ __forceinline__ void ids_of(const P& a, int64_t t, int64_t apart, bool (&live)[N], int32_t (&id)[N]) {
  int64_t at[N], v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int64_t u = t + k * apart;
    const uint32_t c = static_cast<uint32_t>(u < a.tokens ? u : a.tokens - 1), b = c / static_cast<uint32_t>(a.L);
    const uint32_t l = c - b * static_cast<uint32_t>(a.L);
    at[k] = b * a.ids_batch + l;
    live[k] = u < a.tokens;
    if (a.lens) live[k] = live[k] && static_cast<int32_t>(l) < a.lens[b];
  }
  if (a.ids64) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = static_cast<const int64_t*>(a.ids)[at[k]];
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = static_cast<const int32_t*>(a.ids)[at[k]];
  }
#pragma unroll
  for (int k = 0; k < N; ++k) id[k] = live[k] && v[k] >= 0 && v[k] < a.V ? static_cast<int32_t>(v[k]) : -1;
}

}  // namespace gspn
