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
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch takes fewer than 2^32 threads; what is above is cut off without an
// error. Where the host checks admit more workgroups than that, they go out in
// parts of at most kMostBlocks (of up to 512 threads): part(first, count), in
// order; the kernel adds `first`.
constexpr int64_t kMostBlocks = int64_t(1) << 22;
template <typename F> hipError_t in_parts(int64_t blocks, F&& part) {
  for (int64_t first = 0; first < blocks; first += kMostBlocks) {
    part(first, static_cast<unsigned>(std::min(kMostBlocks, blocks - first)));
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

// length of entry b: lens[b] clamped to 0 .. L, or L
__device__ __forceinline__ int64_t seq_len(const int32_t* lens, int64_t b, int64_t L) {
  if (!lens) return L;
  const int64_t n = lens[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

}  // namespace gspn
