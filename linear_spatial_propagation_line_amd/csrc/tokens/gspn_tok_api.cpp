// C ABI of the token-sequence operators: host-side validation (no HIP call
// before an argument is known to be good), workspace checks and launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <exception>

#include "gspn_tokens.hpp"

namespace {

using gspn::set_error;

constexpr int64_t k31 = int64_t(1) << 31;
constexpr int64_t kMaxElems = int64_t(1) << 60;

size_t esize(gspn_dtype dt) { return dt == GSPN_F32 ? 4 : 2; }

// a byte range the call reads or writes
struct Span {
  uintptr_t lo, hi;
};

// Collects what a call reads and writes, and the first thing wrong with it.
class Check {
 public:
  gspn_status status = GSPN_OK;

  gspn_status bad(gspn_status s, const char* detail) {
    if (status == GSPN_OK) status = set_error(s, detail);
    return status;
  }
  bool ok() const { return status == GSPN_OK; }

  // n1 * n2 * ... of non-negative factors, or an error when it grows past
  // what 64-bit byte offsets can address
  int64_t product(std::initializer_list<int64_t> f) {
    int64_t v = 1;
    for (const int64_t x : f) {
      if (x != 0 && v > kMaxElems / x) {
        bad(GSPN_E_SHAPE, "tensor size overflows");
        return 0;
      }
      v *= x;
    }
    return v;
  }
  // contiguous tensor of n elements of size es
  void input(const void* p, int64_t n, size_t es, bool required = true) {
    add(p, n, es, required, false);
  }
  void output(void* p, int64_t n, size_t es, bool required = true) { add(p, n, es, required, true); }
  // strided view: extents and strides, innermost extent last with stride 1
  void view(const void* p, size_t es, std::initializer_list<int64_t> n,
            std::initializer_list<int64_t> stride, bool required = true) {
    int64_t top = 0;
    auto s = stride.begin();
    for (const int64_t x : n) {
      if (x == 0) return;
      const int64_t st = s == stride.end() ? 1 : *s++;
      if (st < 0) {
        bad(GSPN_E_SHAPE, "strides must be >= 0");
        return;
      }
      if (x > 1) {
        if (st > kMaxElems / (x - 1) || top > kMaxElems - (x - 1) * st) {
          bad(GSPN_E_SHAPE, "tensor size overflows");
          return;
        }
        top += (x - 1) * st;
      }
    }
    add(p, top + 1, es, required, false);
  }
  // an input, not required, that update() may name
  void state(const void* p, int64_t n, size_t es) {
    const int before = nin_;
    add(p, n, es, false, false);
    if (nin_ > before) state_in_ = before;
  }
  // an output that may be exactly the memory of the state
  void update(void* p, int64_t n, size_t es) {
    const int before = nout_;
    add(p, n, es, false, true);
    if (nout_ > before) state_out_ = before;
  }
  void scratch(void* ws, size_t bytes, size_t need) {
    if (!ok() || need == 0) return;
    if (!ws || bytes < need) {
      bad(GSPN_E_WORKSPACE, "workspace is NULL or too small");
      return;
    }
    if (reinterpret_cast<uintptr_t>(ws) % 256) {
      bad(GSPN_E_ALIGN, "workspace must be 256-byte aligned");
      return;
    }
    const Span w = span(ws, static_cast<int64_t>(need), 1);
    for (int i = 0; i < nin_; ++i)
      if (meet(w, ins_[i])) bad(GSPN_E_ALIAS, "the workspace overlaps an input");
    for (int i = 0; i < nout_; ++i)
      if (meet(w, outs_[i])) bad(GSPN_E_ALIAS, "the workspace overlaps an output");
  }
  // call after all tensors are named
  void aliases() {
    if (!ok()) return;
    for (int i = 0; i < nout_; ++i) {
      for (int k = 0; k < nin_; ++k) {
        if (!meet(outs_[i], ins_[k])) continue;
        if (i == state_out_ && k == state_in_ && ins_[k].lo == outs_[i].lo) continue;
        bad(GSPN_E_ALIAS, "an output overlaps an input");
      }
      for (int k = i + 1; k < nout_; ++k)
        if (meet(outs_[i], outs_[k])) bad(GSPN_E_ALIAS, "two outputs overlap");
    }
  }

 private:
  static Span span(const void* p, int64_t n, size_t es) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{lo, lo + static_cast<uintptr_t>(n) * es};
  }
  static bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
  void align(const void* p, size_t es) {
    if (reinterpret_cast<uintptr_t>(p) % es)
      bad(GSPN_E_ALIGN, "a pointer is not aligned to its element size");
  }
  void add(const void* p, int64_t n, size_t es, bool required, bool out) {
    if (!ok() || n == 0) return;
    if (!p) {
      if (required) bad(GSPN_E_NULL, "a required pointer is NULL");
      return;
    }
    align(p, es);
    if (out) outs_[nout_++] = span(p, n, es);
    else ins_[nin_++] = span(p, n, es);
  }
  Span ins_[24], outs_[16];
  int nin_ = 0, nout_ = 0, state_in_ = -1, state_out_ = -1;
};

bool dtype_ok(gspn_dtype dt) { return dt == GSPN_F32 || dt == GSPN_BF16; }

// runs `fn(tracer)`; a C entry lets no C++ exception out
template <typename F> gspn_status enqueue(F&& fn) {
  gspn::Tracer tr;
  gspn::trace_begin(&tr);
  const hipError_t e = fn(&tr);
  gspn::trace_end(tr);
  if (e != hipSuccess) return set_error(GSPN_E_HIP, hipGetErrorString(e));
  return GSPN_OK;
}
template <typename F> gspn_status guarded(F&& fn) {
  try {
    gspn::clear_error();
    return fn();
  } catch (const std::exception&) {
    return GSPN_E_NOMEM;   // host memory for an error text or a launch record
  }
}

// ---- convolution ------------------------------------------------------------
void conv_shape(Check& k, int64_t B, int64_t L, int64_t C, int64_t K, gspn_dtype dt) {
  if (!dtype_ok(dt)) k.bad(GSPN_E_DTYPE, "dtype must be GSPN_F32 or GSPN_BF16");
  else if (B < 0 || L < 0 || C < 0 || K < 1 || K > 4)
    k.bad(GSPN_E_SHAPE, "need B, L, C >= 0 and 1 <= K <= 4");
  else if (B >= k31 || L >= k31 || C >= k31 / 8)
    k.bad(GSPN_E_SHAPE, "dimension too large");
  else if (k.product({B, L + K, C, K + 1}) / 32 >= k31 * 32 || k.product({B, L / 128 + 1, C / 64 + 1}) >= k31)
    k.bad(GSPN_E_SHAPE, "tensor too large for one launch");
}
void conv_inputs(Check& k, const gspn_conv_args& a) {
  const size_t es = esize(a.dtype);
  k.view(a.x.p, es, {a.B, a.L, a.C}, {a.x.batch, a.x.row});
  k.input(a.weight, a.C * a.K, es);
  k.input(a.bias, a.C, es, false);
  k.state(a.state, a.B * (a.K - 1) * a.C, es);
  k.input(a.lens, a.B, 4, false);
}

// ---- scan -------------------------------------------------------------------
void scan_shape(Check& k, int64_t B, int64_t L, int64_t C, int64_t N, int64_t G, gspn_dtype dt) {
  if (!dtype_ok(dt)) k.bad(GSPN_E_DTYPE, "dtype must be GSPN_F32 or GSPN_BF16");
  else if (B < 0 || L < 0 || C < 0 || N < 1 || N > 32 || G < 1 || (C % G) != 0)
    k.bad(GSPN_E_SHAPE, "need B, L, C >= 0, 1 <= N <= 32 and G >= 1 dividing C");
  else if (B >= k31 || L >= k31 || C >= k31 / 32)
    k.bad(GSPN_E_SHAPE, "dimension too large");
  else if (k.product({B, L + 1, C + 64, 32}) >= (int64_t(1) << 52) ||
           k.product({B, L / 32 + 1, C / 64 + G}) >= k31 || k.product({B, N, C / 64 + 1}) >= k31 ||
           k.product({B, G, L + 16, 64}) / 256 >= k31)
    k.bad(GSPN_E_SHAPE, "tensor too large for one launch");
}
void scan_inputs(Check& k, const gspn_scan_args& a) {
  const size_t es = esize(a.dtype);
  k.view(a.x.p, es, {a.B, a.L, a.C}, {a.x.batch, a.x.row});
  k.view(a.dt.p, es, {a.B, a.L, a.C}, {a.dt.batch, a.dt.row});
  k.view(a.z.p, es, {a.B, a.L, a.C}, {a.z.batch, a.z.row}, false);
  k.input(a.A, a.C * a.N, 4);
  k.view(a.Bm.p, es, {a.B, a.L, a.G, a.N}, {a.Bm.batch, a.Bm.row, a.Bm.head});
  k.view(a.Cm.p, es, {a.B, a.L, a.G, a.N}, {a.Cm.batch, a.Cm.row, a.Cm.head});
  k.input(a.D, a.C, 4, false);
  k.input(a.dt_bias, a.C, 4, false);
  k.state(a.state, a.B * a.C * a.N, 4);
  k.input(a.lens, a.B, 4, false);
}
void check_saved(Check& k, const void* saved) {
  if (k.ok() && saved && reinterpret_cast<uintptr_t>(saved) % 256)
    k.bad(GSPN_E_ALIGN, "saved must be 256-byte aligned");
}

// ---- attention --------------------------------------------------------------
void attn_shape(Check& k, int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t E,
                gspn_dtype dt) {
  if (!dtype_ok(dt)) k.bad(GSPN_E_DTYPE, "dtype must be GSPN_F32 or GSPN_BF16");
  else if (B < 0 || Lq < 0 || Lk < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || E < 1 || E > 128)
    k.bad(GSPN_E_SHAPE, "need B, Lq, Lk >= 0, Hkv >= 1 dividing Hq, 1 <= E <= 128");
  else if (B >= k31 || Lq >= k31 || Lk >= k31 - 256 || Hq >= k31 || k.product({Lq, Hq}) >= k31 - 256)
    k.bad(GSPN_E_SHAPE, "dimension too large (Lq * Hq and Lk must stay below 2^31)");
  // the last two also keep every launch of tiles below 2^24 workgroups of 256
  else if (k.product({B, Lq + 1, Hq, 128, 4}) >= (int64_t(1) << 52) ||
           k.product({B, Lk + 1, Hkv, 128, 4}) >= (int64_t(1) << 52) ||
           k.product({B, Hkv, Lq * (Hq / Hkv) / 32 + 64}) >= k31 / 64 ||
           k.product({B, Hkv, Lk / 32 + 64}) >= k31 / 64)
    k.bad(GSPN_E_SHAPE, "tensor too large for one launch");
}
void attn_inputs(Check& k, const gspn_attn_args& a) {
  const size_t es = esize(a.dtype);
  if (k.ok() && !(a.scale > 0.0f && std::isfinite(a.scale * 2.0f)))   // the kernels take scale * log2(e)
    k.bad(GSPN_E_SHAPE, "scale must be > 0 and at most half of the largest float");
  k.view(a.q.p, es, {a.B, a.Lq, a.Hq, a.E}, {a.q.batch, a.q.row, a.q.head});
  k.view(a.k.p, es, {a.B, a.Lk, a.Hkv, a.E}, {a.k.batch, a.k.row, a.k.head});
  k.view(a.v.p, es, {a.B, a.Lk, a.Hkv, a.E}, {a.v.batch, a.v.row, a.v.head});
  k.view(a.mask, 1, {a.B, a.Lk}, {a.mask_batch}, false);
}

}  // namespace

extern "C" {

gspn_status gspn_causal_conv(const gspn_conv_args* a, hipStream_t stream) {
  return guarded([&]() -> gspn_status {
    if (!a) return set_error(GSPN_E_NULL, "args must be non-null");
    Check k;
    conv_shape(k, a->B, a->L, a->C, a->K, a->dtype);
    if (!k.ok()) return k.status;
    const size_t es = esize(a->dtype);
    conv_inputs(k, *a);
    k.output(a->out, a->B * a->L * a->C, es);
    k.update(a->state_out, a->B * (a->K - 1) * a->C, es);
    k.aliases();
    if (!k.ok()) return k.status;
    if (a->B == 0 || a->C == 0) return GSPN_OK;
    return enqueue([&](gspn::Tracer* tr) { return gspn::launch_conv(*a, stream, tr); });
  });
}

size_t gspn_causal_conv_backward_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t K,
                                                 gspn_dtype dtype) {
  size_t need = 0;
  guarded([&]() -> gspn_status {
    Check k;
    conv_shape(k, B, L, C, K, dtype);
    if (k.ok()) need = gspn::conv_bwd_workspace_bytes(B, L, C, K);
    return GSPN_OK;
  });
  return need;
}

gspn_status gspn_causal_conv_backward_ws(const gspn_conv_args* a, const gspn_conv_grads* g, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
  return guarded([&]() -> gspn_status {
    if (!a || !g) return set_error(GSPN_E_NULL, "args and grads must be non-null");
    Check k;
    conv_shape(k, a->B, a->L, a->C, a->K, a->dtype);
    if (!k.ok()) return k.status;
    const size_t es = esize(a->dtype);
    conv_inputs(k, *a);
    k.view(g->grad_out.p, es, {a->B, a->L, a->C}, {g->grad_out.batch, g->grad_out.row});
    k.input(g->grad_state, a->B * (a->K - 1) * a->C, es, false);
    k.output(g->x, a->B * a->L * a->C, es);
    k.output(g->weight, a->C * a->K, es);
    k.output(g->bias, a->C, es, false);
    k.output(g->state, a->B * (a->K - 1) * a->C, es, false);
    k.aliases();
    k.scratch(ws, ws_bytes, k.ok() ? gspn::conv_bwd_workspace_bytes(a->B, a->L, a->C, a->K) : 0);
    if (!k.ok()) return k.status;
    if (a->C == 0) return GSPN_OK;
    return enqueue([&](gspn::Tracer* tr) { return gspn::launch_conv_bwd(*a, *g, ws, stream, tr); });
  });
}

gspn_status gspn_selective_scan_ws(const gspn_scan_args* a, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
  return guarded([&]() -> gspn_status {
    if (!a) return set_error(GSPN_E_NULL, "args must be non-null");
    Check k;
    scan_shape(k, a->B, a->L, a->C, a->N, a->G, a->dtype);
    if (!k.ok()) return k.status;
    scan_inputs(k, *a);
    k.output(a->out, a->B * a->L * a->C, esize(a->dtype));
    k.update(a->state_out, a->B * a->C * a->N, 4);
    check_saved(k, a->saved);
    k.output(a->saved, static_cast<int64_t>(gspn::scan_saved_bytes(a->B, a->L, a->C, a->N)), 1, false);
    k.aliases();
    k.scratch(ws, ws_bytes, k.ok() ? gspn::scan_workspace_bytes(a->B, a->L, a->C, a->N, a->G) : 0);
    if (!k.ok()) return k.status;
    if (a->B == 0 || a->C == 0) return GSPN_OK;
    return enqueue([&](gspn::Tracer* tr) { return gspn::launch_scan(*a, ws, stream, tr); });
  });
}

size_t gspn_selective_scan_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G,
                                           gspn_dtype dtype) {
  size_t need = 0;
  guarded([&]() -> gspn_status {
    Check k;
    scan_shape(k, B, L, C, N, G, dtype);
    if (k.ok()) need = gspn::scan_workspace_bytes(B, L, C, N, G);
    return GSPN_OK;
  });
  return need;
}

size_t gspn_selective_scan_saved_bytes(int64_t B, int64_t L, int64_t C, int64_t N) {
  size_t need = 0;
  guarded([&]() -> gspn_status {
    Check k;
    scan_shape(k, B, L, C, N, 1, GSPN_F32);
    if (k.ok()) need = gspn::scan_saved_bytes(B, L, C, N);
    return GSPN_OK;
  });
  return need;
}

gspn_status gspn_selective_scan_backward_ws(const gspn_scan_args* a, const gspn_scan_grads* g,
                                            void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&]() -> gspn_status {
    if (!a || !g) return set_error(GSPN_E_NULL, "args and grads must be non-null");
    Check k;
    scan_shape(k, a->B, a->L, a->C, a->N, a->G, a->dtype);
    if (!k.ok()) return k.status;
    const size_t es = esize(a->dtype);
    const int64_t rows = a->B * a->L * a->C, bc = a->B * a->L * a->G * a->N;
    scan_inputs(k, *a);
    check_saved(k, a->saved);
    k.input(a->saved, static_cast<int64_t>(gspn::scan_saved_bytes(a->B, a->L, a->C, a->N)), 1, false);
    k.view(g->grad_out.p, es, {a->B, a->L, a->C}, {g->grad_out.batch, g->grad_out.row});
    k.input(g->grad_state, a->B * a->C * a->N, 4, false);
    if (k.ok() && rows > 0 && !a->z.p != !g->z)
      k.bad(GSPN_E_NULL, "the gradient of z is wanted exactly when there is a z");
    k.output(g->x, rows, es);
    k.output(g->dt, rows, es);
    k.output(g->z, rows, es, false);
    k.output(g->Bm, bc, es);
    k.output(g->Cm, bc, es);
    k.output(g->A, a->C * a->N, 4);
    k.output(g->D, a->C, 4, false);
    k.output(g->dt_bias, a->C, 4, false);
    k.output(g->state, a->B * a->C * a->N, 4, false);
    k.aliases();
    k.scratch(ws, ws_bytes, k.ok() ? gspn::scan_bwd_workspace_bytes(a->B, a->L, a->C, a->N, a->G) : 0);
    if (!k.ok()) return k.status;
    return enqueue([&](gspn::Tracer* tr) { return gspn::launch_scan_bwd(*a, *g, ws, stream, tr); });
  });
}

size_t gspn_selective_scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N,
                                                    int64_t G, gspn_dtype dtype) {
  size_t need = 0;
  guarded([&]() -> gspn_status {
    Check k;
    scan_shape(k, B, L, C, N, G, dtype);
    if (k.ok()) need = gspn::scan_bwd_workspace_bytes(B, L, C, N, G);
    return GSPN_OK;
  });
  return need;
}

gspn_status gspn_cross_attention_ws(const gspn_attn_args* a, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
  return guarded([&]() -> gspn_status {
    if (!a) return set_error(GSPN_E_NULL, "args must be non-null");
    Check k;
    attn_shape(k, a->B, a->Lq, a->Lk, a->Hq, a->Hkv, a->E, a->dtype);
    if (!k.ok()) return k.status;
    attn_inputs(k, *a);
    k.output(a->out, a->B * a->Lq * a->Hq * a->E, esize(a->dtype));
    k.output(a->lse, a->B * a->Lq * a->Hq, 4, false);
    k.aliases();
    k.scratch(ws, ws_bytes,
              k.ok() ? gspn::attn_workspace_bytes(a->B, a->Lq, a->Lk, a->Hq, a->Hkv, a->E) : 0);
    if (!k.ok()) return k.status;
    if (a->B == 0 || a->Lq == 0) return GSPN_OK;
    return enqueue([&](gspn::Tracer* tr) { return gspn::launch_attn(*a, ws, stream, tr); });
  });
}

size_t gspn_cross_attention_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq,
                                            int64_t Hkv, int64_t E, gspn_dtype dtype) {
  size_t need = 0;
  guarded([&]() -> gspn_status {
    Check k;
    attn_shape(k, B, Lq, Lk, Hq, Hkv, E, dtype);
    if (k.ok()) need = gspn::attn_workspace_bytes(B, Lq, Lk, Hq, Hkv, E);
    return GSPN_OK;
  });
  return need;
}

gspn_status gspn_cross_attention_backward_ws(const gspn_attn_args* a, const gspn_attn_grads* g,
                                             void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&]() -> gspn_status {
    if (!a || !g) return set_error(GSPN_E_NULL, "args and grads must be non-null");
    Check k;
    attn_shape(k, a->B, a->Lq, a->Lk, a->Hq, a->Hkv, a->E, a->dtype);
    if (!k.ok()) return k.status;
    const size_t es = esize(a->dtype);
    const int64_t nq = a->B * a->Lq * a->Hq, nk = a->B * a->Lk * a->Hkv;
    attn_inputs(k, *a);
    k.input(a->out, nq * a->E, es);
    k.input(a->lse, nq, 4);
    k.view(g->grad_out.p, es, {a->B, a->Lq, a->Hq, a->E},
           {g->grad_out.batch, g->grad_out.row, g->grad_out.head});
    k.output(g->q, nq * a->E, es);
    k.output(g->k, nk * a->E, es);
    k.output(g->v, nk * a->E, es);
    k.aliases();
    k.scratch(ws, ws_bytes,
              k.ok() ? gspn::attn_bwd_workspace_bytes(a->B, a->Lq, a->Lk, a->Hq, a->Hkv, a->E) : 0);
    if (!k.ok()) return k.status;
    if (a->B == 0) return GSPN_OK;
    return enqueue([&](gspn::Tracer* tr) { return gspn::launch_attn_bwd(*a, *g, ws, stream, tr); });
  });
}

size_t gspn_cross_attention_backward_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq,
                                                     int64_t Hkv, int64_t E, gspn_dtype dtype) {
  size_t need = 0;
  guarded([&]() -> gspn_status {
    Check k;
    attn_shape(k, B, Lq, Lk, Hq, Hkv, E, dtype);
    if (k.ok()) need = gspn::attn_bwd_workspace_bytes(B, Lq, Lk, Hq, Hkv, E);
    return GSPN_OK;
  });
  return need;
}

}  // extern "C"
