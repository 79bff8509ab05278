/*
 * gspn_tokens.h -- C ABI of the token-sequence operators that stand next to
 * the 2D propagation in a text-conditioned model:
 *
 *   gspn_causal_conv      the short causal convolution of a state space block,
 *   gspn_selective_scan   its selective scan (a 1D linear recurrence with
 *                         input-dependent weights, as the 2D propagation is a
 *                         2D one), for whole prompts and for single tokens,
 *   gspn_cross_attention  attention of image or text tokens to an encoder's
 *                         states of another length,
 *
 * each with its backward pass. Conventions are those of gspn.h: arguments are
 * validated on the host before anything is enqueued, work is asynchronous on
 * `stream`, no pointer is kept after the call returns, status codes and
 * gspn_last_error() report failures, and storage is fp32 or bf16 with fp32
 * arithmetic and one rounding (to nearest even) per output, except where an
 * operator says otherwise.
 *
 * Sequences are token-major: [B, L, C], the C values of a token contiguous.
 * Inputs may be strided views (slices of a wider projection); outputs and
 * parameters are contiguous. All strides are in elements and >= 0.
 *
 * Padding: `lens`, when not NULL, holds B lengths on the device; token t of
 * entry b with t >= lens[b] is padding, whatever it holds (NaN included): its
 * output is 0, it moves no state, and its gradients are 0. Lengths are taken
 * as clamped to 0 .. L.
 *
 * gspn_trace_events() records the launches of these calls as well.
 *
 * An output may overlap neither an input nor another output (GSPN_E_ALIAS),
 * except state_out, which may be the same memory as state (a step in place).
 */
#ifndef GSPN_TOKENS_H
#define GSPN_TOKENS_H

#include "gspn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* [B, L, C] input: value c of token t of entry b is p[b * batch + t * row + c] */
typedef struct {
  const void* p;
  int64_t batch, row;
} gspn_seq;

/* [B, L, H, E] input: value e of head h is p[b * batch + t * row + h * head + e] */
typedef struct {
  const void* p;
  int64_t batch, row, head;
} gspn_heads;

/*
 * gspn_causal_conv -- a causal convolution of every channel with K taps:
 *   pre[b,t,c] = bias[c] + sum_{j<K} weight[c,j] xx[b, t + j, c],
 *   out = silu ? pre * sigmoid(pre) : pre,
 * where xx[b] is state[b] (the K-1 tokens before the first, zeros when state
 * is NULL) followed by x[b]. state_out (or NULL) receives the K-1 tokens
 * before the next one, the last K-1 rows of xx[b] cut after lens[b] tokens;
 * a call with L = 1 and state_out = state is one step of a serving loop.
 *   B, L, C             L = 0 only moves the state; B * C == 0 does nothing
 *   K                   1 .. 4 (GSPN_E_SHAPE)
 *   weight [C, K], bias [C] or NULL, state and state_out [B, K-1, C] or NULL,
 *   out [B, L, C]       all in dtype
 */
typedef struct {
  int64_t B, L, C, K;
  gspn_dtype dtype;
  int32_t silu;
  gspn_seq x;
  const void* weight;
  const void* bias;
  const void* state;
  const int32_t* lens;
  void* out;
  void* state_out;
} gspn_conv_args;

gspn_status gspn_causal_conv(const gspn_conv_args* args, hipStream_t stream);

/*
 * gspn_causal_conv_backward_ws -- gradients given grad_out = dL/dout and,
 * unless NULL, grad_state = dL/dstate_out [B, K-1, C] (what the next chunk of a
 * sequence hands back): of x [B, L, C], weight [C, K], bias [C] (or NULL) and
 * state [B, K-1, C] (or NULL), all in dtype. args as for the forward call (out
 * and state_out are not read). Sums over tokens are in fp32, in a fixed order. Workspace:
 * gspn_causal_conv_backward_workspace_bytes() bytes, 256-byte aligned.
 */
typedef struct {
  gspn_seq grad_out;
  void* x;
  void* weight;
  void* bias;
  void* state;
  const void* grad_state;
} gspn_conv_grads;

gspn_status gspn_causal_conv_backward_ws(const gspn_conv_args* args, const gspn_conv_grads* grads,
                                         void* workspace, size_t ws_bytes, hipStream_t stream);
size_t gspn_causal_conv_backward_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t K,
                                                 gspn_dtype dtype);

/*
 * gspn_selective_scan_ws -- the selective scan of a state space block. For
 * every entry b and channel c, with N states each:
 *   d_t = softplus ? log(1 + exp(dt_t + dt_bias)) : dt_t + dt_bias
 *   h_t[n] = exp(d_t A[c,n]) h_{t-1}[n] + d_t x_t B_t[n],   h_{-1} = state
 *   y_t = sum_n C_t[n] h_t[n] + D[c] x_t,   out_t = y_t * silu(z_t)
 * Channel c reads group c / (C / G) of B and C.
 *   x, dt, z            [B, L, C] in dtype; z.p may be NULL (no gate)
 *   A [C, N], D [C], dt_bias [C], state and state_out [B, C, N]   fp32,
 *                       D, dt_bias, state and state_out may be NULL
 *   Bm, Cm              [B, L, G, N] in dtype
 *   N 1 .. 32, G >= 1 dividing C (GSPN_E_SHAPE)
 *   out [B, L, C]       in dtype
 *   saved               NULL, or gspn_selective_scan_saved_bytes() bytes,
 *                       256-byte aligned: receives the states at every 16th
 *                       token, which the backward pass of the same arguments
 *                       then takes instead of finding them again
 * A call with L = 1 and state_out = state is one step of a serving loop.
 * Workspace: gspn_selective_scan_workspace_bytes() bytes, 256-byte aligned
 * (0 for L <= 4).
 */
typedef struct {
  int64_t B, L, C, N, G;
  gspn_dtype dtype;
  int32_t softplus;
  gspn_seq x, dt, z;
  const float* A;
  gspn_heads Bm, Cm;
  const float* D;
  const float* dt_bias;
  const float* state;
  const int32_t* lens;
  void* out;
  float* state_out;
  void* saved;
} gspn_scan_args;

gspn_status gspn_selective_scan_ws(const gspn_scan_args* args, void* workspace, size_t ws_bytes,
                                   hipStream_t stream);
size_t gspn_selective_scan_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N, int64_t G,
                                           gspn_dtype dtype);
size_t gspn_selective_scan_saved_bytes(int64_t B, int64_t L, int64_t C, int64_t N);

/*
 * gspn_selective_scan_backward_ws -- gradients given grad_out = dL/dout and,
 * unless NULL, grad_state = dL/dstate_out [B, C, N] (fp32): of x, dt, z
 * [B, L, C], Bm, Cm [B, L, G, N] in dtype, of A [C, N], D [C], dt_bias [C]
 * and state [B, C, N] in fp32. z is required with args->z and must be NULL
 * without; D, dt_bias and state may be NULL (skipped). args as for the
 * forward call (out and state_out are not read; saved is read unless NULL).
 * Sums are in fp32, in a fixed order. Workspace:
 * gspn_selective_scan_backward_workspace_bytes() bytes, 256-byte aligned.
 */
typedef struct {
  gspn_seq grad_out;
  const float* grad_state;
  void* x;
  void* dt;
  void* z;
  void* Bm;
  void* Cm;
  float* A;
  float* D;
  float* dt_bias;
  float* state;
} gspn_scan_grads;

gspn_status gspn_selective_scan_backward_ws(const gspn_scan_args* args,
                                            const gspn_scan_grads* grads, void* workspace,
                                            size_t ws_bytes, hipStream_t stream);
size_t gspn_selective_scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t C, int64_t N,
                                                    int64_t G, gspn_dtype dtype);

/*
 * gspn_cross_attention_ws -- attention of Lq queries to the Lk states of an
 * encoder: for every entry b and query head h, with key head h / (Hq / Hkv),
 *   P = softmax over the kept keys of scale * q k^T,   out = P v,
 *   lse = log sum over the kept keys of exp(scale * q k^T).
 * mask (or NULL: keep all) holds one byte per key, [B, Lk] with entry stride
 * mask_batch, 0 = dropped. Keys that are dropped do not take part, whatever
 * they hold (NaN included). An entry that keeps no key (or Lk = 0) gives
 * out = 0 and lse = -inf, and gradients of 0.
 *   q [B, Lq, Hq, E]; k, v [B, Lk, Hkv, E]; out [B, Lq, Hq, E]   in dtype
 *   lse [B, Hq, Lq] fp32, or NULL
 *   E 1 .. 128; Hkv >= 1 dividing Hq; scale > 0 and below 2^127 (GSPN_E_SHAPE)
 * Products run on matrix cores with fp32 accumulation; with bf16 storage the
 * probabilities are an operand of the second product with 16 bits of mantissa.
 * Workspace: gspn_cross_attention_workspace_bytes() bytes, 256-byte aligned
 * (partial results where few queries read many keys; otherwise 0).
 */
typedef struct {
  int64_t B, Lq, Lk, Hq, Hkv, E;
  gspn_dtype dtype;
  float scale;
  gspn_heads q, k, v;
  const uint8_t* mask;
  int64_t mask_batch;
  void* out;
  float* lse;
} gspn_attn_args;

gspn_status gspn_cross_attention_ws(const gspn_attn_args* args, void* workspace, size_t ws_bytes,
                                    hipStream_t stream);
size_t gspn_cross_attention_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq,
                                            int64_t Hkv, int64_t E, gspn_dtype dtype);

/*
 * gspn_cross_attention_backward_ws -- gradients of q, k, v (contiguous, in
 * dtype) given grad_out = dL/dout. args->out and args->lse are read: they
 * hold the forward call's results. Sums over queries and over the heads that
 * share keys are in fp32, in a fixed order; with bf16 storage the
 * probabilities and the score gradients are operands with 16 bits of mantissa.
 * The sum over e of grad_out out, which every score gradient takes, is found
 * from the probabilities where an entry's kept keys lie within 128 (fp32: 32)
 * and from out as it is stored where they do not.
 * Workspace: gspn_cross_attention_backward_workspace_bytes() bytes, 256-byte
 * aligned.
 */
typedef struct {
  gspn_heads grad_out;
  void* q;
  void* k;
  void* v;
} gspn_attn_grads;

gspn_status gspn_cross_attention_backward_ws(const gspn_attn_args* args,
                                             const gspn_attn_grads* grads, void* workspace,
                                             size_t ws_bytes, hipStream_t stream);
size_t gspn_cross_attention_backward_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq,
                                                     int64_t Hkv, int64_t E, gspn_dtype dtype);

#ifdef __cplusplus
}
#endif

#endif /* GSPN_TOKENS_H */
