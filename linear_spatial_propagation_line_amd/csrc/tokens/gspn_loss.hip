// Softmax cross entropy of hidden states over a vocabulary, and its gradients,
// without the logits in memory.
//
//   z = x W^T,  lse = log sum_v exp(z_v),  loss = lse - z_target
//   G = g (softmax(z) - onehot(target)),  dx = G W,  dW = G^T x
//
// Bound by matrix products: 2 T V D operations forward, 6 T V D backward (the
// logits are found again): 8192 x 50001 x 2304 bf16 1510 to 1740 us forward as the
// card's power allows (1080 to 1250 TFLOP/s), 4800 to 5400 backward; a library product
// of the logits alone 1603. Few tokens are bound by reading the weight: 32 x 65536 x
// 2304 bf16 54 us (5.6 TB/s). Forward: each tile of logits, 256 vocabulary rows by
// 256 tokens, leaves its maximum and sum of every token, which a last kernel
// joins. Backward, in pieces of the vocabulary: G of the piece goes to the
// workspace, then one launch takes dW of the piece (complete) and the piece's
// part of dx.
//
// Tokens that count are first packed into whole rows (padding, strides and
// widths that are no multiple of a stage end there).
//
// G is an operand, in bf16 for bf16 storage. Its entries at the targets, g (p - 1),
// are most of its norm, and their rounding would add to a gradient as much as
// the result's own (0.0023 from 64 bits in the norm for 0.00166). So they are 0
// in the operand; they are found apart, one fp32 value per token, and their
// products with W's rows and x's are added to dx and dW in fp32. The other
// entries' rounding stays. They sum to 1 - p(target), so their squares are at most
// the square of the target's entry and add at most half of the result's own rounding's
// square: the distance from 64 bits is the result's own rounding times 1.006 where
// logits have a standard deviation of 2, 1.06 to 1.09 at 4, 1.17 at 8, 1.21 at 16, and
// 1.24 where a softmax is one entry off the target (32 and more; 512 tokens, 4096 rows).
// Two bf16 parts would take all of it away for 10 T V D operations instead of 6. With
// fp32 storage the operand holds the targets as well.
#include "gspn_loss_gemm.hpp"

namespace gspn {

namespace {

constexpr int kTile = 256;       // the largest tile: tokens, vocabulary rows or columns
constexpr int kFewTile = 64;     // tokens of a tile where there are few

// whether G's entries at the targets are kept apart from the operand
template <typename T> constexpr bool apart() { return sizeof(T) == 2; }

// wavefronts of a square tile
constexpr int waves_of(int tile) { return tile == 64 ? 4 : 8; }

template <typename T> constexpr int k_step() { return 128 / static_cast<int>(sizeof(T)); }

// Tokens that count, in order. pos >= count: target -1, g 0, lse 0
struct TokenList {
  int32_t* count;
  int32_t* token;    // [Tp]
  int32_t* target;   // [Tp]
  float* g;          // [Tp] backward: the loss's gradient
  float* lse;        // [Tp]
  float* at;         // [Tp] forward: the target's logit; backward, if apart: G there
  int32_t* pos;      // [T] backward: the token's place, -1 without
};

template <typename T> struct LossP {
  TokenList list;
  const T* x; int64_t xb, xr;
  const T* weight;
  const void* ids; int64_t ids_batch; int64_t ids64;   // the targets
  const int32_t* lens;
  float* loss; float* lse;
  const float* glse; const float* gloss;
  T* packed;           // [Tp][Dp]
  const T* w;          // the weight, or its packed copy
  int64_t wld;
  float2* part;        // maximum and sum of tile m of V and place p: [m * part_m + p * part_p]
  int64_t part_m, part_p;
  int64_t L, V, D, tokens, Tp, Dp;
  int64_t block0;
};

// ---- tokens -----------------------------------------------------------------
// One workgroup: the tokens that count in their order. Forward all but the
// padding (whose results are set to 0 here), backward those with a target. Eight
// tokens per lane and turn, all loaded before the first is used (8192 tokens: 7.7 us,
// one at a time 14).
template <typename P, bool BACK>
__global__ __launch_bounds__(1024) void loss_list_kernel(P a) {
  constexpr int kRows = 8;
  __shared__ int32_t sums[kRows][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t done = 0;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kRows * 1024) {
    bool keep[kRows];
    int32_t target[kRows];
    float g[kRows], lse[kRows];
    ids_of<kRows>(a, t0 + threadIdx.x, 1024, keep, target);
    if constexpr (BACK) {
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t t = t0 + k * 1024 + threadIdx.x, c = t < a.tokens ? t : a.tokens - 1;
        keep[k] = target[k] >= 0;
        g[k] = a.gloss[c];
        lse[k] = a.glse[c];
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const uint64_t mask = __ballot(keep[k]);
      if (lane == 0) sums[k][wave] = __popcll(mask);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t t = t0 + k * 1024 + threadIdx.x;
      const uint64_t mask = __ballot(keep[k]);
      int32_t at = done + __popcll(mask & ((uint64_t(1) << lane) - 1));
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        at += w < wave ? sums[k][w] : 0;
        done += sums[k][w];
      }
      if (keep[k]) {
        a.list.token[at] = static_cast<int32_t>(t);
        a.list.target[at] = target[k];
        if constexpr (BACK) {
          a.list.g[at] = g[k];
          a.list.lse[at] = lse[k];
        }
      } else if (t < a.tokens) {
        if constexpr (!BACK) {
          a.loss[t] = 0.0f;
          if (a.lse) a.lse[t] = 0.0f;
        }
      }
      if constexpr (BACK)
        if (t < a.tokens) a.list.pos[t] = keep[k] ? at : -1;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.list.count = done;
  for (int64_t p = done + threadIdx.x; p < a.Tp; p += 1024) {
    a.list.token[p] = -1;
    a.list.target[p] = -1;
    if constexpr (BACK) {
      a.list.g[p] = 0.0f;
      a.list.lse[p] = 0.0f;
      a.list.at[p] = 0.0f;
    }
  }
}

// Few tokens: list and rows in one launch. Workgroup p finds the tokens that count
// among the first 64 by itself and packs the p-th's row; the first writes the list.
template <typename T>
__global__ __launch_bounds__(256) void loss_few_kernel(LossP<T> a, int wide) {
  constexpr int kPer = 16 / sizeof(T);
  const int lane = threadIdx.x & 63, p = blockIdx.x;
  bool live[1];
  int32_t id[1];
  ids_of<1>(a, lane, 0, live, id);
  const bool keep = live[0];
  const int32_t target = id[0];
  const uint64_t mask = __ballot(keep);
  const int count = __popcll(mask);
  if (p == 0 && threadIdx.x < 64) {
    if (lane == 0) *a.list.count = count;
    if (keep) {
      const int at = __popcll(mask & ((uint64_t(1) << lane) - 1));
      a.list.token[at] = lane;
      a.list.target[at] = target;
    } else if (lane < a.tokens) {
      a.loss[lane] = 0.0f;
      if (a.lse) a.lse[lane] = 0.0f;
    }
    if (lane >= count) a.list.target[lane] = -1;
  }
  uint64_t rest = mask;
  for (int k = 0; k < p; ++k) rest &= rest - 1;
  const bool some = p < count;
  const int64_t t = some ? __builtin_ctzll(rest) : 0, b = t / a.L;
  const T* src = a.x + b * a.xb + (t - b * a.L) * a.xr;
  for (int64_t at = threadIdx.x * kPer; at < a.Dp; at += 256 * kPer)
    *reinterpret_cast<u32x4*>(a.packed + p * a.Dp + at) =
        load16<T, false>(src, static_cast<int>(at), some ? static_cast<int>(a.D) : 0, wide);
}

// Rows packed to Dp values, 16 bytes per lane, zeros past D and for places
// without a token: the tokens', then the weight's (rows as they come).
template <typename T> struct PackP {
  const T* x; int64_t xb, xr;
  const int32_t* token;   // null: rows as they come
  T* out;
  int64_t rows, blocks;
  int wide;
};
template <typename T>
__global__ __launch_bounds__(256) void loss_pack_kernel(PackP<T> tokens, PackP<T> weight, int64_t L, int64_t D, int64_t Dp,
                                                        const int32_t* count, int64_t block0) {
  constexpr int kPer = 16 / sizeof(T);
  int64_t block = block0 + blockIdx.x;
  const bool second = block >= tokens.blocks;
  if (second) block -= tokens.blocks;
  const PackP<T>& k = second ? weight : tokens;
  const int64_t per = Dp / kPer, first = block * 256, p0 = first / per;
  const uint32_t i = static_cast<uint32_t>(first - p0 * per) + threadIdx.x, up = i / static_cast<uint32_t>(per);
  const int64_t p = p0 + up, at = static_cast<int64_t>(i - up * static_cast<uint32_t>(per)) * kPer;
  if (p >= k.rows) return;
  const T* src = k.x + p * k.xr;
  bool some = true;
  if (k.token) {
    const int64_t all = *count;
    if (p >= (all + kTile - 1) / kTile * kTile) return;
    some = p < all;
    const int64_t t = some ? k.token[p] : 0, b = some ? static_cast<uint32_t>(t) / static_cast<uint32_t>(L) : 0;
    src = k.x + b * k.xb + (t - b * L) * k.xr;
  }
  *reinterpret_cast<u32x4*>(k.out + p * Dp + at) =
      load16<T, false>(src, static_cast<int>(at), some ? static_cast<int>(D) : 0, k.wide);
}

// ---- forward ----------------------------------------------------------------
// Tiles of vocabulary rows by tokens, dealt to the eight XCDs in contiguous
// shares (each has its own L2), within a share 8 row tiles by as many token
// tiles as run at once.
struct TilePlace {
  int64_t m, n;
};
__device__ __forceinline__ TilePlace tile_place(int64_t g, int64_t mt, int64_t nt) {
  const int64_t all = mt * nt, per = (all + 7) / 8;
  int64_t o = (g & 7) * per + (g >> 3);
  if ((g >> 3) >= per || o >= all) return TilePlace{-1, 0};
  const int64_t band = o / (8 * nt), in = o - band * 8 * nt;
  const int64_t high = mt - band * 8 < 8 ? mt - band * 8 : 8;
  return TilePlace{band * 8 + in % high, in / high};
}
int64_t tile_blocks(int64_t mt, int64_t nt) { return cdiv(mt * nt, 8) * 8; }

// (top, sum) of exponentials joined with another pair of them
__device__ __forceinline__ void join_sums(float& top, float& sum, float t, float u) {
  const float high = fmaxf(top, t), base = high == -INFINITY ? 0.0f : high;
  sum = sum * __builtin_amdgcn_exp2f((top - base) * kLog2e) + u * __builtin_amdgcn_exp2f((t - base) * kLog2e);
  top = high;
}

template <typename T, int BM, int BN, int WM, int NW>
__global__ __launch_bounds__(64 * NW) void loss_logits_kernel(LossP<T> a, int64_t mt, int64_t nt) {
  using P = Product<T, true, true, BM, BN, WM, NW>;
  __shared__ __align__(16) char lds[P::kLds];
  const TilePlace at = tile_place(a.block0 + blockIdx.x, mt, nt);
  if (at.m < 0 || at.n * BN >= *a.list.count) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / P::WN);
  const int64_t m0 = at.m * BM, n0 = at.n * BN;
  f32x16 acc[P::MI][P::NI] = {};
  P::run(Operand<T>{a.w, a.wld, a.V, a.Dp}, Operand<T>{a.packed, a.Dp, a.Tp, a.Dp}, m0, n0, 0, a.D, lds, acc);
  // every token's maximum and sum over the tile's rows
  float2* red = reinterpret_cast<float2*>(lds);   // [WM][BN]
#pragma unroll
  for (int j = 0; j < P::NI; ++j) {
    const int col = wn + 32 * j + (lane & 31);
    const int target = a.list.target[n0 + col];
    const int64_t want = target - m0 - wm;   // the target's row in the wavefront's
    if (__ballot(target >= 0 && want >= 0 && want < BM / WM)) {
#pragma unroll
      for (int i = 0; i < P::MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (target >= 0 && 32 * i + tile_row(r, lane) == want) a.list.at[n0 + col] = acc[i][j][r];
    }
    if (m0 + BM > a.V) {
#pragma unroll
      for (int i = 0; i < P::MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (m0 + wm + 32 * i + tile_row(r, lane) >= a.V) acc[i][j][r] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < P::MI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, acc[i][j][r]);
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < P::MI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f((acc[i][j][r] - base) * kLog2e);
    sum += __shfl_xor(sum, 32, 64);
    if (lane < 32) red[(wave % WM) * BN + col] = make_float2(top, sum);
  }
  lds_barrier();
  for (int col = threadIdx.x; col < BN; col += 64 * NW) {
    float2 s = red[col];
#pragma unroll
    for (int w = 1; w < WM; ++w) join_sums(s.x, s.y, red[w * BN + col].x, red[w * BN + col].y);
    a.part[at.m * a.part_m + (n0 + col) * a.part_p] = s;
  }
}

template <typename P> __device__ __forceinline__ void write_loss(const P& a, int64_t p, float top, float sum) {
  const float lse = top + __builtin_amdgcn_logf(sum) * kLn2;
  const int64_t t = a.list.token[p];
  a.loss[t] = a.list.target[p] >= 0 ? lse - a.list.at[p] : 0.0f;
  if (a.lse) a.lse[t] = lse;
}

// lse and loss from the tiles' maxima and sums: 64 tokens by 8 wavefronts,
// each an eighth of the tiles
template <typename T>
__global__ __launch_bounds__(512) void loss_join_kernel(LossP<T> a, int64_t mt) {
  __shared__ float2 red[8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t p = (a.block0 + blockIdx.x) * 64 + lane, all = *a.list.count;
  if ((a.block0 + blockIdx.x) * 64 >= all) return;
  const int64_t per = (mt + 7) / 8, m0 = wave * per, m1 = m0 + per < mt ? m0 + per : mt;
  float top = -INFINITY, sum = 0.0f;
  constexpr int kAhead = 8;
  for (int64_t m = m0; m < m1; m += kAhead) {
    float2 s[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) s[k] = a.part[(m + k < m1 ? m + k : m1 - 1) * a.part_m + p];
    float t = top;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) t = fmaxf(t, s[k].x);
    const float base = t == -INFINITY ? 0.0f : t;
    sum *= __builtin_amdgcn_exp2f((top - base) * kLog2e);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      sum += m + k < m1 ? s[k].y * __builtin_amdgcn_exp2f((s[k].x - base) * kLog2e) : 0.0f;
    top = t;
  }
  red[wave][lane] = make_float2(top, sum);
  __syncthreads();
  if (wave != 0 || p >= all) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) {
    join_sums(top, sum, red[w][lane].x, red[w][lane].y);
  }
  write_loss(a, p, top, sum);
}

// The same for few tokens, a workgroup for each: its tiles' values lie side by side
template <typename T>
__global__ __launch_bounds__(256) void loss_join_few_kernel(LossP<T> a, int64_t mt) {
  __shared__ float2 red[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t p = blockIdx.x;
  if (p >= *a.list.count) return;
  float top = -INFINITY, sum = 0.0f;
  for (int64_t m0 = 0; m0 < mt; m0 += 4 * 256) {
    float2 s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t m = m0 + k * 256 + threadIdx.x;
      s[k] = m < mt ? a.part[p * a.part_p + m] : make_float2(-INFINITY, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) join_sums(top, sum, s[k].x, s[k].y);
  }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) {
    const float t = __shfl_xor(top, k, 64), u = __shfl_xor(sum, k, 64);
    join_sums(top, sum, t, u);
  }
  if (lane == 0) red[wave] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) join_sums(top, sum, red[w].x, red[w].y);
  write_loss(a, p, top, sum);
}

// ---- backward ---------------------------------------------------------------
// The logits of a piece again, G to the workspace: [Tp][Vp], token rows, through
// LDS so that memory sees whole lines.
template <typename T, int S>
__global__ __launch_bounds__(64 * waves_of(S)) void loss_g_kernel(LossP<T> a, T* G, int64_t v0, int64_t Vp, int64_t mt,
                                                                  int64_t nt) {
  using P = Product<T, true, true, S, S, 2, waves_of(S)>;
  constexpr int kHalves = S * sizeof(T) > 512 ? 2 : 1;        // rows of 1 KB: a half of them at a time
  constexpr int kRows = S / kHalves;
  constexpr int kPitch = kRows * sizeof(T) + 16;
  constexpr int kOut = S * kPitch;
  __shared__ __align__(16) char lds[P::kLds > kOut ? P::kLds : kOut];
  const TilePlace at = tile_place(a.block0 + blockIdx.x, mt, nt);
  if (at.m < 0 || at.n * S >= *a.list.count) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave % 2) * (S / 2), wn = (wave / 2) * (S / P::WN);
  const int64_t m0 = v0 + at.m * S, n0 = at.n * S;
  f32x16 acc[P::MI][P::NI] = {};
  P::run(Operand<T>{a.w, a.wld, a.V, a.Dp}, Operand<T>{a.packed, a.Dp, a.Tp, a.Dp}, m0, n0, 0, a.D, lds, acc);
#pragma unroll
  for (int half = 0; half < kHalves; ++half) {
    if (kHalves == 1 || wave % 2 == half) {
#pragma unroll
      for (int j = 0; j < P::NI; ++j) {
        const int col = wn + 32 * j + (lane & 31);
        const int target = a.list.target[n0 + col];
        const float g = a.list.g[n0 + col], lse = a.list.lse[n0 + col];
        const int64_t want = target >= 0 ? target - m0 - wm : -1;
        char* row_out = lds + col * kPitch + (kHalves == 1 ? wm : 0) * sizeof(T);
#pragma unroll
        for (int i = 0; i < P::MI; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float y[4];
            const int row = 32 * i + tile_row(4 * q, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float p = __builtin_amdgcn_exp2f((acc[i][j][4 * q + e] - lse) * kLog2e);
              if (m0 + S > a.V) p = m0 + wm + row + e < a.V ? p : 0.0f;
              y[e] = g * p;
            }
            if constexpr (sizeof(T) == 2) {
              *reinterpret_cast<uint2*>(row_out + row * 2) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            } else {
              *reinterpret_cast<float4*>(row_out + row * 4) = make_float4(y[0], y[1], y[2], y[3]);
            }
          }
        lds_wave_sync();
        if (lane < 32 && want >= 0 && want < S / 2) {
          T* target_entry = reinterpret_cast<T*>(row_out) + want;
          Store<T>::put(target_entry, 0, apart<T>() ? 0.0f : to_f32(*target_entry) - g);
        }
      }
    }
    lds_barrier();
    constexpr int kPieces = kRows * sizeof(T) / 16;   // of a token's row
    T* out = G + n0 * Vp + at.m * S + half * kRows;
    for (int c = tid; c < S * kPieces; c += P::kThreads) {
      const int t = c / kPieces, q = c % kPieces;
      *reinterpret_cast<u32x4*>(out + t * Vp + q * (16 / sizeof(T))) =
          *reinterpret_cast<const u32x4*>(lds + t * kPitch + q * 16);
    }
    lds_barrier();
  }
}

struct GradPlan {
  int64_t Vp, pieces, splits;   // vocabulary rows of a piece, pieces, parts of dx's contraction
  int64_t tile, gtile;          // of the gradients, of G
};

// dW of a piece and the piece's part of dx in one launch: the tiles of dx first
// (their contraction is a part of the piece), then those of dW (over all tokens).
template <typename T, int S>
__global__ __launch_bounds__(64 * waves_of(S)) void loss_grads_kernel(LossP<T> a, const T* G, int64_t v0, GradPlan plan, float* dx,
                                                         T* dw, const int32_t* start, const float* rest,
                                                         int64_t xblocks, int64_t ttiles, int64_t dtiles,
                                                         int64_t vtiles) {
  using PX = Product<T, true, false, S, S, 2, waves_of(S)>;
  using PW = Product<T, false, false, S, S, 2, waves_of(S)>;
  __shared__ __align__(16) char lds[PX::kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave % 2) * (S / 2), wn = (wave / 2) * (S / PX::WN);
  const int64_t count = *a.list.count, Vp = plan.Vp;
  int64_t g = a.block0 + blockIdx.x;
  f32x16 acc[PX::MI][PX::NI] = {};
  if (g < xblocks) {
    const TilePlace at = tile_place(g, ttiles, dtiles * plan.splits);
    if (at.m < 0 || at.m * S >= count) return;
    const int64_t slot = at.n / dtiles, m0 = at.m * S, n0 = (at.n - slot * dtiles) * S;
    const int64_t live = a.V - v0 < Vp ? a.V - v0 : Vp;      // the piece's rows
    constexpr int64_t step = k_step<T>();
    const int64_t per = ((live + plan.splits - 1) / plan.splits + step - 1) / step * step;
    const int64_t k = slot * per, kend = k + per < live ? k + per : live;
    PX::run(Operand<T>{G, Vp, a.Tp, Vp}, Operand<T>{a.w + v0 * a.wld, a.wld, live, a.wld}, m0, n0, k, kend, lds, acc);
    float* out = dx + (slot * a.Tp + m0 + wm) * a.Dp;
#pragma unroll
    for (int j = 0; j < PX::NI; ++j) {
      const int64_t col = n0 + wn + 32 * j + (lane & 31);
      if (col >= a.Dp) continue;
#pragma unroll
      for (int i = 0; i < PX::MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float* p = out + (32 * i + tile_row(r, lane)) * a.Dp + col;
          *p = v0 == 0 ? acc[i][j][r] : *p + acc[i][j][r];
        }
    }
    return;
  }
  const TilePlace at = tile_place(g - xblocks, vtiles, dtiles);
  if (at.m < 0) return;
  const int64_t m0 = at.m * S, n0 = at.n * S;
  PW::run(Operand<T>{G, Vp, a.Tp, Vp}, Operand<T>{a.packed, a.Dp, a.Tp, a.Dp}, m0, n0, 0, count, lds, acc);
#pragma unroll
  for (int i = 0; i < PW::MI; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t v = v0 + m0 + wm + 32 * i + tile_row(r, lane);
      if (v >= a.V) continue;
      int64_t s0 = 0;
      bool some = false;
      if constexpr (apart<T>()) {
        s0 = start[v];
        some = start[v + 1] > s0;
      }
#pragma unroll
      for (int j = 0; j < PW::NI; ++j) {
        const int64_t col = n0 + wn + 32 * j + (lane & 31);
        if (col >= a.D) continue;
        const float y = some ? acc[i][j][r] + rest[s0 * a.Dp + col] : acc[i][j][r];
        Store<T>::put(dw, v * a.D + col, y);
      }
    }
}

// G at the targets: g (exp(z - lse) - 1), one wavefront per token
template <typename T>
__global__ __launch_bounds__(256) void loss_target_kernel(LossP<T> a) {
  constexpr int kPer = 16 / sizeof(T);
  const int lane = threadIdx.x & 63;
  const int64_t p = (a.block0 + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (p >= *a.list.count) return;
  const T* x = a.packed + p * a.Dp;
  const T* w = a.w + a.list.target[p] * a.wld;
  float s = 0.0f;
  for (int64_t at = lane * kPer; at < a.wld; at += 64 * kPer) {
    Raw<T, kPer> rx, rw;
    rx.load(x + at);
    rw.load(w + at);
    float dx[kPer], dw[kPer];
    rx.wide(dx);
    rw.wide(dw);
#pragma unroll
    for (int e = 0; e < kPer; ++e) s = __builtin_fmaf(dx[e], dw[e], s);
  }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) s += __shfl_xor(s, k, 64);
  if (lane == 0) a.list.at[p] = a.list.g[p] * expm1_f32(s - a.list.lse[p]);
}

// dx: the splits' sums and the target's part, rounded once; zeros for tokens
// that do not count. V adjacent values per lane.
template <typename T, int V>
__global__ __launch_bounds__(256) void loss_dx_kernel(LossP<T> a, const float* parts, int64_t splits, T* dx) {
  const int64_t per = a.D / V, first = (a.block0 + blockIdx.x) * 256, t0 = first / per;
  const uint32_t i = static_cast<uint32_t>(first - t0 * per) + threadIdx.x;
  const uint32_t up = i / static_cast<uint32_t>(per);
  const int64_t t = t0 + up, col = static_cast<int64_t>(i - up * static_cast<uint32_t>(per)) * V;
  if (t >= a.tokens) return;
  const int64_t p = a.list.pos[t];
  float s[V] = {};
  if (p >= 0) {
    for (int64_t k = 0; k < splits; ++k) {
      float y[V];
      ldv<V>(parts + (k * a.Tp + p) * a.Dp + col, y);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += y[e];
    }
    if constexpr (apart<T>()) {
      float w[V];
      ldv<V>(a.w + a.list.target[p] * a.wld + col, w);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = __builtin_fmaf(a.list.at[p], w[e], s[e]);
    }
  }
  stv<V>(dx + t * a.D + col, s);
}

// ---- host -------------------------------------------------------------------
// rows of no whole pieces, where there are tokens: without one the weight is not read
bool packs_weight(int64_t tokens, int64_t D, size_t es) { return tokens > 0 && D * es % 16 != 0; }
int64_t padded(int64_t D, size_t es) { return cdiv(D, 128 / static_cast<int64_t>(es)) * (128 / static_cast<int64_t>(es)); }
// at least one tile: without a token the weight's gradient is still written
int64_t padded_tokens(int64_t T) { return std::max<int64_t>(1, cdiv(T, kTile)) * kTile; }

// pieces of a workspace, in turn
class Space {
 public:
  explicit Space(void* p) : p_(static_cast<char*>(p)) {}
  template <typename E> E* take(int64_t n) {
    E* r = reinterpret_cast<E*>(p_ + used_);
    used_ += up256(static_cast<size_t>(n) * sizeof(E));
    return r;
  }
  size_t used() const { return used_; }

 private:
  char* p_;
  size_t used_ = 0;
};

// The largest square tile that keeps the compute units busy; large tiles read
// their operands less often. Those of 256 (one workgroup a compute unit) have to
// fill three quarters of whole rounds: logits in us with tiles of 256 and of 128,
// 320 tiles of 256 in fp32 1119 and 787, 260 in bf16 55 and 45, 128 30 and 22;
// 256 67 and 84, 640 168 and 197. Those of 128 (two a compute unit) have to fill
// them once: 120 tiles of 128 in fp32 27 and with tiles of 64 18; 256 14 and 18.
int64_t tile_for(int64_t m, int64_t n) {
  const int64_t large = cdiv(m, 256) * cdiv(n, 256);
  if (4 * large >= 3 * 256 * cdiv(large, 256)) return 256;
  return cdiv(m, 128) * cdiv(n, 128) >= 192 ? 128 : 64;
}

// Vocabulary rows of a tile where there are few tokens: 128, 64 where that leaves
// each compute unit one tile at most (5003 x 333 fp32 11 us, with 128 15.6; 16384 x 2304
// bf16 17.0 and 17.6; 50001 x 2304 41.6 and 35.1).
int64_t few_rows(int64_t V) { return V <= 64 * 256 ? 64 : 128; }

template <typename T> void take_common(Space& s, LossP<T>& p) {
  p.list.count = s.take<int32_t>(1);
  p.list.token = s.take<int32_t>(p.Tp);
  p.list.target = s.take<int32_t>(p.Tp);
  p.list.at = s.take<float>(p.Tp);
  p.packed = s.take<T>(p.Tp * p.Dp);
  const bool packs = packs_weight(p.tokens, p.D, sizeof(T));
  p.w = packs ? s.take<T>(p.V * p.Dp) : p.weight;
  p.wld = packs ? p.Dp : p.D;
}
template <typename T> void take_forward(Space& s, LossP<T>& p) {
  take_common(s, p);
  p.part = s.take<float2>(cdiv(p.V, p.tokens <= kFewTile ? few_rows(p.V) : tile_for(p.V, p.tokens)) * p.Tp);
}

// G of a piece is at most half a GiB (pieces of a quarter or a whole GiB take the
// same time to 5 %: 8192 x 65536 x 1024 bf16 3270, 3110, 2980 us), and pieces are alike. dx's contraction is
// cut where its tiles alone are fewer than the compute units.
GradPlan grad_plan(int64_t T, int64_t V, int64_t D, size_t es) {
  GradPlan g;
  const int64_t Tp = padded_tokens(T), most = std::max<int64_t>(kTile, (int64_t(1) << 29) / (Tp * static_cast<int64_t>(es)));
  g.pieces = cdiv(V, std::max<int64_t>(1, most / kTile) * kTile);
  g.Vp = cdiv(cdiv(V, g.pieces), kTile) * kTile;
  g.pieces = cdiv(V, g.Vp);
  const int64_t rows = std::min(g.Vp, V), tokens = std::max<int64_t>(1, T);
  g.gtile = tile_for(rows, tokens);
  g.tile = tile_for(rows, D);
  const int64_t tiles = cdiv(tokens, g.tile) * cdiv(D, g.tile);
  g.splits = std::max<int64_t>(1, std::min<int64_t>(256 / tiles, g.Vp / 512));
  return g;
}
// calls f with the tile as a constant
template <int S> struct TileOf {
  static constexpr int value = S;
};
template <typename F> void by_tile(int64_t tile, F&& f) {
  if (tile == 256) f(TileOf<256>{});
  else if (tile == 128) f(TileOf<128>{});
  else f(TileOf<64>{});
}
template <typename T> struct BackSpace {
  T* G;
  float* dx;
  float* rest;
  float* rest_part;
  void* sort;
};
template <typename T> BackSpace<T> take_backward(Space& s, LossP<T>& p, const GradPlan& g) {
  BackSpace<T> b{};
  take_common(s, p);
  p.list.g = s.take<float>(p.Tp);
  p.list.lse = s.take<float>(p.Tp);
  p.list.pos = s.take<int32_t>(p.tokens);
  b.G = s.take<T>(p.Tp * g.Vp);
  b.dx = s.take<float>(g.splits * p.Tp * p.Dp);
  if (!apart<T>()) return b;
  b.rest = s.take<float>(p.Tp * p.Dp);
  b.rest_part = reinterpret_cast<float*>(s.take<char>(static_cast<int64_t>(run_part_bytes(p.Tp, p.Dp))));
  b.sort = s.take<char>(static_cast<int64_t>(token_sort_bytes(p.Tp, p.V)));
  return b;
}

template <typename T> LossP<T> loss_sizes(int64_t tokens, int64_t L, int64_t V, int64_t D) {
  LossP<T> p{};
  p.L = L;
  p.V = V;
  p.D = D;
  p.tokens = tokens;
  p.Tp = padded_tokens(tokens);
  p.Dp = padded(D, sizeof(T));
  return p;
}
template <typename T> LossP<T> loss_params(const gspn_loss_args& a) {
  LossP<T> p = loss_sizes<T>(a.B * a.L, a.L, a.V, a.D);
  p.x = static_cast<const T*>(a.x.p);
  p.xb = a.x.batch;
  p.xr = a.x.row;
  p.weight = static_cast<const T*>(a.weight);
  p.ids = a.targets;
  p.ids_batch = a.targets_batch;
  p.ids64 = a.targets64;
  p.lens = a.lens;
  return p;
}

template <typename T, bool BACK> hipError_t gather(LossP<T>& p, hipStream_t stream, Tracer* tr) {
  const bool few = !BACK && p.tokens <= kFewTile;
  const int wide_x = wide_ok(p.x, 16, sizeof(T), {p.xb, p.xr}) && p.D % (16 / static_cast<int64_t>(sizeof(T))) == 0;
  tr->before(stream, few ? "loss_few" : "loss_list", p.tokens);
  if (few) hipLaunchKernelGGL((loss_few_kernel<T>), dim3(kFewTile), dim3(256), 0, stream, p, wide_x);
  else hipLaunchKernelGGL((loss_list_kernel<LossP<T>, BACK>), dim3(1), dim3(1024), 0, stream, p);
  hipError_t e = hipGetLastError();
  tr->after(stream);
  if (e != hipSuccess) return e;
  const int64_t pieces = p.Dp * static_cast<int64_t>(sizeof(T)) / 16;
  PackP<T> x{p.x, p.xb, p.xr, p.list.token, p.packed, few || p.tokens == 0 ? 0 : p.Tp, 0, wide_x};
  PackP<T> w{p.weight, 0, p.D, nullptr, const_cast<T*>(p.w), p.w != p.weight ? p.V : 0, 0, 0};
  x.blocks = cdiv(x.rows * pieces, 256);
  w.blocks = cdiv(w.rows * pieces, 256);
  if (x.blocks + w.blocks == 0) return hipSuccess;
  tr->before(stream, "loss_pack", p.Tp);
  e = in_parts(x.blocks + w.blocks, [&](int64_t first, unsigned count) {
    hipLaunchKernelGGL((loss_pack_kernel<T>), dim3(count), dim3(256), 0, stream, x, w, p.L, p.D, p.Dp, p.list.count, first);
  });
  tr->after(stream);
  return e;
}

template <typename T> hipError_t loss_fwd(const gspn_loss_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  LossP<T> p = loss_params<T>(a);
  p.loss = a.loss;
  p.lse = a.lse;
  Space s(ws);
  take_forward(s, p);
  hipError_t e = gather<T, false>(p, stream, tr);
  if (e != hipSuccess) return e;
  const bool few = p.tokens <= kFewTile;
  const int64_t tile = few ? few_rows(p.V) : tile_for(p.V, p.tokens);
  const int64_t mt = cdiv(p.V, tile), nt = few ? 1 : cdiv(p.tokens, tile);
  p.part_m = few ? 1 : p.Tp;
  p.part_p = few ? mt : 1;
  tr->before(stream, "loss_logits", p.V);
  e = in_parts(tile_blocks(mt, nt), [&](int64_t first, unsigned count) {
    p.block0 = first;
    if (few && tile == 128) hipLaunchKernelGGL((loss_logits_kernel<T, 128, kFewTile, 4, 8>), dim3(count), dim3(512), 0, stream, p, mt, nt);
    else if (tile == 256) hipLaunchKernelGGL((loss_logits_kernel<T, 256, 256, 2, 8>), dim3(count), dim3(512), 0, stream, p, mt, nt);
    else if (tile == 128) hipLaunchKernelGGL((loss_logits_kernel<T, 128, 128, 2, 8>), dim3(count), dim3(512), 0, stream, p, mt, nt);
    else hipLaunchKernelGGL((loss_logits_kernel<T, 64, 64, 2, 4>), dim3(count), dim3(256), 0, stream, p, mt, nt);
  });
  tr->after(stream);
  if (e != hipSuccess) return e;
  if (few) {
    tr->before(stream, "loss_join_few", p.tokens);
    hipLaunchKernelGGL((loss_join_few_kernel<T>), dim3(static_cast<unsigned>(p.tokens)), dim3(256), 0, stream, p, mt);
    e = hipGetLastError();
    tr->after(stream);
    return e;
  }
  tr->before(stream, "loss_join", p.tokens);
  e = in_parts(cdiv(p.tokens, 64), [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((loss_join_kernel<T>), dim3(count), dim3(512), 0, stream, p, mt);
  });
  tr->after(stream);
  return e;
}

template <typename T>
hipError_t loss_bwd(const gspn_loss_args& a, const gspn_loss_grads& g, void* ws, hipStream_t stream, Tracer* tr) {
  LossP<T> p = loss_params<T>(a);
  p.glse = g.lse;
  p.gloss = g.grad_loss;
  const GradPlan plan = grad_plan(p.tokens, p.V, p.D, sizeof(T));
  Space s(ws);
  const BackSpace<T> b = take_backward(s, p, plan);
  hipError_t e = gather<T, true>(p, stream, tr);
  if (e != hipSuccess) return e;
  TokenSort sorted{};
  const int64_t ttiles = cdiv(p.tokens, plan.tile), dtiles = cdiv(p.D, plan.tile), gtiles = cdiv(p.tokens, plan.gtile);
  auto launch = [&](const char* name, int64_t blocks, auto&& kernel) {
    tr->before(stream, name, p.tokens);
    const hipError_t r = in_parts(blocks, [&](int64_t first, unsigned count) {
      p.block0 = first;
      kernel(dim3(count));
    });
    tr->after(stream);
    return r;
  };
  if (apart<T>()) {
    // G at the targets, and times the tokens' rows, summed for each target
    e = sort_tokens(p.list.target, 0, 0, nullptr, 1, p.Tp, p.V, b.sort, &sorted, stream, tr);
    if (e != hipSuccess) return e;
    e = launch("loss_target", cdiv(p.tokens, 4), [&](dim3 n) { hipLaunchKernelGGL((loss_target_kernel<T>), n, dim3(256), 0, stream, p); });
    if (e != hipSuccess) return e;
    RunSum sum{};
    sum.sort = sorted;
    sum.dtype = a.dtype;
    sum.x = p.packed;
    sum.row = p.Dp;
    sum.L = sum.tokens = p.Tp;
    sum.weight = p.list.at;
    sum.scale = 1.0f;
    sum.out = b.rest;
    sum.by_place = 1;
    sum.part = b.rest_part;
    sum.V = p.V;
    sum.D = p.Dp;
    if ((e = run_sums(sum, stream, tr)) != hipSuccess) return e;
  }
  for (int64_t k = 0; k < plan.pieces; ++k) {
    const int64_t v0 = k * plan.Vp, rows = std::min(plan.Vp, p.V - v0);
    const int64_t mtiles = cdiv(rows, plan.gtile), vtiles = cdiv(rows, plan.tile);
    e = launch("loss_g", tile_blocks(mtiles, gtiles), [&](dim3 n) {
      auto go = [&](auto s) {
        constexpr int S = decltype(s)::value;
        hipLaunchKernelGGL((loss_g_kernel<T, S>), n, dim3(64 * waves_of(S)), 0, stream, p, b.G, v0, plan.Vp, mtiles, gtiles);
      };
      by_tile(plan.gtile, go);
    });
    if (e != hipSuccess) return e;
    const int64_t xblocks = tile_blocks(ttiles, dtiles * plan.splits);
    e = launch("loss_grads", xblocks + tile_blocks(vtiles, dtiles), [&](dim3 n) {
      auto go = [&](auto s) {
        constexpr int S = decltype(s)::value;
        hipLaunchKernelGGL((loss_grads_kernel<T, S>), n, dim3(64 * waves_of(S)), 0, stream, p, b.G, v0, plan, b.dx,
                           static_cast<T*>(g.weight), sorted.start, b.rest, xblocks, ttiles, dtiles, vtiles);
      };
      by_tile(plan.tile, go);
    });
    if (e != hipSuccess) return e;
  }
  // whole pieces of x's gradient where its rows allow them
  constexpr int kPer = 16 / sizeof(T);
  const bool wide = p.D % kPer == 0 && wide_ok(g.x, 16, sizeof(T), {});
  return launch("loss_dx", cdiv(p.tokens * (wide ? p.D / kPer : p.D), 256), [&](dim3 n) {
    if (wide) hipLaunchKernelGGL((loss_dx_kernel<T, kPer>), n, dim3(256), 0, stream, p, b.dx, plan.splits, static_cast<T*>(g.x));
    else hipLaunchKernelGGL((loss_dx_kernel<T, 1>), n, dim3(256), 0, stream, p, b.dx, plan.splits, static_cast<T*>(g.x));
  });
}

template <typename T> size_t loss_bytes(int64_t B, int64_t L, int64_t V, int64_t D, bool back) {
  LossP<T> p = loss_sizes<T>(B * L, L, V, D);
  if (p.tokens == 0 && !back) return 0;
  Space s(nullptr);
  if (back) take_backward(s, p, grad_plan(p.tokens, V, D, sizeof(T)));
  else take_forward(s, p);
  return s.used();
}

}  // namespace

size_t loss_workspace_bytes(int64_t B, int64_t L, int64_t V, int64_t D, gspn_dtype dt) {
  return dt == GSPN_F32 ? loss_bytes<float>(B, L, V, D, false) : loss_bytes<bf16_t>(B, L, V, D, false);
}
hipError_t launch_loss(const gspn_loss_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return loss_fwd<float>(a, ws, stream, tr);
  return loss_fwd<bf16_t>(a, ws, stream, tr);
}
size_t loss_bwd_workspace_bytes(int64_t B, int64_t L, int64_t V, int64_t D, gspn_dtype dt) {
  return dt == GSPN_F32 ? loss_bytes<float>(B, L, V, D, true) : loss_bytes<bf16_t>(B, L, V, D, true);
}
hipError_t launch_loss_bwd(const gspn_loss_args& a, const gspn_loss_grads& g, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return loss_bwd<float>(a, g, ws, stream, tr);
  return loss_bwd<bf16_t>(a, g, ws, stream, tr);
}

}  // namespace gspn
