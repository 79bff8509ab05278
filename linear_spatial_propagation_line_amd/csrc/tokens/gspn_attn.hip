// Cross attention, forward: out = softmax(scale q k^T over the kept keys) v.
//
// One pass over the keys with the running maximum and sum of the softmax: a
// wavefront holds query rows in tiles of 32 (their fragments and the 32 x E
// result stay in registers) and takes 32 keys at a time, X^T = K Q^T,
// probabilities, then O^T += V^T P^T, with one lane per query row, so that the
// row's maximum and sum need one exchange between half-wavefronts. The query heads that share
// a key head are rows of one problem, so their K and V are read once.
#include "gspn_attn.hpp"

namespace gspn {

namespace {

constexpr int kThreads = 256;

template <typename T> struct AttnP {
  const T *q, *k, *v;
  RowMap qm, km, vm;
  const uint8_t* mask;
  int64_t mask_batch;
  T* out;
  float* lse;
  float* part;         // [splits][B * Hkv][rows][EP] unnormalised results,
  float* part_ml;      // [splits][B * Hkv][rows][2] their maxima and sums
  int64_t B, Lq, Lk, rows;
  int Hq, Hkv, share, E, splits, key_tiles, row_tiles, tiles_each;
  float c;             // scale * log2(e)
  bool wide_q, wide_kv, wide_o;
};

template <typename T> struct Keys {   // K, V and the kept keys of one (entry, key head)
  const T *k, *v;
  const uint8_t* mask;
  __device__ __forceinline__ Keys(const AttnP<T>& a, int64_t b, int hk)
      : k(a.k + b * a.km.batch + hk * a.km.head), v(a.v + b * a.vm.batch + hk * a.vm.head),
        mask(a.mask ? a.mask + b * a.mask_batch : nullptr) {}
  __device__ __forceinline__ int64_t clamp(const AttnP<T>& a, int64_t key) const {
    return key < a.Lk ? key : a.Lk - 1;
  }
  __device__ __forceinline__ bool kept(const AttnP<T>& a, int64_t key) const {
    return key < a.Lk && (!mask || mask[key] != 0);
  }
};

// The running maximum may lag behind the true one by this much (base 2): the
// probabilities then reach 2^8, which neither fp32 sums nor bf16 operands
// mind, and the result so far is rescaled only when it has to be.
constexpr float kLag = 8.0f;

// One step of the running softmax over 32 keys: w becomes the probabilities
// (unnormalised, base 2 exponent against m), m and l follow, and the result
// so far is rescaled when the maximum moved far.
template <int N>
__device__ __forceinline__ void softmax_step(float (&w)[16], float c, float& m, float& l, f32x16 (&o)[N]) {
  float top = w[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) top = fmaxf(top, w[i]);
  top = column_max(top) * c;
  if (__any(top > m + kLag)) {
    const float mn = fmaxf(m, top);
    const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
    m = mn;
    l *= f;
#pragma unroll
    for (int et = 0; et < N; ++et) o[et] *= f;
  }
  const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(w[i], c, -base));
    l += w[i];
  }
}

// A row tile's result: into out and lse, or, where the keys are split, as it
// stands into this split's partial results.
template <typename T, int EP, bool FULL>
__device__ __forceinline__ void finish_rows(const AttnP<T>& a, int split, int64_t bh, int64_t b, int hk, uint32_t r,
                                            const f32x16 (&o)[EP / 32], float m, float l, int lane) {
  const bool row_ok = r < a.rows;
  const QRow w = q_row(a, hk, r);
  l = column_sum(l);
  if (a.splits > 1) {
    const int64_t at = (split * a.B * a.Hkv + bh) * a.rows + r;
    store_col<float, EP, true>(a.part + at * EP, row_ok, true, EP, true, o, 1.0f, lane);
    if (row_ok && lane < 32) {
      a.part_ml[at * 2] = m;
      a.part_ml[at * 2 + 1] = l;
    }
  } else {
    store_col<T, EP, FULL>(a.out + ((b * a.Lq + w.q) * a.Hq + w.h) * a.E, row_ok, true, a.E, a.wide_o, o,
                           softmax_scale(l), lane);
    if (a.lse && row_ok && lane < 32) a.lse[(b * a.Hq + w.h) * a.Lq + w.q] = softmax_lse(m, l);
  }
}

// ---- long key axes, many rows, fp32 --------------------------------------------
// Four wavefronts of 32 rows each; K and V pass through LDS 32 keys at a time.
// Bound by the fp32 products (an eighth of bf16's rate).
template <int EP, bool FULL>
__global__ __launch_bounds__(kThreads) void attn_fwd_kernel(AttnP<float> a) {
  using T = float;
  extern __shared__ __align__(16) char lds[];
  constexpr int TK = 32;
  char* kt = lds;
  char* vt = lds + TK * tile_pitch<T, EP>();
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t blk = blockIdx.x;
  const int rt = static_cast<int>(blk % a.row_tiles);
  blk /= a.row_tiles;
  const int split = static_cast<int>(blk % a.splits);
  const int64_t bh = blk / a.splits, b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const uint32_t r = (static_cast<uint32_t>(rt) * 4 + wave) * 32 + (lane & 31);
  const QRow w_ = q_row(a, hk, r);
  const Keys<T> keys(a, b, hk);

  Mma<T>::Frag qf[EP / Mma<T>::kChunk];
  row_frags<T, EP, FULL>(a.q + b * a.qm.batch + w_.q * a.qm.row + w_.h * a.qm.head, true, a.E, a.wide_q, qf);
  f32x16 o[EP / 32] = {};
  float m = -INFINITY, l = 0.0f;
  int64_t k_lo, k_hi;
  key_range(keys.mask, a.Lk, tid, &k_lo, &k_hi);
  const int t_first = max(split * a.tiles_each, static_cast<int>(k_lo / TK));
  const int t_last = min((split + 1) * a.tiles_each, static_cast<int>((k_hi + TK - 1) / TK));
  Stage<T, EP, TK, kThreads> ks, vs;
  auto fetch = [&](int t) {
    const int64_t k0 = static_cast<int64_t>(t) * TK;
    ks.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return keys.k + keys.clamp(a, k0 + i) * a.km.row; });
    vs.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return keys.v + keys.clamp(a, k0 + i) * a.vm.row; });
  };
  if (t_first < t_last) fetch(t_first);
  for (int t = t_first; t < t_last; ++t) {
    const int64_t k0 = static_cast<int64_t>(t) * TK;
    ks.template write<FULL>(kt, tid, a.E, [&](int i) { return keys.kept(a, k0 + i); });
    vs.template write<FULL>(vt, tid, a.E, [&](int i) { return keys.kept(a, k0 + i); });
    __syncthreads();
    if (t + 1 < t_last) fetch(t + 1);
    const uint32_t bits = static_cast<uint32_t>(__ballot(keys.kept(a, k0 + (lane & 31))));
    if (bits != 0) {
      const f32x16 x = tile_dot<T, EP>(kt, 0, qf, lane);
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = x[i];
      drop_keys(w, bits, lane);
      softmax_step(w, a.c, m, l, o);
      tile_accum<EP>(vt, 0, w, o, lane, T{});
    }
    __syncthreads();
  }
  finish_rows<T, EP, FULL>(a, split, bh, b, hk, r, o, m, l, lane);
}

// ---- long key axes, many rows, bf16 ----------------------------------------------
// Four wavefronts of 32 rows each. The products of P and V lag one subtile of
// 32 keys behind, and those of K and Q run one ahead, of the exponentials that
// stand between them, so that a wavefront's own products and exponentials can
// overlap. Tiles of 64 keys in two LDS buffers. Two column tiles (64 rows) per
// wavefront halve what is read from LDS per product, but cost the wavefronts
// that fill each other's waits (with P in bf16 alone, 4x4096x2048 with ragged
// masks, 16 heads of 64: 184 us with two, 130 with one; 2x4096x2048, 16 heads of
// 128: 250 with two and accumulation registers, 190 with one). Now 153 us and
// 175: 500 and 550 TFLOP/s of the products with kept keys (0.55 and 0.70 of all),
// P's second part not counted. The matrix units work for two fifths of the time;
// a wavefront's exponentials and its products still wait for each other.
template <int EP, bool FULL>
__global__ __launch_bounds__(kThreads, 2) void attn_wide_kernel(AttnP<bf16_t> a) {
  using T = bf16_t;
  extern __shared__ __align__(16) char lds[];
  constexpr int kTile = 64 * tile_pitch<T, EP>(), kN = EP / 32;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t blk = blockIdx.x;
  const int rt = static_cast<int>(blk % a.row_tiles);
  blk /= a.row_tiles;
  const int split = static_cast<int>(blk % a.splits);
  const int64_t bh = blk / a.splits, b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const Keys<T> keys(a, b, hk);
  const uint32_t r = (static_cast<uint32_t>(rt) * 4 + wave) * 32 + (lane & 31);
  Mma<T>::Frag qf[EP / 16];
  {
    const QRow w = q_row(a, hk, r);
    row_frags<T, EP, FULL>(a.q + b * a.qm.batch + w.q * a.qm.row + w.h * a.qm.head, true, a.E, a.wide_q, qf);
  }
  int64_t k_lo, k_hi;
  key_range(keys.mask, a.Lk, tid, &k_lo, &k_hi);
  const int t0 = max(split * a.tiles_each, static_cast<int>(k_lo / 64));
  const int t1 = min((split + 1) * a.tiles_each, static_cast<int>((k_hi + 63) / 64));

  f32x16 o[kN] = {};
  float m = -INFINITY, l = 0.0f;
  Stage<T, EP, 64, kThreads> ks, vs;
  bool keep = false;
  auto fetch = [&](int t) {
    const int64_t k0 = static_cast<int64_t>(t) * 64;
    keep = keys.kept(a, k0 + lane);
    ks.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return keys.k + keys.clamp(a, k0 + i) * a.km.row; });
    vs.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return keys.v + keys.clamp(a, k0 + i) * a.vm.row; });
  };
  uint64_t bits = 0, bits_next = 0;   // kept keys of this tile and of the one in staging
  auto stage = [&](int t) {
    bits_next = __ballot(keep);
    char* k = lds + (t & 1) * 2 * kTile;
    ks.template write<FULL>(k, tid, a.E, [&](int i) { return (bits_next >> i) & 1u; });
    vs.template write<FULL>(k + kTile, tid, a.E, [&](int i) { return (bits_next >> i) & 1u; });
  };
  f32x16 x;        // scores of the subtile at hand
  uint32_t p[8], rest[8];   // probabilities of the subtile before, in two bf16 parts
  auto scores = [&](int t, int s) { x = tile_dot<T, EP>(lds + (t & 1) * 2 * kTile, s * 32, qf, lane); };
  auto values = [&](int t, int s) {   // o += V^T P of subtile s of tile t
    tile_accum_split<EP>(lds + (t & 1) * 2 * kTile + kTile, s * 32, p, rest, o, lane);
  };
  if (t0 < t1) {
    fetch(t0);
    stage(t0);
    __syncthreads();
    if (t0 + 1 < t1) fetch(t0 + 1);
    scores(t0, 0);
  }
  for (int t = t0; t < t1; ++t) {
    bits = bits_next;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = x[i];
      drop_keys(w, static_cast<uint32_t>(bits >> (32 * s)), lane);
      // the subtile before: its values are in this tile's buffer or the other
      if (s == 1) values(t, 0);
      else if (t > t0) values(t - 1, 1);
      float top = w[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, w[i]);
      top = column_max(top) * a.c;
      if (s == 0) {
        // all wavefronts are through with the other buffer
        lds_barrier();
        if (t + 1 < t1) stage(t + 1);
        if (t + 2 < t1) fetch(t + 2);
      } else {
        lds_barrier();   // and now it holds the next tile
      }
      if (__any(top > m + kLag)) {
        asm volatile("");   // a branch: these products are not to be done every time
        const float mn = fmaxf(m, top);
        const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
        m = mn;
        l *= f;
#pragma unroll
        for (int et = 0; et < kN; ++et) o[et] *= f;
      }
      if (s == 0) scores(t, 1);
      else if (t + 1 < t1) scores(t + 1, 0);
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(w[i], a.c, -base));
        l += w[i];
      }
      split_bf16(w, p, rest);
    }
  }
  if (t0 < t1) values(t1 - 1, 1);
  finish_rows<T, EP, FULL>(a, split, bh, b, hk, r, o, m, l, lane);
}

// ---- at most 128 keys -----------------------------------------------------------
// All keys of an (entry, key head) stay in LDS while each wavefront walks row
// tiles of its own, with no barrier after the keys are staged: all scores of
// a row are in registers, so its maximum is known before the first exponential.
// Bound by the rows' bytes (q in, out back), nearly matched by the products and
// exponentials of a row; the next tile's q is loaded ahead. 2097152 rows, 77 keys,
// 5 heads of 64, bf16: 625 to 645 us by box, 4.2 TB/s (a copy 4.86, and this
// kernel 4.8 with P in bf16 alone).
template <typename T, int EP, int NT, bool FULL>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void attn_short_kernel(AttnP<T> a) {
  extern __shared__ __align__(16) char lds[];
  char* kt = lds;
  char* vt = lds + NT * 32 * tile_pitch<T, EP>();
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // adjacent workgroups take the heads of the same rows, which share lines
  // and memory pages; splits: of the rows
  const uint32_t heads = static_cast<uint32_t>(a.B) * a.Hkv, bh = blockIdx.x % heads, part = blockIdx.x / heads;
  const int64_t b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const Keys<T> keys(a, b, hk);
  __shared__ __align__(16) float bias[NT * 32];   // 0 for a kept key, -inf for a dropped one
  bool kept = false;
  {
    Stage<T, EP, NT * 32, kThreads> ks;
    Stage<T, EP, NT * 32, kThreads> vs;
    ks.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return keys.k + keys.clamp(a, i) * a.km.row; });
    vs.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return keys.v + keys.clamp(a, i) * a.vm.row; });
    ks.template write<FULL>(kt, tid, a.E, [&](int i) { return keys.kept(a, i); });
    vs.template write<FULL>(vt, tid, a.E, [&](int i) { return keys.kept(a, i); });
    if (tid < NT * 32) {
      kept = keys.kept(a, tid);
      bias[tid] = kept ? 0.0f : -INFINITY;
    }
  }
  const bool any = __syncthreads_or(kept);   // a barrier too
  // Rows pass through LDS in both directions, so that every access to memory
  // is of whole 128-byte lines: fragments straight from memory take a line in
  // four 32-byte parts, and with the lines of all wavefronts in flight the
  // first-level cache does not hold one that long.
  constexpr int kRow = tile_pitch<T, EP>();
  char* mine = lds + 2 * NT * 32 * kRow + wave * 32 * kRow;
  const int t_last = min((part + 1) * a.tiles_each, static_cast<uint32_t>(a.row_tiles));
  int E = a.E;
  using Rows = Stage<T, EP, 32, 64>;
  // 16 bytes of a row of the result
  auto put = [&](const RowTile& rows, int row, int e0, u32x4 v) {
    if (rows.r0 + row >= a.rows) return;
    const QRow u = rows.at(row);
    T* out = a.out + ((b * a.Lq + u.q) * a.Hq + u.h) * E;
    if (FULL || (a.wide_o && e0 < E)) {
      *reinterpret_cast<u32x4*>(out + e0) = v;
    } else {
      const T* from = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int k = 0; k < 16 / static_cast<int>(sizeof(T)); ++k)
        if (e0 + k < E) out[e0 + k] = from[k];
    }
  };
  int t = part * a.tiles_each + wave;
  if (!any) {   // no key kept: 0 whatever q holds (an infinity against the staged zeros would be NaN)
    for (; t < t_last; t += 4) {
      const RowTile rows(a, hk, static_cast<uint32_t>(t) * 32);
#pragma unroll
      for (int i = 0; i < Rows::kEach; ++i) put(rows, Rows::row(lane, i), Rows::e0(lane, i), u32x4{0u, 0u, 0u, 0u});
      if (a.lse && lane < 32 && rows.r0 + lane < a.rows) {
        const QRow u = rows.at(lane);
        a.lse[(b * a.Hq + u.h) * a.Lq + u.q] = -INFINITY;
      }
    }
    return;
  }
  Rows qs;
  auto fetch = [&](int t) {
    const RowTile rows(a, hk, static_cast<uint32_t>(t) * 32);
    qs.template load<FULL>(lane, E, a.wide_q, [&](int i) {
      const QRow w = rows.at(i);
      return a.q + b * a.qm.batch + w.q * a.qm.row + w.h * a.qm.head;
    });
  };
  if (t < t_last) fetch(t);
  for (; t < t_last; t += 4) {
    // The keys' fragments and the comparisons with E are the same for every
    // tile; kept in registers they would cost the occupancy that hides the
    // rows' latency, so they are taken anew.
    asm volatile("" : "+s"(E) : : "memory");
    const RowTile rows(a, hk, static_cast<uint32_t>(t) * 32);
    qs.template write<FULL>(mine, lane, E, [](int) { return true; });
    lds_wave_sync();
    typename Mma<T>::Frag qf[EP / Mma<T>::kChunk];
#pragma unroll
    for (int j = 0; j < EP / Mma<T>::kChunk; ++j) qf[j] = tile_frag<T, EP>(mine, 0, j, lane);
    if (t + 4 < t_last) fetch(t + 4);
    float w[NT][16], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      const f32x16 x = tile_dot<T, EP>(kt, s * 32, qf, lane);
      // dropped keys are zeros in LDS, so a finite row's x is 0 there (an
      // infinity or a NaN in the row makes it NaN by its kept keys anyway)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(bias + s * 32 + 8 * j + 4 * (lane >> 5));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[s][4 * j + i] = __builtin_fmaf(x[4 * j + i], a.c, y[i]);
          m = fmaxf(m, w[s][4 * j + i]);
        }
      }
    }
    m = column_max(m);
    const float base = m == -INFINITY ? 0.0f : m;
    f32x16 o[EP / 32] = {};
#pragma unroll
    for (int s = 0; s < NT; ++s) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[s][i] = __builtin_amdgcn_exp2f(w[s][i] - base);
        l += w[s][i];
      }
      tile_accum<EP>(vt, s * 32, w[s], o, lane, T{});
    }
    l = column_sum(l);
    if (a.lse && lane < 32 && rows.r0 + lane < a.rows) {
      const QRow u = rows.at(lane);
      a.lse[(b * a.Hq + u.h) * a.Lq + u.q] = softmax_lse(m, l);
    }
    const float f = softmax_scale(l);
    lds_wave_sync();   // the queries' fragments have been read
    T* to = reinterpret_cast<T*>(mine + (lane & 31) * kRow) + 4 * (lane >> 5);
#pragma unroll
    for (int et = 0; et < EP / 32; ++et) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v[4] = {o[et][4 * j] * f, o[et][4 * j + 1] * f, o[et][4 * j + 2] * f, o[et][4 * j + 3] * f};
        V4<T>::store(to, et * 32 + 8 * j, v);
      }
    }
    lds_wave_sync();
#pragma unroll
    for (int i = 0; i < Rows::kEach; ++i) {
      const int row = Rows::row(lane, i), e0 = Rows::e0(lane, i);
      put(rows, row, e0, *reinterpret_cast<const u32x4*>(mine + row * kRow + e0 * static_cast<int>(sizeof(T))));
    }
    lds_wave_sync();   // before the next tile's queries go there
  }
}

// ---- at most 32 rows share a key head, more keys ---------------------------------
// Bound by the bytes of K and V (8 x 8192 keys, 8 key heads of 128, 4 rows
// each, bf16: 62 to 66 us from memory by box, 4.1 TB/s; 47 us where the last-level
// cache holds them). What the mask drops is loaded too: with padding to between
// half and all of the keys and one empty entry, a third of these bytes. Each wavefront walks 32 keys at a time of its
// own through its own part of LDS, without barriers, so that wavefronts drift
// apart and loads stay in flight; the four are joined at the end, and the
// workgroups of an (entry, key head) by attn_join_kernel.
template <typename T, int EP, bool FULL>
__global__ __launch_bounds__(kThreads) void attn_few_kernel(AttnP<T> a) {
  extern __shared__ __align__(16) char lds[];
  constexpr int kMine = 2 * 32 * tile_pitch<T, EP>();
  static_assert(kMine >= 32 * EP * 4, "the result fits where the tiles were");
  __shared__ float sm[4][32], sl[4][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  char* kt = lds + wave * kMine;
  char* vt = kt + 32 * tile_pitch<T, EP>();
  const uint32_t bh = blockIdx.x / a.splits;
  const int split = blockIdx.x % a.splits;
  const int64_t b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const uint32_t r = lane & 31;
  const QRow w_ = q_row(a, hk, r);
  const Keys<T> keys(a, b, hk);
  typename Mma<T>::Frag qf[EP / Mma<T>::kChunk];
  row_frags<T, EP, FULL>(a.q + b * a.qm.batch + w_.q * a.qm.row + w_.h * a.qm.head, true, a.E, a.wide_q, qf);
  f32x16 o[EP / 32] = {};
  float m = -INFINITY, l = 0.0f;
  const int t_last = min((split + 1) * a.tiles_each, a.key_tiles);
  Stage<T, EP, 32, 64> ks, vs;
  bool keep = false;   // of key lane % 32
  auto fetch = [&](int t) {
    const int64_t k0 = static_cast<int64_t>(t) * 32;
    keep = keys.kept(a, k0 + (lane & 31));
    ks.template load<FULL>(lane, a.E, a.wide_kv, [&](int i) { return keys.k + keys.clamp(a, k0 + i) * a.km.row; });
    vs.template load<FULL>(lane, a.E, a.wide_kv, [&](int i) { return keys.v + keys.clamp(a, k0 + i) * a.vm.row; });
  };
  int t = split * a.tiles_each + wave;
  if (t < t_last) fetch(t);
  for (; t < t_last; t += 4) {
    const uint32_t bits = static_cast<uint32_t>(__ballot(keep));
    ks.template write<FULL>(kt, lane, a.E, [&](int i) { return (bits >> i) & 1u; });
    vs.template write<FULL>(vt, lane, a.E, [&](int i) { return (bits >> i) & 1u; });
    lds_wave_sync();
    if (t + 4 < t_last) fetch(t + 4);
    if (bits != 0) {
      const f32x16 x = tile_dot<T, EP>(kt, 0, qf, lane);
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = x[i];
      drop_keys(w, bits, lane);
      softmax_step(w, a.c, m, l, o);
      tile_accum<EP>(vt, 0, w, o, lane, T{});
    }
    lds_wave_sync();
  }
  l = column_sum(l);
  float* mine = reinterpret_cast<float*>(kt);
#pragma unroll
  for (int et = 0; et < EP / 32; ++et) {
#pragma unroll
    for (int i = 0; i < 16; ++i) mine[(lane & 31) * EP + et * 32 + (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5)] = o[et][i];
  }
  if (lane < 32) {
    sm[wave][lane] = m;
    sl[wave][lane] = l;
  }
  __syncthreads();
  const int rows = static_cast<int>(a.rows);
  for (int i = tid; i < rows * EP; i += kThreads) {
    const int row = i / EP, e = i - row * EP;
    float top = sm[0][row];
#pragma unroll
    for (int q = 1; q < 4; ++q) top = fmaxf(top, sm[q][row]);
    const float base = top == -INFINITY ? 0.0f : top;
    float v = 0.0f, sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f = __builtin_amdgcn_exp2f(sm[q][row] - base);
      sum = __builtin_fmaf(f, sl[q][row], sum);
      v = __builtin_fmaf(f, reinterpret_cast<const float*>(lds + q * kMine)[i], v);
    }
    const QRow u = q_row(a, hk, row);
    if (a.splits > 1) {
      const int64_t at = (static_cast<int64_t>(split) * a.B * a.Hkv + bh) * rows + row;
      a.part[at * EP + e] = v;
      if (e == 0) {
        a.part_ml[at * 2] = top;
        a.part_ml[at * 2 + 1] = sum;
      }
    } else {
      if (e < a.E) Store<T>::put(a.out, ((b * a.Lq + u.q) * a.Hq + u.h) * a.E + e, v * softmax_scale(sum));
      if (e == 0 && a.lse) a.lse[(b * a.Hq + u.h) * a.Lq + u.q] = softmax_lse(top, sum);
    }
  }
}

// Joins the at most 64 parts of a row, in order: one wavefront per row, lane s
// holding part s's maximum and sum, lanes over the values.
template <typename T, int EP>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnP<T> a) {
  const int lane = threadIdx.x & 63;
  const int64_t i = blockIdx.x * int64_t(kThreads / 64) + (threadIdx.x >> 6);
  const int64_t total = a.B * a.Hkv * a.rows;
  if (i >= total) return;
  const int64_t bh = i / a.rows, b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const QRow u = q_row(a, hk, static_cast<uint32_t>(i - bh * a.rows));
  const bool in = lane < a.splits;
  const float pm = in ? a.part_ml[(lane * total + i) * 2] : -INFINITY;
  float m = pm;
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
  const float f = __builtin_amdgcn_exp2f(pm - (m == -INFINITY ? 0.0f : m));
  float l = in ? f * a.part_ml[(lane * total + i) * 2 + 1] : 0.0f;
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) l += __shfl_xor(l, d);
  constexpr int kV = (EP + 63) / 64;
  float v[kV] = {};
  const float* p = a.part + i * EP + lane;
#pragma unroll 8
  for (int s = 0; s < a.splits; ++s) {
    const float fs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), s));
#pragma unroll
    for (int k = 0; k < kV; ++k)
      if (lane + 64 * k < EP) v[k] = __builtin_fmaf(fs, p[s * total * EP + 64 * k], v[k]);
  }
  const float scale = softmax_scale(l);
#pragma unroll
  for (int k = 0; k < kV; ++k)
    if (lane + 64 * k < a.E)
      Store<T>::put(a.out, ((b * a.Lq + u.q) * a.Hq + u.h) * a.E + lane + 64 * k, v[k] * scale);
  if (a.lse && lane == 0) a.lse[(b * a.Hq + u.h) * a.Lq + u.q] = softmax_lse(m, l);
}

// out = 0, lse = -inf when there is no key at all
template <typename T>
__global__ __launch_bounds__(kThreads) void attn_empty_kernel(T* out, int64_t n, float* lse, int64_t rows,
                                                              int64_t block0) {
  const int64_t i = (block0 + blockIdx.x) * kThreads + threadIdx.x;
  if (i < n) Store<T>::put(out, i, 0.0f);
  if (lse && i < rows) lse[i] = -INFINITY;
}

// ---- host -------------------------------------------------------------------
enum class AttnPlan { kShort, kFew, kRows };
// rows of K and V in LDS for attn_short: its keys, and 32 query rows (half as
// many of both) for each of four wavefronts
constexpr int short_rows(int nt) { return 32 * nt + 64; }
struct AttnCut {
  AttnPlan plan;
  int splits, parts, key_tiles, row_tiles, tiles_each;
};
AttnCut cut_attn(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t E, size_t es, bool full) {
  AttnCut k{};
  const int64_t rows = Lq * (Hq / Hkv), heads = std::max<int64_t>(1, B * Hkv);
  int64_t splits = 1;
  // LDS bytes of a key's K and V, and of attn_short's workgroup
  const int64_t row = 2 * (attn_ep(E) * static_cast<int64_t>(es) + (es == 2 ? 32 : 16));
  const int64_t bytes = short_rows(static_cast<int>(cdiv(Lk, 32))) * row + 512;
  if (Lk <= 128 && (bytes <= 81920 || (bytes <= 163840 && heads * cdiv(rows, 128) < 256))) {
    // Taken where two workgroups fit a compute unit's LDS, or the chip would
    // not be full anyway and splitting the keys would cost a second launch.
    // us here and through the kernels below: 262144 rows, 5 heads of 64, 77 keys
    // 92, 131; 131072 rows, 64 heads of 64, 128 keys 173, 186 (16384 rows 28, 27);
    // of 96, 96 keys 34, 38; of 128, 64 keys 33, 34, 128 keys (one workgroup per
    // compute unit) 59, 44; 512 rows, 16 heads of 128, 128 keys 11.7, 11.6.
    // Row tiles of 32; a workgroup's four wavefronts take up to 32 each, so
    // that staging the keys is a small part, but all compute units get some.
    k.plan = AttnPlan::kShort;
    k.row_tiles = static_cast<int>(cdiv(rows, 32));
    const int64_t each = std::max<int64_t>(4, std::min<int64_t>(128, heads * k.row_tiles / 1024));
    splits = cdiv(k.row_tiles, each);
    k.tiles_each = static_cast<int>(cdiv(k.row_tiles, splits));
    k.splits = static_cast<int>(cdiv(k.row_tiles, k.tiles_each));
    return k;
  }
  if (rows <= 32) {
    // (8 x 8192 keys, 8 key heads of 128, cached: 4 rows each 48 us here, 62 as
    // row tiles of 128; 32 rows each 52, 63.)
    // Keys in tiles of 32, four at a time per workgroup. One workgroup per
    // compute unit reads at the memory's rate (64 heads, from memory: 128
    // workgroups 91 us, 256 65, 512 65, 1024 71); a second, shorter round costs
    // more than idle units do (160 heads of 4096: unsplit 69, split in two 85).
    k.plan = AttnPlan::kFew;
    k.key_tiles = static_cast<int>(cdiv(Lk, 32));
    splits = std::max<int64_t>(1, std::min<int64_t>(64, std::min<int64_t>(cdiv(k.key_tiles, 8), 256 / heads)));
    k.tiles_each = static_cast<int>(cdiv(cdiv(k.key_tiles, splits), 4) * 4);
    k.splits = static_cast<int>(cdiv(k.key_tiles, k.tiles_each));
  } else {
    // Row tiles of 128; where these are few the key axis is split, as often as
    // two workgroups per compute unit allow. (2048 keys, 16 heads, us split and
    // whole: bf16 of 128, 64 tiles 37, 68; 144 tiles, in three, 55, 69. fp32 of
    // 72, 1024 keys, 128 tiles 81, 124; 144 tiles, in three, 104, 126.) In two it
    // pays only where padded bf16 rows make the loads long (bf16 of 64, 256 tiles
    // 51, 48; of 72 68, 79; fp32 of 72, 240 tiles 146, 127).
    k.plan = AttnPlan::kRows;
    k.key_tiles = static_cast<int>(cdiv(Lk, es == 2 ? 64 : 32));
    k.row_tiles = static_cast<int>(cdiv(rows, 128));
    splits = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(k.key_tiles, 64), 512 / (heads * k.row_tiles)));
    if (splits == 2 && (full || es == 4)) splits = 1;
    k.tiles_each = static_cast<int>(cdiv(k.key_tiles, splits));
    k.splits = static_cast<int>(cdiv(k.key_tiles, k.tiles_each));
  }
  k.parts = k.splits > 1 ? k.splits : 0;
  return k;
}

template <typename T> AttnP<T> attn_params(const gspn_attn_args& a) {
  AttnP<T> p{};
  p.q = static_cast<const T*>(a.q.p); p.qm = {a.q.batch, a.q.row, a.q.head};
  p.k = static_cast<const T*>(a.k.p); p.km = {a.k.batch, a.k.row, a.k.head};
  p.v = static_cast<const T*>(a.v.p); p.vm = {a.v.batch, a.v.row, a.v.head};
  p.mask = a.mask; p.mask_batch = a.mask_batch;
  p.out = static_cast<T*>(a.out);
  p.lse = a.lse;
  p.B = a.B; p.Lq = a.Lq; p.Lk = a.Lk;
  p.Hq = static_cast<int>(a.Hq); p.Hkv = static_cast<int>(a.Hkv);
  p.share = p.Hq / p.Hkv;
  p.rows = a.Lq * p.share;
  p.E = static_cast<int>(a.E);
  p.c = a.scale * kLog2e;
  constexpr int per = 16 / sizeof(T);
  const bool whole = a.E % per == 0;
  p.wide_q = whole && wide_ok(a.q.p, 16, sizeof(T), {a.q.batch, a.q.row, a.q.head});
  p.wide_kv = whole && wide_ok(a.k.p, 16, sizeof(T), {a.k.batch, a.k.row, a.k.head}) &&
              wide_ok(a.v.p, 16, sizeof(T), {a.v.batch, a.v.row, a.v.head});
  p.wide_o = a.E % 8 == 0 && wide_ok(a.out, 16, sizeof(T), {});
  return p;
}

template <typename T>
hipError_t run(void (*kern)(AttnP<T>), const char* name, int bytes, int64_t grid, const AttnP<T>& p,
               hipStream_t stream, Tracer* tr) {
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  tr->before(stream, name, p.B * p.Hkv);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), bytes, stream, p);
  tr->after(stream);
  return hipGetLastError();
}

template <typename T, int EP, bool FULL>
hipError_t attn_plan_run(AttnP<T>& p, const AttnCut& k, hipStream_t stream, Tracer* tr) {
  constexpr int row = 2 * tile_pitch<T, EP>();   // LDS bytes of a key's K and V
  const int64_t heads = p.B * p.Hkv;
  if (k.plan == AttnPlan::kShort) {
    const int nt = static_cast<int>(cdiv(p.Lk, 32)), bytes = short_rows(nt) * row;
    auto kern = nt == 1 ? attn_short_kernel<T, EP, 1, FULL> : nt == 2 ? attn_short_kernel<T, EP, 2, FULL>
              : nt == 3 ? attn_short_kernel<T, EP, 3, FULL> : attn_short_kernel<T, EP, 4, FULL>;
    return run<T>(kern, "attn_short", bytes, heads * k.splits, p, stream, tr);
  }
  if (k.plan == AttnPlan::kFew)
    return run<T>(attn_few_kernel<T, EP, FULL>, "attn_few", 128 * row, heads * k.splits, p, stream, tr);
  const int64_t grid = heads * k.splits * k.row_tiles;
  if constexpr (sizeof(T) == 2) return run<T>(attn_wide_kernel<EP, FULL>, "attn_wide", 128 * row, grid, p, stream, tr);
  else return run<T>(attn_fwd_kernel<EP, FULL>, "attn_fwd", 32 * row, grid, p, stream, tr);
}

template <typename T, int EP>
hipError_t attn_ep_run(const gspn_attn_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  AttnP<T> p = attn_params<T>(a);
  // whole 16-byte pieces everywhere and no padding of the head
  const bool full = p.E == EP && p.wide_q && p.wide_kv && p.wide_o;
  const AttnCut k = cut_attn(a.B, a.Lq, a.Lk, a.Hq, a.Hkv, a.E, sizeof(T), full);
  p.splits = k.splits; p.key_tiles = k.key_tiles; p.row_tiles = k.row_tiles;
  p.tiles_each = k.tiles_each;
  const int64_t total = p.B * p.Hkv * p.rows;
  if (k.parts) {
    p.part = static_cast<float*>(ws);
    p.part_ml = p.part + k.parts * total * EP;
  }
  hipError_t e;
  if (full) e = attn_plan_run<T, EP, true>(p, k, stream, tr);
  else e = attn_plan_run<T, EP, false>(p, k, stream, tr);
  if (e != hipSuccess || !k.parts) return e;
  return run<T>(attn_join_kernel<T, EP>, "attn_join", 0, cdiv(total, kThreads / 64), p, stream, tr);
}

template <typename T> hipError_t attn_dt(const gspn_attn_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.Lk == 0) {
    const int64_t rows = a.B * a.Lq * a.Hq, n = rows * a.E;
    tr->before(stream, "attn_empty", a.B);
    const hipError_t e = in_parts(cdiv(n, kThreads), [&](int64_t first, unsigned count) {
      hipLaunchKernelGGL(attn_empty_kernel<T>, dim3(count), dim3(kThreads), 0, stream, static_cast<T*>(a.out), n,
                         a.lse, rows, first);
    });
    tr->after(stream);
    return e;
  }
  switch (attn_ep(a.E)) {
    case 32: return attn_ep_run<T, 32>(a, ws, stream, tr);
    case 64: return attn_ep_run<T, 64>(a, ws, stream, tr);
    case 96: return attn_ep_run<T, 96>(a, ws, stream, tr);
    default: return attn_ep_run<T, 128>(a, ws, stream, tr);
  }
}

}  // namespace

size_t attn_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t E) {
  if (B == 0 || Lq == 0 || Lk == 0) return 0;
  size_t most = 0;
  // the larger of the two element types' needs; a `full` call needs no more
  for (const size_t es : {size_t(2), size_t(4)}) {
    const AttnCut k = cut_attn(B, Lq, Lk, Hq, Hkv, E, es, false);
    most = std::max(most, static_cast<size_t>(k.parts * B * Lq * Hq * (attn_ep(E) + 2)) * sizeof(float));
  }
  return most;
}

hipError_t launch_attn(const gspn_attn_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return attn_dt<float>(a, ws, stream, tr);
  return attn_dt<bf16_t>(a, ws, stream, tr);
}

}  // namespace gspn
