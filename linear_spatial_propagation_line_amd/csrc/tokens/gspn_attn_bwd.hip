// Cross attention, backward. With P from the forward pass's lse, dP = dO V^T and
// D[row] = sum_e grad_out out (= sum over keys of P dP):
//
//   dV = P^T dO,   dS = P (dP - D),   dQ = scale dS K,   dK = scale dS^T Q
//
// Two passes recompute P: one owns rows and walks the keys, one owns keys (a
// wavefront 32 of them, their K and V fragments and their dK, dV in registers)
// and walks the rows. Each sum then has one owner, so nothing is added
// atomically; where few keys leave the chip idle, the rows of the second
// pass are split and the parts added in order.
#include "gspn_attn.hpp"

namespace gspn {

namespace {

constexpr int kThreads = 256;

template <typename T> struct BwdP {
  const T *q, *k, *v, *gy, *out;
  RowMap qm, km, vm, gm;
  const uint8_t* mask;
  int64_t mask_batch;
  const float* lse;
  float* delta;        // [B][Hq][Lq]
  T *dq, *dk, *dv;
  float* part;         // [2][splits][B][Lk][Hkv][E], or null
  int64_t B, Lq, Lk, rows;
  int Hq, Hkv, share, E, splits, key_tiles, row_tiles, tiles_each;
  float c, scale;      // scale * log2(e), scale
  uint32_t block0;     // attn_delta: first workgroup of this launch
  bool wide_q, wide_kv, wide_g, wide_dq, wide_dkv, full;
};

// D of a row is sum_e grad_out out = sum_j P dP. The first takes the rounding of
// out with it, which is large against score gradients that are small differences
// of few terms (bf16, rms of dQ's error in units of its own rounding: 2 keys 1.6,
// 17 keys 1.4, 77 keys 1.06; 2048 keys 1.00). The second needs all of a row's
// keys before the first score gradient. So attn_dq walks the kept keys twice
// where they lie in at most this many tiles of 32, and leaves D for attn_dkv; the
// launch that reads grad_out and out falls away where no entry can have more
// (262144 rows, 77 keys, 5 heads of 64, training step 464 us, 550 by out; with
// both 572). fp32 rounds out as finely as all else: one tile, which costs nothing.
template <typename T> constexpr int exact_tiles() { return sizeof(T) == 2 ? 4 : 1; }

// delta[b][h][q] = sum_e grad_out out: 16 lanes per row
template <typename T>
__global__ __launch_bounds__(kThreads) void attn_delta_kernel(BwdP<T> a) {
  const int64_t i = ((static_cast<int64_t>(a.block0) + blockIdx.x) * kThreads + threadIdx.x) / 16;
  const int64_t total = a.B * a.Hq * a.Lq;
  const int64_t ic = i < total ? i : total - 1;
  const int64_t q = ic % a.Lq, bh = ic / a.Lq, b = bh / a.Hq, h = bh - b * a.Hq;
  const T* g = a.gy + b * a.gm.batch + q * a.gm.row + h * a.gm.head;
  const T* o = a.out + ((b * a.Lq + q) * a.Hq + h) * a.E;
  float s = 0.0f;
  for (int e = threadIdx.x % 16; e < a.E; e += 16) s = __builtin_fmaf(ld1(g + e), ld1(o + e), s);
#pragma unroll
  for (int m = 8; m >= 1; m /= 2) s += __shfl_xor(s, m);
  if (i < total && threadIdx.x % 16 == 0) a.delta[i] = s;
}

// ---- dK, dV: 128 keys per workgroup, rows 32 at a time through LDS ----------
// Four products per tile, S^T and dP^T from the keys' side, then dV and dK. A
// tile's products wait for its exponentials and for LDS (47 % of the cycles are
// waits, the matrix units work for 44 %). 2x4096x2048 with ragged masks, 16
// heads of 128 on 4, bf16: 460 us.
// Results and fragments of K and V are 6 E registers; where that leaves no
// room for two wavefronts per SIMD the fragments of V stay in LDS (with them
// in registers the loop spills; training step, 4x2048x1024, 16 heads of 96:
// 359 us against 347).
template <typename T, int EP> constexpr bool dkv_v_in_lds() { return EP * sizeof(T) >= 192; }
template <typename T, int EP> constexpr int dkv_lds() {
  return (4 * 32 + (dkv_v_in_lds<T, EP>() ? 128 : 0)) * tile_pitch<T, EP>() + 2 * 64 * 4;
}
template <typename T, int EP, bool FULL>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void attn_dkv_kernel(BwdP<T> a) {
  extern __shared__ __align__(16) char lds[];
  constexpr int TR = 32;
  // two tiles of rows (Q, grad_out, and their lse and delta), one being
  // computed with while the next is written: one barrier per tile
  constexpr int kTile = 2 * TR * tile_pitch<T, EP>() + 2 * TR * 4;
  char* vt = lds + 2 * kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, hh = lane >> 5;
  uint32_t blk = xcd_block(blockIdx.x, gridDim.x);
  const int kt = static_cast<int>(blk % a.key_tiles);
  blk /= a.key_tiles;
  const int split = static_cast<int>(blk % a.splits);
  const int64_t bh = blk / a.splits, b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const int64_t key = static_cast<int64_t>(kt) * 128 + wave * 32 + (lane & 31);
  const bool in = key < a.Lk;
  const int64_t kc = in ? key : a.Lk - 1;
  const bool keep = in && (!a.mask || a.mask[b * a.mask_batch + kc] != 0);

  typename Mma<T>::Frag kf[EP / Mma<T>::kChunk], vf[EP / Mma<T>::kChunk];
  row_frags<T, EP, FULL>(a.k + b * a.km.batch + kc * a.km.row + hk * a.km.head, keep, a.E, a.wide_kv, kf);
  row_frags<T, EP, FULL>(a.v + b * a.vm.batch + kc * a.vm.row + hk * a.vm.head, keep, a.E, a.wide_kv, vf);
  if constexpr (dkv_v_in_lds<T, EP>()) {
#pragma unroll
    for (int j = 0; j < EP / Mma<T>::kChunk; ++j)
      *reinterpret_cast<typename Mma<T>::Frag*>(vt + (wave * 32 + (lane & 31)) * tile_pitch<T, EP>() + j * 32 + hh * 16) = vf[j];
  }

  f32x16 dk[EP / 32] = {}, dv[EP / 32] = {};
  // nothing to add up where the workgroup's keys are all dropped
  const int t_first = split * a.tiles_each;
  const int t_last = __syncthreads_or(keep) ? min(t_first + a.tiles_each, a.row_tiles) : t_first;
  Stage<T, EP, TR, kThreads> qs, gs;
  float stat = 0.0f;
  auto fetch = [&](int t) {
    const int64_t r0 = static_cast<int64_t>(t) * TR;
    const RowTile rows(a, hk, static_cast<uint32_t>(r0));
    qs.template load<FULL>(tid, a.E, a.wide_q, [&](int i) {
      const QRow w = rows.at(i);
      return a.q + b * a.qm.batch + w.q * a.qm.row + w.h * a.qm.head;
    });
    gs.template load<FULL>(tid, a.E, a.wide_g, [&](int i) {
      const QRow w = rows.at(i);
      return a.gy + b * a.gm.batch + w.q * a.gm.row + w.h * a.gm.head;
    });
    if (tid < 2 * TR) {
      // rows past the end get lse = +inf, hence P = 0; the rows of one key
      // head are adjacent in lse and delta
      const int64_t r = r0 + (tid & (TR - 1));
      const int64_t at = (b * a.Hq + hk * a.share) * a.Lq + r;
      stat = tid < TR ? (r < a.rows ? a.lse[at] * kLog2e : INFINITY) : (r < a.rows ? a.delta[at] : 0.0f);
    }
  };
  auto put = [&](int t) {
    char* to = lds + (t & 1) * kTile;
    const int64_t left = a.rows - static_cast<int64_t>(t) * TR;
    qs.template write<FULL>(to, tid, a.E, [&](int i) { return i < left; });
    gs.template write<FULL>(to + TR * tile_pitch<T, EP>(), tid, a.E, [&](int i) { return i < left; });
    if (tid < 2 * TR) reinterpret_cast<float*>(to + 2 * TR * tile_pitch<T, EP>())[tid] = stat;
  };
  if (t_first < t_last) {
    fetch(t_first);
    put(t_first);
  }
  lds_barrier();
  for (int t = t_first; t < t_last; ++t) {
    const char* qt = lds + (t & 1) * kTile;
    const char* gt = qt + TR * tile_pitch<T, EP>();
    const float* st = reinterpret_cast<const float*>(gt + TR * tile_pitch<T, EP>());
    if (t + 1 < t_last) fetch(t + 1);
    // the softmax of the tile between the two products, so that lse and delta
    // are not held at once
    const f32x16 x = tile_dot<T, EP>(qt, 0, kf, lane);
    float p[16], ds[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)   // a dropped key's column is finite (zeros) and not stored
      p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], a.c, -st[(i & 3) + 8 * (i >> 2) + 4 * hh]));
    f32x16 y;
    if constexpr (dkv_v_in_lds<T, EP>()) {
      y = f32x16{};
#pragma unroll
      for (int j = 0; j < EP / Mma<T>::kChunk; ++j) {
        y = Mma<T>::mma(tile_frag<T, EP>(gt, 0, j, lane), tile_frag<T, EP>(vt, wave * 32, j, lane), y);
        if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // not all fragments at once
      }
    } else {
      y = tile_dot<T, EP>(gt, 0, vf, lane);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 16; ++i) ds[i] = p[i] * (y[i] - st[TR + (i & 3) + 8 * (i >> 2) + 4 * hh]);
    tile_accum<EP>(gt, 0, p, dv, lane, T{});
    tile_accum<EP>(qt, 0, ds, dk, lane, T{});
    if (t + 1 < t_last) put(t + 1);
    lds_barrier();
  }
  const int64_t at = ((b * a.Lk + key) * a.Hkv + hk) * a.E;
  if (a.part) {
    const int64_t n = a.B * a.Lk * a.Hkv * a.E;
    store_col<float, EP, FULL>(a.part + split * n + at, in, keep, a.E, a.E % 8 == 0, dk, a.scale, lane);
    store_col<float, EP, FULL>(a.part + (a.splits + split) * n + at, in, keep, a.E, a.E % 8 == 0, dv, 1.0f, lane);
  } else {
    store_col<T, EP, FULL>(a.dk + at, in, keep, a.E, a.wide_dkv, dk, a.scale, lane);
    store_col<T, EP, FULL>(a.dv + at, in, keep, a.E, a.wide_dkv, dv, 1.0f, lane);
  }
}

// the row splits' parts of dK and dV, added in order
template <typename T>
__global__ __launch_bounds__(kThreads) void attn_dkv_join_kernel(BwdP<T> a) {
  const int64_t n = a.B * a.Lk * a.Hkv * a.E;
  const int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x;
  if (i >= 2 * n) return;
  const bool second = i >= n;
  const int64_t k = second ? i - n : i;
  const float* p = a.part + (second ? a.splits * n : 0) + k;
  float s = 0.0f;
  for (int j = 0; j < a.splits; ++j) s += p[j * n];
  Store<T>::put(second ? a.dv : a.dk, k, s);
}

// ---- dQ: 128 rows per workgroup, keys 32 at a time through LDS --------------
// Bound by the products (the matrix units work half of the time): 250 us at the
// same size.
template <typename T, int EP, bool FULL>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void attn_dq_kernel(BwdP<T> a) {
  extern __shared__ __align__(16) char lds[];
  constexpr int TK = 32, kTile = 2 * TK * tile_pitch<T, EP>();
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rts = static_cast<int>((a.rows + 127) / 128);
  const uint32_t blk = blockIdx.x;
  const int rt = static_cast<int>(blk % rts);
  const int64_t bh = blk / rts, b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const int64_t r = static_cast<int64_t>(rt) * 128 + wave * 32 + (lane & 31);
  const bool row_ok = r < a.rows;
  const QRow w = q_row(a, hk, static_cast<uint32_t>(r));
  typename Mma<T>::Frag qf[EP / Mma<T>::kChunk], gf[EP / Mma<T>::kChunk];
  row_frags<T, EP, FULL>(a.q + b * a.qm.batch + w.q * a.qm.row + w.h * a.qm.head, true, a.E, a.wide_q, qf);
  row_frags<T, EP, FULL>(a.gy + b * a.gm.batch + w.q * a.gm.row + w.h * a.gm.head, true, a.E, a.wide_g, gf);
  const int64_t at = (b * a.Hq + w.h) * a.Lq + w.q;
  const float lse = row_ok ? a.lse[at] * kLog2e : INFINITY;

  const T* kp = a.k + b * a.km.batch + hk * a.km.head;
  const T* vp = a.v + b * a.vm.batch + hk * a.vm.head;
  const uint8_t* mp = a.mask ? a.mask + b * a.mask_batch : nullptr;
  auto kept = [&](int64_t key) { return key < a.Lk && (!mp || mp[key] != 0); };
  f32x16 dq[EP / 32] = {};
  Stage<T, EP, TK, kThreads> ks, vs;
  int64_t k_lo, k_hi;
  key_range(mp, a.Lk, tid, &k_lo, &k_hi);
  const int t_first = static_cast<int>(k_lo / TK), t_last = static_cast<int>((k_hi + TK - 1) / TK);
  bool keep = false;         // of key lane % 32 of the tile on its way
  uint32_t bits = 0, next = 0;
  auto fetch = [&](int t) {
    const int64_t k0 = static_cast<int64_t>(t) * TK;
    keep = kept(k0 + (lane & 31));
    ks.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return kp + (k0 + i < a.Lk ? k0 + i : a.Lk - 1) * a.km.row; });
    vs.template load<FULL>(tid, a.E, a.wide_kv, [&](int i) { return vp + (k0 + i < a.Lk ? k0 + i : a.Lk - 1) * a.vm.row; });
  };
  auto put = [&](int t) {
    char* to = lds + (t & 1) * kTile;
    next = static_cast<uint32_t>(__ballot(keep));
    ks.template write<FULL>(to, tid, a.E, [&](int i) { return (next >> i) & 1u; });
    vs.template write<FULL>(to + TK * tile_pitch<T, EP>(), tid, a.E, [&](int i) { return (next >> i) & 1u; });
  };
  // use(K tile, V tile) for every tile that keeps a key
  auto walk = [&](auto&& use) {
    if (t_first < t_last) {
      fetch(t_first);
      put(t_first);
    }
    lds_barrier();
    for (int t = t_first; t < t_last; ++t) {
      const char* kt = lds + (t & 1) * kTile;
      bits = next;
      if (t + 1 < t_last) fetch(t + 1);
      if (bits != 0) use(kt, kt + TK * tile_pitch<T, EP>());
      if (t + 1 < t_last) put(t + 1);
      lds_barrier();
    }
  };
  auto probabilities = [&](const char* kt, float (&p)[16]) {
    const f32x16 x = tile_dot<T, EP>(kt, 0, qf, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = x[i];
    drop_keys(p, bits, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], a.c, -lse));
  };
  float delta;
  if (t_last - t_first > exact_tiles<T>()) {
    delta = row_ok ? a.delta[at] : 0.0f;
  } else {
    float sum = 0.0f;
    walk([&](const char* kt, const char* vt) {
      float p[16];
      probabilities(kt, p);
      const f32x16 y = tile_dot<T, EP>(vt, 0, gf, lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(p[i], y[i], sum);
    });
    delta = column_sum(sum);
    if (row_ok && lane < 32) a.delta[at] = delta;
  }
  walk([&](const char* kt, const char* vt) {
    float ds[16];
    probabilities(kt, ds);
    const f32x16 y = tile_dot<T, EP>(vt, 0, gf, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i) ds[i] *= y[i] - delta;
    tile_accum<EP>(kt, 0, ds, dq, lane, T{});
  });
  store_col<T, EP, FULL>(a.dq + ((b * a.Lq + w.q) * a.Hq + w.h) * a.E, row_ok, true, a.E, a.wide_dq, dq, a.scale, lane);
}

// ---- host -------------------------------------------------------------------
struct BwdCut {
  int key_tiles, row_tiles, splits, tiles_each;
};
// Row splits of the dK, dV pass: as many as the workgroups that run at once
// allow, two per compute unit, one for fp32. (2048 rows, 16 heads of 128, bf16,
// whole training step, us split and whole: 32 groups 81, 206; 128 groups 166,
// 257; 240 groups in two 272, 315, in three 303. fp32 of 64, 1024 rows, 64 groups: in
// four 160, in eight 158, whole 278.)
BwdCut cut_bwd(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, size_t es) {
  BwdCut k;
  k.key_tiles = static_cast<int>(cdiv(Lk, 128));
  k.row_tiles = static_cast<int>(cdiv(Lq * (Hq / Hkv), 32));
  const int64_t groups = std::max<int64_t>(1, B * Hkv * k.key_tiles);
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(k.row_tiles, (es == 2 ? 512 : 256) / groups));
  k.tiles_each = static_cast<int>(cdiv(std::max(1, k.row_tiles), splits));
  k.splits = static_cast<int>(cdiv(std::max(1, k.row_tiles), k.tiles_each));
  return k;
}

template <typename K> hipError_t more_lds(K kern, int bytes) {
  if (bytes <= 65536) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int EP>
hipError_t bwd_ep(const BwdP<T>& p, hipStream_t stream, Tracer* tr) {
  hipError_t e;
  if (p.rows > 0 && cdiv(p.Lk, 32) > exact_tiles<T>()) {   // some entry may keep keys in more tiles
    tr->before(stream, "attn_delta", p.B);
    e = in_parts(cdiv(p.B * p.Hq * p.Lq, kThreads / 16), [&](int64_t first, unsigned count) {
      BwdP<T> d = p;
      d.block0 = static_cast<uint32_t>(first);
      hipLaunchKernelGGL(attn_delta_kernel<T>, dim3(count), dim3(kThreads), 0, stream, d);
    });
    tr->after(stream);
    if (e != hipSuccess) return e;
  }
  if (p.rows > 0) {
    auto kern = p.full ? attn_dq_kernel<T, EP, true> : attn_dq_kernel<T, EP, false>;
    constexpr int bytes = 4 * 32 * tile_pitch<T, EP>();
    if ((e = more_lds(kern, bytes)) != hipSuccess) return e;
    tr->before(stream, "attn_dq", p.B * p.Hkv);
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(p.B * p.Hkv * cdiv(p.rows, 128))),
                       dim3(kThreads), bytes, stream, p);
    tr->after(stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (p.Lk > 0) {
    auto kern = p.full ? attn_dkv_kernel<T, EP, true> : attn_dkv_kernel<T, EP, false>;
    constexpr int bytes = dkv_lds<T, EP>();
    if ((e = more_lds(kern, bytes)) != hipSuccess) return e;
    tr->before(stream, "attn_dkv", p.B * p.Hkv);
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(p.B * p.Hkv * p.splits * p.key_tiles)),
                       dim3(kThreads), bytes, stream, p);
    tr->after(stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (p.part) {
      tr->before(stream, "attn_dkv_join", p.B * p.Hkv);
      hipLaunchKernelGGL(attn_dkv_join_kernel<T>,
                         dim3(static_cast<unsigned>(cdiv(2 * p.B * p.Lk * p.Hkv * p.E, kThreads))),
                         dim3(kThreads), 0, stream, p);
      tr->after(stream);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

template <typename T>
hipError_t bwd_dt(const gspn_attn_args& a, const gspn_attn_grads& g, void* ws, hipStream_t stream,
                  Tracer* tr) {
  BwdP<T> p{};
  const BwdCut k = cut_bwd(a.B, a.Lq, a.Lk, a.Hq, a.Hkv, sizeof(T));
  p.q = static_cast<const T*>(a.q.p); p.qm = {a.q.batch, a.q.row, a.q.head};
  p.k = static_cast<const T*>(a.k.p); p.km = {a.k.batch, a.k.row, a.k.head};
  p.v = static_cast<const T*>(a.v.p); p.vm = {a.v.batch, a.v.row, a.v.head};
  p.gy = static_cast<const T*>(g.grad_out.p);
  p.gm = {g.grad_out.batch, g.grad_out.row, g.grad_out.head};
  p.out = static_cast<const T*>(a.out);
  p.mask = a.mask; p.mask_batch = a.mask_batch;
  p.lse = a.lse;
  p.dq = static_cast<T*>(g.q); p.dk = static_cast<T*>(g.k); p.dv = static_cast<T*>(g.v);
  p.B = a.B; p.Lq = a.Lq; p.Lk = a.Lk;
  p.Hq = static_cast<int>(a.Hq); p.Hkv = static_cast<int>(a.Hkv);
  p.share = p.Hq / p.Hkv;
  p.rows = a.Lq * p.share;
  p.E = static_cast<int>(a.E);
  p.splits = k.splits; p.key_tiles = k.key_tiles; p.row_tiles = k.row_tiles;
  p.tiles_each = k.tiles_each;
  p.scale = a.scale;
  p.c = a.scale * kLog2e;
  p.delta = static_cast<float*>(ws);
  if (k.splits > 1)
    p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + up256(static_cast<size_t>(a.B * a.Hq * a.Lq) * 4));
  constexpr int per = 16 / sizeof(T);
  const bool whole = a.E % per == 0, eight = a.E % 8 == 0;
  const size_t es = sizeof(T);
  p.wide_q = whole && wide_ok(a.q.p, 16, es, {a.q.batch, a.q.row, a.q.head});
  p.wide_kv = whole && wide_ok(a.k.p, 16, es, {a.k.batch, a.k.row, a.k.head}) &&
              wide_ok(a.v.p, 16, es, {a.v.batch, a.v.row, a.v.head});
  p.wide_g = whole && wide_ok(p.gy, 16, es, {p.gm.batch, p.gm.row, p.gm.head});
  p.wide_dq = eight && wide_ok(p.dq, 16, es, {});
  p.wide_dkv = eight && wide_ok(p.dk, 16, es, {}) && wide_ok(p.dv, 16, es, {});
  // whole 16-byte pieces everywhere and no padding of the head
  p.full = p.E == attn_ep(a.E) && p.wide_q && p.wide_kv && p.wide_g && p.wide_dq && p.wide_dkv;
  switch (attn_ep(a.E)) {
    case 32: return bwd_ep<T, 32>(p, stream, tr);
    case 64: return bwd_ep<T, 64>(p, stream, tr);
    case 96: return bwd_ep<T, 96>(p, stream, tr);
    default: return bwd_ep<T, 128>(p, stream, tr);
  }
}

}  // namespace

size_t attn_bwd_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t E) {
  if (B == 0) return 0;
  const BwdCut k = cut_bwd(B, Lq, Lk, Hq, Hkv, 2);
  size_t n = up256(static_cast<size_t>(B * Hq * Lq) * sizeof(float));
  if (k.splits > 1) n += static_cast<size_t>(2 * k.splits * B * Lk * Hkv * E) * sizeof(float);
  return n;
}

hipError_t launch_attn_bwd(const gspn_attn_args& a, const gspn_attn_grads& g, void* ws,
                           hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return bwd_dt<float>(a, g, ws, stream, tr);
  return bwd_dt<bf16_t>(a, g, ws, stream, tr);
}

}  // namespace gspn
