// Cross attention, forward: out = softmax(scale q k^T over the kept keys) v.
//
// One pass over the keys with the running maximum and sum of the softmax: a
// wavefront holds 32 query rows (their fragments and the 32 x E result stay
// in registers) and takes 32 keys at a time, X^T = K Q^T, probabilities, then
// O^T += V^T P^T, with one lane per query row, so that the row's maximum and
// sum need one exchange between half-wavefronts. The query heads that share
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

// WR wavefronts take different rows; with WR = 1 the four wavefronts take
// different keys of the same 32 rows, each as a split of its own.
template <typename T, int EP, int WR, int TK>
__global__ __launch_bounds__(kThreads) void attn_fwd_kernel(AttnP<T> a) {
  extern __shared__ __align__(16) char lds[];
  constexpr int kKeysEach = WR == 1 ? TK / 4 : TK;   // keys of a tile that one wavefront takes
  char* kt = lds;
  char* vt = lds + TK * tile_pitch<T, EP>();
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t blk = blockIdx.x;
  const int rt = static_cast<int>(blk % a.row_tiles);
  blk /= a.row_tiles;
  const int split = static_cast<int>(blk % a.splits);
  const int64_t bh = blk / a.splits, b = bh / a.Hkv;
  const int hk = static_cast<int>(bh - b * a.Hkv);

  const int64_t r = (static_cast<int64_t>(rt) * WR + (WR == 1 ? 0 : wave)) * 32 + (lane & 31);
  const bool row_ok = r < a.rows;
  const int64_t rc = row_ok ? r : a.rows - 1;
  const int64_t hs = rc / a.Lq, qi = rc - hs * a.Lq;
  const int64_t h = hk * a.share + hs;

  typename Mma<T>::Frag qf[EP / Mma<T>::kChunk];
  row_frags<T, EP>(a.q + b * a.qm.batch + qi * a.qm.row + h * a.qm.head, row_ok, a.E, a.wide_q, qf);

  const T* kp = a.k + b * a.km.batch + hk * a.km.head;
  const T* vp = a.v + b * a.vm.batch + hk * a.vm.head;
  const uint8_t* mp = a.mask ? a.mask + b * a.mask_batch : nullptr;
  auto kept = [&](int64_t key) { return key < a.Lk && (!mp || mp[key] != 0); };

  f32x16 o[EP / 32] = {};
  float m = -INFINITY, l = 0.0f;
  const int t_first = split * a.tiles_each;
  const int t_last = t_first + a.tiles_each < a.key_tiles ? t_first + a.tiles_each : a.key_tiles;

  Stage<T, EP, TK, kThreads> ks, vs;
  auto fetch = [&](int t) {
    const int64_t k0 = static_cast<int64_t>(t) * TK;
    ks.load(tid, a.E, a.wide_kv, [&](int i) { return k0 + i < a.Lk ? kp + (k0 + i) * a.km.row : nullptr; });
    vs.load(tid, a.E, a.wide_kv, [&](int i) { return k0 + i < a.Lk ? vp + (k0 + i) * a.vm.row : nullptr; });
  };
  if (t_first < t_last) fetch(t_first);
  for (int t = t_first; t < t_last; ++t) {
    const int64_t k0 = static_cast<int64_t>(t) * TK;
    ks.write(kt, tid, [&](int i) { return kept(k0 + i); });
    vs.write(vt, tid, [&](int i) { return kept(k0 + i); });
    __syncthreads();
    if (t + 1 < t_last) fetch(t + 1);
#pragma unroll
    for (int s = 0; s < kKeysEach / 32; ++s) {
      const int row0 = (WR == 1 ? wave * kKeysEach : 0) + s * 32;
      const uint32_t bits = static_cast<uint32_t>(__ballot(kept(k0 + row0 + (lane & 31))));
      if (bits == 0) continue;
      const f32x16 x = tile_dot<T, EP>(kt, row0, qf, lane);
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = x[i];
      if (bits != 0xffffffffu) {
        const uint32_t mine = bits >> (4 * (lane >> 5));
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = (mine >> ((i & 3) + 8 * (i >> 2))) & 1u ? w[i] : -INFINITY;
      }
      float top = w[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, w[i]);
      top = fmaxf(top, other_half(top)) * a.c;
      if (__any(top > m)) {
        const float mn = fmaxf(m, top);
        const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
        m = mn;
        l *= f;
#pragma unroll
        for (int et = 0; et < EP / 32; ++et) o[et] *= f;
      }
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(w[i], a.c, -base));
        l += w[i];
      }
      tile_accum<EP>(vt, row0, w, o, lane, T{});
    }
    __syncthreads();
  }
  l += other_half(l);
  const int64_t n = a.rows;
  if (WR == 1 || a.splits > 1) {
    const int64_t sp = WR == 1 ? split * 4 + wave : split;
    const int64_t at = (sp * a.B * a.Hkv + bh) * n + r;
    store_col<float, EP>(a.part + at * EP, row_ok, true, EP, true, o, 1.0f, lane);
    if (row_ok && lane < 32) {
      a.part_ml[at * 2] = m;
      a.part_ml[at * 2 + 1] = l;
    }
  } else {
    const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    store_col<T, EP>(a.out + ((b * a.Lq + qi) * a.Hq + h) * a.E, row_ok, true, a.E, a.wide_o, o, f, lane);
    if (a.lse && row_ok && lane < 32)
      a.lse[(b * a.Hq + h) * a.Lq + qi] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

// Joins the splits of a row: one wavefront per row, lanes over the values.
template <typename T>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnP<T> a, int parts, int EP) {
  const int lane = threadIdx.x & 63;
  const int64_t i = blockIdx.x * int64_t(kThreads / 64) + (threadIdx.x >> 6);
  const int64_t total = a.B * a.Hkv * a.rows;
  if (i >= total) return;
  const int64_t bh = i / a.rows, r = i - bh * a.rows;
  const int64_t b = bh / a.Hkv, hs = r / a.Lq, qi = r - hs * a.Lq;
  const int64_t h = (bh - b * a.Hkv) * a.share + hs;
  float m = -INFINITY;
  for (int s = 0; s < parts; ++s) m = fmaxf(m, a.part_ml[(s * total + i) * 2]);
  const float base = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, v[2] = {0.0f, 0.0f};
  for (int s = 0; s < parts; ++s) {
    const int64_t at = s * total + i;
    const float f = __builtin_amdgcn_exp2f(a.part_ml[at * 2] - base);
    l = __builtin_fmaf(f, a.part_ml[at * 2 + 1], l);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lane + 64 * k < EP) v[k] = __builtin_fmaf(f, a.part[at * EP + lane + 64 * k], v[k]);
  }
  const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane + 64 * k < a.E)
      Store<T>::put(a.out, ((b * a.Lq + qi) * a.Hq + h) * a.E + lane + 64 * k, v[k] * f);
  if (a.lse && lane == 0)
    a.lse[(b * a.Hq + h) * a.Lq + qi] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// out = 0, lse = -inf when there is no key at all
template <typename T>
__global__ __launch_bounds__(kThreads) void attn_empty_kernel(T* out, int64_t n, float* lse, int64_t rows) {
  const int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x;
  if (i < n) Store<T>::put(out, i, 0.0f);
  if (lse && i < rows) lse[i] = -INFINITY;
}

// ---- host -------------------------------------------------------------------
struct AttnCut {
  bool few;          // at most 32 rows share a key head: wavefronts over keys
  int tk, splits, parts, key_tiles, row_tiles, tiles_each;
};
// With few rows the wavefronts take different keys; the key axis is split
// further until about two workgroups per compute unit run.
AttnCut cut_attn(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, size_t es) {
  AttnCut k{};
  const int64_t rows = Lq * (Hq / Hkv);
  k.few = rows <= 32;
  k.tk = k.few ? 128 : (es == 2 ? 64 : 32);
  k.key_tiles = static_cast<int>(cdiv(Lk, k.tk));
  k.row_tiles = static_cast<int>(cdiv(rows, k.few ? 32 : 128));
  const int64_t groups = std::max<int64_t>(1, B * Hkv * k.row_tiles);
  int64_t splits = 1;
  if (groups < 256) splits = std::min<int64_t>(k.key_tiles, cdiv(512, groups));
  splits = std::max<int64_t>(1, std::min<int64_t>(splits, 64));
  k.tiles_each = static_cast<int>(cdiv(std::max(1, k.key_tiles), splits));
  k.splits = static_cast<int>(cdiv(std::max(1, k.key_tiles), k.tiles_each));
  k.parts = k.few ? 4 * k.splits : (k.splits > 1 ? k.splits : 0);
  return k;
}

template <typename T> AttnP<T> attn_params(const gspn_attn_args& a, const AttnCut& k) {
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
  p.splits = k.splits; p.key_tiles = k.key_tiles; p.row_tiles = k.row_tiles;
  p.tiles_each = k.tiles_each;
  p.c = a.scale * kLog2e;
  constexpr int per = 16 / sizeof(T);
  const bool whole = a.E % per == 0;
  p.wide_q = whole && wide_ok(a.q.p, 16, sizeof(T), {a.q.batch, a.q.row, a.q.head});
  p.wide_kv = whole && wide_ok(a.k.p, 16, sizeof(T), {a.k.batch, a.k.row, a.k.head}) &&
              wide_ok(a.v.p, 16, sizeof(T), {a.v.batch, a.v.row, a.v.head});
  p.wide_o = a.E % 8 == 0 && wide_ok(a.out, 16, sizeof(T), {});
  return p;
}

template <typename T, int EP, int WR, int TK>
hipError_t run_fwd(const AttnP<T>& p, hipStream_t stream, Tracer* tr) {
  auto kern = attn_fwd_kernel<T, EP, WR, TK>;
  constexpr int bytes = 2 * TK * tile_pitch<T, EP>();
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  const int64_t grid = p.B * p.Hkv * p.splits * p.row_tiles;
  tr->before(stream, "attn_fwd", p.B * p.Hkv);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), bytes, stream, p);
  tr->after(stream);
  return hipGetLastError();
}

template <typename T, int EP>
hipError_t attn_ep_run(const gspn_attn_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  const AttnCut k = cut_attn(a.B, a.Lq, a.Lk, a.Hq, a.Hkv, sizeof(T));
  AttnP<T> p = attn_params<T>(a, k);
  const int64_t total = p.B * p.Hkv * p.rows;
  if (k.parts) {
    p.part = static_cast<float*>(ws);
    p.part_ml = p.part + k.parts * total * EP;
  }
  hipError_t e = k.few ? run_fwd<T, EP, 1, 128>(p, stream, tr)
                       : run_fwd<T, EP, 4, sizeof(T) == 2 ? 64 : 32>(p, stream, tr);
  if (e != hipSuccess || !k.parts) return e;
  tr->before(stream, "attn_join", total);
  hipLaunchKernelGGL(attn_join_kernel<T>, dim3(static_cast<unsigned>(cdiv(total, kThreads / 64))),
                     dim3(kThreads), 0, stream, p, k.parts, EP);
  tr->after(stream);
  return hipGetLastError();
}

template <typename T> hipError_t attn_dt(const gspn_attn_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.Lk == 0) {
    const int64_t rows = a.B * a.Lq * a.Hq, n = rows * a.E;
    tr->before(stream, "attn_empty", a.B);
    hipLaunchKernelGGL(attn_empty_kernel<T>, dim3(static_cast<unsigned>(cdiv(n, kThreads))),
                       dim3(kThreads), 0, stream, static_cast<T*>(a.out), n, a.lse, rows);
    tr->after(stream);
    return hipGetLastError();
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
  for (const size_t es : {size_t(2), size_t(4)}) {   // the larger of the two element types' needs
    const AttnCut k = cut_attn(B, Lq, Lk, Hq, Hkv, es);
    most = std::max(most, static_cast<size_t>(k.parts * B * Lq * Hq * (attn_ep(E) + 2)) * sizeof(float));
  }
  return most;
}

hipError_t launch_attn(const gspn_attn_args& a, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return attn_dt<float>(a, ws, stream, tr);
  return attn_dt<bf16_t>(a, ws, stream, tr);
}

}  // namespace gspn
