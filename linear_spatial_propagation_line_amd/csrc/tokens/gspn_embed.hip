// Token embedding and its gradient.
//
//   out[t] = scale * weight[ids[t]],   dweight[v] = scale * sum_{t: ids[t] = v} grad_out[t]
//
// Both are bound by memory: a multiplication for two values moved. The lookup
// takes 16 bytes per lane. The gradient sums in fp32 and in token order
// without atomics on values: tokens are sorted by id (a stable counting sort),
// a row of the table then owns a run of them. Most rows have no token, a few have
// thousands, so the work is dealt out by sorted tokens: a wavefront owns kChunk
// of them, finishes the runs that lie within, and leaves a part of those that do
// not, which are joined in order. Rows without a token are filled with zeros.
// 32768 tokens (half of them padding), 65536 rows of 2304 bf16 values: lookup 51 us,
// 4.4 TB/s; sort 12, sums and zeros 73 (5.2 TB/s), join 10. A large copy: 5.1 TB/s.
#include "gspn_mfma.hpp"
#include "gspn_tokens.hpp"

namespace gspn {

namespace {

constexpr int kChunk = 16;        // sorted tokens that a wavefront sums
constexpr int kSortWaves = 16;
constexpr int kRangeBits = 10;
constexpr int kMaxRange = 1 << kRangeBits;   // table rows that one sorting workgroup owns, at most
constexpr int kBlock = 256;

// How a sort is dealt out. A wavefront's share of the tokens: up to a turn of
// kTurn * 64 in steps of 64, from there on whole turns, to which the rows are
// padded with -1, so that no load asks where the end is; in up to four parts of
// whole turns. Table rows of a workgroup: at least a wavefront's worth, so many
// that there is about one workgroup per compute unit, each of which reads all tokens.
constexpr int kTurn = 8;
struct SortPlan {
  int64_t share;    // tokens of a wavefront
  int parts, range;
  int64_t blocks;
  int64_t padded() const { return share * kSortWaves * parts; }
  bool direct() const { return share <= kTurn * 64 && parts == 1; }
};
SortPlan sort_plan(int64_t tokens, int64_t V) {
  SortPlan s{cdiv(tokens, kSortWaves * 64) * 64, 1, 64, 0};
  constexpr int64_t turn = kTurn * 64;
  if (s.share > turn) {
    s.parts = s.share > 2 * turn ? 4 : 2;
    s.share = cdiv(cdiv(tokens, s.parts * kSortWaves), turn) * turn;
  }
  while (s.range < kMaxRange && cdiv(V, s.range) * s.parts > 256) s.range *= 2;
  s.blocks = cdiv(V, s.range) * s.parts;
  return s;
}

template <typename T> struct EmbedP {
  const void* ids;
  int64_t ids_batch;
  const int32_t* lens;
  const T* weight;
  T* out;
  int64_t L, V, D, tokens;
  int64_t pieces;         // pieces of a row
  int64_t block0;         // first workgroup of this launch
  float scale;
  int ids64;
};

// How rows are dealt to wavefronts: `per` rows to one, a row's pieces in
// `slices` shares where there are few rows. Row, id and run are the same for the
// whole wavefront, so that a piece costs little more than its load and store
// (a piece per lane with its own row: sums of 65536 rows of 2304 108 us, 72). Shares
// where wavefronts would be fewer than two a SIMD: 32 rows of 2304 3.4 us, without
// 4.4; 3063 rows of 1153 single values 6.8 without, 7.9 in three.
struct Deal {
  int64_t rows;
  int32_t slices, per;
};
constexpr int kAtOnce = 4;   // pieces that a lane has in flight
Deal deal(int64_t rows, int64_t pieces) {
  Deal d{rows, 1, 1};
  const int64_t turns = cdiv(pieces, 64);
  while (rows * d.slices < 2048 && d.slices < turns) ++d.slices;
  while (d.per < 4 && rows / d.per > 65536) d.per *= 2;
  return d;
}
int64_t deal_blocks(const Deal& d) { return cdiv(cdiv(d.rows, d.per) * d.slices, kBlock / 64); }
// this wavefront's first row and its lane's first piece
struct Share {
  int64_t row;
  int64_t piece;
};
__device__ __forceinline__ Share share_of(const Deal& d, int64_t block) {
  const int64_t g = block * (kBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t r = g / d.slices;
  return Share{r * d.per, (g - r * d.slices) * 64 + (threadIdx.x & 63)};
}

template <typename T, int V>
__global__ __launch_bounds__(kBlock) void embed_kernel(EmbedP<T> a, Deal deal) {
  const Share w = share_of(deal, a.block0 + blockIdx.x);
  const int64_t step = deal.slices * int64_t(64);
  for (int k = 0; k < deal.per; ++k) {
    const int64_t t = w.row + k;
    if (t >= a.tokens) return;
    bool live[1];
    int32_t one[1];
    ids_of<1>(a, t, 0, live, one);
    const int64_t row = one[0];
    const T* src = a.weight + (row < 0 ? 0 : row) * a.D;
    T* dst = a.out + t * a.D;
    for (int64_t p = w.piece; p < a.pieces; p += step * kAtOnce) {
      float d[kAtOnce][V];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
#pragma unroll
        for (int e = 0; e < V; ++e) d[q][e] = 0.0f;
        if (row >= 0 && p + q * step < a.pieces) ldv<V>(src + (p + q * step) * V, d[q]);
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        if (p + q * step >= a.pieces) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) d[q][e] *= a.scale;
        stv<V>(dst + (p + q * step) * V, d[q]);
      }
    }
  }
}

// rows of all tokens as 32-bit numbers, -1 for those without and for the padding
template <typename P>
__global__ __launch_bounds__(kBlock) void embed_rows_kernel(P a, int32_t* rows, int64_t padded) {
  const int64_t t = (a.block0 + blockIdx.x) * kBlock + threadIdx.x;
  bool live[1];
  int32_t row[1];
  ids_of<1>(a, t, 0, live, row);
  if (t < padded) rows[t] = row[0];
}

// Stable counting sort. A workgroup owns table rows v0 = range * (its number / parts)
// .. and one of `parts` equal parts of the tokens. It counts all tokens of its rows,
// those of its own part by wavefront (in LDS; integer counts do not depend on
// the order of the additions), and finds how many tokens belong to rows below v0;
// then, with every row's and wavefront's first place known, it places those of its
// own part. Parts, since a few rows hold half of a text's tokens and one workgroup
// would place them all (32768 tokens, 65536 rows: one part 24 us, four 14).
// Equal rows among 64 tokens are found by comparing the bits of the row
// numbers, so that a lane's place is its wavefront's next one plus the lanes
// of the same row before it. DIRECT: one turn per wavefront, whose rows every
// workgroup finds from the ids itself; more tokens come as rows that another
// kernel has found once (a launch more, which few tokens would wait for).
template <bool DIRECT, typename P>
__global__ __launch_bounds__(kSortWaves * 64) void embed_sort_kernel(
    P a, const int32_t* rows, int64_t share, int64_t V, int range, int parts, int32_t* start, int2* place_of) {
  __shared__ int32_t counts[(kSortWaves + 2) * kMaxRange];   // [wavefront][row], of the parts before, after
  __shared__ int32_t sums[kSortWaves], below[kSortWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int32_t* mine_next = counts + wave * range;
  const int64_t block = a.block0 + blockIdx.x;
  const int part = static_cast<int>(block % parts);
  const int32_t v0 = static_cast<int32_t>(block / parts) * range;
  for (int i = threadIdx.x; i < (kSortWaves + 2) * range; i += kSortWaves * 64) counts[i] = 0;
  __syncthreads();
  const int32_t* own = rows + (part * kSortWaves + wave) * share;
  int32_t lower = 0;
  uint32_t r[kTurn];
  if constexpr (DIRECT) {
    bool live[kTurn];
    int32_t own_rows[kTurn] = {};
    if (share > 0) ids_of<kTurn>(a, wave * share + lane, 64, live, own_rows);
#pragma unroll
    for (int k = 0; k < kTurn; ++k) r[k] = 64 * k < share ? own_rows[k] : -1;
  }
  for (int q = 0; q < parts; ++q) {
    const int32_t* from = rows + (q * kSortWaves + wave) * share;
    int32_t* count = q == part ? mine_next : counts + (kSortWaves + (q < part ? 0 : 1)) * range;
    for (int64_t turn = 0; turn < share; turn += kTurn * 64) {
      if constexpr (!DIRECT) {
#pragma unroll
        for (int k = 0; k < kTurn; ++k) r[k] = from[turn + 64 * k + lane];
      }
#pragma unroll
      for (int k = 0; k < kTurn; ++k) {
        lower += r[k] < static_cast<uint32_t>(v0) ? 1 : 0;   // -1 is the largest
        const uint32_t i = r[k] - v0;
        if (i < static_cast<uint32_t>(range)) atomicAdd(&count[i], 1);
      }
    }
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) lower += __shfl_xor(lower, s, 64);
  if (lane == 0) below[wave] = lower;
  __syncthreads();
  // thread i: row v0 + i
  const int i = threadIdx.x;
  int32_t total = 0;
  if (i < range)
#pragma unroll
    for (int w = 0; w < kSortWaves + 2; ++w) total += counts[w * range + i];
  int32_t before = total;   // inclusive sum over the wavefront's rows
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int32_t u = __shfl_up(before, s, 64);
    if (lane >= s) before += u;
  }
  if (lane == 63) sums[wave] = before;
  __syncthreads();
  int32_t at = before - total;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) at += below[w] + (w < wave ? sums[w] : 0);
  if (i < range) {
    if (part == 0 && v0 + static_cast<int64_t>(i) < V) start[v0 + i] = at;
    if (part == 0 && v0 + static_cast<int64_t>(i) == V - 1) start[V] = at + total;
    at += counts[kSortWaves * range + i];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t n = counts[w * range + i];
      counts[w * range + i] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t turn = 0; turn < share; turn += kTurn * 64) {
    uint32_t lo[kTurn], hi[kTurn];   // lanes whose row numbers agree in every bit
    if constexpr (!DIRECT) {
#pragma unroll
      for (int k = 0; k < kTurn; ++k) r[k] = own[turn + 64 * k + lane];
    }
#pragma unroll
    for (int k = 0; k < kTurn; ++k) {
      const uint32_t i = r[k] - v0;
      const uint64_t in = __ballot(i < static_cast<uint32_t>(range));
      lo[k] = static_cast<uint32_t>(in);
      hi[k] = static_cast<uint32_t>(in >> 32);
      if (in == 0) continue;
#pragma unroll
      for (int b = 0; b < kRangeBits; ++b) {
        const int32_t set = __builtin_amdgcn_sbfe(i, b, 1);   // 0 or -1
        const uint64_t have = __ballot(set != 0);
        lo[k] &= ~(static_cast<uint32_t>(have) ^ set);
        hi[k] &= ~(static_cast<uint32_t>(have >> 32) ^ set);
      }
    }
    // a wavefront's LDS accesses take effect in their order, so a row's last lane
    // moves its place on without a wait
#pragma unroll
    for (int k = 0; k < kTurn; ++k) {
      const uint32_t i = r[k] - v0;
      if (i < static_cast<uint32_t>(range)) {
        const uint64_t same = static_cast<uint64_t>(hi[k]) << 32 | lo[k];
        const int32_t first = mine_next[i], place = first + __popcll(same & ((uint64_t(1) << lane) - 1));
        __builtin_amdgcn_wave_barrier();
        if ((same >> lane) == 1) mine_next[i] = place + 1;
        place_of[place] = make_int2(static_cast<int32_t>((part * kSortWaves + wave) * share + turn + 64 * k + lane), r[k]);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// ---- sums of runs -----------------------------------------------------------
template <typename T, typename O> struct RunP {
  const int32_t* start;
  const int2* place;
  const T* x;
  int64_t batch, stride, L;
  const float* weight;   // of every token, or null
  float scale;
  O* out;
  int by_place;          // a run's sum goes to row `start` of out, not to its table row
  float* part;           // [chunks][2][D]: parts of a run begun before the chunk, begun in it
  int64_t V, D, pieces, chunks;
  int64_t block0, chunk_blocks;
};

template <int V, typename T, typename O>
__device__ __forceinline__ void finish_run(const RunP<T, O>& a, int64_t v, int64_t r0, int64_t at, float (&s)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] *= a.scale;
  stv<V>(a.out + (a.by_place ? r0 : v) * a.D + at, s);
}

// Workgroups 0 .. chunk_blocks - 1: a chunk's tokens, 64 pieces of their rows
// per wavefront, eight tokens loaded ahead. The others fill rows that no token
// names.
template <typename T, typename O, int V>
__global__ __launch_bounds__(kBlock) void run_sums_kernel(RunP<T, O> a, Deal deal) {
  const int64_t g = a.block0 + blockIdx.x;
  const int lane = threadIdx.x & 63;
  if (g >= a.chunk_blocks) {
    const Share w = share_of(deal, g - a.chunk_blocks);
    const int64_t step = deal.slices * int64_t(64);
    const float zero[V] = {};
    for (int k = 0; k < deal.per; ++k) {
      const int64_t v = w.row + k;
      if (v >= a.V) return;
      if (a.start[v + 1] != a.start[v]) continue;
      for (int64_t p = w.piece; p < a.pieces; p += step) stv<V>(a.out + v * a.D + p * V, zero);
    }
    return;
  }
  const int64_t w = g * (kBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t slice = w / a.chunks, c = w - slice * a.chunks;
  const int64_t piece = slice * 64 + lane, at = piece * V;
  const int64_t all = a.start[a.V], p0 = c * kChunk;
  if (p0 >= all || piece >= a.pieces) return;
  const int64_t p1 = p0 + kChunk < all ? p0 + kChunk : all;
  float s[V] = {}, f[kChunk];
  int64_t from[kChunk];
  int32_t v[kChunk], r0[kChunk], r1[kChunk];
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    const int2 tr = a.place[p0 + k < p1 ? p0 + k : p1 - 1];
    const int64_t t = tr.x, b = static_cast<uint32_t>(t) / static_cast<uint32_t>(a.L);
    from[k] = b * a.batch + (t - b * a.L) * a.stride;
    v[k] = tr.y;
    f[k] = a.weight ? a.weight[t] : 1.0f;
  }
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    r0[k] = a.start[v[k]];
    r1[k] = a.start[v[k] + 1];
  }
  constexpr int kAhead = 8;
#pragma unroll
  for (int k0 = 0; k0 < kChunk; k0 += kAhead) {
    if (p0 + k0 >= p1) break;
    float d[kAhead][V];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ldv<V>(a.x + from[k0 + k] + at, d[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int n = k0 + k;
      if (p0 + n >= p1) break;
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = __builtin_fmaf(f[n], d[k][e], s[e]);
      if (p0 + n + 1 < p1 && p0 + n + 1 < r1[n]) continue;
      // the run ends here, or goes on after the chunk
      if (r0[n] >= p0 && r1[n] <= p1) finish_run<V>(a, v[n], r0[n], at, s);
      else stv<V>(a.part + (c * 2 + (r0[n] >= p0 ? 1 : 0)) * a.D + at, s);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = 0.0f;
    }
  }
}

// Joins the run that begins in chunk c and goes on after it (one at most) from
// its parts, V values per lane; wavefront w sums the w-th quarter of them, in order.
template <typename T, typename O, int V>
__global__ __launch_bounds__(kBlock) void run_join_kernel(RunP<T, O> a) {
  __shared__ float acc[4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t g = a.block0 + blockIdx.x, slices = cdiv(a.D, 64 * V);
  const int64_t c = g / slices, at = ((g - c * slices) * 64 + lane) * V;
  const int64_t all = a.start[a.V], p0 = c * kChunk, p1 = p0 + kChunk;
  if (p1 >= all) return;
  const int64_t v = a.place[p1 - 1].y, r0 = a.start[v], r1 = a.start[v + 1];
  if (r0 < p0 || r1 <= p1) return;
  const int64_t n = (r1 - 1) / kChunk - c + 1;   // chunks that hold it
  const int64_t per = cdiv(n, 4), k0 = wave * per, k1 = k0 + per < n ? k0 + per : n;
  float s[V] = {};
  if (at < a.D) {
    constexpr int kAhead = 8;
    for (int64_t k = k0; k < k1; k += kAhead) {
      float d[kAhead][V];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t q = k + j < k1 ? k + j : k1 - 1;
        ldv<V>(a.part + ((c + q) * 2 + (q == 0 ? 1 : 0)) * a.D + at, d[j]);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] += k + j < k1 ? d[j][e] : 0.0f;
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) acc[wave][lane * V + e] = s[e];
  __syncthreads();
  if (wave == 0 && at < a.D) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      s[e] = ((acc[0][lane * V + e] + acc[1][lane * V + e]) + acc[2][lane * V + e]) + acc[3][lane * V + e];
    finish_run<V>(a, v, r0, at, s);
  }
}

template <typename T, typename O, int V>
hipError_t run_sums_of(const RunSum& r, hipStream_t stream, Tracer* tr) {
  RunP<T, O> p{};
  p.start = r.sort.start;
  p.place = r.sort.place;
  p.x = static_cast<const T*>(r.x);
  p.batch = r.batch;
  p.stride = r.row;
  p.L = r.L;
  p.weight = r.weight;
  p.scale = r.scale;
  p.out = static_cast<O*>(r.out);
  p.by_place = r.by_place;
  p.part = r.part;
  p.V = r.V;
  p.D = r.D;
  p.pieces = r.D / V;
  p.chunks = cdiv(r.tokens, kChunk);
  p.chunk_blocks = cdiv(p.chunks * cdiv(p.pieces, 64), kBlock / 64);
  const Deal d = deal(r.V, p.pieces);
  tr->before(stream, "run_sums", r.V);
  hipError_t e = in_parts(p.chunk_blocks + (r.by_place ? 0 : deal_blocks(d)), [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((run_sums_kernel<T, O, V>), dim3(count), dim3(kBlock), 0, stream, p, d);
  });
  tr->after(stream);
  if (e != hipSuccess || r.tokens <= kChunk) return e;   // no run goes past a chunk
  tr->before(stream, "run_join", p.chunks);
  e = in_parts(p.chunks * cdiv(p.D, 64 * V), [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((run_join_kernel<T, O, V>), dim3(count), dim3(kBlock), 0, stream, p);
  });
  tr->after(stream);
  return e;
}
template <typename T, typename O> hipError_t run_sums_dt(const RunSum& r, hipStream_t stream, Tracer* tr) {
  constexpr int V = 16 / sizeof(T);
  if (r.D % V == 0 && wide_ok(r.out, 16, sizeof(O), {}) &&
      (r.tokens == 0 || wide_ok(r.x, 16, sizeof(T), {r.batch, r.row})))
    return run_sums_of<T, O, V>(r, stream, tr);
  // rows of no whole 16 bytes: bf16 in pairs, if that
  if constexpr (sizeof(T) == 2)
    if (r.D % 2 == 0 && wide_ok(r.out, 2 * sizeof(O), sizeof(O), {}) &&
        (r.tokens == 0 || wide_ok(r.x, 4, sizeof(T), {r.batch, r.row})))
      return run_sums_of<T, O, 2>(r, stream, tr);
  return run_sums_of<T, O, 1>(r, stream, tr);
}

template <typename T> EmbedP<T> embed_params(const gspn_embed_args& a) {
  EmbedP<T> p{};
  p.ids = a.ids;
  p.ids_batch = a.ids_batch;
  p.lens = a.lens;
  p.weight = static_cast<const T*>(a.weight);
  p.out = static_cast<T*>(a.out);
  p.L = a.L;
  p.V = a.V;
  p.D = a.D;
  p.tokens = a.B * a.L;
  p.scale = a.scale;
  p.ids64 = a.ids64;
  return p;
}

template <typename T, int V> hipError_t embed_run(EmbedP<T> p, hipStream_t stream, Tracer* tr) {
  p.pieces = p.D / V;
  const Deal d = deal(p.tokens, p.pieces);
  tr->before(stream, "embed", p.tokens);
  const hipError_t e = in_parts(deal_blocks(d), [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((embed_kernel<T, V>), dim3(count), dim3(kBlock), 0, stream, p, d);
  });
  tr->after(stream);
  return e;
}
template <typename T> hipError_t embed_dt(const gspn_embed_args& a, hipStream_t stream, Tracer* tr) {
  constexpr int V = 16 / sizeof(T);
  const EmbedP<T> p = embed_params<T>(a);
  if (a.D % V == 0 && wide_ok(a.weight, 16, sizeof(T), {}) && wide_ok(a.out, 16, sizeof(T), {}))
    return embed_run<T, V>(p, stream, tr);
  if constexpr (sizeof(T) == 2)
    if (a.D % 2 == 0 && wide_ok(a.weight, 4, sizeof(T), {}) && wide_ok(a.out, 4, sizeof(T), {}))
      return embed_run<T, 2>(p, stream, tr);
  return embed_run<T, 1>(p, stream, tr);
}

}  // namespace

size_t token_sort_bytes(int64_t tokens, int64_t V) {
  return up256(static_cast<size_t>(sort_plan(tokens, V).padded()) * 4) + up256(static_cast<size_t>(tokens) * 8) +
         up256(static_cast<size_t>(V + 1) * 4);
}

hipError_t sort_tokens(const void* ids, int ids64, int64_t ids_batch, const int32_t* lens, int64_t B, int64_t L,
                       int64_t V, void* ws, TokenSort* out, hipStream_t stream, Tracer* tr) {
  const int64_t tokens = B * L;
  const SortPlan s = sort_plan(tokens, V);
  const int64_t padded = s.padded();
  const size_t each = up256(static_cast<size_t>(padded) * 4);
  char* w = static_cast<char*>(ws);
  int32_t* rows = reinterpret_cast<int32_t*>(w);
  int2* place = reinterpret_cast<int2*>(w + each);
  int32_t* start = reinterpret_cast<int32_t*>(w + each + up256(static_cast<size_t>(tokens) * 8));
  *out = TokenSort{start, place};
  EmbedP<bf16_t> p{};
  p.ids = ids;
  p.ids_batch = ids_batch;
  p.lens = lens;
  p.L = L;
  p.V = V;
  p.tokens = tokens;
  p.ids64 = ids64;
  hipError_t e = hipSuccess;
  if (!s.direct()) {
    tr->before(stream, "embed_rows", tokens);
    e = in_parts(cdiv(padded, kBlock), [&](int64_t first, unsigned count) {
      p.block0 = first;
      hipLaunchKernelGGL((embed_rows_kernel<EmbedP<bf16_t>>), dim3(count), dim3(kBlock), 0, stream, p, rows, padded);
    });
    tr->after(stream);
    if (e != hipSuccess) return e;
  }
  tr->before(stream, "embed_sort", tokens);
  e = in_parts(s.blocks, [&](int64_t first, unsigned count) {
    p.block0 = first;
    const dim3 block(kSortWaves * 64);
    if (s.direct())
      hipLaunchKernelGGL((embed_sort_kernel<true, EmbedP<bf16_t>>), dim3(count), block, 0, stream, p, rows, s.share, V,
                         s.range, s.parts, start, place);
    else
      hipLaunchKernelGGL((embed_sort_kernel<false, EmbedP<bf16_t>>), dim3(count), block, 0, stream, p, rows, s.share, V,
                         s.range, s.parts, start, place);
  }, kMostBlocks / 2);
  tr->after(stream);
  return e;
}

hipError_t launch_embed(const gspn_embed_args& a, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return embed_dt<float>(a, stream, tr);
  return embed_dt<bf16_t>(a, stream, tr);
}

size_t run_part_bytes(int64_t tokens, int64_t D) {
  return up256(static_cast<size_t>(cdiv(tokens, kChunk)) * 2 * static_cast<size_t>(D) * 4);
}
hipError_t run_sums(const RunSum& r, hipStream_t stream, Tracer* tr) {
  if (r.dtype == GSPN_F32) return run_sums_dt<float, float>(r, stream, tr);
  if (r.by_place) return run_sums_dt<bf16_t, float>(r, stream, tr);
  return run_sums_dt<bf16_t, bf16_t>(r, stream, tr);
}

size_t embed_bwd_workspace_bytes(int64_t B, int64_t L, int64_t V, int64_t D) {
  return token_sort_bytes(B * L, V) + run_part_bytes(B * L, D);
}
hipError_t launch_embed_bwd(const gspn_embed_args& a, const gspn_embed_grads& g, void* ws, hipStream_t stream, Tracer* tr) {
  RunSum r{};
  const hipError_t e = sort_tokens(a.ids, a.ids64, a.ids_batch, a.lens, a.B, a.L, a.V, ws, &r.sort, stream, tr);
  if (e != hipSuccess) return e;
  r.dtype = a.dtype;
  r.x = g.grad_out.p;
  r.batch = g.grad_out.batch;
  r.row = g.grad_out.row;
  r.L = a.L;
  r.tokens = a.B * a.L;
  r.scale = a.scale;
  r.out = g.weight;
  r.part = reinterpret_cast<float*>(static_cast<char*>(ws) + token_sort_bytes(r.tokens, a.V));
  r.V = a.V;
  r.D = a.D;
  return run_sums(r, stream, tr);
}

}  // namespace gspn
