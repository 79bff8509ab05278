// Token embedding and its gradient.
//
//   out[t] = scale * weight[ids[t]],   dweight[v] = scale * sum_{t: ids[t] = v} grad_out[t]
//
// Both are bound by memory: a multiplication for two values moved. The lookup
// takes 16 bytes per lane. The gradient sums in fp32 and in token order
// without atomics on values: tokens are sorted by id (a stable counting sort),
// a row of the table then owns a run of them. Most rows have few or no tokens,
// a few rows have thousands, so runs of more than kChunk tokens are summed in
// parts by workgroups that own kChunk sorted tokens each, and joined in order.
#include "gspn_mfma.hpp"
#include "gspn_tokens.hpp"

namespace gspn {

namespace {

constexpr int kChunk = 32;        // sorted tokens per part of a long run
constexpr int kSortWaves = 16;
constexpr int kMaxRange = 1024;   // table rows that one sorting workgroup owns, at most
constexpr int kBlock = 256;

// Rows per sorting workgroup: about one workgroup per compute unit, each of
// which reads all ids, at least a wavefront's worth of rows.
int sort_range(int64_t V) {
  int r = 64;
  while (r < kMaxRange && cdiv(V, r) > 256) r *= 2;
  return r;
}

template <typename T> struct EmbedP {
  const void* ids;
  int64_t ids_batch;
  const int32_t* lens;
  const T* weight;
  T* out;
  const T* gy;
  int64_t gb, gr;
  T* dw;
  const int32_t* start;   // [V + 1]: row v owns sorted tokens start[v] .. start[v + 1] - 1
  const int32_t* token;   // [tokens]: sorted tokens
  const int32_t* row;     // [tokens]: their rows
  float* part;            // [chunks][2][D]: sums of long runs, begun before the chunk or in it
  int64_t L, V, D, tokens;
  int64_t pieces;         // pieces of a row
  int64_t block0;         // first workgroup of this launch
  int64_t long_blocks;    // workgroups of long runs' parts, before those of rows
  float scale;
  int ids64;
};

__device__ __forceinline__ int64_t id_at(const void* ids, int ids64, int64_t i) {
  return ids64 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// entry of token t (fewer than 2^31 tokens)
template <typename P> __device__ __forceinline__ int64_t entry_of(const P& a, int64_t t) {
  return static_cast<uint32_t>(t) / static_cast<uint32_t>(a.L);
}
// the table row of token t, -1 for padding and for ids outside the table
template <typename P> __device__ __forceinline__ int64_t row_of(const P& a, int64_t t) {
  const int64_t b = entry_of(a, t), l = t - b * a.L;
  if (l >= seq_len(a.lens, b, a.L)) return -1;
  const int64_t id = id_at(a.ids, a.ids64, b * a.ids_batch + l);
  return id >= 0 && id < a.V ? id : -1;
}

// A workgroup copies kCopies * 256 pieces of the output, whole rows or not
constexpr int kCopies = 4;
template <typename T, int V>
__global__ __launch_bounds__(kBlock) void embed_kernel(EmbedP<T> a) {
  const int64_t first = (a.block0 + blockIdx.x) * (kBlock * kCopies);
  const int64_t t0 = first / a.pieces;
  const int64_t left = first - t0 * a.pieces;
  float d[kCopies][V];
  int64_t to[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    const int64_t i = left + k * kBlock + threadIdx.x;
    // a row of fewer than 2^31 pieces: the quotient fits 32 bits
    const uint32_t up = static_cast<uint32_t>(i) / static_cast<uint32_t>(a.pieces);
    const int64_t t = t0 + up, at = (i - static_cast<int64_t>(up) * a.pieces) * V;
    to[k] = -1;
#pragma unroll
    for (int e = 0; e < V; ++e) d[k][e] = 0.0f;
    if (t < a.tokens) {
      const int64_t row = row_of(a, t);
      to[k] = t * a.D + at;
      if (row >= 0) ldv<V>(a.weight + row * a.D + at, d[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    if (to[k] < 0) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) d[k][e] *= a.scale;
    stv<V>(a.out + to[k], d[k]);
  }
}

// rows of all tokens as 32-bit numbers, -1 for those without
template <typename P>
__global__ __launch_bounds__(kBlock) void embed_rows_kernel(P a, int32_t* rows) {
  const int64_t t = (a.block0 + blockIdx.x) * kBlock + threadIdx.x;
  if (t < a.tokens) rows[t] = static_cast<int32_t>(row_of(a, t));
}

// Stable counting sort. Workgroup g owns table rows v0 = g * range .. and
// walks all tokens twice, wavefront w the w-th sixteenth of them: first it
// counts (per wavefront and row, in LDS; integer counts do not depend on the
// order of the additions) and finds how many tokens belong to rows below v0,
// then, with every row's and wavefront's first place known, it places them.
// Equal rows among 64 tokens are found by comparing the bits of the row
// numbers, so that a lane's place is its wavefront's next one plus the lanes
// of the same row before it.
__global__ __launch_bounds__(kSortWaves * 64) void embed_sort_kernel(
    const int32_t* rows, int64_t tokens, int64_t V, int range, int32_t* start, int32_t* token, int32_t* row) {
  __shared__ int32_t counts[kSortWaves * kMaxRange];   // [wavefront][row]
  __shared__ int32_t sums[kSortWaves], below[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t* mine_next = counts + wave * range;
  const int32_t v0 = static_cast<int32_t>(blockIdx.x) * range;
  for (int i = threadIdx.x; i < kSortWaves * range; i += kSortWaves * 64) counts[i] = 0;
  __syncthreads();
  const int64_t share = cdiv(cdiv(tokens, kSortWaves), 64) * 64;
  const int64_t t0 = wave * share, t1 = t0 + share < tokens ? t0 + share : tokens;
  constexpr int kAhead = 16;
  int32_t lower = 0;
  for (int64_t t = t0 + lane; t < t1; t += 64 * kAhead) {
    int32_t r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) r[k] = t + 64 * k < t1 ? rows[t + 64 * k] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      lower += r[k] >= 0 && r[k] < v0 ? 1 : 0;
      const int32_t i = r[k] - v0;
      if (r[k] >= 0 && i >= 0 && i < range) atomicAdd(&mine_next[i], 1);
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
    for (int w = 0; w < kSortWaves; ++w) total += counts[w * range + i];
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
    if (v0 + static_cast<int64_t>(i) < V) start[v0 + i] = at;
    if (v0 + static_cast<int64_t>(i) == V - 1) start[V] = at + total;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t n = counts[w * range + i];
      counts[w * range + i] = at;
      at += n;
    }
  }
  __syncthreads();
  const int bits = 31 - __builtin_clz(range);
  for (int64_t t = t0; t < t1; t += 64 * kAhead) {
    int32_t r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) r[k] = t + 64 * k + lane < t1 ? rows[t + 64 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int32_t i = r[k] - v0;
      const bool mine = r[k] >= 0 && i >= 0 && i < range;
      uint64_t same = __ballot(mine);
      if (same == 0) continue;
      for (int b = 0; b < bits; ++b) {
        const bool set = (i >> b) & 1;
        const uint64_t have = __ballot(set);
        same &= set ? have : ~have;
      }
      if (mine) {
        const int32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
        const int32_t place = mine_next[i] + rank;
        token[place] = static_cast<int32_t>(t + 64 * k + lane);
        row[place] = r[k];
      }
      lds_wave_sync();
      if (mine && (same >> lane) == 1) mine_next[i] += __popcll(same);   // the row's last lane
      lds_wave_sync();
    }
  }
}

// sum of grad_out over sorted tokens p0 .. p1 - 1 at values `at` ..
template <typename T, int V>
__device__ __forceinline__ void sum_tokens(const EmbedP<T>& a, int64_t p0, int64_t p1, int64_t at, float (&s)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = 0.0f;
  constexpr int kAhead = V > 4 ? 4 : 8;
  for (int64_t p = p0; p < p1; p += kAhead) {
    float d[kAhead][V];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t t = a.token[p + k < p1 ? p + k : p1 - 1], b = entry_of(a, t);
      ldv<V>(a.gy + b * a.gb + (t - b * a.L) * a.gr + at, d[k]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += p + k < p1 ? d[k][e] : 0.0f;
  }
}

// Workgroups 0 .. long_blocks - 1: the parts of long runs, 256 pieces of one
// chunk of sorted tokens. A chunk meets at most two long runs: one that its
// first token continues or begins, one that begins later and reaches its end.
// The other workgroups: kPut * 256 pieces of the gradient, each with its row's run.
constexpr int kPut = 4;
template <typename T, int V>
__global__ __launch_bounds__(kBlock) void embed_grad_kernel(EmbedP<T> a) {
  int64_t g = a.block0 + blockIdx.x;
  float s[V];
  if (g < a.long_blocks) {
    const int64_t slices = cdiv(a.pieces, kBlock);
    const int64_t c = g / slices, piece = (g - c * slices) * kBlock + threadIdx.x;
    const int64_t all = a.start[a.V], p0 = c * kChunk;
    if (p0 >= all) return;
    const int64_t p1 = p0 + kChunk < all ? p0 + kChunk : all;
    const int64_t va = a.row[p0], vb = a.row[p1 - 1];
    const int64_t a0 = a.start[va], a1 = a.start[va + 1], b0 = a.start[vb], b1 = a.start[vb + 1];
    if (piece >= a.pieces) return;
    if (a1 - a0 > kChunk) {
      sum_tokens<T, V>(a, p0, a1 < p1 ? a1 : p1, piece * V, s);
      stv<V>(a.part + (c * 2 + (a0 < p0 ? 0 : 1)) * a.D + piece * V, s);
    }
    if (vb != va && b1 - b0 > kChunk) {
      sum_tokens<T, V>(a, b0, p1, piece * V, s);
      stv<V>(a.part + (c * 2 + 1) * a.D + piece * V, s);
    }
    return;
  }
  g -= a.long_blocks;
  const int64_t first = g * (kBlock * kPut), v0 = first / a.pieces;
  const uint32_t left = static_cast<uint32_t>(first - v0 * a.pieces), pieces = static_cast<uint32_t>(a.pieces);
  int32_t p0[kPut], p1[kPut];
  int64_t to[kPut];
  uint32_t at[kPut];
#pragma unroll
  for (int k = 0; k < kPut; ++k) {
    const uint32_t i = left + k * kBlock + threadIdx.x, up = i / pieces;
    const int64_t v = v0 + up;
    at[k] = (i - up * pieces) * V;
    to[k] = v * a.D + at[k];
    p0[k] = 0;
    p1[k] = kChunk + 1;   // past the table: not written
    if (v < a.V) {
      p0[k] = a.start[v];
      p1[k] = a.start[v + 1];
    }
  }
#pragma unroll
  for (int k = 0; k < kPut; ++k) {
    if (p1[k] - p0[k] > kChunk) continue;   // joined from its parts
    sum_tokens<T, V>(a, p0[k], p1[k], at[k], s);
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] *= a.scale;
    stv<V>(a.dw + to[k], s);
  }
}

// Joins the long run that begins in chunk c (one at most: it reaches the
// chunk's end) from its parts, V values per lane; wavefront w sums the w-th
// quarter of them, in order.
template <typename T, int V>
__global__ __launch_bounds__(kBlock) void embed_join_kernel(EmbedP<T> a) {
  __shared__ float acc[4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t g = a.block0 + blockIdx.x, slices = cdiv(a.D, 64 * V);
  const int64_t c = g / slices, at = ((g - c * slices) * 64 + lane) * V;
  const int64_t all = a.start[a.V], p0 = c * kChunk;
  if (p0 >= all) return;
  const int64_t p1 = p0 + kChunk < all ? p0 + kChunk : all;
  const int64_t v = a.row[p1 - 1], r0 = a.start[v], r1 = a.start[v + 1];
  if (r0 < p0 || r1 - r0 <= kChunk) return;
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
      s[e] = (((acc[0][lane * V + e] + acc[1][lane * V + e]) + acc[2][lane * V + e]) + acc[3][lane * V + e]) * a.scale;
    stv<V>(a.dw + v * a.D + at, s);
  }
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
  tr->before(stream, "embed", p.tokens);
  const hipError_t e = in_parts(cdiv(p.tokens * p.pieces, kBlock * kCopies), [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((embed_kernel<T, V>), dim3(count), dim3(kBlock), 0, stream, p);
  });
  tr->after(stream);
  return e;
}
template <typename T> hipError_t embed_dt(const gspn_embed_args& a, hipStream_t stream, Tracer* tr) {
  constexpr int V = 16 / sizeof(T);
  const EmbedP<T> p = embed_params<T>(a);
  if (a.D % V == 0 && wide_ok(a.weight, 16, sizeof(T), {}) && wide_ok(a.out, 16, sizeof(T), {}))
    return embed_run<T, V>(p, stream, tr);
  return embed_run<T, 1>(p, stream, tr);
}

template <typename T, int V> hipError_t embed_grad_run(EmbedP<T> p, hipStream_t stream, Tracer* tr) {
  p.pieces = p.D / V;
  const int64_t chunks = cdiv(p.tokens, kChunk);
  p.long_blocks = chunks * cdiv(p.pieces, kBlock);
  tr->before(stream, "embed_grad", p.V);
  hipError_t e = in_parts(p.long_blocks + cdiv(p.V * p.pieces, kBlock * kPut), [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((embed_grad_kernel<T, V>), dim3(count), dim3(kBlock), 0, stream, p);
  });
  tr->after(stream);
  if (e != hipSuccess || p.tokens <= kChunk) return e;   // no run is longer than the tokens
  tr->before(stream, "embed_join", chunks);
  constexpr int J = V == 1 ? 1 : 4;
  e = in_parts(chunks * cdiv(p.D, 64 * J), [&](int64_t first, unsigned count) {
    p.block0 = first;
    hipLaunchKernelGGL((embed_join_kernel<T, J>), dim3(count), dim3(kBlock), 0, stream, p);
  });
  tr->after(stream);
  return e;
}
template <typename T>
hipError_t embed_grad_dt(const gspn_embed_args& a, const gspn_embed_grads& g, void* ws, hipStream_t stream, Tracer* tr) {
  constexpr int V = 16 / sizeof(T);
  EmbedP<T> p = embed_params<T>(a);
  p.gy = static_cast<const T*>(g.grad_out.p);
  p.gb = g.grad_out.batch;
  p.gr = g.grad_out.row;
  p.dw = static_cast<T*>(g.weight);
  TokenSort s;
  const hipError_t e = sort_tokens(a.ids, a.ids64, a.ids_batch, a.lens, a.B, a.L, a.V, ws, &s, stream, tr);
  if (e != hipSuccess) return e;
  p.start = s.start;
  p.token = s.token;
  p.row = s.row;
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + token_sort_bytes(p.tokens, a.V));
  if (a.D % V == 0 && wide_ok(p.dw, 16, sizeof(T), {}) && (p.tokens == 0 || wide_ok(p.gy, 16, sizeof(T), {p.gb, p.gr})))
    return embed_grad_run<T, V>(p, stream, tr);
  return embed_grad_run<T, 1>(p, stream, tr);
}

}  // namespace

size_t token_sort_bytes(int64_t tokens, int64_t V) {
  return 3 * up256(static_cast<size_t>(tokens) * 4) + up256(static_cast<size_t>(V + 1) * 4);
}

hipError_t sort_tokens(const void* ids, int ids64, int64_t ids_batch, const int32_t* lens, int64_t B, int64_t L,
                       int64_t V, void* ws, TokenSort* out, hipStream_t stream, Tracer* tr) {
  const int64_t tokens = B * L;
  const size_t each = up256(static_cast<size_t>(tokens) * 4);
  char* w = static_cast<char*>(ws);
  int32_t* rows = reinterpret_cast<int32_t*>(w);
  int32_t* token = reinterpret_cast<int32_t*>(w + each);
  int32_t* row = reinterpret_cast<int32_t*>(w + 2 * each);
  int32_t* start = reinterpret_cast<int32_t*>(w + 3 * each);
  *out = TokenSort{start, token, row};
  EmbedP<bf16_t> p{};
  p.ids = ids;
  p.ids_batch = ids_batch;
  p.lens = lens;
  p.L = L;
  p.V = V;
  p.tokens = tokens;
  p.ids64 = ids64;
  hipError_t e = hipSuccess;
  if (tokens > 0) {
    tr->before(stream, "embed_rows", tokens);
    e = in_parts(cdiv(tokens, kBlock), [&](int64_t first, unsigned count) {
      p.block0 = first;
      hipLaunchKernelGGL((embed_rows_kernel<EmbedP<bf16_t>>), dim3(count), dim3(kBlock), 0, stream, p, rows);
    });
    tr->after(stream);
    if (e != hipSuccess) return e;
  }
  const int range = sort_range(V);
  tr->before(stream, "embed_sort", tokens);
  hipLaunchKernelGGL(embed_sort_kernel, dim3(static_cast<unsigned>(cdiv(V, range))), dim3(kSortWaves * 64), 0, stream,
                     rows, tokens, V, range, start, token, row);
  e = hipGetLastError();
  tr->after(stream);
  return e;
}

hipError_t launch_embed(const gspn_embed_args& a, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return embed_dt<float>(a, stream, tr);
  return embed_dt<bf16_t>(a, stream, tr);
}

size_t embed_bwd_workspace_bytes(int64_t B, int64_t L, int64_t V, int64_t D) {
  return token_sort_bytes(B * L, V) + static_cast<size_t>(cdiv(B * L, kChunk)) * 2 * static_cast<size_t>(D) * 4;
}

hipError_t launch_embed_bwd(const gspn_embed_args& a, const gspn_embed_grads& g, void* ws, hipStream_t stream, Tracer* tr) {
  if (a.dtype == GSPN_F32) return embed_grad_dt<float>(a, g, ws, stream, tr);
  return embed_grad_dt<bf16_t>(a, g, ws, stream, tr);
}

}  // namespace gspn
