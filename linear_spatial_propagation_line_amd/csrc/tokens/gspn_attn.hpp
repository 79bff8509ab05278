// Tiles shared by the cross attention kernels (gspn_attn.hip,
// gspn_attn_bwd.hip): 32 x 32 products on matrix cores whose result feeds the
// next product from registers.
//
// Every product is taken as X = M1 M2^T or X = M1^T W with 32 x 32 results
// (v_mfma_f32_32x32x16_bf16, or four v_mfma_f32_32x32x2_f32 for fp32):
// lane l holds column l % 32 of the result, rows (i % 4) + 8 (i / 4) + 4 (l / 32)
// in its 16 registers i. A result W[row][col] is then already a B operand
// (lane: one column, consecutive contraction rows) if the contraction runs
// over its rows in the order in which the registers hold them; the other
// operand, M1^T, is read from LDS in that same order, for bf16 by the
// transposing LDS read. So probabilities and score gradients never pass
// through LDS.
#pragma once

#include "gspn_mfma.hpp"
#include "gspn_tokens.hpp"

namespace gspn {

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct RowMap {
  int64_t batch, row, head;   // strides in elements
};

// The rows that share one key head: row r of (entry, key head hk) is query
// r % Lq of head hk * share + r / Lq; P is a problem with Lq, share and rows.
struct QRow {
  int64_t h, q;
};
template <typename P> __device__ __forceinline__ QRow q_row(const P& a, int hk, uint32_t r) {
  const uint32_t rc = r < a.rows ? r : static_cast<uint32_t>(a.rows) - 1;   // clamped to the last
  const uint32_t hs = rc / static_cast<uint32_t>(a.Lq);
  return QRow{static_cast<int64_t>(hk) * a.share + hs, static_cast<int64_t>(rc - hs * static_cast<uint32_t>(a.Lq))};
}
// 32 adjacent rows starting at row r0: one division for all of them unless
// the queries are few
struct RowTile {
  uint32_t r0, h, q, Lq, left, share, hk;
  template <typename P>
  __device__ __forceinline__ RowTile(const P& a, int hk_, uint32_t r0_)
      : r0(r0_), Lq(static_cast<uint32_t>(a.Lq)), left(static_cast<uint32_t>(a.rows) - 1 - r0_),
        share(a.share), hk(hk_) {
    h = r0 / Lq;
    q = r0 - h * Lq;
    h += hk * share;
  }
  // row i of the tile, clamped to the last row
  __device__ __forceinline__ QRow at(int i) const {
    const uint32_t k = static_cast<uint32_t>(i) < left ? i : left;
    if (Lq < 32) {
      const uint32_t hs = (r0 + k) / Lq;
      return QRow{static_cast<int64_t>(hk) * share + hs, static_cast<int64_t>(r0 + k - hs * Lq)};
    }
    const uint32_t u = q + k;
    return u < Lq ? QRow{h, u} : QRow{static_cast<int64_t>(h) + 1, u - Lq};
  }
};

template <typename T> struct Mma;

template <> struct Mma<bf16_t> {
  static constexpr int kChunk = 16;    // contraction length of one fragment pair
  static constexpr int kPer = 8;       // elements a lane holds of it
  typedef bf16x8 Frag;
  __device__ static __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mma<float> {
  static constexpr int kChunk = 8;
  static constexpr int kPer = 4;
  typedef f32x4 Frag;
  __device__ static __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
    for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[k], b[k], c, 0, 0, 0);
    return c;
  }
};

// LDS row pitch in bytes: 16 bytes of padding spread a column of 16-byte
// pieces over the banks
template <typename T, int EP> constexpr int tile_pitch() {
  return EP * static_cast<int>(sizeof(T)) + (sizeof(T) == 2 ? 32 : 16);
}

// 16 bytes of row values e0 .. : whole when `wide`, else value by value with
// the row's end honoured (a value past E is 0). FULL: the row holds all the
// values that a tile has room for and is 16-byte aligned, no questions asked.
template <typename T, bool FULL>
__device__ __forceinline__ u32x4 load16(const T* row, int e0, int E, bool wide) {
  constexpr int kPer = 16 / sizeof(T);
  if constexpr (FULL) return *reinterpret_cast<const u32x4*>(row + e0);
  u32x4 v = {0u, 0u, 0u, 0u};
  if (wide) {
    if (e0 < E) v = *reinterpret_cast<const u32x4*>(row + e0);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (e0 + k < E) {
        if constexpr (sizeof(T) == 4) v[k] = __float_as_uint(to_f32(row[e0 + k]));
        else v[k / 2] |= static_cast<uint32_t>(row[e0 + k].bits) << (16 * (k & 1));
      }
    }
  }
  return v;
}

// a lane's fragments of one row in global memory (zeros when !keep; with FULL
// the row is always read, so it has to be one that exists)
template <typename T, int EP, bool FULL>
__device__ __forceinline__ void row_frags(const T* row, bool keep, int E, bool wide,
                                          typename Mma<T>::Frag (&f)[EP / Mma<T>::kChunk]) {
  const int hh = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int j = 0; j < EP / Mma<T>::kChunk; ++j) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if constexpr (FULL) {
      const u32x4 u = load16<T, true>(row, j * Mma<T>::kChunk + hh * Mma<T>::kPer, E, wide);
      v = keep ? u : v;
    } else if (keep) {
      v = load16<T, false>(row, j * Mma<T>::kChunk + hh * Mma<T>::kPer, E, wide);
    }
    f[j] = __builtin_bit_cast(typename Mma<T>::Frag, v);
  }
}

// fragment j of the lane's row (row0 + l % 32) of an LDS tile
template <typename T, int EP>
__device__ __forceinline__ typename Mma<T>::Frag tile_frag(const char* tile, int row0, int j, int lane) {
  return *reinterpret_cast<const typename Mma<T>::Frag*>(
      tile + (row0 + (lane & 31)) * tile_pitch<T, EP>() + j * 32 + (lane >> 5) * 16);
}

// X[32 rows of the tile][32 lane columns] = tile rows . the lanes' fragments
template <typename T, int EP>
__device__ __forceinline__ f32x16 tile_dot(const char* tile, int row0,
                                           const typename Mma<T>::Frag (&f)[EP / Mma<T>::kChunk],
                                           int lane) {
  f32x16 x = {};
#pragma unroll
  for (int j = 0; j < EP / Mma<T>::kChunk; ++j)
    x = Mma<T>::mma(tile_frag<T, EP>(tile, row0, j, lane), f[j], x);
  return x;
}

// Probabilities and score gradients are operands of the second products. In
// bf16 alone (8 bits of mantissa) their rounding would be as large as the
// result's own: outputs, dK and dV 0.00235 from 64 bits in the norm, where
// rounding an exact result gives 0.00166. So they are taken as two bf16 parts,
// the value rounded and what that left (16 bits together), at the price of one
// more matrix product: 4x4096x2048 with ragged masks, 16 heads of 64, forward 153 us against
// 126; 2x4096x2048, 16 heads of 128 on 4, training step 819 against 730;
// 2097152 rows, 77 keys, 5 heads of 64, 626 against 553; few rows on long keys, none.
__device__ __forceinline__ void split_bf16(const float (&w)[16], uint32_t (&p)[8], uint32_t (&rest)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    p[k] = pack_bf16x2(w[2 * k], w[2 * k + 1]);
    rest[k] = pack_bf16x2(w[2 * k] - __uint_as_float(p[k] << 16), w[2 * k + 1] - __uint_as_float(p[k] & 0xffff0000u));
  }
}
// acc[et][32 e of slab et][lane column] += tile rows^T W, W[32 rows][lane
// column] in the result layout above as bf16 pairs in two parts
template <int EP>
__device__ __forceinline__ void tile_accum_split(const char* tile, int row0, const uint32_t (&p)[8],
                                                 const uint32_t (&rest)[8], f32x16 (&acc)[EP / 32], int lane) {
  const int hh = lane >> 5, g = (lane >> 4) & 1, c = lane & 15;
  constexpr int pitch = tile_pitch<bf16_t, EP>();
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    const bf16x8 b = __builtin_bit_cast(bf16x8, u32x4{p[4 * kb], p[4 * kb + 1], p[4 * kb + 2], p[4 * kb + 3]});
    const bf16x8 d = __builtin_bit_cast(bf16x8, u32x4{rest[4 * kb], rest[4 * kb + 1], rest[4 * kb + 2], rest[4 * kb + 3]});
    const char* q = tile + (row0 + 16 * kb + 4 * hh + (c >> 2)) * pitch + (g * 16 + 4 * (c & 3)) * 2;
#pragma unroll
    for (int et = 0; et < EP / 32; ++et) {
      const v4i16 lo = lds_read_tr(reinterpret_cast<const uint16_t*>(q + et * 64));
      const v4i16 hi = lds_read_tr(reinterpret_cast<const uint16_t*>(q + et * 64 + 8 * pitch));
      const bf16x8 a = __builtin_bit_cast(bf16x8, v8i16{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w});
      acc[et] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[et], 0, 0, 0);
      acc[et] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, d, acc[et], 0, 0, 0);
    }
  }
}
// the same from fp32 W
template <int EP>
__device__ __forceinline__ void tile_accum(const char* tile, int row0, const float (&w)[16],
                                           f32x16 (&acc)[EP / 32], int lane, bf16_t) {
  uint32_t p[8], rest[8];
  split_bf16(w, p, rest);
  tile_accum_split<EP>(tile, row0, p, rest, acc, lane);
}
template <int EP>
__device__ __forceinline__ void tile_accum(const char* tile, int row0, const float (&w)[16],
                                           f32x16 (&acc)[EP / 32], int lane, float) {
  constexpr int pitch = tile_pitch<float, EP>();
  const char* q = tile + (row0 + 4 * (lane >> 5)) * pitch + (lane & 31) * 4;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int et = 0; et < EP / 32; ++et) {
      const float a = *reinterpret_cast<const float*>(q + ((i & 3) + 8 * (i >> 2)) * pitch + et * 128);
      acc[et] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, w[i], acc[et], 0, 0, 0);
    }
  }
}

// a column's maximum and sum over both half-wavefronts
__device__ __forceinline__ float column_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// scores of 32 keys with the dropped ones (bits: kept keys) at -inf
__device__ __forceinline__ void drop_keys(float (&w)[16], uint32_t bits, int lane) {
  if (bits != 0xffffffffu) {
    const uint32_t mine = bits >> (4 * (lane >> 5));
#pragma unroll
    for (int i = 0; i < 16; ++i) {   // all ones or zeros from the key's bit, then a bitwise select
      const uint32_t m = static_cast<uint32_t>(__builtin_amdgcn_sbfe(static_cast<int>(mine), (i & 3) + 8 * (i >> 2), 1));
      w[i] = __uint_as_float((__float_as_uint(w[i]) & m) | (0xff800000u & ~m));
    }
  }
}

// The first and one past the last key of [0, Lk) that the mask keeps (0, 0 if
// none), found by the whole workgroup; tiles outside need not be looked at.
__device__ __forceinline__ void key_range(const uint8_t* mask, int64_t Lk, int tid, int64_t* first,
                                          int64_t* last) {
  __shared__ int lo[4], hi[4];
  int a = static_cast<int>(Lk), b = 0;
  if (mask) {
    for (int k = tid; k < Lk; k += 256) {
      const bool on = mask[k] != 0;
      a = on && k < a ? k : a;
      b = on ? k + 1 : b;
    }
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) {
      const int u = __shfl_xor(a, d), v = __shfl_xor(b, d);
      a = u < a ? u : a;
      b = v > b ? v : b;
    }
    if ((tid & 63) == 0) {
      lo[tid >> 6] = a;
      hi[tid >> 6] = b;
    }
    __syncthreads();
    a = min(min(lo[0], lo[1]), min(lo[2], lo[3]));
    b = max(max(hi[0], hi[1]), max(hi[2], hi[3]));
  } else {
    a = 0;
    b = static_cast<int>(Lk);
  }
  *first = a < b ? a : 0;
  *last = b;
}

// Workgroups go to the eight XCDs in turn, each with an L2 of its own: the
// logical block of a launch of n blocks such that each XCD works on
// neighbours, which read the same rows. (Where the work of an entry depends on
// its mask, taking the blocks in turn balances the XCDs better than sharing
// keys helps: 2x4096x2048 with ragged masks, 16 heads of 128 on 4 key heads,
// P in bf16 alone, forward 204 us against 188, dQ 242 against 228.)
__device__ __forceinline__ uint32_t xcd_block(uint32_t blk, uint32_t n) {
  const uint32_t each = n / 8, left = n % 8, x = blk % 8;
  return x * each + (x < left ? x : left) + blk / 8;
}

// 1 / l for the softmax's sum: 0 for a row that kept no key, NaN stays NaN
__device__ __forceinline__ float softmax_scale(float l) { return l > 0.0f || l != l ? 1.0f / l : 0.0f; }
// the log of the softmax's sum from the running maximum (base 2) and sum
__device__ __forceinline__ float softmax_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// A lane column of acc (EP values of one row) times f into row[0 .. E), or
// zeros when !live, whatever acc holds; nothing when !keep. Halves of the
// wavefront swap register groups so that each lane stores 8 adjacent values;
// `wide` needs E % 8 == 0 and a 16-byte aligned row.
template <typename T, int EP, bool FULL>
__device__ __forceinline__ void store_col(T* row, bool keep, bool live, int E, bool wide,
                                          const f32x16 (&acc)[EP / 32], float f, int lane) {
  const int hh = lane >> 5;
#pragma unroll
  for (int et = 0; et < EP / 32; ++et) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[et][8 * h + k] * f),
                                                        __float_as_uint(acc[et][8 * h + 4 + k] * f),
                                                        false, false);
        v[k] = live ? __uint_as_float(r[0]) : 0.0f;
        v[4 + k] = live ? __uint_as_float(r[1]) : 0.0f;
      }
      const int e0 = et * 32 + h * 16 + hh * 8;
      if (!keep || (!FULL && e0 >= E)) continue;
      if (FULL || wide) {
        run_st<8>(row, e0, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (e0 + k < E) Store<T>::put(row, e0 + k, v[k]);
      }
    }
  }
}

// Rows of a [rows][E] operand on their way into an LDS tile of ROWS rows, by
// THREADS threads: 16-byte pieces held in registers between the load and the
// write.
template <typename T, int EP, int ROWS, int THREADS> struct Stage {
  static constexpr int kPieces = EP * static_cast<int>(sizeof(T)) / 16;   // of one row
  static constexpr int kEach = (ROWS * kPieces + THREADS - 1) / THREADS;
  static constexpr bool kExact = ROWS * kPieces % THREADS == 0;
  u32x4 v[kEach];
  __device__ static __forceinline__ int row(int tid, int i) { return (tid + i * THREADS) / kPieces; }
  __device__ static __forceinline__ int e0(int tid, int i) {
    return (tid + i * THREADS) % kPieces * (16 / static_cast<int>(sizeof(T)));
  }
  // at(r): the address of row r of the tile, which has to exist. Whole pieces
  // past the row's end are read from its start, and zeroed by write(): a
  // branch per piece, or a look at what is still on its way, would end the
  // loads in flight (8192 rows, 2048 keys, 16
  // heads of 72, forward: 217 us with them, 150 without).
  template <bool FULL, typename F> __device__ __forceinline__ void load(int tid, int E, bool wide, F&& at) {
    if (FULL || wide) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = row(tid, i), e = e0(tid, i);
        v[i] = load16<T, true>(at(kExact || r < ROWS ? r : ROWS - 1), FULL || e < E ? e : 0, E, true);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = row(tid, i);
        v[i] = load16<T, false>(at(kExact || r < ROWS ? r : ROWS - 1), e0(tid, i), E, false);
      }
    }
  }
  // keep(r): whether the row's values are kept (zeros otherwise)
  template <bool FULL, typename F> __device__ __forceinline__ void write(char* tile, int tid, int E, F&& keep) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int r = row(tid, i), e = e0(tid, i);
      if (kExact || r < ROWS)
        *reinterpret_cast<u32x4*>(tile + r * tile_pitch<T, EP>() + e * static_cast<int>(sizeof(T))) =
            keep(r) && (FULL || e < E) ? v[i] : u32x4{0u, 0u, 0u, 0u};
    }
  }
};

// the kernels' EP for a head of E values
inline int attn_ep(int64_t E) { return E <= 32 ? 32 : (E <= 64 ? 64 : (E <= 96 ? 96 : 128)); }

}  // namespace gspn
