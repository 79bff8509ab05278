// The matrix products of the vocabulary loss: C = A B on matrix cores, with
// either operand stored along the contraction or across it.
//
// A workgroup of eight wavefronts (four for tiles of 64 x 64) owns BM x BN of C. The contraction advances
// 128 bytes of a row at a time (64 bf16 values, 32 fp32) through LDS in two
// buffers: while one is multiplied, the next stage's 16-byte pieces are on their
// way into registers and are written to the other buffer after it, so there
// is one barrier per stage. An operand stored along the contraction lies in LDS
// as [row][128 bytes], its 16-byte pieces swizzled by bits 1 to 3 of the
// row, so that 16 rows' pieces of a column meet every bank once; one stored across
// it lies as it is in memory, [k][BM or BN values], and is read by the
// transposing LDS read (bf16, runs of 64 bytes swizzled by the row) or value by value (fp32).
//
// Matrix units are busy 70 to 78 % of the cycles of tiles of 256 in bf16, and the
// card's power then holds the clock near 1.6 GHz, which is what bounds it: loads in a
// row instead of woven in 1825 us against 1589 (8192 x 50001 x 2304).
//
// Results are 32 x 32 tiles (v_mfma_f32_32x32x16_bf16, or v_mfma_f32_32x32x2_f32):
// lane l holds column l % 32 and the rows (i % 4) + 8 (i / 4) + 4 (l / 32), i < 16.
#pragma once

#include "gspn_attn.hpp"

namespace gspn {

// An operand: rows of `ld` values. Along the contraction (kAlong): element
// (m, k) is p[m * ld + k], m < outer, k < inner. Across it: element (m, k) is
// p[k * ld + m], k < outer, m < inner. Rows begin on 16 bytes, and `inner` is a
// multiple of 16 bytes. Pieces past the contraction's end are zeros, pieces past
// the result's edge are some others of the same tensor.
template <typename T> struct Operand {
  const T* p;
  int64_t ld;
  int64_t outer, inner;
};

__device__ __forceinline__ int tile_row(int i, int lane) { return (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5); }

template <typename T, bool A_ALONG, bool B_ALONG, int BM, int BN, int WM, int kWaves = 8> struct Product {
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kStep = 128 / sizeof(T);       // contraction of a stage
  static constexpr int kPer = 16 / sizeof(T);         // values in 16 bytes
  static constexpr int WN = kWaves / WM;              // wavefronts over M, over N
  static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;   // a wavefront's tiles
  static constexpr int kA = BM * 128, kStage = (BM + BN) * 128;
  static constexpr int kLds = 2 * kStage;
  static constexpr int kPA = BM * 8 / kThreads, kPB = BN * 8 / kThreads;   // pieces per thread and stage
  using Frag = typename Mma<T>::Frag;
  static_assert(BM % (32 * WM) == 0 && BN % (32 * WN) == 0 && BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0, "tiles");

  // what a row's pieces are swizzled by in LDS, of an operand across the contraction
  template <int W> __device__ static __forceinline__ int swizzle(int row) {
    if constexpr (sizeof(T) == 4) return ((row >> 2) & 1) << 3;
    else if constexpr (W == 64) return ((row >> 1) & 1) << 2;
    else return (row & 3) << 2;
  }

  // which piece of a stage this thread moves: row and first value of the n-th
  template <bool ALONG, int W> __device__ static __forceinline__ void piece(int n, int tid, int& row, int& at) {
    if constexpr (ALONG) {
      const int o = n * kThreads + tid;
      row = o >> 3;
      at = ((o & 7) ^ ((row >> 1) & 7)) * kPer;
    } else {
      constexpr int per = W * static_cast<int>(sizeof(T)) / 16;   // pieces of a row
      const int o = n * kThreads + tid;
      row = o / per;
      const int s = o % per;
      at = (s ^ swizzle<W>(row)) * kPer;
    }
  }

  // Moves an operand's stages from memory. Loads go through a buffer
  // descriptor whose range check gives zeros for a lane that asks past the end,
  // so the contraction's last stage needs no branch.
  template <bool ALONG, int W, int N> struct Mover {
    static constexpr uint32_t kRange = 0xfffffff0u;
    // rows of a stage between a thread's pieces (across: contraction indexes)
    static constexpr int kApart = ALONG ? kThreads / 8 : kThreads / (W * static_cast<int>(sizeof(T)) / 16);
    const char* base;      // the tile's first row at the stage's first contraction index
    uint32_t off[N];       // the thread's pieces from there
    int64_t step;          // bytes per stage
    int k0;                // contraction index of the first piece within a stage
    int left;              // contraction indexes left

    __device__ __forceinline__ void set(const Operand<T>& o, int64_t first, int64_t k, int64_t kend, int tid) {
      if constexpr (ALONG) base = reinterpret_cast<const char*>(o.p + first * o.ld + k);
      else base = reinterpret_cast<const char*>(o.p + k * o.ld + first);
      step = (ALONG ? kStep : kStep * o.ld) * static_cast<int64_t>(sizeof(T));
      left = static_cast<int>(kend - k);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        int row, at;
        piece<ALONG, W>(n, tid, row, at);
        if (n == 0) k0 = ALONG ? at : row;
        if constexpr (ALONG) {
          const int64_t r = first + row < o.outer ? row : o.outer - 1 - first;
          off[n] = static_cast<uint32_t>((r * o.ld + at) * static_cast<int64_t>(sizeof(T)));
        } else {
          const int64_t c = first + at < o.inner ? at : 0;
          off[n] = static_cast<uint32_t>((row * o.ld + c) * static_cast<int64_t>(sizeof(T)));
        }
      }
    }
    // piece n of the stage from memory, of the last stage to LDS
    __device__ __forceinline__ u32x4 load(int n) const {
      const auto buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, kRange, 0x00027000);
      const uint32_t at = (ALONG ? k0 : k0 + n * kApart) < left ? off[n] : 0xffffffffu;
      return __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, 0);
    }
    __device__ __forceinline__ void advance() {
      base += step;
      left -= kStep;
    }
    __device__ static __forceinline__ void store(char* lds, int n, const u32x4& r, int tid) {
      *reinterpret_cast<u32x4*>(lds + (n * kThreads + tid) * 16) = r;
    }
  };

  // fragment kk (of four in a stage) of the 32 rows from r0
  template <bool ALONG, int W> __device__ static __forceinline__ Frag frag(const char* lds, int r0, int kk, int lane) {
    if constexpr (ALONG) {
      const int row = r0 + (lane & 31);
      return *reinterpret_cast<const Frag*>(lds + row * 128 + (((2 * kk + (lane >> 5)) ^ ((lane >> 1) & 7)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      const int c = lane & 15, g = (lane >> 4) & 1, h = lane >> 5;
      const int row = 16 * kk + 8 * h + (c >> 2), col = r0 + 16 * g + 4 * (c & 3);
      const uint16_t* q = reinterpret_cast<const uint16_t*>(
          lds + row * (W * 2) + (((col >> 3) ^ swizzle<W>(row)) << 4) + (col & 7) * 2);
      const v4i16 lo = lds_read_tr(q), hi = lds_read_tr(q + 4 * W);
      return __builtin_bit_cast(Frag, v8i16{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w});
    } else {
      Frag f;
      const int col = r0 + (lane & 31), h = lane >> 5;
      const char* q = lds + (8 * kk + 4 * h) * (W * 4) + (((col >> 2) ^ swizzle<W>(4 * h)) << 4) + (col & 3) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const float*>(q + j * W * 4);
      return f;
    }
  }

  struct Frags {
    Frag a[2][MI], b[2][NI];
  };
  // fragments of quarter kk of a stage
  __device__ static __forceinline__ void read(const char* lds, int kk, int wm, int wn, int lane, Frags& f) {
#pragma unroll
    for (int i = 0; i < MI; ++i) f.a[kk & 1][i] = frag<A_ALONG, BM>(lds, wm + 32 * i, kk, lane);
#pragma unroll
    for (int j = 0; j < NI; ++j) f.b[kk & 1][j] = frag<B_ALONG, BN>(lds + kA, wn + 32 * j, kk, lane);
  }
  __device__ static __forceinline__ void multiply(int kk, const Frags& f, f32x16 (&acc)[MI][NI]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = Mma<T>::mma(f.a[kk & 1][i], f.b[kk & 1][j], acc[i][j]);
  }

  // The order of a quarter's instructions: its reads go out among the first
  // products, two before each, the stage's pieces (one write to LDS, one load)
  // among the others, so that none of them holds the matrix unit up.
  static constexpr int kReads = (MI * (A_ALONG ? 1 : (sizeof(T) == 2 ? 2 : 4)) + NI * (B_ALONG ? 1 : (sizeof(T) == 2 ? 2 : 4)));
  static constexpr int kProducts = MI * NI * (sizeof(T) == 2 ? 1 : 4);
  static constexpr int kEach = 2 * kReads > kProducts ? (2 * kReads + kProducts - 1) / kProducts : 1;
  template <int READS, int PIECES, int PRODUCTS> __device__ static __forceinline__ void weave() {
    if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS < kEach ? READS : kEach, 0);
    if constexpr (PRODUCTS > 0) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr bool move = PIECES > 0 && (PRODUCTS <= PIECES || READS <= kEach);
    if constexpr (move) {
      __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    if constexpr (READS > 0 || PIECES > 0 || PRODUCTS > 0)
      weave<(READS > kEach ? READS - kEach : 0), (move ? PIECES - 1 : PIECES), (PRODUCTS > 0 ? PRODUCTS - 1 : 0)>();
  }

  // acc += A[m0 ..][k .. kend) B[k .. kend)[n0 ..]; all threads of the workgroup.
  // A stage in four quarters, the fragments of the next one read before the
  // products of each. In the first three the next stage, loaded a whole stage
  // ago, goes to the other buffer and the one after it is asked for; the barrier
  // comes before the last quarter's products, whose fragments are in registers by
  // then, and they cover the first reads of the next stage.
  __device__ static __forceinline__ void run(const Operand<T>& A, const Operand<T>& B, int64_t m0, int64_t n0,
                                             int64_t k, int64_t kend, char* lds, f32x16 (&acc)[MI][NI]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
    if (kend <= k) return;
    Mover<A_ALONG, BM, kPA> ma;
    Mover<B_ALONG, BN, kPB> mb;
    ma.set(A, m0, k, kend, tid);
    mb.set(B, n0, k, kend, tid);
    const int stages = static_cast<int>((kend - k + kStep - 1) / kStep);
    constexpr int kPieces = kPA + kPB;
    u32x4 r[kPieces];
    auto load = [&](int n) { r[n] = n < kPA ? ma.load(n < kPA ? n : 0) : mb.load(n < kPA ? 0 : n - kPA); };
    auto store = [&](char* to, int n) {
      if (n < kPA) ma.store(to, n, r[n], tid);
      else mb.store(to + kA, n - kPA, r[n], tid);
    };
    auto fence = []() { __builtin_amdgcn_sched_barrier(0); };
    Frags f;
    int cur = 0;   // the stage in use: LDS offset
#pragma unroll
    for (int n = 0; n < kPieces; ++n) load(n);
    ma.advance();
    mb.advance();
#pragma unroll
    for (int n = 0; n < kPieces; ++n) store(lds, n);
#pragma unroll
    for (int n = 0; n < kPieces; ++n) load(n);   // past the end: zeros
    ma.advance();
    mb.advance();
    lds_barrier();
    read(lds, 0, wm, wn, lane, f);
    fence();
    constexpr int kThird = (kPieces + 2) / 3, kLast = kPieces - 2 * kThird;
    static_assert(kLast >= 0, "pieces over three quarters");
    for (int s = 1; s < stages; ++s) {
      const char* now = lds + cur;
      cur ^= kStage;
      char* next = lds + cur;
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        read(now, q + 1, wm, wn, lane, f);
#pragma unroll
        for (int n = q * kThird; n < (q + 1) * kThird && n < kPieces; ++n) {
          store(next, n);
          load(n);
        }
        multiply(q, f, acc);
        if (q < 2) weave<kReads, kThird, kProducts>();
        else weave<kReads, kLast, kProducts>();
        fence();
      }
      ma.advance();
      mb.advance();
      lds_barrier();
      read(next, 0, wm, wn, lane, f);
      multiply(3, f, acc);
      weave<kReads, 0, kProducts>();
      fence();
    }
    read(lds + cur, 1, wm, wn, lane, f);
    multiply(0, f, acc);
    read(lds + cur, 2, wm, wn, lane, f);
    multiply(1, f, acc);
    read(lds + cur, 3, wm, wn, lane, f);
    multiply(2, f, acc);
    multiply(3, f, acc);
    lds_barrier();
  }
};

}  // namespace gspn
