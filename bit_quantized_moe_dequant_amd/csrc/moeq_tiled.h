// A tiled product W X^T of two row-major operands whose rows run along K, for the matrix
// instructions of shape 32 x 32 that take 16 bytes a lane (lane L: 16 bytes of row L % 32 at
// byte 16 (L / 32) of K; output register r: row (r % 4) + 8 (r / 4) + 4 (L / 32) of the
// first operand, row L % 32 of the second): int8 and bf16.
//
// A work-group holds BM x BN outputs. Both operands' next G_BK bytes of K are copied to LDS
// by the memory pipe itself (no registers), into a ring of STAGES buffers. A row's 16-byte
// chunks are stored at chunk ^ key(row): sixteen lanes that read the same chunk of sixteen
// rows touch all 64 banks once (with the row's low three bits as the key, half of the LDS
// cycles were bank conflicts: two 128-byte rows share the banks, and a row's parity and its
// key went together).
//
// One barrier per step: before the last batch of a step's operands is multiplied, all of
// them already in registers, every wave waits for its copies of the next step and for its
// own reads; past the barrier the buffer just read is free for the copy STAGES steps on
// and the next step's first operands are read, both under the last batch's products. The
// loop over whole steps has no branches (they cost a third of a 64 x 64 tile's time).
#pragma once
#include "moeq_device.h"
#include "moeq_wave.h"

namespace moeq {

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct MmaI8 {
  typedef i32x16 Acc;
  __device__ static __forceinline__ Acc mma(i32x4 a, i32x4 b, Acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
};
struct MmaBf16 {
  typedef f32x16 Acc;
  __device__ static __forceinline__ Acc mma(i32x4 a, i32x4 b, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};

// Tile of a work-group. Work-groups go to the eight XCDs in turn; each XCD is given a
// contiguous run of tiles, eight channel tiles wide, so that the tiles it works on at a
// time share operand rows in its L2.
__device__ __forceinline__ void tile_of(int b, int nbm, int nbn, int& bm, int& bn) {
  const int total = nbm * nbn, per = total / 8, rem = total % 8, xcd = b % 8;
  const int l = xcd * per + min(xcd, rem) + b / 8;
  constexpr int GM = 8;
  const int group = l / (GM * nbn), first = group * GM, width = min(GM, nbm - first), in = l - group * GM * nbn;
  bm = first + in % width;
  bn = in / width;
}

// 16 bytes per lane from base + off + step into LDS at dst + 16 lane (dst the wave's own).
__device__ __forceinline__ void copy16(const int8_t* base, int off, int step, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base), (short)0, 0x7FFFFFFF, 0x00020000),
      (__attribute__((address_space(3))) void*)dst, 16, off, step, 0, 0);
}

template <int N> struct Count {
  static constexpr int value = N;
};

// Spread a batch's R operand reads and V copies among its M products instead of all before
// them: a copy waits for its turn at the memory pipe, and what follows it waits with it.
template <int R, int V, int M, int I = 0>
__device__ __forceinline__ void interleave() {
  if constexpr (I < M) {
    constexpr int reads = (I + 1) * R / M - I * R / M, copies = (I + 1) * V / M - I * V / M;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one matrix instruction
    if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
    if constexpr (copies > 0) __builtin_amdgcn_sched_group_barrier(0x020, copies, 0);
    interleave<R, V, M, I + 1>();
  }
}

// acc = the tile's sums over K bytes (a multiple of 16, at least 16) of rows `pitch` bytes
// apart: wrows rows from wbase (channels), xrows from xbase (tokens); rows past them repeat
// the last. lds: tiled_lds<...>() bytes.
template <int WM, int WN, int TM, int TN, int STAGES, int G_BK>
constexpr int tiled_lds() {
  return STAGES * 32 * (WM * TM + WN * TN) * G_BK;
}

// after(s) is called behind step s's products and may change acc.
// PAIR (TM = 2): two first operands at once, whose rows take turns in blocks of 32:
// acc[0] holds the sums of wbase's rows, acc[1] those of w2base's at the same place; wrows
// counts the rows of one, of which a tile takes BM / 2.
struct Nothing {
  __device__ __forceinline__ void operator()(int) const {}
};
template <class M, int WM, int WN, int TM, int TN, int STAGES, int G_BK, int Q, int SPREAD, class After = Nothing,
          bool PAIR = false>
__device__ __forceinline__ void tiled_product(const int8_t* wbase, int wrows, const int8_t* xbase, int xrows, int pitch,
                                              int K, uint8_t* lds, typename M::Acc (&acc)[TM][TN], After after = {},
                                              const int8_t* w2base = nullptr) {
  static_assert(!PAIR || TM == 2, "a wave holds a block of each");
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32, WAVES = WM * WN;
  constexpr int ROWS = BM + BN;                 // rows of one buffer: channels, then tokens
  constexpr int CPR = G_BK / 16, RPC = 64 / CPR;  // chunks of a row, rows of a copy
  constexpr int WL = BM / RPC / WAVES, XL = BN / RPC / WAVES;  // a wave's copies per step
  constexpr int LOADS = WL + XL;
  constexpr int NB = G_BK / 32 / Q;             // operand batches of a step, Q matrix-instruction depths each
  static_assert(BM % (RPC * WAVES) == 0 && BN % (RPC * WAVES) == 0 && (G_BK == 128 || G_BK == 256), "whole copies");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // a copy: RPC rows of one operand, lane l the 16 bytes that are stored at row l / CPR, position l % CPR
  const int wrow = RPC * WL * wave, xrow = RPC * XL * wave;  // this wave's first rows of the tiles
  int off[LOADS];  // rows past the operand's end read its last row
  auto key = [](int row) { return G_BK == 128 ? (row >> 1) & 7 : row & 15; };
  auto c16 = [&](int row) { return 16 * ((lane & (CPR - 1)) ^ key(row)); };  // chunk at this lane's position
#pragma unroll
  for (int j = 0; j < WL; j++) {
    const int row = wrow + RPC * j + lane / CPR;
    off[j] = min(PAIR ? (row >> 6) * 32 + (row & 31) : row, wrows - 1) * pitch + c16(row);
  }
  // a copy's rows lie in one block of 32
  auto base = [&](int j) { return j >= WL ? xbase : PAIR && ((wrow + RPC * j) & 32) ? w2base : wbase; };
#pragma unroll
  for (int j = 0; j < XL; j++) {
    const int row = xrow + RPC * j + lane / CPR;
    off[WL + j] = min(row, xrows - 1) * pitch + c16(row);
  }
  const int full = K / G_BK, steps = (K + G_BK - 1) / G_BK;
  constexpr int BUF = ROWS * G_BK;
  // part `part` of step s, wholly inside K, into the buffer at byte `at` of the ring
  auto copy = [&](int s, int at, int part) {
#pragma unroll
    for (int j = part * LOADS / SPREAD; j < (part + 1) * LOADS / SPREAD; j++)
      copy16(base(j), off[j], s * G_BK, lds + at + (j < WL ? wrow + RPC * j : BM + xrow + RPC * (j - WL)) * G_BK);
  };
  // any step, none past the end; in the last, partial one chunks past K are zeros
  auto copy_any = [&](int s, int at, int part) {
    if (s < full) {
      copy(s, at, part);
    } else if (s < steps) {
#pragma unroll
      for (int j = part * LOADS / SPREAD; j < (part + 1) * LOADS / SPREAD; j++) {
        const int row = j < WL ? wrow + RPC * j : xrow + RPC * (j - WL);
        u32x4 v = u32x4{0u, 0u, 0u, 0u};
        if (s * G_BK + c16(row + lane / CPR) < K) v = ld16(base(j) + off[j] + (size_t)s * G_BK);
        *reinterpret_cast<u32x4*>(lds + at + (j < WL ? row : BM + row) * G_BK + 16 * lane) = v;
      }
    }
  };

  const int wm = wave % WM, wn = wave / WM;
  const int n = lane & 31, g = lane >> 5;
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = typename M::Acc{};
  i32x4 a[2][Q][TM], x[2][Q][TN];
  const uint8_t* la = lds + (wm * TM * 32 + n) * G_BK;
  const uint8_t* lx = lds + (BM + wn * TN * 32 + n) * G_BK;
  auto read = [&](int ring, int b, int to) {  // operands of batch b of the step in the buffer at `ring`
#pragma unroll
    for (int q = 0; q < Q; q++) {
      // operand tiles start at multiples of 32 rows
      const int at = ring + 16 * ((2 * (b * Q + q) + g) ^ key(n));
#pragma unroll
      for (int i = 0; i < TM; i++) a[to][q][i] = *reinterpret_cast<const i32x4*>(la + at + i * 32 * G_BK);
#pragma unroll
      for (int j = 0; j < TN; j++) x[to][q][j] = *reinterpret_cast<const i32x4*>(lx + at + j * 32 * G_BK);
    }
  };
  auto multiply = [&](int from) {
#pragma unroll
    for (int q = 0; q < Q; q++)
#pragma unroll
      for (int j = 0; j < TN; j++)
#pragma unroll
        for (int i = 0; i < TM; i++)
          acc[i][j] = M::mma(a[from][q][i], x[from][q][j], acc[i][j]);
  };
  // The compiler does not see that copies write LDS: a wave waits for its own by count.
  // `flying`: the steps whose copies may still be on their way.
  auto landed = [&](auto flying) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(flying)::value) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto next = [](int ring) { return ring + BUF == STAGES * BUF ? 0 : ring + BUF; };

#pragma unroll
  for (int s = 0; s < STAGES; s++)
#pragma unroll
    for (int part = 0; part < (s + 1 < STAGES ? SPREAD : 1); part++) copy_any(s, s * BUF, part);
  if (STAGES <= full) landed(Count<(STAGES - 2) * LOADS + LOADS / SPREAD>{});
  else landed(Count<0>{});
  read(0, 0, 0);
  int ring = 0, last = (STAGES - 1) * BUF;  // step s's buffer, and the one before
  // FULL: every copy made so far and the ones made here are of whole steps
  auto step = [&](int s, int at, auto FULL) {  // at: the register set that holds batch 0
#pragma unroll
    for (int b = 0; b < NB; b++) {
      const int cur = (at + b) & 1;
      const int part = b + 1 == NB ? 0 : b + 1;  // of step s - 1 + STAGES until the barrier, then of the next one
      if (b + 1 < NB) {
        read(ring, b + 1, cur ^ 1);
      } else {
        if constexpr (decltype(FULL)::value) landed(Count<(STAGES - 2) * LOADS>{});  // steps s + 2 .. s + STAGES - 1
        else landed(Count<0>{});
        last = ring;
        ring = next(ring);
        read(ring, 0, cur ^ 1);  // past the end: a buffer's old bytes, not used
      }
      if (part < SPREAD) {
        if constexpr (decltype(FULL)::value) copy(s + STAGES - (part ? 1 : 0), last, part);
        else copy_any(s + STAGES - (part ? 1 : 0), last, part);
      }
      multiply(cur);
      if constexpr (Q == 1) interleave<TM + TN, LOADS / SPREAD, TM * TN>();
    }
  };
  static_assert(SPREAD <= NB && LOADS % SPREAD == 0, "a step's copies are made within a step");
  constexpr int SWAP = NB % 2;  // one batch per step: the register sets swap roles every step
  int s = 0;
  for (; s + STAGES + 1 < full; s += 2) {
    step(s, 0, Count<1>{});
    after(s);
    step(s + 1, SWAP, Count<1>{});
    after(s + 1);
  }
  for (; s < steps; s += 2) {
    step(s, 0, Count<0>{});
    after(s);
    if (s + 1 < steps) {
      step(s + 1, SWAP, Count<0>{});
      after(s + 1);
    }
  }

}

}  // namespace moeq
