// Products of INT4 weights with many activation rows (layout of the weights: moeq_int4.h).
//
//   y_tr = sum_g s_rg sum_{k in g} (q_rk - z_rg) x_tk
//
// on the fp16 matrix instruction (16 x 16 x 32). Codes become fp16 integers q - z, exact: the
// nibble is laid into the mantissa of 1024 (or of 64, four bits higher) by a mask-and-or, and a
// packed addition takes 1024 + z away, nine vector operations for eight values. Activations come
// as fp16, every row times a power of two of its own (k_int4_rows): a bf16 value keeps all its
// bits down to 2^-31 of its row's largest (fp16's last bit, 2^-24, is the eighth of 2^-17 there, and
// the largest is 2^14 or more) and is rounded by up to 2^-39 of it below; the intermediate h, fp32, is
// two fp16 terms, 22 bits down to 2^-17 of its row's largest, by up to 2^-39 of it off below.
// A group's sum, of exact products, is multiplied by its scale in fp32 and added up (a vector
// operation per output and group); sums are fp32. The scale multiplied into the weight instead,
// rounded to fp16, would save those operations (bf16 outputs, tiles of 256 x 128: 2048 x 4096 x 4096
// 76 us a call instead of 83-92, 8192 x 8192 x 4096 565 instead of 710-755), but every weight would be off by up to
// 2^-11 and a token's outputs would differ with the batch it is in, by 8e-4.
//
// Activations are operand A (its rows: tokens), so a lane's outputs belong to one weight row and
// need one scale per group. A work-group's waves stand WM x WN, each with NM row tiles of weights
// and 16 NT of its tokens, which lie in LDS in steps of 128 columns (three buffers; a row's 16-byte
// chunks at chunk ^ (row % 16), so that the sixteen rows of an operand touch all banks once).
// Weights go from memory to registers, a step ahead.
//
// One barrier per step, before the products of its last 32 columns, whose operands are in
// registers by then: behind it the step's buffer is free for the copy three steps on, and the
// next step's first operands are read under those products. A wave decodes the next fragment of
// weights between the products of one, as spread by the scheduling groups: left to the compiler,
// the vector unit's and the matrix unit's work took turns.
//
// Measured: linear 2048 x 4096 x 4096, groups of 128, 81 us (0.84 PFLOP/s; its rows 7), 8192 x 8192 x
// 4096, groups of 64, zero points, about 690 in a stream of calls: the vector unit's work beside the
// products, decoding and scales, is what bounds it. Tiles of 96 and 128 tokens instead of 64 were
// slower (2048 x 4096 x 4096 107 and 111 us a call; 8192 x 8192 x 4096 640, two rounds fewer, and 964,
// where registers spill). 256 experts of 4096 x 2048, 6 to a token, 2048 tokens, groups of 128:
// gate/up 650, down 590. For few tokens to an expert the weight stream bounds it: 16 tokens, groups
// of 32, 4.9 TB/s.
#pragma once
#include <hip/hip_ext.h>

#include "moeq_int4.h"
#include "moeq_int8.h"
#include "moeq_tiled.h"

namespace moeq {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- product

constexpr int I4_STAGES = 3;  // buffers of activations, and sets of weights in registers

__device__ __forceinline__ uint32_t pk_add(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, a) + __builtin_bit_cast(f16x2_t, b));
}
__device__ __forceinline__ uint32_t pk_half(float v) {
  const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)v);
  return h | (h << 16);
}

// Spread V vector operations among M matrix instructions, and R operand reads behind the first.
template <int M, int V, int R, int I = 0>
__device__ __forceinline__ void spread() {
  if constexpr (I < M) {
    constexpr int v = (I + 1) * V / M - I * V / M;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (I < R) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x002, v, 0);
    spread<M, V, R, I + 1>();
  }
}

// One work-group's tile: row block bm of expert e, activation rows first .. + count (LINEAR), or
// the pairs perm[0 .. count); count at most 16 NT WN. WK: waves that share an output, each with
// every WK-th step of columns; a step below is then WK of those, and the first wave adds up.
template <int KIND, int GP, bool ZEROS, int WM, int WN, int NM, int NT, int WK = 1>
__device__ __forceinline__ void int4_tile(const Int4Rows& P, uint8_t* lds, int bm, int e, int first, int count,
                                          const int32_t* perm) {
  constexpr int TOK = 16 * NT * WN;
  constexpr int TERMS = KIND == I4_DOWN_PART ? 2 : 1, ROWS = WK * TERMS * TOK, STAGE = ROWS * 256;
  constexpr int WAVES = WM * WN * WK;
  static_assert(WK == 1 || KIND == I4_LINEAR, "steps shared by waves");
  // copies of a wave per step, four LDS rows each (the waves past the last row repeat the first)
  constexpr int COPIES = (ROWS / 4 + WAVES - 1) / WAVES;
  static_assert(ROWS % (4 * COPIES) == 0, "no copy passes the end");
  constexpr int PAIRS = KIND == I4_GATE_UP ? 2 : 1;  // matrices side by side
  constexpr int RT = NM / PAIRS;               // row tiles of a wave
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ktiles = int4_ktiles(P.cols), kpad = ktiles * 128, rtiles = int4_rtiles(P.rows);
  const int wm = wave % WM, wn = wave / WM % WN, wk = wave / (WM * WN);
  const int row0 = 4 * COPIES * wave % ROWS;
  const int steps = (ktiles + WK - 1) / WK, last = steps - 1;

  // this lane's part of a wave's copies: LDS row row0 + 4 i + lane / 16, term by term
  const uint16_t* abase = P.act + (size_t)first * kpad;  // LINEAR
  int off[COPIES];
  const uint8_t* from[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; i++) {
    const int row = row0 + 4 * i + (lane >> 4), term = row / TOK % TERMS, t = min(row % TOK, count - 1);
    const int chunk = 16 * ((lane & 15) ^ (row & 15));
    if constexpr (KIND == I4_LINEAR) {
      off[i] = t * kpad * 2 + chunk;
    } else {
      const size_t a = KIND == I4_GATE_UP ? perm[t] / P.top_k : perm[t];
      from[i] = reinterpret_cast<const uint8_t*>(P.act + (a * TERMS + term) * kpad) + chunk;
    }
  }
  auto column = [&](int k, int s) { return WK == 1 ? s : min(s * WK + k, ktiles - 1); };  // in tiles of 128
  auto copy = [&](int s, int to) {  // step s into buffer `to`
    uint8_t* dst = lds + to * STAGE + 256 * row0;
#pragma unroll
    for (int i = 0; i < COPIES; i++) {
      if constexpr (KIND == I4_LINEAR)
        copy16(reinterpret_cast<const int8_t*>(abase), off[i], column((row0 + 4 * i) / TOK, s) * 256, dst + 1024 * i);
      else
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from[i] + (size_t)s * 256),
                                         (__attribute__((address_space(3))) void*)(dst + 1024 * i), 16, 0, 0);
    }
  };

  // row tiles of this wave; past the end the last one, whose outputs are not stored
  const uint8_t* wp[NM];
  const uint8_t* sp[NM];
  const uint8_t* zp[NM];
#pragma unroll
  for (int m = 0; m < NM; m++) {
    const WeightRef& w = P.w[PAIRS == 2 ? m / RT : 0];
    const size_t tile = (size_t)min((bm * WM + wm) * RT + m % RT, rtiles - 1) * ktiles;
    wp[m] = w.data + (size_t)e * w.estride + tile * 1024 + 16 * lane;
    const uint8_t* s = w.scales + (size_t)e * w.sestride;
    sp[m] = s + (tile * 16 + n) * GP * 2;
    zp[m] = s + int4_zeros_at(P.fmt, P.rows, P.cols) + (tile * 16 + n) * GP;
  }
  struct Step {
    u32x4 w[NM];
    u32x2 s[NM];
    uint32_t z[NM];
  };
  auto fetch = [&](int step, Step& v) {
    const int s = column(wk, step);
#pragma unroll
    for (int m = 0; m < NM; m++) {
      v.w[m] = ld16(wp[m] + (size_t)s * 1024);
      const uint8_t* q = sp[m] + (size_t)s * 32 * GP;
      if constexpr (GP == 1) v.s[m][0] = *reinterpret_cast<const uint16_t*>(q);
      else if constexpr (GP == 2) v.s[m][0] = *reinterpret_cast<const uint32_t*>(q);
      else v.s[m] = *reinterpret_cast<const u32x2*>(q);
      if constexpr (ZEROS) {
        const uint8_t* z = zp[m] + (size_t)s * 16 * GP;
        if constexpr (GP == 1) v.z[m] = *z;
        else if constexpr (GP == 2) v.z[m] = *reinterpret_cast<const uint16_t*>(z);
        else v.z[m] = *reinterpret_cast<const uint32_t*>(z);
      }
    }
  };

  f32x4_t tot[NM][NT], acc[NM][NT];
#pragma unroll
  for (int m = 0; m < NM; m++)
#pragma unroll
    for (int t = 0; t < NT; t++) tot[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // masks and the numbers whose mantissas take the nibbles, held in registers: one v_and_or each
  uint32_t m0 = 0x000F000Fu, m1 = 0x00F000F0u, o0 = 0x64006400u, o1 = 0x54005400u;
  asm volatile("" : "+s"(m0), "+s"(m1), "+v"(o0), "+v"(o1));
  Step w[I4_STAGES];
  f16x8_t xv[2][TERMS][NT];  // operands of these 32 columns and the next
  u32x4 d;                   // the next fragment of weights
  auto read = [&](int buf, int j, int to) {
    const uint8_t* x = lds + buf * STAGE + (wk * TOK + wn * NT * 16 + n) * 256 + 16 * ((4 * j + g) ^ n);
#pragma unroll
    for (int a = 0; a < TERMS; a++)
#pragma unroll
      for (int t = 0; t < NT; t++) xv[to][a][t] = *reinterpret_cast<const f16x8_t*>(x + (a * TOK + t * 16) * 256);
  };
  auto decode = [&](const Step& v, int j, int m) {
    const int gi = j * GP / 4;
    const float z = ZEROS ? (float)(v.z[m] >> (8 * gi) & 255u) : 8.0f;
    const uint32_t c0 = pk_half(-1024.0f - z), c1 = pk_half(-64.0f - z), lo = v.w[m][j], hi = lo >> 8;
    d = u32x4{pk_add((lo & m0) | o0, c0), pk_add((lo & m1) | o1, c1), pk_add((hi & m0) | o0, c0), pk_add((hi & m1) | o1, c1)};
  };
  // Copies and fetches past the last step repeat it (into buffers that nobody reads), so that
  // every wait counts the same. Waits for copies count the copies behind them alone.
#pragma unroll
  for (int i = 0; i < I4_STAGES; i++) {
    if (i < I4_STAGES - 1) fetch(min(i, last), w[i]);
    asm volatile("" ::: "memory");
    copy(min(i, last), i);
    asm volatile("" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * COPIES) : "memory");  // copy 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  read(0, 0, 0);
  decode(w[0], 0, 0);
  auto step = [&](int s, auto B) {  // B: s % I4_STAGES
    constexpr int b = decltype(B)::value, nb = (b + 1) % I4_STAGES;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const bool begin = j % (4 / GP) == 0, end = (j + 1) % (4 / GP) == 0;
      if (j < 3) {
        read(b, j + 1, (j + 1) & 1);
      } else {
        // the next step's copies, and all reads of this one's; the copies behind may be on their way
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(COPIES) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        fetch(min(s + 2, last), w[(b + 2) % I4_STAGES]);
        asm volatile("" ::: "memory");
        copy(min(s + 3, last), b);
        read(nb, 0, 0);
      }
#pragma unroll
      for (int m = 0; m < NM; m++) {
        const f16x8_t now = __builtin_bit_cast(f16x8_t, d);
        if (m + 1 < NM) decode(w[b], j, m + 1);
        else if (j < 3) decode(w[b], j + 1, 0);
        else decode(w[nb], 0, 0);
#pragma unroll
        for (int t = 0; t < NT; t++) {
          f32x4_t c = begin ? f32x4_t{0.f, 0.f, 0.f, 0.f} : acc[m][t];
          c = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[j & 1][0][t], now, c, 0, 0, 0);
          if constexpr (TERMS == 2) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[j & 1][TERMS - 1][t], now, c, 0, 0, 0);
          acc[m][t] = c;
        }
        if (end) {
          float f = half_bits_f32(w[b].s[m][(j * GP / 4) / 2] >> (16 * (j * GP / 4 & 1)));
          if (WK > 1 && s * WK + wk >= ktiles) f = 0.f;  // past the end: the last step again
#pragma unroll
          for (int t = 0; t < NT; t++)
#pragma unroll
            for (int r = 0; r < 4; r++) tot[m][t][r] = __builtin_fmaf(f, acc[m][t][r], tot[m][t][r]);
        }
      }
      if (end) spread<NM * NT * TERMS, NM * (11 + 4 * NT), TERMS * NT>();
      else spread<NM * NT * TERMS, NM * 11, TERMS * NT>();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int s = 0; s < steps; s += I4_STAGES) {
    step(s, Count<0>{});
    if (s + 1 < steps) step(s + 1, Count<1>{});
    if (s + 2 < steps) step(s + 2, Count<2>{});
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives the work-group
  if constexpr (WK > 1) {
    static_assert((WK - 1) * WM * WN * NM * NT * 1024 <= I4_STAGES * STAGE, "the other waves' sums");
    auto sums = [&](int k, int m, int t) {
      return reinterpret_cast<f32x4_t*>(lds) + ((((k - 1) * WN * WM + wn * WM + wm) * NM + m) * NT + t) * 64 + lane;
    };
    __syncthreads();
    if (wk > 0)
#pragma unroll
      for (int m = 0; m < NM; m++)
#pragma unroll
        for (int t = 0; t < NT; t++) *sums(wk, m, t) = tot[m][t];
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int k = 1; k < WK; k++)
#pragma unroll
      for (int m = 0; m < NM; m++)
#pragma unroll
        for (int t = 0; t < NT; t++) tot[m][t] += *sums(k, m, t);
  }

  // lane (n, g), register r of token tile t: token 16 t + 4 g + r, weight row n of the tile. Of the
  // token's and the tensor's powers of two, a sum takes the token's first where the tensor's is 1 or
  // more, and last where it is less: one by itself may carry it out of fp32's range and the other back.
  const int t0 = wn * NT * 16 + 4 * g;
  float s2[PAIRS];
#pragma unroll
  for (int m = 0; m < PAIRS; m++) s2[m] = P.w[m].scale2[e];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    float c[PAIRS][4][2];
    size_t at[4];
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int i = min(t0 + 16 * t + r, count - 1);
      const size_t a = KIND == I4_LINEAR ? (size_t)(first + i) : (size_t)perm[i];
      float as = P.act_scale[KIND == I4_GATE_UP ? a / P.top_k : a];
      if constexpr (KIND == I4_DOWN_PART) as *= P.rw[a];
#pragma unroll
      for (int m = 0; m < PAIRS; m++) {
        c[m][r][0] = s2[m] >= 1.f ? as : s2[m];
        c[m][r][1] = s2[m] >= 1.f ? s2[m] : as;
      }
      at[r] = a * P.rows;
    }
#pragma unroll
    for (int m = 0; m < RT; m++) {
      const int row = ((bm * WM + wm) * RT + m) * 16 + n;
      if (row >= P.rows) continue;
      float bias = 0.f;
      if constexpr (KIND == I4_LINEAR)
        if (P.bias) bias = P.bias[row];
#pragma unroll
      for (int r = 0; r < 4; r++) {
        if (t0 + 16 * t + r >= count) continue;
        float v = tot[m][t][r] * c[0][r][0] * c[0][r][1];
        if constexpr (PAIRS == 2) v = silu_mul(v, tot[RT + m][t][r] * c[1][r][0] * c[1][r][1]);
        if constexpr (KIND == I4_LINEAR) {
          v += bias;
          if (P.out_bf16) {
            ((uint16_t*)P.y)[at[r] + row] = (uint16_t)f32_bf16_rne_nan(v);
            continue;
          }
        }
        ((float*)P.y)[at[r] + row] = v;
      }
    }
  }
}

template <int GP, bool ZEROS, int WM, int WN, int NM, int NT, int WK>
__global__ __launch_bounds__(64 * WM * WN * WK, WM * WN * WK / 4) void k_int4_linear(Int4Rows P) {
  constexpr int TOK = 16 * NT * WN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[I4_STAGES * WK * TOK * 256];
  int bm, bn;
  tile_of(blockIdx.x, (int4_rtiles(P.rows) + WM * NM - 1) / (WM * NM), (P.T + TOK - 1) / TOK, bm, bn);
  int4_tile<I4_LINEAR, GP, ZEROS, WM, WN, NM, NT, WK>(P, lds, bm, P.expert, bn * TOK, min(TOK, P.T - bn * TOK), nullptr);
}

// A chunk of up to PREFILL_MC pairs of an expert, 16 NT of them at a time; as many token tiles are
// multiplied as there are. WAVES: to a SIMD.
template <int KIND, int GP, bool ZEROS, int WM, int NM, int NT, int WAVES>
__global__ __launch_bounds__(64 * WM, WAVES) void k_int4_experts(Int4Rows P) {
  static_assert(NT == 1 || NT == 2 || NT == 4, "token tiles below");
  constexpr int TOK = 16 * NT, RT = NM / (KIND == I4_GATE_UP ? 2 : 1);
  __shared__ __attribute__((aligned(16))) uint8_t lds[I4_STAGES * (KIND == I4_DOWN_PART ? 2 : 1) * TOK * 256];
  const int nbm = (int4_rtiles(P.rows) + WM * RT - 1) / (WM * RT);
  // the row blocks of a chunk of tokens on one XCD: they share the tokens in its L2
  const int l = blockIdx.x / 8, q = l / nbm * 8 + (int)(blockIdx.x % 8), bm = l % nbm;
  if (q >= P.route.n_chunks()[0]) return;
  const int e = P.route.chunk_e()[q];
  const int p0 = P.route.offsets()[e], m0 = P.route.chunk_m0()[q];
  const int count = min(PREFILL_MC, P.route.offsets()[e + 1] - p0 - m0);
  const int32_t* perm = P.route.perm() + p0 + m0;
  if (e >= P.n_experts) {  // ids out of range: their h, or parts, are zeros
    for (int i = threadIdx.x; i < count * 16 * WM * RT; i += 64 * WM) {
      const int r = bm * 16 * WM * RT + i % (16 * WM * RT);
      if (r < P.rows) ((float*)P.y)[(size_t)perm[i / (16 * WM * RT)] * P.rows + r] = 0.f;
    }
    return;
  }
  for (int m = 0; m < count; m += TOK) {
    const int here = min(TOK, count - m);
    if (m > 0) __syncthreads();  // the tile before has been read
    if (NT == 1 || here <= 16) int4_tile<KIND, GP, ZEROS, WM, 1, NM, 1>(P, lds, bm, e, 0, here, perm + m);
    else if (NT == 2 || here <= 32) int4_tile<KIND, GP, ZEROS, WM, 1, NM, NT == 1 ? 1 : 2>(P, lds, bm, e, 0, here, perm + m);
    else if (here <= 48) int4_tile<KIND, GP, ZEROS, WM, 1, NM, NT == 4 ? 3 : 1>(P, lds, bm, e, 0, here, perm + m);
    else int4_tile<KIND, GP, ZEROS, WM, 1, NM, NT>(P, lds, bm, e, 0, here, perm + m);
  }
}

template <int GP, int WM, int WN, int NM, int NT, int WK = 1>
hipError_t linear(const Int4Rows& p, hipStream_t s) {
  const long rows = 16 * WM * NM, tok = 16 * WN * NT;
  const dim3 g((unsigned)((p.rows + rows - 1) / rows * ((p.T + tok - 1) / tok))), b(64 * WM * WN * WK);
  if (int4_zeros(p.fmt)) hipLaunchKernelGGL((k_int4_linear<GP, true, WM, WN, NM, NT, WK>), g, b, 0, s, p);
  else hipLaunchKernelGGL((k_int4_linear<GP, false, WM, WN, NM, NT, WK>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int KIND, int GP, int WM, int NM, int NT, int WAVES>
hipError_t experts(const Int4Rows& p, hipStream_t s, const LaunchEvents* ev = nullptr) {
  constexpr int RT = NM / (KIND == I4_GATE_UP ? 2 : 1);
  const long items = RouteView::max_chunks(p.n_experts, p.T * p.top_k);
  const dim3 g((unsigned)((int4_rtiles(p.rows) + WM * RT - 1) / (WM * RT) * ((items + 7) / 8 * 8)));
  auto k = int4_zeros(p.fmt) ? k_int4_experts<KIND, GP, true, WM, NM, NT, WAVES> : k_int4_experts<KIND, GP, false, WM, NM, NT, WAVES>;
  if (ev) hipExtLaunchKernelGGL(k, g, dim3(64 * WM), 0, s, ev->start, ev->stop, 0, p);
  else hipLaunchKernelGGL(k, g, dim3(64 * WM), 0, s, p);
  return hipGetLastError();
}

}  // namespace

}  // namespace moeq
