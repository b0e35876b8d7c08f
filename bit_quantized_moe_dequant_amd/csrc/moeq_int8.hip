// 8-bit integer linear: per-token quantisation and the product on the integer matrix
// instructions.
//
//   quantise  s_t = fl32(max_k |x_tk| / 127),  q_tk = clamp(rne(fl32(x_tk / s_t)), -127, 127)
//             (an all-zero token: s = 0, codes 0; one with an infinity or a NaN: s = NaN,
//             codes 0, so that its outputs are NaN and no other token's are)
//   product   y_tr = (sum_k q_tk W_rk) s_t w_r (+ b_r)
//
// The sum runs in int32 and is exact: |q W| <= 2^14 and cols <= 65536 keep it below
// 2^31 in any order, so every split of K below gives the same bits. The scales
// multiply the sum once, in fp32: int32 -> fp32 is the first rounding, two products
// and the bias follow, and bf16 outputs are rounded once more at the store.
#include "moeq_grid.h"
#include "moeq_int8.h"
#include "moeq_tiled.h"

namespace moeq {

namespace {

// ---------------------------------------------------------------- quantisation
// One work-group per token, 16 values per thread and step (two 16-byte loads for
// bf16, four for fp32; one 16-byte store of codes). The maximum is taken over the
// values' bits with the sign cleared, as integers: that orders finite values like
// their magnitudes and puts infinities and NaNs above all of them.
constexpr int Q_THREADS = 256;
constexpr int Q_HOLD = 2;  // steps whose values stay in registers between the two passes (K <= 8192)

template <int IN_F32> struct QVals {
  static constexpr int NV = IN_F32 ? 4 : 2;
  u32x4 v[NV];
  __device__ __forceinline__ void load(const void* x, size_t i) {
#pragma unroll
    for (int j = 0; j < NV; j++) v[j] = ld16((const uint8_t*)x + i * (IN_F32 ? 4 : 2) + 16 * j);
  }
  __device__ __forceinline__ uint32_t amax_bits(uint32_t m) const {
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int k = 0; k < 4; k++) {
        if (IN_F32) {
          m = max(m, v[j][k] & 0x7FFFFFFFu);
        } else {
          m = max(m, (v[j][k] << 16) & 0x7FFF0000u);
          m = max(m, v[j][k] & 0x7FFF0000u);
        }
      }
    return m;
  }
  __device__ __forceinline__ float at(int i) const {
    if (IN_F32) return u2f(v[i / 4][i % 4]);
    const uint32_t w = v[i / 8][(i % 8) / 2];
    return u2f((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ u32x4 codes(float s, float r) const {
    float f[16];
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 16; i++) f[i] = at(i);
    int8_codes(f, s, r, w);
    return u32x4{w[0], w[1], w[2], w[3]};
  }
};

template <int IN_F32>
__global__ __launch_bounds__(Q_THREADS) void k_quant_int8(const void* x, int K, int8_t* q, float* scale) {
  __shared__ uint32_t red[Q_THREADS / 64];
  const int tid = threadIdx.x;
  const size_t row = (size_t)blockIdx.x * K;
  const int n = K / 16;  // chunks of 16 values
  QVals<IN_F32> held[Q_HOLD];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < Q_HOLD; j++)
    if (tid + j * Q_THREADS < n) held[j].load(x, row + 16 * (size_t)(tid + j * Q_THREADS));
#pragma unroll
  for (int j = 0; j < Q_HOLD; j++)
    if (tid + j * Q_THREADS < n) m = held[j].amax_bits(m);
  for (int c = tid + Q_HOLD * Q_THREADS; c < n; c += Q_THREADS) {
    QVals<IN_F32> v;
    v.load(x, row + 16 * (size_t)c);
    m = v.amax_bits(m);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < Q_THREADS / 64; w++) m = max(m, red[w]);
  const float s = int8_scale(m), r = 1.0f / s;
  if (tid == 0) scale[blockIdx.x] = s;
#pragma unroll
  for (int j = 0; j < Q_HOLD; j++) {
    const int c = tid + j * Q_THREADS;
    if (c < n) *reinterpret_cast<u32x4*>(q + row + 16 * (size_t)c) = held[j].codes(s, r);
  }
  for (int c = tid + Q_HOLD * Q_THREADS; c < n; c += Q_THREADS) {
    QVals<IN_F32> v;
    v.load(x, row + 16 * (size_t)c);
    *reinterpret_cast<u32x4*>(q + row + 16 * (size_t)c) = v.codes(s, r);
  }
}

// ---------------------------------------------------------------- few tokens
// v_mfma_i32_16x16x64_i8: lane L holds 16 bytes of row L % 16 at K = 16 (L / 16) +
// [0, 16) of a 64-wide step, on both operands; output lane L register r is operand
// A's row 4 (L / 16) + r times operand B's row L % 16. Operand A is 16 weight rows,
// operand B 16 tokens, so a lane ends with four consecutive channels of one token.
// A work-group takes 16 weight rows and NT tiles of 16 tokens; its waves take
// contiguous runs of K steps and their int32 partials meet in LDS.
// MATS = 2: a gate/up pair, h = silu(gate) * up in fp32.
template <int MATS, int NT, int U, int S_WAVES>
__global__ __launch_bounds__(64 * S_WAVES) void k_int8_few(Int8Params P) {
  __shared__ int32_t red[MATS][S_WAVES][16 * NT][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * 16;
  const int t0 = blockIdx.y * 16 * NT;
  const int K = P.cols;
  const int steps = (K + 63) / 64;
  const int spw = (steps + S_WAVES - 1) / S_WAVES;
  const int s0 = wave * spw, s1 = min(s0 + spw, steps);
  const int8_t* wr[MATS];
#pragma unroll
  for (int m = 0; m < MATS; m++) wr[m] = (m ? P.w2 : P.w) + (size_t)min(r0 + n, P.rows - 1) * K;
  const int8_t* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) xr[t] = P.xq + (size_t)min(t0 + 16 * t + n, P.T - 1) * K;
  i32x4 acc[MATS][NT];
#pragma unroll
  for (int m = 0; m < MATS; m++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[m][t] = i32x4{0, 0, 0, 0};
  for (int s = s0; s < s1; s += U) {
    u32x4 wv[U][MATS], xv[U][NT];
    // K steps past the end and the last step's bytes past K: the last 16 bytes again
    // (in bounds), with zeros in the weights' place
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int m = 0; m < MATS; m++) wv[u][m] = ld16(wr[m] + min(64 * (s + u) + 16 * g, K - 16));
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int t = 0; t < NT; t++) xv[u][t] = ld16(xr[t] + min(64 * (s + u) + 16 * g, K - 16));
#pragma unroll
    for (int u = 0; u < U; u++) {
#pragma unroll
      for (int m = 0; m < MATS; m++) {
        if (s + u >= s1 || 64 * (s + u) + 16 * g >= K) wv[u][m] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int t = 0; t < NT; t++)
          acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv[u][m]),
                                                             __builtin_bit_cast(i32x4, xv[u][t]), acc[m][t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MATS; m++)
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int r = 0; r < 4; r++) red[m][wave][16 * t + n][4 * g + r] = acc[m][t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * NT; i += 64 * S_WAVES) {
    const int tk = i >> 4, c = i & 15;
    if (t0 + tk < P.T && r0 + c < P.rows) {
      int v[MATS];
#pragma unroll
      for (int m = 0; m < MATS; m++) {
        v[m] = 0;
#pragma unroll
        for (int w = 0; w < S_WAVES; w++) v[m] += red[m][w][tk][c];
      }
      const float xs = P.xs[t0 + tk];
      float f = (float)v[0] * xs * P.ws[r0 + c];
      if constexpr (MATS == 2) f = silu_mul(f, (float)v[1] * xs * P.ws2[r0 + c]);
      else f = finish(P, t0 + tk, r0 + c, f);
      store_out(P, t0 + tk, r0 + c, f);
    }
  }
}

// Four consecutive channels r .. r + 3 of token t from their sums.
__device__ __forceinline__ void store4(const Int8Params& P, int t, int r, float xs, int v0, int v1, int v2, int v3) {
  if (t >= P.T || r >= P.rows) return;
  const int v[4] = {v0, v1, v2, v3};
  if (P.vec4) {  // rows a multiple of 4 and aligned outputs: all four exist, one store
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; e++) f[e] = finish(P, t, r + e, (float)v[e] * xs * P.ws[r + e]);
    if (P.out_bf16) {
      const u32x2 o = {f32_bf16_rne_nan(f[0]) | (f32_bf16_rne_nan(f[1]) << 16),
                       f32_bf16_rne_nan(f[2]) | (f32_bf16_rne_nan(f[3]) << 16)};
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(P.y) + (size_t)t * P.rows + r) = o;
    } else {
      const u32x4 o = {f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3])};
      *reinterpret_cast<u32x4*>(reinterpret_cast<float*>(P.y) + (size_t)t * P.rows + r) = o;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; e++)
    if (r + e < P.rows) store_out(P, t, r + e, finish(P, t, r + e, (float)v[e] * xs * P.ws[r + e]));
}

// ---------------------------------------------------------------- many tokens
// RUNS 1: bf16 outputs without bias or added term; 2: the others; for both rows a multiple
// of 8 and everything 16-byte aligned. 0: any.
template <int WM, int WN, int TM, int TN, int STAGES, int G_BK, int Q, int SPREAD, int RUNS>
__global__ __launch_bounds__(64 * WM * WN) void k_int8_tiled(Int8Params P) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  __shared__ __attribute__((aligned(16))) uint8_t lds[tiled_lds<WM, WN, TM, TN, STAGES, G_BK>()];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = P.cols;
  int bm, bn;
  tile_of(blockIdx.x, (P.rows + BM - 1) / BM, (P.T + BN - 1) / BN, bm, bn);
  const int r0 = bm * BM, t0 = bn * BN;
  i32x16 acc[TM][TN];
  tiled_product<MmaI8, WM, WN, TM, TN, STAGES, G_BK, Q, SPREAD>(P.w + (size_t)r0 * K, P.rows - r0, P.xq + (size_t)t0 * K,
                                                               P.T - t0, K, K, lds, acc);
  const int wm = wave % WM, wn = wave / WM;
  const int n = lane & 31, g = lane >> 5;
  if constexpr (RUNS == 1) {
    // Through LDS, 32 tokens at a time and each wave for itself (past the last barrier nobody
    // reads operands any more), so that a store writes whole runs of channels: stored from
    // the registers, 8 bytes to a lane, a wave's store touches 32 rows (2048 x 4096 x 4096:
    // 44.6 against 38.3 us).
    constexpr int CH = TM * 32, PITCH = 2 * CH + 16;
    static_assert(WM * WN * 32 * PITCH <= sizeof(lds), "the outputs of 32 tokens fit");
    uint8_t* mine = lds + wave * 32 * PITCH;
    const int rb = r0 + wm * CH;
#pragma unroll
    for (int j = 0; j < TN; j++) {
      const int tb = t0 + (wn * TN + j) * 32, t = min(tb + n, P.T - 1);
      const float xs = P.xs[t];
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int c = i * 32 + 8 * q + 4 * g;
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int r = min(rb + c + e, P.rows - 1);
            f[e] = (float)acc[i][j][4 * q + e] * xs * P.ws[r];
          }
          *reinterpret_cast<u32x2*>(mine + n * PITCH + 2 * c) =
              u32x2{f32_bf16_rne_nan(f[0]) | (f32_bf16_rne_nan(f[1]) << 16),
                    f32_bf16_rne_nan(f[2]) | (f32_bf16_rne_nan(f[3]) << 16)};
          __builtin_amdgcn_sched_barrier(0);  // the scales of all channels at once would spill
        }
      constexpr int LPR = CH / 8;  // lanes to a row
#pragma unroll
      for (int k = 0; k < 32 * LPR / 64; k++) {
        const int row = k * (64 / LPR) + lane / LPR, c = 8 * (lane % LPR);
        const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * PITCH + 2 * c);
        if (tb + row < P.T && rb + c < P.rows)
          *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(P.y) + (size_t)(tb + row) * P.rows + rb + c) = v;
      }
    }
  } else if constexpr (RUNS == 2) {
    // The same in fp32, 64 channels at a time, so that bias and added term are read in whole
    // runs too (2048 x 4096 x 2048 with an added term: 56.7 us from the registers, 35 so; fp32
    // outputs of 2048 x 4096 x 4096 48 and 43, of 8192^3 534 and 505).
    constexpr int CB = (TM < 2 ? TM : 2) * 32, PITCH = 4 * CB + 16;
    static_assert(WM * WN * 32 * PITCH <= sizeof(lds), "the outputs of 32 tokens fit");
    uint8_t* mine = lds + wave * 32 * PITCH;
#pragma unroll
    for (int j = 0; j < TN; j++) {
      const int tb = t0 + (wn * TN + j) * 32;
      const float xs = P.xs[min(tb + n, P.T - 1)];
#pragma unroll
      for (int i0 = 0; i0 < TM; i0 += CB / 32) {
        const int rb = r0 + (wm * TM + i0) * 32;
#pragma unroll
        for (int i = 0; i < CB / 32; i++)
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const int c = i * 32 + 8 * q + 4 * g;
            u32x4 f;
#pragma unroll
            for (int e = 0; e < 4; e++) f[e] = f2u((float)acc[i0 + i][j][4 * q + e] * xs * P.ws[min(rb + c + e, P.rows - 1)]);
            *reinterpret_cast<u32x4*>(mine + n * PITCH + 4 * c) = f;
            __builtin_amdgcn_sched_barrier(0);
          }
        constexpr int LPR = CB / 8;  // lanes to a row
#pragma unroll
        for (int k = 0; k < 32 * LPR / 64; k++) {
          const int row = k * (64 / LPR) + lane / LPR, t = tb + row, r = rb + 8 * (lane % LPR);
          const u32x4 v[2] = {*reinterpret_cast<const u32x4*>(mine + row * PITCH + 32 * (lane % LPR)),
                              *reinterpret_cast<const u32x4*>(mine + row * PITCH + 32 * (lane % LPR) + 16)};
          if (t < P.T && r < P.rows) {
            u32x4 o[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
              u32x4 b = u32x4{0u, 0u, 0u, 0u}, a = b;
              if (P.bias) b = ld16(P.bias + r + 4 * h);
              if (P.add) a = ld16(P.add + (size_t)t * P.rows + r + 4 * h);
#pragma unroll
              for (int e = 0; e < 4; e++) {
                float f = u2f(v[h][e]);
                if (P.bias) f += u2f(b[e]);
                if (P.add) f += u2f(a[e]);
                o[h][e] = P.out_bf16 ? f32_bf16_rne_nan(f) : f2u(f);
              }
            }
            const size_t at = (size_t)t * P.rows + r;
            if (P.out_bf16) {
              *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(P.y) + at) =
                  u32x4{o[0][0] | (o[0][1] << 16), o[0][2] | (o[0][3] << 16), o[1][0] | (o[1][1] << 16), o[1][2] | (o[1][3] << 16)};
            } else {
              *reinterpret_cast<u32x4*>(reinterpret_cast<float*>(P.y) + at) = o[0];
              *reinterpret_cast<u32x4*>(reinterpret_cast<float*>(P.y) + at + 4) = o[1];
            }
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < TN; j++) {
      const int t = t0 + (wn * TN + j) * 32 + n;
      const float xs = t < P.T ? P.xs[t] : 0.f;
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int q = 0; q < 4; q++)  // four consecutive channels
          store4(P, t, r0 + (wm * TM + i) * 32 + 8 * q + 4 * g, xs, acc[i][j][4 * q], acc[i][j][4 * q + 1],
                 acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
    }
  }
}

// A gate/up pair: h = silu(gate) * up, fp32, rows a multiple of 4, y 16-byte aligned. A wave
// ends with the gate and the up sums of the same 32 channels.
template <int WM, int WN, int TN, int STAGES, int G_BK, int Q, int SPREAD>
__global__ __launch_bounds__(64 * WM * WN) void k_gu_int8_tiled(Int8Params P) {
  constexpr int BM = WM * 32, BN = WN * TN * 32;  // channels, tokens
  __shared__ __attribute__((aligned(16))) uint8_t lds[tiled_lds<WM, WN, 2, TN, STAGES, G_BK>()];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = P.cols;
  int bm, bn;
  tile_of(blockIdx.x, (P.rows + BM - 1) / BM, (P.T + BN - 1) / BN, bm, bn);
  const int r0 = bm * BM, t0 = bn * BN;
  i32x16 acc[2][TN];
  tiled_product<MmaI8, WM, WN, 2, TN, STAGES, G_BK, Q, SPREAD, Nothing, true>(
      P.w + (size_t)r0 * K, P.rows - r0, P.xq + (size_t)t0 * K, P.T - t0, K, K, lds, acc, {}, P.w2 + (size_t)r0 * K);
  const int wm = wave % WM, wn = wave / WM;
  const int n = lane & 31, g = lane >> 5;
#pragma unroll
  for (int j = 0; j < TN; j++) {
    const int t = t0 + (wn * TN + j) * 32 + n;
    const float xs = P.xs[min(t, P.T - 1)];
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int r = r0 + wm * 32 + 8 * q + 4 * g;
      if (t < P.T && r < P.rows) {
        u32x4 f;
#pragma unroll
        for (int e = 0; e < 4; e++)
          f[e] = f2u(silu_mul((float)acc[0][j][4 * q + e] * xs * P.ws[r + e], (float)acc[1][j][4 * q + e] * xs * P.ws2[r + e]));
        *reinterpret_cast<u32x4*>(reinterpret_cast<float*>(P.y) + (size_t)t * P.rows + r) = f;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// ---------------------------------------------------------------- exact weights
__global__ __launch_bounds__(256) void k_dequant_int8(const int8_t* w, const float* ws, int rows, int cols, float* out) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < (size_t)rows * cols; i += (size_t)gridDim.x * 256)
    out[i] = (float)w[i] * ws[i / cols];
}

template <int WM, int WN, int TM, int TN, int STAGES, int BK, int Q, int SPREAD>
hipError_t go_tiled(const Int8Params& p, hipStream_t s) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  const long blocks = (long)((p.rows + BM - 1) / BM) * ((p.T + BN - 1) / BN);
  if (blocks > GRID_MAX_BLOCKS) return hipErrorInvalidValue;
  const dim3 g((unsigned)blocks), b(64 * WM * WN);
  const bool runs = p.rows % 8 == 0 && ((uintptr_t)p.y | (uintptr_t)p.bias | (uintptr_t)p.add) % 16 == 0;
  if (runs && p.out_bf16 && !p.bias && !p.add)
    hipLaunchKernelGGL((k_int8_tiled<WM, WN, TM, TN, STAGES, BK, Q, SPREAD, 1>), g, b, 0, s, p);
  else if (runs)
    hipLaunchKernelGGL((k_int8_tiled<WM, WN, TM, TN, STAGES, BK, Q, SPREAD, 2>), g, b, 0, s, p);
  else
    hipLaunchKernelGGL((k_int8_tiled<WM, WN, TM, TN, STAGES, BK, Q, SPREAD, 0>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int WM, int WN, int TN, int STAGES, int BK, int Q, int SPREAD>
hipError_t go_gu_tiled(const Int8Params& p, hipStream_t s) {
  constexpr int BM = WM * 32, BN = WN * TN * 32;
  const long blocks = (long)((p.rows + BM - 1) / BM) * ((p.T + BN - 1) / BN);
  if (blocks > GRID_MAX_BLOCKS) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_gu_int8_tiled<WM, WN, TN, STAGES, BK, Q, SPREAD>), dim3((unsigned)blocks), dim3(64 * WM * WN), 0, s, p);
  return hipGetLastError();
}

template <int MATS, int NT, int U, int S_WAVES = 8>
hipError_t go_few(const Int8Params& p, hipStream_t s) {
  const dim3 g((unsigned)((p.rows + 15) / 16), (unsigned)((p.T + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((k_int8_few<MATS, NT, U, S_WAVES>), g, dim3(64 * S_WAVES), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_int8(int in_f32, const void* x, int T, int K, int8_t* q, float* scale, hipStream_t s) {
  if (T < 1 || K < 16 || K % 16) return hipErrorInvalidValue;
  for (long t = 0; t < T; t += 1 << 22) {  // a grid holds below 2^32 threads
    const dim3 g((unsigned)(T - t < (1 << 22) ? T - t : 1 << 22));
    const uint8_t* xt = (const uint8_t*)x + (size_t)t * K * (in_f32 ? 4 : 2);
    if (in_f32) hipLaunchKernelGGL(k_quant_int8<1>, g, dim3(Q_THREADS), 0, s, xt, K, q + (size_t)t * K, scale + t);
    else hipLaunchKernelGGL(k_quant_int8<0>, g, dim3(Q_THREADS), 0, s, xt, K, q + (size_t)t * K, scale + t);
  }
  return hipGetLastError();
}

hipError_t launch_dequant_int8(const int8_t* w, const float* ws, int rows, int cols, float* out, hipStream_t s) {
  const size_t n = (size_t)rows * cols;
  hipLaunchKernelGGL(k_dequant_int8, dim3((unsigned)(n < (1u << 28) ? (n + 255) / 256 : 1 << 20)), dim3(256), 0, s, w, ws, rows, cols, out);
  return hipGetLastError();
}

// T up to 16, rounded up to a power of two times cols at most 65536 (16 chunks to a lane).
bool few_bf16_fits(int T, int cols) {
  if (T < 1 || T > 16) return false;
  const FewPlan f = few_plan(T, cols, 8);
  return f.tpw * f.cpl <= 16;
}

namespace {
template <int MATS, int TPW, int CPL, int IN_F32>
__global__ __launch_bounds__(512) void k_int8_few_x(Int8Params P) { int8_few<MATS, TPW, CPL, 8, IN_F32>(P, blockIdx.x); }

template <int MATS, int IN_F32>
hipError_t few_x(const Int8Params& p0, hipStream_t s) {
  Int8Params p = p0;
  const FewPlan f = few_plan(p.T, p.cols, 8);
  p.wpt = f.wpt;
  const dim3 g((unsigned)((p.rows + 15) / 16)), b(512);
  if (f.tpw == 1 && f.cpl <= 1) hipLaunchKernelGGL((k_int8_few_x<MATS, 1, 1, IN_F32>), g, b, 0, s, p);
  else if (f.tpw == 1 && f.cpl <= 4) hipLaunchKernelGGL((k_int8_few_x<MATS, 1, 4, IN_F32>), g, b, 0, s, p);
  else if (f.tpw == 1) hipLaunchKernelGGL((k_int8_few_x<MATS, 1, 16, IN_F32>), g, b, 0, s, p);
  else if (f.cpl <= 2) hipLaunchKernelGGL((k_int8_few_x<MATS, 2, 2, IN_F32>), g, b, 0, s, p);
  else hipLaunchKernelGGL((k_int8_few_x<MATS, 2, 8, IN_F32>), g, b, 0, s, p);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_linear_int8_few(const Int8Params& p, bool in_f32, hipStream_t s) {
  if (!few_bf16_fits(p.T, p.cols) || p.rows < 1 || p.rows > INT8_MAX_ROWS || p.cols < 16 || p.cols % 16) return hipErrorInvalidValue;
  return in_f32 ? few_x<1, 1>(p, s) : few_x<1, 0>(p, s);
}

namespace {
hipError_t linear_int8(Int8Params p, hipStream_t s) {
  p.vec4 = p.rows % 4 == 0 && (uintptr_t)p.y % (p.out_bf16 ? 8 : 16) == 0;
  if (p.T <= 16) return go_few<1, 1, 8>(p, s);
  if (p.T <= 32) return go_few<1, 2, 8>(p, s);
  // The tile with the smallest estimate. A step of 128 bytes of K takes a CU, by how many
  // work-groups it holds (measured, us): 32 x 64 0.21, 0.29, 0.39, then 0.13 each; 64 x 64
  // 0.25, 0.44, then 0.22 each; 128 x 64 0.41, 0.72, then 0.36 each; 256 x 128 1.1 each and
  // 256 x 256 2.0 each, one at a time. At 4096 x 4096 (us): T = 64 10.0 with 32 x 64 and 11.7
  // with 64 x 64; T = 256 12.9, 12.2 and 17.2 with 128 x 64; T = 1000 -, 30.7, 26.2 and 30.5
  // with 256 x 128; T = 2048 48 with 128 x 64, 38.4 with 256 x 128, 54 with 256 x 256; T =
  // 4096 75 and 67.
  auto per_cu = [&](int bm, int bn) {
    return (double)(((long)((p.rows + bm - 1) / bm) * ((p.T + bn - 1) / bn) + 255) / 256);
  };
  const double n0 = per_cu(32, 64), n1 = per_cu(64, 64), n2 = per_cu(128, 64);
  const double c[5] = {n0 <= 1 ? 0.21 : n0 <= 2 ? 0.29 : 0.13 * n0, n1 <= 1 ? 0.25 : 0.22 * n1,
                       n2 <= 1 ? 0.41 : 0.36 * n2, 1.1 * per_cu(256, 128), 2.0 * per_cu(256, 256)};
  int best = 0;
  for (int i = 1; i < 5; i++)
    if (c[i] < c[best]) best = i;
  switch (best) {
    case 0: return go_tiled<1, 2, 1, 1, 4, 128, 4, 1>(p, s);
    case 1: return go_tiled<2, 2, 1, 1, 4, 128, 4, 1>(p, s);
    case 2: return go_tiled<4, 2, 1, 1, 3, 128, 4, 1>(p, s);
    case 3: return go_tiled<4, 2, 2, 2, 3, 128, 1, 2>(p, s);
  }
  return go_tiled<2, 4, 4, 2, 2, 128, 1, 2>(p, s);
}
}  // namespace

hipError_t launch_linear_int8(const Int8Params& p, hipStream_t s) {
  if (p.T < 1 || p.rows < 1 || p.rows > INT8_MAX_ROWS || p.cols < 16 || p.cols % 16 || p.cols > INT8_MAX_COLS)
    return hipErrorInvalidValue;
  const long most = int8_tokens(p.rows);
  for (long t0 = 0; t0 < p.T; t0 += most) {
    Int8Params q = p;
    q.T = (int)(p.T - t0 < most ? p.T - t0 : most);
    q.xq += (size_t)t0 * p.cols;
    q.xs += t0;
    q.y = (uint8_t*)p.y + (size_t)t0 * p.rows * (p.out_bf16 ? 2 : 4);
    if (p.add) q.add = p.add + (size_t)t0 * p.rows;
    const hipError_t e = linear_int8(q, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

namespace {
hipError_t gate_up_int8(const Int8Params& p, hipStream_t s) {
  if (p.T <= 16) return go_few<2, 1, 4>(p, s);
  if (p.T <= 32) return go_few<2, 2, 4>(p, s);
  auto per_cu = [&](int bm, int bn) {
    return (double)(((long)((p.rows + bm - 1) / bm) * ((p.T + bn - 1) / bn) + 255) / 256);
  };
  // The tile (channels x tokens) with the smallest estimate, as in linear_int8: a step of 128
  // bytes takes a CU that holds n work-groups 0.23 + 0.22 n us with 32 x 64, 0.35 + 0.34 n
  // with 64 x 64, 0.93 n with 128 x 64 and 1.2 n with 128 x 128. At 2 x 2048 x 4096 (us), with
  // go_few's tile of 16 x 64 first: T = 64 16.0, 14.7, 21.5, 29.4, 31.7; T = 256 29.6, 14.5,
  // 22.5, 28.5, 34.2; T = 1024 108, 36.0, 32.9, 29.8, 35.1; T = 2048 216, 63.8, 54.8, 53.6,
  // 39.8. T = 32: 11.8 with go_few's tile of 16 x 32, 14.2 with 32 x 64.
  const double c[4] = {0.23 + 0.22 * per_cu(32, 64), 0.35 + 0.34 * per_cu(64, 64), 0.93 * per_cu(128, 64),
                       1.2 * per_cu(128, 128)};
  int best = 0;
  for (int i = 1; i < 4; i++)
    if (c[i] < c[best]) best = i;
  switch (best) {
    case 0: return go_gu_tiled<1, 2, 1, 4, 128, 4, 1>(p, s);
    case 1: return go_gu_tiled<2, 2, 1, 3, 128, 4, 1>(p, s);
    case 2: return go_gu_tiled<4, 2, 1, 3, 128, 4, 1>(p, s);
  }
  return go_gu_tiled<4, 2, 2, 3, 128, 1, 2>(p, s);
}
}  // namespace

hipError_t launch_gate_up_int8(const Int8Params& p, hipStream_t s) {
  if (p.T < 1 || p.rows < 1 || p.rows > INT8_MAX_ROWS || p.cols < 16 || p.cols % 16 || p.cols > INT8_MAX_COLS ||
      p.rows % 4 || (uintptr_t)p.y % 16)
    return hipErrorInvalidValue;
  const long most = int8_tokens(p.rows);
  for (long t0 = 0; t0 < p.T; t0 += most) {
    Int8Params q = p;
    q.T = (int)(p.T - t0 < most ? p.T - t0 : most);
    q.xq += (size_t)t0 * p.cols;
    q.xs += t0;
    q.y = (float*)p.y + (size_t)t0 * p.rows;
    const hipError_t e = gate_up_int8(q, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

__global__ __launch_bounds__(256) void k_to_bf16(const float* x, size_t n, uint16_t* y) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
    y[i] = (uint16_t)f32_bf16_rne_nan(x[i]);
}

hipError_t launch_to_bf16(const float* x, size_t n, uint16_t* y, hipStream_t s) {
  const size_t b = (n + 255) / 256;
  hipLaunchKernelGGL(k_to_bf16, dim3((unsigned)(b < 4096 ? b : 4096)), dim3(256), 0, s, x, n, y);
  return hipGetLastError();
}

}  // namespace moeq
