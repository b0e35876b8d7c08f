// Device side of the INT8 linears that more than one kernel uses: the epilogue, and the
// product of a few tokens that are quantised where they are used.
#pragma once
#include "moeq_device.h"
#include "moeq_kernels.h"
#include "moeq_wave.h"

namespace moeq {

// fp32 -> bf16 bits, round to nearest even, for any input: NaNs stay NaN (quiet), infinities
// are kept.
__device__ __forceinline__ uint32_t f32_bf16_rne_nan(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  return (u & 0x7FFFFFFFu) > 0x7F800000u ? ((u >> 16) | 0x40u) : f32_bf16_rne(f);
}

// Token scale of the int8 quantisation from the bits of the row's largest magnitude,
// and the code of one value under it (IEEE divisions: the codes are defined by them).
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  return amax_bits >= 0x7F800000u ? u2f(0x7FC00000u) : u2f(amax_bits) / 127.0f;
}
__device__ __forceinline__ int int8_code(float v, float s) {
  const float q = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(v / s), -127.0f), 127.0f);
  return s > 0.f ? (int)q : 0;
}
// N codes at a time, four to a word, r = 1 / s. The product v r is within 127.5 * 2^-23 of
// fl(v / s), so its nearest integer is the code unless it lies that near a half: then (and
// where r is not finite: s zero, NaN or tiny) the divisions are made. Adding 1.5 * 2^23
// rounds to the nearest integer, ties to even, and leaves it in the low bits.
template <int N>
__device__ __forceinline__ void int8_codes(const float (&v)[N], float s, float r, uint32_t (&out)[N / 4]) {
  constexpr float MAGIC = 12582912.0f;
  float far = 0.f;
#pragma unroll
  for (int j = 0; j < N / 4; j++) {
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float m = __builtin_fmaf(v[4 * j + k], r, MAGIC);
      far = __builtin_fmaxf(far, __builtin_fabsf(__builtin_fmaf(v[4 * j + k], r, MAGIC - m)));
      t[k] = f2u(m);
    }
    out[j] = __builtin_amdgcn_perm(t[1], t[0], 0x0C0C0400u) | __builtin_amdgcn_perm(t[3], t[2], 0x04000C0Cu);
  }
  if (!(far < 0.499976f) || !(r <= 3.402823466e38f)) {
#pragma unroll
    for (int j = 0; j < N / 4; j++) {
      out[j] = 0;
#pragma unroll
      for (int k = 0; k < 4; k++) out[j] |= ((uint32_t)int8_code(v[4 * j + k], s) & 255u) << (8 * k);
    }
  }
}

// The bias and the added term of one output; not fused with the product before, which other
// forms of the store keep in memory in between: every form gives the same bits.
__device__ __forceinline__ float finish(const Int8Params& P, size_t t, int r, float v) {
#pragma clang fp contract(off)
  if (P.bias) v += P.bias[r];
  if (P.add) v += P.add[t * P.rows + r];
  return v;
}

__device__ __forceinline__ void store_out(const Int8Params& P, size_t t, int r, float v) {
  if (P.out_bf16) reinterpret_cast<uint16_t*>(P.y)[t * P.rows + r] = (uint16_t)f32_bf16_rne_nan(v);
  else reinterpret_cast<float*>(P.y)[t * P.rows + r] = v;
}

// y[t] (+)= W q(x[t]) for up to 16 bf16 or fp32 tokens (dynamic quantisation), or a gate/up
// pair's silu(gate) * up (MATS = 2), by one work-group of W waves for 16 weight rows. Every
// work-group makes the codes of its tokens itself, in LDS, while its weight loads are on
// their way: a second launch and a round trip of the codes through memory cost more at
// these sizes than the repeated conversion (one token, 4096 x 4096, in a graph over twenty
// weights: 8.7 us in two launches, 6.1 in one; 7.7 and 4.4 where the weight stays in L2;
// sixteen tokens, 2048 x 4096: 9.2 and 9.0). Wave w works on tokens w / wpt + (W / wpt) j (wpt waves to a token, TPW
// tokens to a wave), lane l on chunks of 8 values l, l + 64 wpt, ... (CPL of them), so the
// codes take at most 512 W TPW CPL bytes. The product is that of k_int8_few.
template <int MATS, int TPW, int CPL, int W, int IN_F32>
__device__ __forceinline__ void int8_few(const Int8Params& P, int block) {
  constexpr int U = 8;               // K steps of weights in flight
  constexpr int NV = IN_F32 ? 2 : 1;  // 16-byte loads of a chunk
  constexpr int TOK = W * TPW < 16 ? W * TPW : 16;
  __shared__ __attribute__((aligned(16))) uint8_t code[512 * W * TPW * CPL + 16 * TOK + 64];  // rows K + 16 apart
  __shared__ int32_t red[MATS][W][16][17];
  __shared__ uint32_t top[W][2];
  __shared__ float sc[16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = block * 16;
  const int K = P.cols, pitch = K + 16;
  const int wpt = P.wpt, per = W / wpt;  // waves to a token, tokens at a time
  const int sub = wave % wpt;

  // tokens first, then the weights: the conversion waits for the former only
  u32x4 v[TPW][CPL][NV];
#pragma unroll
  for (int j = 0; j < TPW; j++) {
    const int t = min(wave / wpt + per * j, P.T - 1);
#pragma unroll
    for (int c = 0; c < CPL; c++)
#pragma unroll
      for (int i = 0; i < NV; i++)  // chunks past the row's end repeat its last one
        v[j][c][i] = ld16((const uint8_t*)P.x + ((size_t)t * K + 8 * min(lane + 64 * (sub + wpt * c), K / 8 - 1)) * (IN_F32 ? 4 : 2) + 16 * i);
  }
  __builtin_amdgcn_sched_barrier(0);
  const int steps = (K + 63) / 64;
  const int spw = (steps + W - 1) / W;
  const int s0 = wave * spw, s1 = min(s0 + spw, steps);
  const int8_t* wr[MATS];
#pragma unroll
  for (int m = 0; m < MATS; m++) wr[m] = (m ? P.w2 : P.w) + (size_t)min(r0 + n, P.rows - 1) * K;
  u32x4 wv[U][MATS];
  auto load = [&](int s) {
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int m = 0; m < MATS; m++) wv[u][m] = ld16(wr[m] + min(64 * (s + u) + 16 * g, K - 16));
  };
  load(s0);
  __builtin_amdgcn_sched_barrier(0);

  uint32_t m[TPW];
#pragma unroll
  for (int j = 0; j < TPW; j++) {
    m[j] = 0;
#pragma unroll
    for (int c = 0; c < CPL; c++)
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int k = 0; k < 4; k++) {
          if (IN_F32) m[j] = max(m[j], v[j][c][i][k] & 0x7FFFFFFFu);
          else m[j] = max(max(m[j], (v[j][c][i][k] << 16) & 0x7FFF0000u), v[j][c][i][k] & 0x7FFF0000u);
        }
    m[j] = wave_max(m[j]);
    if (lane == 0) top[wave][j] = m[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < TPW; j++) {
    const int t = wave / wpt + per * j;
    for (int w = 0; w < wpt; w++) m[j] = max(m[j], top[wave - sub + w][j]);
    const float s = int8_scale(m[j]), r = 1.0f / s;
    if (t < P.T) {  // uniform
      if (sub == 0 && lane == 0) sc[t] = s;
#pragma unroll
      for (int c = 0; c < CPL; c++) {
        const int ch = lane + 64 * (sub + wpt * c);
        float f[8];
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 8; k++) {
          if (IN_F32) f[k] = u2f(v[j][c][k / 4][k % 4]);
          else f[k] = u2f(k & 1 ? v[j][c][0][k / 2] & 0xFFFF0000u : v[j][c][0][k / 2] << 16);
        }
        int8_codes(f, s, r, q);
        if (ch < K / 8) *reinterpret_cast<u32x2*>(&code[t * pitch + 8 * ch]) = u32x2{q[0], q[1]};
      }
    }
  }
  __syncthreads();

  const uint8_t* xr = code + min(n, P.T - 1) * pitch + 16 * g;
  i32x4 acc[MATS];
#pragma unroll
  for (int mt = 0; mt < MATS; mt++) acc[mt] = i32x4{0, 0, 0, 0};
  for (int s = s0; s < s1; s += U) {
    if (s > s0) load(s);
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (s + u < s1) {  // uniform; in the last step weights past K are zeros (and the codes there old bytes)
        const i32x4 xv = *reinterpret_cast<const i32x4*>(xr + 64 * (s + u));
#pragma unroll
        for (int mt = 0; mt < MATS; mt++) {
          if (64 * (s + u) + 16 * g >= K) wv[u][mt] = u32x4{0u, 0u, 0u, 0u};
          acc[mt] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv[u][mt]), xv, acc[mt], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MATS; mt++)
#pragma unroll
    for (int r = 0; r < 4; r++) red[mt][wave][n][4 * g + r] = acc[mt][r];
  __syncthreads();
  const int tk = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (threadIdx.x < 256 && tk < P.T && r0 + c < P.rows) {
    int sum[MATS];
#pragma unroll
    for (int mt = 0; mt < MATS; mt++) {
      sum[mt] = 0;
#pragma unroll
      for (int w = 0; w < W; w++) sum[mt] += red[mt][w][tk][c];
    }
    const float xs = sc[tk];
    float f = (float)sum[0] * xs * P.ws[r0 + c];
    if constexpr (MATS == 2) f = silu_mul(f, (float)sum[1] * xs * P.ws2[r0 + c]);
    else f = finish(P, tk, r0 + c, f);
    store_out(P, tk, r0 + c, f);
  }
}

// How T tokens of K values are shared out over W waves: a power of two of waves to a token;
// chunks per lane as the kernels are built for (0: more than any).
struct FewPlan {
  int wpt, tpw, cpl;
};
inline FewPlan few_plan(int T, int K, int W) {
  FewPlan f{W, 1, 0};
  while (f.wpt > 1 && W / f.wpt < T) f.wpt /= 2;
  f.tpw = (T + W / f.wpt - 1) / (W / f.wpt);
  f.cpl = (K / 8 + 64 * f.wpt - 1) / (64 * f.wpt);
  return f;
}

}  // namespace moeq
