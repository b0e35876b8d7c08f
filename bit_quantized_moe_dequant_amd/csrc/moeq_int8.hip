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
#include "moeq_device.h"
#include "moeq_kernels.h"

namespace moeq {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// The bias and the added term of one output.
__device__ __forceinline__ float finish(const Int8Params& P, size_t t, int r, float v) {
  if (P.bias) v += P.bias[r];
  if (P.add) v += P.add[t * P.rows + r];
  return v;
}

__device__ __forceinline__ void store_out(const Int8Params& P, size_t t, int r, float v) {
  if (P.out_bf16) reinterpret_cast<uint16_t*>(P.y)[t * P.rows + r] = (uint16_t)f32_bf16_rne_nan(v);
  else reinterpret_cast<float*>(P.y)[t * P.rows + r] = v;
}

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
  __device__ __forceinline__ u32x4 codes(float s) const {
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t w = 0;
#pragma unroll
      for (int k = 0; k < 4; k++) w |= ((uint32_t)int8_code(at(4 * j + k), s) & 255u) << (8 * k);
      q[j] = w;
    }
    return q;
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
  const float s = int8_scale(m);
  if (tid == 0) scale[blockIdx.x] = s;
#pragma unroll
  for (int j = 0; j < Q_HOLD; j++) {
    const int c = tid + j * Q_THREADS;
    if (c < n) *reinterpret_cast<u32x4*>(q + row + 16 * (size_t)c) = held[j].codes(s);
  }
  for (int c = tid + Q_HOLD * Q_THREADS; c < n; c += Q_THREADS) {
    QVals<IN_F32> v;
    v.load(x, row + 16 * (size_t)c);
    *reinterpret_cast<u32x4*>(q + row + 16 * (size_t)c) = v.codes(s);
  }
}

// ---------------------------------------------------------------- few tokens
// v_mfma_i32_16x16x64_i8: lane L holds 16 bytes of row L % 16 at K = 16 (L / 16) +
// [0, 16) of a 64-wide step, on both operands; output lane L register r is operand
// A's row 4 (L / 16) + r times operand B's row L % 16. Operand A is 16 weight rows,
// operand B 16 tokens, so a lane ends with four consecutive channels of one token.
// A work-group takes 16 weight rows and NT tiles of 16 tokens; its waves take
// contiguous runs of K steps and their int32 partials meet in LDS.
constexpr int S_WAVES = 8;

// MATS = 2: a gate/up pair, h = silu(gate) * up in fp32.
template <int MATS, int NT, int U>
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

// ---------------------------------------------------------------- many tokens
// A tiled product on v_mfma_i32_32x32x32_i8 (lane L: 16 bytes of row L % 32 at K =
// 16 (L / 32); output register r: row (r % 4) + 8 (r / 4) + 4 (L / 32) of A, row
// L % 32 of B). A work-group holds BM channels x BN tokens; per 128-byte step of K
// both tiles are copied to LDS by the memory pipe itself (no registers), into one
// of two buffers while the other is multiplied. A row's eight 16-byte chunks are
// stored at chunk ^ (row & 7), so eight lanes reading the same chunk of eight rows
// touch all banks once.
constexpr int G_BK = 128;

template <int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64 * WM * WN) void k_int8_tiled(Int8Params P) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32, WAVES = WM * WN;
  constexpr int ROWS = BM + BN;                 // rows of one buffer: channels, then tokens
  constexpr int LOADS = ROWS / 8 / WAVES;       // copies per wave and step, eight rows each
  static_assert(ROWS % (8 * WAVES) == 0 && BM % 8 == 0, "whole copies");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * ROWS * G_BK];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = P.cols;
  const int nbm = (P.rows + BM - 1) / BM;
  const int bm = blockIdx.x % nbm, bn = blockIdx.x / nbm;
  const int r0 = bm * BM, t0 = bn * BN;

  // copy j of this wave: buffer rows 8 (wave LOADS + j) + lane / 8, chunk lane % 8
  const int8_t* src[LOADS];
#pragma unroll
  for (int j = 0; j < LOADS; j++) {
    const int row = 8 * (wave * LOADS + j) + (lane >> 3);
    const int c = (lane & 7) ^ (row & 7);
    src[j] = (row < BM ? P.w + (size_t)min(r0 + row, P.rows - 1) * K : P.xq + (size_t)min(t0 + row - BM, P.T - 1) * K) + 16 * c;
  }
  const int full = K / G_BK, steps = (K + G_BK - 1) / G_BK;
  auto copy = [&](int s, int buf) {
    uint8_t* dst = lds + buf * ROWS * G_BK;
    if (s < full) {
#pragma unroll
      for (int j = 0; j < LOADS; j++)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src[j] + (size_t)s * G_BK),
                                         (__attribute__((address_space(3))) void*)(dst + 8 * (wave * LOADS + j) * G_BK), 16, 0, 0);
    } else {  // the last, partial step: chunks past K are zeros
#pragma unroll
      for (int j = 0; j < LOADS; j++) {
        const int row = 8 * (wave * LOADS + j) + (lane >> 3);
        const int c = (lane & 7) ^ (row & 7);
        u32x4 v = u32x4{0u, 0u, 0u, 0u};
        if (s * G_BK + 16 * c < K) v = ld16(src[j] + (size_t)s * G_BK);
        *reinterpret_cast<u32x4*>(dst + row * G_BK + 16 * (lane & 7)) = v;
      }
    }
  };

  const int wm = wave % WM, wn = wave / WM;
  const int n = lane & 31, g = lane >> 5;
  i32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = i32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};

  copy(0, 0);
  for (int s = 0; s < steps; s++) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's copies of step s have landed
    __syncthreads();                                  // everybody's have, and step s - 1 has been read
    if (s + 1 < steps) copy(s + 1, (s + 1) & 1);
    const uint8_t* b = lds + (s & 1) * ROWS * G_BK;
#pragma unroll
    for (int k = 0; k < G_BK / 32; k++) {
      const int pos = 16 * ((2 * k + g) ^ (n & 7));  // tile rows start at multiples of 32: row & 7 = n & 7
      i32x4 a[TM], x[TN];
#pragma unroll
      for (int i = 0; i < TM; i++) a[i] = *reinterpret_cast<const i32x4*>(b + ((wm * TM + i) * 32 + n) * G_BK + pos);
#pragma unroll
      for (int j = 0; j < TN; j++) x[j] = *reinterpret_cast<const i32x4*>(b + (BM + (wn * TN + j) * 32 + n) * G_BK + pos);
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], x[j], acc[i][j], 0, 0, 0);
    }
  }

#pragma unroll
  for (int j = 0; j < TN; j++) {
    const int t = t0 + (wn * TN + j) * 32 + n;
    const float xs = t < P.T ? P.xs[t] : 0.f;
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {  // four consecutive channels
        const int r = r0 + (wm * TM + i) * 32 + 8 * q + 4 * g;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          if (t < P.T && r + e < P.rows) {
            store_out(P, t, r + e, finish(P, t, r + e, (float)acc[i][j][4 * q + e] * xs * P.ws[r + e]));
          }
        }
      }
  }
}

// ---------------------------------------------------------------- exact weights
__global__ __launch_bounds__(256) void k_dequant_int8(const int8_t* w, const float* ws, int rows, int cols, float* out) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < (size_t)rows * cols; i += (size_t)gridDim.x * 256)
    out[i] = (float)w[i] * ws[i / cols];
}

template <int WM, int WN, int TM, int TN>
hipError_t go_tiled(const Int8Params& p, hipStream_t s) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  const int blocks = ((p.rows + BM - 1) / BM) * ((p.T + BN - 1) / BN);
  hipLaunchKernelGGL((k_int8_tiled<WM, WN, TM, TN>), dim3((unsigned)blocks), dim3(64 * WM * WN), 0, s, p);
  return hipGetLastError();
}

template <int MATS, int NT, int U>
hipError_t go_few(const Int8Params& p, hipStream_t s) {
  const dim3 g((unsigned)((p.rows + 15) / 16), (unsigned)((p.T + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((k_int8_few<MATS, NT, U>), g, dim3(64 * S_WAVES), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_int8(int in_f32, const void* x, int T, int K, int8_t* q, float* scale, hipStream_t s) {
  if (T < 1 || K < 16 || K % 16) return hipErrorInvalidValue;
  if (in_f32) hipLaunchKernelGGL(k_quant_int8<1>, dim3((unsigned)T), dim3(Q_THREADS), 0, s, x, K, q, scale);
  else hipLaunchKernelGGL(k_quant_int8<0>, dim3((unsigned)T), dim3(Q_THREADS), 0, s, x, K, q, scale);
  return hipGetLastError();
}

hipError_t launch_dequant_int8(const int8_t* w, const float* ws, int rows, int cols, float* out, hipStream_t s) {
  const size_t n = (size_t)rows * cols;
  hipLaunchKernelGGL(k_dequant_int8, dim3((unsigned)(n < (1u << 28) ? (n + 255) / 256 : 1 << 20)), dim3(256), 0, s, w, ws, rows, cols, out);
  return hipGetLastError();
}

hipError_t launch_linear_int8(const Int8Params& p, hipStream_t s) {
  if (p.T < 1 || p.rows < 1 || p.cols < 16 || p.cols % 16 || p.cols > INT8_MAX_COLS) return hipErrorInvalidValue;
  if (p.T <= 16) return go_few<1, 1, 8>(p, s);
  if (p.T <= 64) return go_few<1, 4, 4>(p, s);
  if (p.T <= 128) return go_few<1, 8, 2>(p, s);
  const long tiles = (long)((p.rows + 255) / 256) * ((p.T + 255) / 256);
  if (tiles >= 200) return go_tiled<2, 4, 4, 2>(p, s);
  return go_tiled<2, 2, 2, 2>(p, s);
}

hipError_t launch_gate_up_int8(const Int8Params& p, hipStream_t s) {
  if (p.T < 1 || p.rows < 1 || p.cols < 16 || p.cols % 16 || p.cols > INT8_MAX_COLS) return hipErrorInvalidValue;
  // token tiles are grid rows
  for (int t0 = 0; t0 < p.T; t0 += 1 << 20) {
    Int8Params q = p;
    q.T = p.T - t0 < (1 << 20) ? p.T - t0 : 1 << 20;
    q.xq += (size_t)t0 * p.cols;
    q.xs += t0;
    q.y = (float*)p.y + (size_t)t0 * p.rows;
    const hipError_t e = q.T <= 16 ? go_few<2, 1, 4>(q, s) : go_few<2, 4, 2>(q, s);
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
