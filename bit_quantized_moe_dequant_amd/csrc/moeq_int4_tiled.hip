// Launches of the tiled INT4 products (moeq_int4_tiled.h), and the activation rows they take.
// The kernels with scaled weights are compiled apart (moeq_int4_scaled.hip), where the compiler
// keeps their sums in accumulation registers; here the vector unit reads them.
#include "moeq_int4_tiled.h"

namespace moeq {

namespace {

// ---------------------------------------------------------------- activation rows

// fp16 terms [n][TERMS][kpad] of bf16 or fp32 rows times 2^(15 - e), 2^e just above the row's
// largest magnitude, and scale[row] = 2^(e - 15). Columns past the end are zeros; a row that
// holds an infinity or a NaN is zeros with scale NaN. One work-group to a row.
template <int TERMS, bool IN_F32>
__global__ __launch_bounds__(256) void k_int4_rows(const void* x, int cols, int kpad, uint16_t* out, float* scale) {
  __shared__ uint32_t part[4];
  const size_t row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto get = [&](int k, float (&v)[8]) {
    if constexpr (IN_F32) {
      const float* p = (const float*)x + row * cols + k;
      const u32x4 a = ld16(p), b = ld16(p + 4);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[i] = u2f(a[i]);
        v[4 + i] = u2f(b[i]);
      }
    } else {
      const u32x4 a = ld16((const uint16_t*)x + row * cols + k);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[2 * i] = u2f(a[i] << 16);
        v[2 * i + 1] = u2f(a[i] & 0xFFFF0000u);
      }
    }
  };
  uint32_t m = 0;
  for (int k = 8 * (int)threadIdx.x; k < cols; k += 2048) {
    float v[8];
    get(k, v);
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, f2u(v[i]) & 0x7FFFFFFFu);
  }
  m = wave_max(m);
  if (lane == 0) part[wave] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const bool finite = m < 0x7F800000u;
  int e = 0;
  if (m != 0 && finite) (void)frexpf(u2f(m), &e);
  if (threadIdx.x == 0) scale[row] = finite ? ldexpf(1.0f, e - 15) : u2f(0x7FC00000u);
  uint16_t* o = out + row * TERMS * kpad;
  for (int k = 8 * (int)threadIdx.x; k < kpad; k += 2048) {
    f16x8_t hi{}, lo{};
    if (k < cols && finite) {
      float v[8];
      get(k, v);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float f = __builtin_ldexpf(v[i], 15 - e);
        hi[i] = (_Float16)f;
        if constexpr (TERMS == 2) lo[i] = (_Float16)(f - (float)hi[i]);
      }
    }
    *reinterpret_cast<f16x8_t*>(o + k) = hi;
    if constexpr (TERMS == 2) *reinterpret_cast<f16x8_t*>(o + kpad + k) = lo;
  }
}

#ifndef MOEQ_I4_WIDE
#define MOEQ_I4_WIDE 12
#endif
#ifndef MOEQ_I4_NT
#define MOEQ_I4_NT 1
#endif
template <int GP>
hipError_t tiled_kind(int kind, const Int4Rows& p, hipStream_t s) {
  auto blocks = [&](int rows, int tok) { return (p.rows + (long)rows - 1) / rows * ((p.T + tok - 1) / tok); };
  if (kind == I4_LINEAR) {
    if (p.out_bf16 && blocks(256, 128) >= 192) return launch_int4_scaled(p, s);
    if (blocks(256, 64) >= 192) return linear<GP, false, 8, 1, 2, 4>(p, s);
    if (p.T > 32) return linear<GP, false, 4, 1, 1, 4>(p, s);
    return linear<GP, false, 4, 1, 1, 2>(p, s);
  }
  const bool wide = (long)p.T * p.top_k >= (long)MOEQ_I4_WIDE * p.n_experts;
  if (kind == I4_GATE_UP) return wide ? experts<I4_GATE_UP, GP, 2, 4, 2>(p, s) : experts<I4_GATE_UP, GP, 2, MOEQ_I4_NT, 4>(p, s);
  return wide ? experts<I4_DOWN_PART, GP, 2, 4, 2>(p, s) : experts<I4_DOWN_PART, GP, 2, MOEQ_I4_NT, 4>(p, s);
}

}  // namespace

size_t int4_rows_bytes(size_t n_rows, int terms, int cols) { return n_rows * terms * int4_ktiles(cols) * 256; }

hipError_t launch_int4_rows(bool in_f32, const void* x, size_t n_rows, int cols, uint16_t* out, float* scale, hipStream_t s) {
  if (n_rows < 1 || cols < 32 || cols % 32) return hipErrorInvalidValue;
  const int kpad = int4_ktiles(cols) * 128;
  for (size_t r0 = 0; r0 < n_rows; r0 += 1 << 22) {  // work-groups to a grid
    const unsigned n = (unsigned)(n_rows - r0 < 1 << 22 ? n_rows - r0 : 1 << 22);
    if (in_f32)
      hipLaunchKernelGGL((k_int4_rows<2, true>), dim3(n), dim3(256), 0, s, (const float*)x + r0 * cols, cols, kpad,
                         out + r0 * 2 * kpad, scale + r0);
    else
      hipLaunchKernelGGL((k_int4_rows<1, false>), dim3(n), dim3(256), 0, s, (const uint16_t*)x + r0 * cols, cols, kpad,
                         out + r0 * kpad, scale + r0);
  }
  return hipGetLastError();
}

hipError_t launch_int4_tiled(int kind, const Int4Rows& p, hipStream_t s) {
  if (!is_int4(p.fmt) || p.T < 1 || p.rows < 1 || p.rows > INT4_MAX_ROWS || p.cols < 32 || p.cols > INT4_MAX_COLS ||
      p.cols % int4_group(p.fmt))
    return hipErrorInvalidValue;
  auto run = [&](const Int4Rows& q) {
    switch (int4_group(q.fmt)) {
      case 32: return tiled_kind<4>(kind, q, s);
      case 64: return tiled_kind<2>(kind, q, s);
      default: return tiled_kind<1>(kind, q, s);
    }
  };
  if (kind != I4_LINEAR) return run(p);
  // tokens to a launch: 2^23 work-groups of the smallest tile, 64 rows x 32 tokens, at most
  const long per = (((long)1 << 23) / ((p.rows + 63) / 64)) * 32;
  const int kpad = int4_ktiles(p.cols) * 128;
  for (long t0 = 0; t0 < p.T; t0 += per) {
    Int4Rows q = p;
    q.T = (int)(p.T - t0 < per ? p.T - t0 : per);
    q.act += (size_t)t0 * kpad;
    q.act_scale += t0;
    q.y = (uint8_t*)p.y + (size_t)t0 * p.rows * (p.out_bf16 ? 2 : 4);
    const hipError_t e = run(q);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moeq
