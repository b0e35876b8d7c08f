// Launches of the tiled INT4 products (moeq_int4_tiled.h), and the activation rows they take.
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

// Pairs to an expert, on average, from which gate/up takes tiles of 64 pairs with three waves to a
// SIMD (weights are decoded once for up to 64) instead of 32 with four. Kernel times in us (256
// experts, 4096 columns, 2048 rows of gate and up, groups of 128), 32 | 64: 12 pairs 437 | 456,
// 18 452 | 483, 24 511 | 521, 30 620 | 549, 48 947 | 693. Eight waves to a work-group instead of four
// took 864 at 48 pairs. With 16 pairs or fewer both multiply one tile of tokens.
constexpr long WIDE_PAIRS = 27;
// And those from which down (4096 rows, 2048 columns, two terms to a value) takes 32 pairs instead
// of 16, whose buffers of LDS are half as large: 0.4 pairs 81 (16) | 93 (32), 3 pairs 221 | 230,
// 9 pairs 247 | 255, 12 pairs 273 | 261, 48 pairs 800 | 615; tiles of 64 are no faster there.
constexpr long MID_PAIRS = 10;

template <int GP>
hipError_t tiled_kind(int kind, const Int4Rows& p, hipStream_t s, const LaunchEvents* ev) {
  auto blocks = [&](int rows, int tok) { return (p.rows + (long)rows - 1) / rows * ((p.T + tok - 1) / tok); };
  if (kind == I4_LINEAR) {
    if (blocks(256, 64) >= 192) return linear<GP, 8, 1, 2, 4>(p, s);
    // Too few tiles of 256 rows x 64 tokens to fill the chip: 64 x 32, with two waves to an output,
    // or four where all tokens lie in one tile. us, against one wave and tiles of 64 tokens (of 32):
    // 100 tokens x 5003 x 4128, groups of 32, 21.0 (25.6); 256 x 4096 x 4096, groups of 128, 18.6
    // (22.0); 24 x 2048 x 4096 11.4 (14.3). More buffers in place of waves changed nothing: what
    // binds a step is the vector unit (four waves to a CU or eight alike), not memory.
    if (p.T > 32) return linear<GP, 4, 1, 1, 2, 2>(p, s);
    return linear<GP, 4, 1, 1, 2, 4>(p, s);
  }
  const long pairs = (long)p.T * p.top_k;
  if (kind == I4_GATE_UP)
    return pairs >= WIDE_PAIRS * p.n_experts ? experts<I4_GATE_UP, GP, 4, 2, 4, 3>(p, s, ev)
                                             : experts<I4_GATE_UP, GP, 4, 2, 2, 4>(p, s, ev);
  return pairs >= MID_PAIRS * p.n_experts ? experts<I4_DOWN_PART, GP, 8, 2, 2, 4>(p, s)
                                          : experts<I4_DOWN_PART, GP, 8, 2, 1, 4>(p, s);
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

hipError_t launch_int4_tiled(int kind, const Int4Rows& p, hipStream_t s, const LaunchEvents* ev) {
  if (!is_int4(p.fmt) || p.T < 1 || p.rows < 1 || p.rows > INT4_MAX_ROWS || p.cols < 32 || p.cols > INT4_MAX_COLS ||
      p.cols % int4_group(p.fmt))
    return hipErrorInvalidValue;
  auto run = [&](const Int4Rows& q) {
    switch (int4_group(q.fmt)) {
      case 32: return tiled_kind<4>(kind, q, s, ev);
      case 64: return tiled_kind<2>(kind, q, s, ev);
      default: return tiled_kind<1>(kind, q, s, ev);
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
