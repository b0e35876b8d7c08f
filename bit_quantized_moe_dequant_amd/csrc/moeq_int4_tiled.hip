// Products of INT4 weights with many activation rows (layout of the weights: moeq_int4.h).
//
//   y_tr = sum_g s_rg sum_{k in g} (q_rk - z_rg) x_tk
//
// on the fp16 matrix instruction (16 x 16 x 32). Codes become fp16 integers q - z, exact: the
// nibble is laid into the mantissa of 1024 (or of 64, four bits higher) by a mask-and-or, and a
// packed addition takes 1024 + z away, nine vector operations for eight values. Activations come
// as fp16, every row times a power of two of its own (k_int4_rows): a bf16 value keeps all its
// bits down to 2^-39 of its row's largest; the intermediate h, fp32, is two fp16 terms, 22 bits.
// Products are exact and sums fp32; a group's sum is multiplied by its scale in fp32.
//
// Activations are operand A (its rows: tokens), so a lane's outputs belong to one weight row and
// need one scale per group. A work-group's four waves have NM row tiles each (so every weight is
// decoded once in a work-group) and all of its 16 NT tokens, which lie in LDS in steps of 128
// columns (three buffers; a row's 16-byte chunks at chunk ^ (row % 16), so that the sixteen rows
// of an operand touch all banks once). Weights go from memory to registers, a step ahead.
#include "moeq_int4.h"
#include "moeq_int8.h"
#include "moeq_tiled.h"

namespace moeq {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

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

// ---------------------------------------------------------------- product

__device__ __forceinline__ uint32_t pk_add(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, a) + __builtin_bit_cast(f16x2_t, b));
}
__device__ __forceinline__ uint32_t pk_half(float v) {
  const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)v);
  return h | (h << 16);
}

// 16 bytes per lane from base + off + step into LDS at dst + 16 lane.
__device__ __forceinline__ void copy16u(const uint16_t* base, int off, int step, uint8_t* dst) {
  copy16(reinterpret_cast<const int8_t*>(base), off, step, dst);
}

constexpr int I4_STAGES = 3;
template <int TERMS, int NT>
constexpr int i4_stage() {
  return TERMS * NT * 16 * 256;
}

template <int KIND, int GP, int NM, int NT>
__global__ __launch_bounds__(256, 1) void k_int4_tiled(Int4Rows P) {
  constexpr int TERMS = KIND == I4_DOWN_PART ? 2 : 1, ROWS = TERMS * NT * 16, STAGE = i4_stage<TERMS, NT>();
  constexpr int COPIES = ROWS / 16;            // of a wave per step, four LDS rows each
  constexpr int PAIRS = KIND == I4_GATE_UP ? 2 : 1;  // matrices side by side
  constexpr int RT = NM / PAIRS;               // row tiles of a wave
  __shared__ __attribute__((aligned(16))) uint8_t lds[I4_STAGES * STAGE];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ktiles = int4_ktiles(P.cols), kpad = ktiles * 128, rtiles = int4_rtiles(P.rows);
  const int nbm = (rtiles + 4 * RT - 1) / (4 * RT);

  // tile of this work-group: row block bm, activation rows `first` .. + count
  int bm, e, first, count;
  const int32_t* perm = nullptr;
  if constexpr (KIND == I4_LINEAR) {
    int bn;
    tile_of(blockIdx.x, nbm, (P.T + 16 * NT - 1) / (16 * NT), bm, bn);
    first = bn * 16 * NT;
    count = min(16 * NT, P.T - first);
    e = P.expert;
  } else {
    // the row blocks of a chunk of tokens on one XCD: they share the tokens in its L2
    static_assert(16 * NT == PREFILL_MC, "chunks of the routing");
    const int l = blockIdx.x / 8, q = l / nbm * 8 + (int)(blockIdx.x % 8);
    bm = l % nbm;
    if (q >= P.route.n_chunks()[0]) return;
    e = P.route.chunk_e()[q];
    const int p0 = P.route.offsets()[e], m0 = P.route.chunk_m0()[q];
    count = min(16 * NT, P.route.offsets()[e + 1] - p0 - m0);
    perm = P.route.perm() + p0 + m0;
    first = 0;
    if (e >= P.n_experts) {  // ids out of range
      if constexpr (KIND == I4_DOWN_PART)
        for (int i = threadIdx.x; i < count * 64 * RT; i += 256) {
          const int r = bm * 64 * RT + i % (64 * RT);
          if (r < P.rows) ((float*)P.y)[(size_t)perm[i / (64 * RT)] * P.rows + r] = 0.f;
        }
      return;
    }
  }

  // this lane's part of a wave's copies: LDS row 4 (COPIES wave + i) + lane / 16, term by term
  const uint16_t* abase = P.act + (KIND == I4_LINEAR ? (size_t)first * kpad : 0);
  int off[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; i++) {
    const int row = 4 * (COPIES * wave + i) + (lane >> 4), term = row / (16 * NT), t = min(row % (16 * NT), count - 1);
    int a = t;
    if constexpr (KIND == I4_GATE_UP) a = perm[t] / P.top_k;
    if constexpr (KIND == I4_DOWN_PART) a = perm[t];
    off[i] = (a * TERMS + term) * kpad * 2 + 16 * ((lane & 15) ^ (row & 15));
  }
  auto copy = [&](int s) {
    uint8_t* dst = lds + s % I4_STAGES * STAGE + 1024 * COPIES * wave;
#pragma unroll
    for (int i = 0; i < COPIES; i++) copy16u(abase, off[i], s * 256, dst + 1024 * i);
  };

  // row tiles of this wave; past the end the last one, whose outputs are not stored
  const uint8_t* wp[NM];
  const uint8_t* sp[NM];
  const uint8_t* zp[NM];
  const bool zeros = int4_zeros(P.fmt);
#pragma unroll
  for (int m = 0; m < NM; m++) {
    const WeightRef& w = P.w[PAIRS == 2 ? m / RT : 0];
    const size_t tile = (size_t)min((bm * 4 + wave) * RT + m % RT, rtiles - 1) * ktiles;
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
  auto fetch = [&](int s, Step& v) {
#pragma unroll
    for (int m = 0; m < NM; m++) {
      v.w[m] = ld16(wp[m] + (size_t)s * 1024);
      const uint8_t* q = sp[m] + (size_t)s * 32 * GP;
      if constexpr (GP == 1) v.s[m][0] = *reinterpret_cast<const uint16_t*>(q);
      else if constexpr (GP == 2) v.s[m][0] = *reinterpret_cast<const uint32_t*>(q);
      else v.s[m] = *reinterpret_cast<const u32x2*>(q);
      if (zeros) {
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

  Step next;
  copy(0);
  fetch(0, next);
  if (ktiles > 1) copy(1);
  for (int s = 0; s < ktiles; s++) {
    // step s's copies and weights are there; those of step s + 1's copies may be on their way
    if (s + 1 < ktiles) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(COPIES) : "memory");
    else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const Step now = next;
    if (s + 1 < ktiles) fetch(s + 1, next);
    if (s + 2 < ktiles) copy(s + 2);
    const uint8_t* x = lds + s % I4_STAGES * STAGE + n * 256;
    uint32_t c0[NM], c1[NM];  // -(1024 + z) and -(64 + z), twice each
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const bool begin = j % (4 / GP) == 0, end = (j + 1) % (4 / GP) == 0;
      const int gi = j * GP / 4;
      if (begin) {
#pragma unroll
        for (int m = 0; m < NM; m++) {
          const float z = zeros ? (float)(now.z[m] >> (8 * gi) & 255u) : 8.0f;
          c0[m] = pk_half(-1024.0f - z);
          c1[m] = pk_half(-64.0f - z);
        }
      }
      f16x8_t xv[TERMS][NT];
#pragma unroll
      for (int a = 0; a < TERMS; a++)
#pragma unroll
        for (int t = 0; t < NT; t++)
          xv[a][t] = *reinterpret_cast<const f16x8_t*>(x + (a * NT + t) * 4096 + 16 * ((4 * j + g) ^ n));
#pragma unroll
      for (int m = 0; m < NM; m++) {
        const uint32_t w = now.w[m][j], v = w >> 8;
        const u32x4 d = {pk_add((w & 0x000F000Fu) | 0x64006400u, c0[m]), pk_add((w & 0x00F000F0u) | 0x54005400u, c1[m]),
                         pk_add((v & 0x000F000Fu) | 0x64006400u, c0[m]), pk_add((v & 0x00F000F0u) | 0x54005400u, c1[m])};
        const f16x8_t b = __builtin_bit_cast(f16x8_t, d);
#pragma unroll
        for (int t = 0; t < NT; t++) {
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[0][t], b, begin ? f32x4_t{0.f, 0.f, 0.f, 0.f} : acc[m][t], 0, 0, 0);
          if constexpr (TERMS == 2) acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[TERMS - 1][t], b, acc[m][t], 0, 0, 0);
        }
      }
      if (end) {
#pragma unroll
        for (int m = 0; m < NM; m++) {
          const float sc = half_bits_f32(now.s[m][gi / 2] >> (16 * (gi & 1)));
#pragma unroll
          for (int t = 0; t < NT; t++)
#pragma unroll
            for (int r = 0; r < 4; r++) tot[m][t][r] = __builtin_fmaf(sc, acc[m][t][r], tot[m][t][r]);
        }
      }
    }
  }

  // lane (n, g), register r of token tile t: token 16 t + 4 g + r, weight row n of the tile
#pragma unroll
  for (int t = 0; t < NT; t++) {
    float as[4];
    size_t at[4];
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int i = min(16 * t + 4 * g + r, count - 1);
      const size_t a = KIND == I4_LINEAR ? (size_t)(first + i) : (size_t)perm[i];
      as[r] = P.act_scale[KIND == I4_GATE_UP ? a / P.top_k : a];
      if constexpr (KIND == I4_DOWN_PART) as[r] *= P.rw[a];
      at[r] = a * P.rows;
    }
    const float s0 = P.w[0].scale2[e], s1 = PAIRS == 2 ? P.w[1].scale2[e] : 0.f;
#pragma unroll
    for (int m = 0; m < RT; m++) {
      const int row = ((bm * 4 + wave) * RT + m) * 16 + n;
      if (row >= P.rows) continue;
      float bias = 0.f;
      if constexpr (KIND == I4_LINEAR)
        if (P.bias) bias = P.bias[row];
#pragma unroll
      for (int r = 0; r < 4; r++) {
        if (16 * t + 4 * g + r >= count) continue;
        float v = tot[m][t][r] * s0 * as[r];
        if constexpr (PAIRS == 2) v = silu_mul(v, tot[RT + m][t][r] * s1 * as[r]);
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

template <int KIND, int GP, int NM, int NT>
hipError_t tiled(const Int4Rows& p, long blocks, hipStream_t s) {
  hipLaunchKernelGGL((k_int4_tiled<KIND, GP, NM, NT>), dim3((unsigned)blocks), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int GP>
hipError_t tiled_kind(int kind, const Int4Rows& p, hipStream_t s) {
  const long rt = int4_rtiles(p.rows);
  auto blocks = [&](int nm, int nt) { return (rt + 4 * nm - 1) / (4 * nm) * ((p.T + 16 * nt - 1) / (16 * nt)); };
  if (kind == I4_LINEAR) {
    if (blocks(4, 8) >= 192) return tiled<I4_LINEAR, GP, 4, 8>(p, blocks(4, 8), s);
    if (blocks(2, 4) >= 192 && p.T > 32) return tiled<I4_LINEAR, GP, 2, 4>(p, blocks(2, 4), s);
    if (p.T > 32) return tiled<I4_LINEAR, GP, 1, 4>(p, blocks(1, 4), s);
    return tiled<I4_LINEAR, GP, 1, 2>(p, blocks(1, 2), s);
  }
  const int pairs = p.T * p.top_k;
  const long chunks = (RouteView::max_chunks(p.n_experts, pairs) + 7) / 8 * 8;
  if (kind == I4_GATE_UP) return tiled<I4_GATE_UP, GP, 4, 4>(p, (rt + 7) / 8 * chunks, s);
  return tiled<I4_DOWN_PART, GP, 4, 4>(p, (rt + 15) / 16 * chunks, s);
}

}  // namespace

// Byte offsets of gathered rows are 32-bit.
bool int4_rows_fit(size_t n_rows, int terms, int cols) { return n_rows * terms * int4_ktiles(cols) * 256 < (size_t)1 << 31; }

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
  if (kind != I4_LINEAR && !int4_rows_fit((size_t)p.T * (kind == I4_DOWN_PART ? p.top_k : 1), kind == I4_DOWN_PART ? 2 : 1, p.cols))
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
