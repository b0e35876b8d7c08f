// 4-bit integer weights with group scales (layout: moeq_int4.h): packing, dequantisation, and
// the products for a few activation rows to a tensor.
//
//   y_tr = sum_g s_rg sum_{k in g} (q_rk - z_rg) x_tk
//
// The codes enter the bf16 matrix instruction as 16 + q, exact in bf16: the nibble in the upper
// mantissa bits of a number with exponent 2^4, a shift and a mask-and-or for two values. The
// group's sum then holds (16 + z) sum_k x_tk too much. That sum comes from one more matrix
// instruction, activations times ones, in the registers where the product of the same tokens is:
//
//   y_tr = sum_g s_rg (acc_g - (16 + z_rg) sx_g)
//
// Products are exact and sums are fp32; scales are applied to fp32 sums. The activations are
// operand A (rows: tokens) and the weights B (columns: weight rows), so that a lane's outputs
// belong to one weight row and need one scale per group. Tokens are spread over A's rows so that
// T tokens fill the first output register of four lanes first (token i of a tile in row 4 i):
// for up to four tokens a group's end costs two vector operations instead of eight.
//
// What bounds it: the weight stream, and where that is short the launch and one round of loads.
// Measured, groups of 128: linear 1 x 4096 x 4096 5.3 us, 16 x 2048 x 4096 7.5 (groups of 64, zero
// points); 6 experts of 4096 x 2048 for one token 13.4 + 10.4 us (3.8 and 2.5 TB/s), for eight
// tokens 75 to 87 + 55 (4.8 to 5.5 and 3.8 TB/s; from card to card). The one-token down is short of the
// stream because each of its 256 work-groups first stages all of h, 74 KB, for its 98 KB of weights.
// A tile of 512 weights costs a SIMD 8 vector operations (32 clocks) and one matrix instruction of 16.
#include <hip/hip_ext.h>

#include <algorithm>
#include <type_traits>

#include "moeq_grid.h"
#include "moeq_int4.h"
#include "moeq_int8.h"

namespace moeq {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- packing

// Largest finite |scale| of each tensor as fp32 bits, into scale2 (cleared before).
__global__ __launch_bounds__(256) void k_int4_max(const uint16_t* scales, int bf16, size_t per, uint32_t* out) {
  const uint16_t* s = scales + (size_t)blockIdx.y * per;
  uint32_t m = 0;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < per; i += (size_t)gridDim.x * 256) {
    const float v = bf16 ? u2f((uint32_t)s[i] << 16) : half_bits_f32(s[i]);
    const uint32_t b = f2u(v) & 0x7FFFFFFFu;
    if (b < 0x7F800000u) m = max(m, b);
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) atomicMax(out + blockIdx.y, m);
}

// The power of two that leaves the largest scale in [64, 128), where the kernels' fp16 products
// with codes up to 255 neither overflow nor, down to 2^-20 of it, lose bits.
__device__ __forceinline__ int int4_exponent(uint32_t max_bits) {
  if (max_bits == 0) return 0;
  int e;
  (void)frexpf(u2f(max_bits), &e);  // max in [2^(e - 1), 2^e)
  return max(e - 7, -120);
}

__global__ __launch_bounds__(256) void k_int4_pack(int group, const uint8_t* codes, const uint16_t* scales, int bf16,
                                                   const uint8_t* zeros, int rows, int cols, uint8_t* data, uint8_t* out,
                                                   size_t data_bytes, size_t scale_bytes, size_t zeros_at,
                                                   const uint32_t* max_bits, size_t block0) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, kt_n = int4_ktiles(cols);
  const size_t tile = (block0 + blockIdx.x) * 4 + (threadIdx.x >> 6), e = blockIdx.y;
  if (tile >= int4_tiles(rows, cols)) return;
  const int r = (int)(tile / kt_n) * 16 + n, k0 = (int)(tile % kt_n) * 128;
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int k = k0 + 32 * j + 8 * g;
    uint32_t v = 0;
    if (r < rows && k < cols) {
      const uint8_t* p = codes + (e * rows + r) * ((size_t)cols / 2) + k / 2;
#pragma unroll
      for (int i = 0; i < 4; i++)
        v |= ((uint32_t)(p[i] & 15) << (4 * i)) | ((uint32_t)(p[i] >> 4) << (16 + 4 * i));
    }
    w[j] = v;
  }
  *reinterpret_cast<u32x4*>(data + e * data_bytes + tile * 1024 + 16 * lane) = w;
  const int per = 128 / group;  // scales of a row of the tile
  if (lane < 16 * per) {
    const int row = (int)(tile / kt_n) * 16 + lane / per, k = k0 + group * (lane % per);
    uint16_t s = 0;
    uint8_t z = 8;
    if (row < rows && k < cols) {
      const size_t at = (e * rows + row) * ((size_t)cols / group) + k / group;
      const float v = bf16 ? u2f((uint32_t)scales[at] << 16) : half_bits_f32(scales[at]);
      s = __builtin_bit_cast(uint16_t, (_Float16)ldexpf(v, -int4_exponent(max_bits[e])));
      if (zeros) z = zeros[at];
    }
    *reinterpret_cast<uint16_t*>(out + e * scale_bytes + (tile * 16 * per + lane) * 2) = s;
    if (zeros) out[e * scale_bytes + zeros_at + tile * 16 * per + lane] = z;
  }
}

__global__ void k_int4_scale2(float* scale2, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) scale2[i] = ldexpf(1.0f, int4_exponent(f2u(scale2[i])));
}

// One thread per 8 columns of a row.
__global__ __launch_bounds__(256) void k_int4_dequant(int group, const uint8_t* data, const uint8_t* scales, size_t zeros_at,
                                                      bool zeros, const float* scale2, int rows, int cols, float* out,
                                                      size_t block0) {
  const size_t i = (block0 + blockIdx.x) * 256 + threadIdx.x;
  const int per_row = cols / 8;
  if (i >= (size_t)rows * per_row) return;
  const int r = (int)(i / per_row), k = (int)(i % per_row) * 8;
  const size_t tile = (size_t)(r / 16) * int4_ktiles(cols) + k / 128;
  const int j = (k & 127) / 32, g = (k & 31) / 8;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(data + tile * 1024 + 16 * ((r & 15) + 16 * g) + 4 * j);
  const size_t at = tile * 16 * (128 / group) + (size_t)(r & 15) * (128 / group) + (k & 127) / group;
  const float s = half_bits_f32(reinterpret_cast<const uint16_t*>(scales)[at]) * scale2[0];
  const int z = zeros ? scales[zeros_at + at] : 8;
  float* o = out + (size_t)r * cols + k;
#pragma unroll
  for (int p = 0; p < 4; p++) {
    o[2 * p] = s * (float)((int)(w >> (4 * p) & 15) - z);
    o[2 * p + 1] = s * (float)((int)(w >> (16 + 4 * p) & 15) - z);
  }
}

// An fp32 value as the sum of three bf16 ones of eight bits each: exact (but for subnormals).
__device__ __forceinline__ void bf16_terms(float h, uint32_t (&b)[3]) {
#pragma unroll
  for (int a = 0; a < 3; a++) {
    const uint32_t top = f2u(h) & 0xFFFF0000u;
    b[a] = top >> 16;
    h -= u2f(top);  // not a number behind an infinity
  }
}

__global__ __launch_bounds__(256) void k_int4_terms(const float* h, size_t n, int cols, uint16_t* planes) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const size_t row = i / cols, k = i % cols;
  const u32x4 v = ld16(h + i);
  uint32_t t[3][4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    uint32_t b[3];
    bf16_terms(u2f(v[j]), b);
#pragma unroll
    for (int a = 0; a < 3; a++) t[a][j] = b[a];
  }
  uint16_t* o = planes + row * 3 * cols + k;
#pragma unroll
  for (int a = 0; a < 3; a++)
    *reinterpret_cast<u32x2*>(o + (size_t)a * cols) = u32x2{t[a][0] | (t[a][1] << 16), t[a][2] | (t[a][3] << 16)};
}

// ---------------------------------------------------------------- products

constexpr int FEW_WAVES = 8;

// A row's scales and zero points of one tile.
template <int GP, bool ZEROS, int NMAT>
struct Side {
  u32x2 s[NMAT];
  uint32_t z[NMAT];
};

// Tile `tile` of expert e: codes of this lane, and the side data of its row.
template <int GP, bool ZEROS, int NMAT>
__device__ __forceinline__ void int4_load(const Int4Params& P, int e, size_t tile, int lane, u32x4 (&w)[NMAT], Side<GP, ZEROS, NMAT>& side) {
#pragma unroll
  for (int m = 0; m < NMAT; m++) {
    w[m] = ld16(P.w[m].data + (size_t)e * P.w[m].estride + tile * 1024 + 16 * lane);
    const uint8_t* sp = P.w[m].scales + (size_t)e * P.w[m].sestride;
    const size_t at = (tile * 16 + (lane & 15)) * GP;
    if constexpr (GP == 1) side.s[m][0] = *reinterpret_cast<const uint16_t*>(sp + 2 * at);
    else if constexpr (GP == 2) side.s[m][0] = *reinterpret_cast<const uint32_t*>(sp + 2 * at);
    else side.s[m] = *reinterpret_cast<const u32x2*>(sp + 2 * at);
    if constexpr (ZEROS) {
      const uint8_t* zp = sp + int4_zeros_at(P.fmt, P.rows, P.cols) + at;
      if constexpr (GP == 1) side.z[m] = *zp;
      else if constexpr (GP == 2) side.z[m] = *reinterpret_cast<const uint16_t*>(zp);
      else side.z[m] = *reinterpret_cast<const uint32_t*>(zp);
    }
  }
}

__device__ __forceinline__ f32x4_t mfma(u32x4 x, u32x4 w, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, w), c, 0, 0, 0);
}
__device__ __forceinline__ u32x4 ones() { return u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}; }

// Keeps every register of the matrix instructions' results a and b until `v`, computed from them,
// is there. Where only some of them are used, the compiler gives the others to other operations
// behind the instruction, and in early forms of these kernels not always after the eight wait states
// that this takes: sums were wrong now and then. It costs nothing.
__device__ __forceinline__ void hold(float& v, const f32x4_t& a, const f32x4_t& b) {
  asm volatile("" : "+v"(v) : "v"(a), "v"(b));
}

// Eight codes as 16 + q in bf16.
__device__ __forceinline__ u32x4 int4_operand(uint32_t w) {
  return u32x4{((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
               ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u};
}

// scale of group gi of a tile, and what is too much in its sum for every unit of sum x
template <int GP, bool ZEROS, int NMAT>
__device__ __forceinline__ float int4_scale(const Side<GP, ZEROS, NMAT>& side, int m, int gi) {
  return half_bits_f32(side.s[m][gi / 2] >> (16 * (gi & 1)));
}
template <int GP, bool ZEROS, int NMAT>
__device__ __forceinline__ float int4_offset(const Side<GP, ZEROS, NMAT>& side, int m, int gi) {
  return ZEROS ? 16.0f + (float)(side.z[m] >> (8 * gi) & 255u) : 24.0f;
}

// What becomes of the sums v (one per matrix) of weight row r and activation row t of the tile:
// `pair` is its (token, slot) pair, or the token.
template <int KIND, int NMAT>
__device__ __forceinline__ void int4_store(const Int4Params& P, bool ok, size_t pair, int r, const float (&v)[NMAT]) {
  if constexpr (KIND == I4_LINEAR) {
    const size_t at = pair * P.rows + r;
    float f = v[0];
    if (P.bias) f += P.bias[r];
    if (P.out_bf16) ((uint16_t*)P.y)[at] = (uint16_t)f32_bf16_rne_nan(f);
    else ((float*)P.y)[at] = f;
  } else if constexpr (KIND == I4_GATE_UP) {
    const float h = ok ? silu_mul(v[0], v[NMAT - 1]) : 0.f;
    if (P.out_terms) {
      uint32_t b[3];
      bf16_terms(h, b);
      uint16_t* out = (uint16_t*)P.y + pair * 3 * P.rows + r;
#pragma unroll
      for (int a = 0; a < 3; a++) out[(size_t)a * P.rows] = (uint16_t)b[a];
    } else {
      ((float*)P.y)[pair * P.rows + r] = h;
    }
  } else {
    ((float*)P.y)[pair * P.rows + r] = v[0];
  }
}

// Waves of a work-group of k_int4_one: a token's down has no more work-groups than row tiles.
constexpr int one_waves(int kind) { return kind == I4_DOWN_SUM ? 16 : FEW_WAVES; }

// One token or pair (I4_DOWN_SUM: a token's pairs one behind the other), or up to four tokens of a
// linear, in LDS. A work-group takes rb tiles of 16 weight rows (of the gate and of
// the up matrix), one after another, and all of K, whose tiles its waves take in turn; the waves'
// sums meet in LDS (two buffers, one barrier to a row tile) and are added in the order of the waves.
// A wave's next DEPTH tiles are always on their way, those of the next row tile among them; the
// first are asked for behind the activations' loads and before these are waited for. TERMS: bf16
// terms of an activation. The lanes of operand A's unused rows read zeros.
template <int GP, bool ZEROS, int TERMS, int KIND, int DEPTH>
__global__ __launch_bounds__(64 * one_waves(KIND)) void k_int4_one(Int4Params P, int rb) {
  constexpr int NMAT = KIND == I4_GATE_UP ? 2 : 1, NR = TERMS, TOK = KIND == I4_DOWN_SUM ? 1 : 4;
  constexpr int STAGE = KIND == I4_DOWN_SUM ? 5 : KIND == I4_LINEAR ? 4 : 1;  // 16-byte pieces of the rows to a thread
  extern __shared__ __attribute__((aligned(16))) uint8_t xs[];  // 16 bytes of zeros, then the rows
  __shared__ float red[2][one_waves(KIND)][NMAT][TOK][16];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int rt0 = blockIdx.x * rb, rt1 = min(rt0 + rb, int4_rtiles(P.rows));
  const int item = blockIdx.y, ktiles = int4_ktiles(P.cols);
  const int parts = KIND == I4_DOWN_SUM ? P.top_k : 1, steps = parts * ktiles;

  const int here = KIND == I4_LINEAR ? P.T : 1;

  // the rows, token by token or part by part, and term by term, `pitch` bytes apart
  const int kpad = ktiles * 128, pitch = kpad * 2 + 16;
  const int chunks = (KIND == I4_DOWN_SUM ? parts : here) * TERMS * (kpad / 8);
  auto get = [&](int i) {
    i = min(i, chunks - 1);
    const int row = i / (kpad / 8), k = i % (kpad / 8) * 8;
    size_t a = row / TERMS;
    if constexpr (KIND == I4_DOWN_SUM) a += (size_t)item * P.top_k;
    if constexpr (KIND == I4_GATE_UP) a = item / P.top_k;
    u32x4 v = ld16(P.act + a * P.pitch + row % TERMS * P.term + min(k, P.cols - 8));
    if (k >= P.cols) v = u32x4{0u, 0u, 0u, 0u};
    return v;
  };
  auto put = [&](int i, u32x4 v) {
    i = min(i, chunks - 1);
    *reinterpret_cast<u32x4*>(xs + 16 + (size_t)(i / (kpad / 8)) * pitch + i % (kpad / 8) * 16) = v;
  };
  u32x4 rv[STAGE];
#pragma unroll
  for (int q = 0; q < STAGE; q++) rv[q] = get(threadIdx.x + q * blockDim.x);
  if (threadIdx.x < 4) reinterpret_cast<uint32_t*>(xs)[threadIdx.x] = 0;
  __builtin_amdgcn_sched_barrier(0);

  // the expert; I4_DOWN_SUM: lane k holds part k's, and the factor of its sums (-1: skipped)
  int e = KIND == I4_LINEAR ? P.expert : 0;
  float fac = 0.f;
  bool ok = true;
  if constexpr (KIND == I4_GATE_UP) {
    e = P.ids[item];
    ok = e >= 0 && e < P.n_experts;
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.err, 1u);
    if (!ok) e = 0;
  }
  if constexpr (KIND == I4_DOWN_SUM) {
    e = -1;
    if (lane < parts) {
      e = P.ids[(size_t)item * P.top_k + lane];
      if (e < 0 || e >= P.n_experts) {
        if (blockIdx.x == 0 && wave == 0) atomicOr(P.err, 1u);
        e = -1;
      } else {
        fac = P.rw[(size_t)item * P.top_k + lane] * P.w[0].scale2[e];
      }
    }
  }

  // scale2, in every group's scale: the stored ones, 64 to 128, would carry the sums out of range first
  float s2[NMAT];
#pragma unroll
  for (int m = 0; m < NMAT; m++) s2[m] = KIND == I4_DOWN_SUM ? 1.f : P.w[m].scale2[e];

  // A wave's tiles: row tile by row tile, step wave, wave + waves, ... of each
  struct At {
    int rt, u;
  };
  auto step = [&](At& a) {
    a.u += waves;
    if (a.u >= steps) {
      a.u = wave;
      a.rt++;
    }
  };
  u32x4 wv[DEPTH][NMAT];
  Side<GP, ZEROS, NMAT> side[DEPTH];
  auto load = [&](At a, int d) {
    if (a.rt >= rt1) return;
    int kt = a.u, ex = e;
    if constexpr (KIND == I4_DOWN_SUM) {
      const int k = a.u / ktiles;
      kt = a.u % ktiles;
      ex = max(__builtin_amdgcn_readlane(e, k), 0);
    }
    int4_load(P, ex, (size_t)a.rt * ktiles + kt, lane, wv[d], side[d]);
  };
  At ahead = {rt0, wave}, at = {rt0, wave};
  if (wave >= steps) ahead.rt = at.rt = rt1;  // (a wave without tiles keeps the barriers)
#pragma unroll
  for (int d = 0; d < DEPTH; d++) {
    load(ahead, d);
    step(ahead);
  }
  __builtin_amdgcn_sched_barrier(0);

#pragma unroll
  for (int q = 0; q < STAGE; q++) put(threadIdx.x + q * blockDim.x, rv[q]);
  for (int i = threadIdx.x + STAGE * blockDim.x; i < chunks; i += blockDim.x) put(i, get(i));
  __syncthreads();
  // this lane's row of operand A: row 4 i + a holds term a of token i
  const bool a_on = (n & 3) < TERMS && n / 4 < here;
  const int a0 = a_on ? 16 + (n / 4 * TERMS + (n & 3)) * pitch + 16 * g : 0, a_step = a_on ? 1 : 0;

  int buf = 0;
  float tot[NMAT][NR];
#pragma unroll
  for (int m = 0; m < NMAT; m++)
#pragma unroll
    for (int r = 0; r < NR; r++) tot[m][r] = 0.f;
  auto finish = [&](int rt) {  // a row tile's end
#pragma unroll
    for (int m = 0; m < NMAT; m++) {
      float v = tot[m][0];
#pragma unroll
      for (int a = 1; a < TERMS; a++) v += tot[m][a];
      if (g < TOK) red[buf][wave][m][g][n] = v;
#pragma unroll
      for (int r = 0; r < NR; r++) tot[m][r] = 0.f;
    }
    __syncthreads();
    if ((int)threadIdx.x < here * 16) {
      const int t = threadIdx.x >> 4, r = rt * 16 + n;
      float v[NMAT];
#pragma unroll
      for (int m = 0; m < NMAT; m++) {
        v[m] = 0.f;
        for (int w = 0; w < waves; w++) v[m] += red[buf][w][m][t][n];
      }
      if (r < P.rows) int4_store<KIND, NMAT>(P, ok, KIND == I4_LINEAR ? t : item, r, v);
    }
    buf ^= 1;
  };
  while (at.rt < rt1) {
#pragma unroll
    for (int d = 0; d < DEPTH; d++) {
      if (at.rt >= rt1) break;
      bool live = ok;
      float f = 1.f;  // I4_DOWN_SUM: its factor, scale2 in it
      int k = 0, kt = at.u;
      if constexpr (KIND == I4_DOWN_SUM) {
        k = at.u / ktiles;
        kt = at.u % ktiles;
        live = __builtin_amdgcn_readlane(e, k) >= 0;
        f = u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(fac), k));
      }
      if (live) {
        const uint8_t* x = xs + a0 + a_step * (k * TERMS * pitch + kt * 256);
        f32x4_t acc[NMAT], sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < NMAT; m++) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const u32x4 xv = *reinterpret_cast<const u32x4*>(x + a_step * 64 * j);
          sx = mfma(xv, ones(), sx);
#pragma unroll
          for (int m = 0; m < NMAT; m++) acc[m] = mfma(xv, int4_operand(wv[d][m][j]), acc[m]);
          if ((j + 1) % (4 / GP) == 0) {  // a group's end
            const int gi = j * GP / 4;
#pragma unroll
            for (int m = 0; m < NMAT; m++) {
              const float s = int4_scale(side[d], m, gi) * (KIND == I4_DOWN_SUM ? f : s2[m]);
              const float c = int4_offset(side[d], m, gi);
#pragma unroll
              for (int r = 0; r < NR; r++) tot[m][r] = __builtin_fmaf(s, __builtin_fmaf(-c, sx[r], acc[m][r]), tot[m][r]);
              hold(tot[m][NR - 1], acc[m], sx);
              acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
            sx = f32x4_t{0.f, 0.f, 0.f, 0.f};
          }
        }
      }
      load(ahead, d);
      step(ahead);
      const int rt = at.rt;
      step(at);
      if (at.rt != rt) finish(rt);
    }
  }
  if (wave >= steps)
    for (int rt = rt0; rt < rt1; rt++) finish(rt);
}

// Five to sixteen tokens of a linear (or fewer, with more columns than fit k_int4_one's LDS). A
// work-group: 16 weight rows and all of K, whose tiles its waves take in turn, KT of them at a
// time, with their activations in registers; the waves' sums meet in LDS and are added in the
// order of the waves. NR: output registers in use, so a tile of operand A holds 4 NR tokens.
template <int GP, bool ZEROS, int NR, int KT>
__global__ __launch_bounds__(64 * FEW_WAVES, 2) void k_int4_few(Int4Params P) {
  constexpr int TOK = 4 * NR;
  __shared__ float red[FEW_WAVES][TOK][16];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rt = blockIdx.x, ktiles = int4_ktiles(P.cols);
  // this lane's row of operand A: token `ai`
  const int ai = (n & 3) + (n >> 2) * NR;
  const bool a_on = (n & 3) < NR && ai < P.T;
  const uint16_t* ap = P.act + (size_t)(a_on ? ai : 0) * P.pitch + 8 * g;
  const float s2 = P.w[0].scale2[P.expert];
  float tot[NR];
#pragma unroll
  for (int r = 0; r < NR; r++) tot[r] = 0.f;
  for (int k1 = wave; k1 < ktiles; k1 += FEW_WAVES * KT) {
    u32x4 wv[KT][1], xv[KT][4];
    Side<GP, ZEROS, 1> side[KT];
#pragma unroll
    for (int i = 0; i < KT; i++)
      int4_load(P, P.expert, (size_t)rt * ktiles + min(k1 + i * FEW_WAVES, ktiles - 1), lane, wv[i], side[i]);
#pragma unroll
    for (int i = 0; i < KT; i++) {
      const int k0 = (k1 + i * FEW_WAVES) * 128;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        xv[i][j] = u32x4{0u, 0u, 0u, 0u};
        if (a_on && k0 + 32 * j < P.cols) xv[i][j] = ld16(ap + k0 + 32 * j);
      }
    }
#pragma unroll
    for (int i = 0; i < KT; i++) {
      if (k1 + i * FEW_WAVES >= ktiles) break;
#pragma unroll
      for (int q = 0; q < GP; q++) {
        f32x4_t acc = {0.f, 0.f, 0.f, 0.f}, sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = q * (4 / GP); j < (q + 1) * (4 / GP); j++) {
          sx = mfma(xv[i][j], ones(), sx);
          acc = mfma(xv[i][j], int4_operand(wv[i][0][j]), acc);
        }
        const float s = int4_scale(side[i], 0, q) * s2, c = int4_offset(side[i], 0, q);
#pragma unroll
        for (int r = 0; r < NR; r++) tot[r] = __builtin_fmaf(s, __builtin_fmaf(-c, sx[r], acc[r]), tot[r]);
        hold(tot[NR - 1], acc, sx);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < NR; r++) red[wave][g * NR + r][n] = tot[r];
  __syncthreads();
  const int t = threadIdx.x >> 4, r = rt * 16 + n;
  if (t < P.T && r < P.rows) {
    float v[1] = {0.f};
#pragma unroll
    for (int w = 0; w < FEW_WAVES; w++) v[0] += red[w][t][n];
    int4_store<I4_LINEAR, 1>(P, true, t, r, v);
  }
}

// LDS of k_int4_one's rows (each term one); more than this and the other kernels take them. A linear
// of up to four tokens: longer rows are faster in k_int4_few (4 x 4096 x 14336, 112 KB, 10.0 us there
// and 11.9 here; 4 x 8192 x 16384 20.5 and 28.3). A down's parts may fill a CU (160 KB, the sums' LDS among
// them): where more than half of that leaves one work-group to a CU, the caller decides.
constexpr size_t ONE_LDS = 96 << 10, ONE_LDS_DOWN = 150 << 10;
size_t one_lds(int rows, int cols) { return 16 + (size_t)rows * (int4_ktiles(cols) * 256 + 16); }

template <int GP, int TERMS, int KIND, int DEPTH>
hipError_t one(const Int4Params& p, int items, int rows, hipStream_t s, const LaunchEvents* ev) {
  const int steps = int4_ktiles(p.cols) * (KIND == I4_DOWN_SUM ? p.top_k : 1);
  // Row tiles of a work-group: one while every CU has up to three work-groups, then more (at most
  // 16), which saves their beginnings: 8 tokens of 4096 x 2048 experts (6 of 256) 130 us then, 169 with
  // one each. (With 512, 1024 and 1536 work-groups instead of 768: 140, 147 and 138.)
  const long rt = int4_rtiles(p.rows);
  const int rb = (int)std::min(16l, std::max(1l, rt * items / 768));
  const dim3 g((unsigned)((rt + rb - 1) / rb), (unsigned)items), b(64 * std::min(steps, one_waves(KIND)));
  const unsigned lds = (unsigned)one_lds(rows, p.cols);
  auto go = [&](auto k) {
    if (ev) hipExtLaunchKernelGGL(k, g, b, lds, s, ev->start, ev->stop, 0, p, rb);
    else hipLaunchKernelGGL(k, g, b, lds, s, p, rb);
    return hipGetLastError();
  };
  return int4_zeros(p.fmt) ? go(k_int4_one<GP, true, TERMS, KIND, DEPTH>) : go(k_int4_one<GP, false, TERMS, KIND, DEPTH>);
}

template <int GP, int NR>
hipError_t few(const Int4Params& p, hipStream_t s) {
  const dim3 g((unsigned)int4_rtiles(p.rows)), b(64 * FEW_WAVES);
  const int kt = (int4_ktiles(p.cols) + FEW_WAVES - 1) / FEW_WAVES;
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, g, b, 0, s, p);
    return hipGetLastError();
  };
  if (int4_zeros(p.fmt)) return kt <= 2 ? go(k_int4_few<GP, true, NR, 2>) : go(k_int4_few<GP, true, NR, 4>);
  return kt <= 2 ? go(k_int4_few<GP, false, NR, 2>) : go(k_int4_few<GP, false, NR, 4>);
}

// DEPTH: fewer tiles on their way leave more waves on a CU, which counts for more (gate/up of one
// token, two against four: 12.4 and 15.6 us).
template <int GP>
hipError_t few_kind(int kind, const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  switch (kind) {
    case I4_LINEAR:
      if (p.T <= 4 && one_lds(p.T, p.cols) <= ONE_LDS) return one<GP, 1, I4_LINEAR, 4>(p, 1, p.T, s, ev);
      return p.T <= 8 ? few<GP, 2>(p, s) : few<GP, 4>(p, s);
    case I4_GATE_UP: return one<GP, 1, I4_GATE_UP, 2>(p, items, 1, s, ev);
    case I4_DOWN_SUM: return one<GP, 3, I4_DOWN_SUM, 3>(p, items, 3 * p.top_k, s, ev);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool int4_one_fits(int kind, int top_k, int cols) {
  return kind == I4_DOWN_SUM ? one_lds(3 * top_k, cols) <= ONE_LDS_DOWN : one_lds(1, cols) <= ONE_LDS;
}

bool int4_down_two_to_a_cu(int top_k, int cols) { return one_lds(3 * top_k, cols) <= 78 << 10; }

hipError_t launch_int4_few(int kind, const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  if (!is_int4(p.fmt) || p.T < 1 || items < 1 || items > 65535 || p.rows < 1 || p.rows > INT4_MAX_ROWS || p.cols < 32 ||
      p.cols > INT4_MAX_COLS || p.cols % int4_group(p.fmt) || p.pitch % 8 || p.term % 8)
    return hipErrorInvalidValue;
  if (kind != I4_LINEAR && !int4_one_fits(kind, p.top_k, p.cols)) return hipErrorInvalidValue;
  if (kind == I4_LINEAR && p.T > INT4_FEW_T) return hipErrorInvalidValue;
  switch (int4_group(p.fmt)) {
    case 32: return few_kind<4>(kind, p, items, s, ev);
    case 64: return few_kind<2>(kind, p, items, s, ev);
    default: return few_kind<1>(kind, p, items, s, ev);
  }
}

hipError_t launch_int4_terms(const float* h, size_t n_rows, int cols, uint16_t* planes, hipStream_t s) {
  const size_t n = n_rows * cols;
  if (cols % 4) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_int4_terms, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, s, h, n, cols, planes);
  return hipGetLastError();
}

hipError_t launch_pack_int4(int fmt, const uint8_t* codes, const uint16_t* scales, bool scales_bf16, const uint8_t* zeros,
                            int rows, int cols, int n, uint8_t* data, uint8_t* out_scales, float* scale2, hipStream_t s) {
  if (!is_int4(fmt) || rows < 1 || rows > INT4_MAX_ROWS || cols < 32 || cols > INT4_MAX_COLS || cols % int4_group(fmt))
    return hipErrorInvalidValue;
  const int group = int4_group(fmt);
  const size_t per = (size_t)rows * (cols / group), tiles = int4_tiles(rows, cols);
  const size_t db = int4_data_bytes(rows, cols), sb = int4_scale_bytes(fmt, rows, cols);
  hipError_t rc = launch_clear_words((uint32_t*)scale2, n, s);
  if (rc != hipSuccess) return rc;
  for (int e0 = 0; e0 < n; e0 += 65535) {  // grid rows
    const int m = n - e0 < 65535 ? n - e0 : 65535;
    const uint8_t* c = codes + (size_t)e0 * rows * (cols / 2);
    const uint16_t* sc = scales + (size_t)e0 * per;
    const unsigned mb = (unsigned)(per + 4095 < 4096 * 64 ? (per + 4095) / 4096 : 64);
    hipLaunchKernelGGL(k_int4_max, dim3(mb, m), dim3(256), 0, s, sc, (int)scales_bf16, per, (uint32_t*)scale2 + e0);
    const size_t blocks = (tiles + 3) / 4;
    for (size_t b0 = 0; b0 < blocks; b0 += INT4_BLOCKS)
      hipLaunchKernelGGL(k_int4_pack, dim3((unsigned)std::min<size_t>(blocks - b0, INT4_BLOCKS), m), dim3(256), 0, s, group, c, sc,
                         (int)scales_bf16, zeros ? zeros + (size_t)e0 * per : nullptr, rows, cols, data + e0 * db,
                         out_scales + e0 * sb, db, sb, int4_zeros_at(fmt, rows, cols), (const uint32_t*)scale2 + e0, b0);
  }
  hipLaunchKernelGGL(k_int4_scale2, dim3((n + 255) / 256), dim3(256), 0, s, scale2, n);
  return hipGetLastError();
}

hipError_t launch_dequant_int4(int fmt, const WeightRef& w, int rows, int cols, int expert, float* out, hipStream_t s) {
  const size_t blocks = ((size_t)rows * (cols / 8) + 255) / 256;
  for (size_t b0 = 0; b0 < blocks; b0 += INT4_BLOCKS)
    hipLaunchKernelGGL(k_int4_dequant, dim3((unsigned)std::min<size_t>(blocks - b0, INT4_BLOCKS)), dim3(256), 0, s, int4_group(fmt),
                       w.data + (size_t)expert * w.estride, w.scales + (size_t)expert * w.sestride,
                       int4_zeros_at(fmt, rows, cols), int4_zeros(fmt), w.scale2 + expert, rows, cols, out, b0);
  return hipGetLastError();
}

}  // namespace moeq
