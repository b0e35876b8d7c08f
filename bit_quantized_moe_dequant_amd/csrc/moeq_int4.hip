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
// What bounds it: the weight stream. A tile of 512 weights costs a SIMD 8 vector operations
// (32 clocks) and one matrix instruction of 16.
#include <hip/hip_ext.h>

#include <algorithm>
#include <type_traits>

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
                                                   const uint32_t* max_bits) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, kt_n = int4_ktiles(cols);
  const size_t tile = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6), e = blockIdx.y;
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
                                                      bool zeros, const float* scale2, int rows, int cols, float* out) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
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
// is there. Where only some of them are used, the compiler gives the others to vector operations
// between the instruction and its end without the wait that this takes, and the result lands in them.
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
__device__ __forceinline__ void int4_store(const Int4Params& P, int e, bool ok, size_t pair, int r, const float (&v)[NMAT]) {
  if constexpr (KIND == I4_LINEAR) {
    const size_t at = pair * P.rows + r;
    float f = v[0] * P.w[0].scale2[e];
    if (P.bias) f += P.bias[r];
    if (P.out_bf16) ((uint16_t*)P.y)[at] = (uint16_t)f32_bf16_rne_nan(f);
    else ((float*)P.y)[at] = f;
  } else if constexpr (KIND == I4_GATE_UP) {
    const float h = ok ? silu_mul(v[0] * P.w[0].scale2[e], v[NMAT - 1] * P.w[1].scale2[e]) : 0.f;
    if (P.out_terms) {
      uint32_t b[3];
      bf16_terms(h, b);
      uint16_t* out = (uint16_t*)P.y + pair * 3 * P.rows + r;
#pragma unroll
      for (int a = 0; a < 3; a++) out[(size_t)a * P.rows] = (uint16_t)b[a];
    } else {
      ((float*)P.y)[pair * P.rows + r] = h;
    }
  } else if constexpr (KIND == I4_DOWN_SUM) {
    ((float*)P.y)[pair * P.rows + r] = v[0];
  } else {
    ((float*)P.y)[pair * P.rows + r] = ok ? v[0] * P.w[0].scale2[e] * P.rw[pair] : 0.f;
  }
}

// One token (or pair; I4_DOWN_SUM: a token's pairs one behind the other) or up to four of a
// linear, whose rows lie in LDS. A work-group: 16 weight rows (of the gate and of the up matrix),
// all of K, whose tiles its waves take in turn, DEPTH of them with their loads in flight at once,
// issued before the activations are waited for; the waves' sums meet in LDS and are added in the
// order of the waves. TERMS: bf16 terms of an activation. The lanes of operand A's unused rows
// read zeros.
template <int GP, bool ZEROS, int TERMS, int KIND, int DEPTH>
__global__ __launch_bounds__(64 * FEW_WAVES) void k_int4_one(Int4Params P) {
  constexpr int NMAT = KIND == I4_GATE_UP ? 2 : 1, NR = TERMS, TOK = TERMS == 1 ? 4 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t xs[];  // 16 bytes of zeros, then the rows
  __shared__ float red[FEW_WAVES][NMAT][TOK][16];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int rt = blockIdx.x, item = blockIdx.y, ktiles = int4_ktiles(P.cols);
  const int parts = KIND == I4_DOWN_SUM ? P.top_k : 1, steps = parts * ktiles;
  const int tok = KIND == I4_LINEAR ? P.T : 1;

  int e = KIND == I4_LINEAR ? P.expert : 0;
  bool ok = true;
  if constexpr (KIND == I4_GATE_UP) {
    e = P.ids[item];
    ok = e >= 0 && e < P.n_experts;
    if (!ok && rt == 0 && threadIdx.x == 0) atomicOr(P.err, 1u);
    if (!ok) e = 0;
  }

  u32x4 wv[DEPTH][NMAT];
  Side<GP, ZEROS, NMAT> side[DEPTH];
  float fac[DEPTH];
  bool live[DEPTH];
  auto load = [&](int u0) {
#pragma unroll
    for (int d = 0; d < DEPTH; d++) {
      const int u = min(u0 + d * waves, steps - 1);
      live[d] = u0 + d * waves < steps && ok;
      int kt = u;
      if constexpr (KIND == I4_DOWN_SUM) {
        const int k = u / ktiles;
        kt = u % ktiles;
        e = P.ids[(size_t)item * P.top_k + k];
        const bool good = e >= 0 && e < P.n_experts;
        if (!good && rt == 0 && lane == 0 && kt == 0 && live[d]) atomicOr(P.err, 1u);
        live[d] = live[d] && good;
        e = good ? e : 0;
        fac[d] = P.rw[(size_t)item * P.top_k + k] * P.w[0].scale2[e];
      }
      int4_load(P, e, (size_t)rt * ktiles + kt, lane, wv[d], side[d]);
    }
  };
  load(wave);

  // the rows: token by token, or part by part and term by term, `pitch` bytes apart
  const int kpad = ktiles * 128, pitch = kpad * 2 + 16, rows = KIND == I4_DOWN_SUM ? parts * TERMS : tok;
  if (threadIdx.x < 4) reinterpret_cast<uint32_t*>(xs)[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < rows * (kpad / 8); i += blockDim.x) {
    const int row = i / (kpad / 8), k = i % (kpad / 8) * 8;
    const uint16_t* a = P.act;
    if constexpr (KIND == I4_DOWN_SUM) a += ((size_t)item * P.top_k + row / TERMS) * P.pitch + row % TERMS * P.term;
    else if constexpr (KIND == I4_GATE_UP) a += (size_t)(item / P.top_k) * P.pitch;
    else a += (size_t)row * P.pitch;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k < P.cols) v = ld16(a + k);
    *reinterpret_cast<u32x4*>(xs + 16 + (size_t)row * pitch + 2 * k) = v;
  }
  __syncthreads();
  // this lane's row of operand A: token n / 4 in row 0, 4, 8, 12, or term n
  const bool a_on = TERMS == 1 ? (n & 3) == 0 && n / 4 < tok : n < TERMS;
  const int a0 = a_on ? 16 + (TERMS == 1 ? n / 4 : n) * pitch + 16 * g : 0, a_step = a_on ? 1 : 0;

  float tot[NMAT][NR];
#pragma unroll
  for (int m = 0; m < NMAT; m++)
#pragma unroll
    for (int r = 0; r < NR; r++) tot[m][r] = 0.f;
  for (int u0 = wave; u0 < steps; u0 += waves * DEPTH) {
    if (u0 != wave) load(u0);
#pragma unroll
    for (int d = 0; d < DEPTH; d++) {
      if (!live[d]) continue;
      const int u = u0 + d * waves, kt = KIND == I4_DOWN_SUM ? u % ktiles : u;
      const uint8_t* x = xs + a0 + a_step * ((KIND == I4_DOWN_SUM ? u / ktiles * TERMS * pitch : 0) + kt * 256);
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
            float s = int4_scale(side[d], m, gi);
            if constexpr (KIND == I4_DOWN_SUM) s *= fac[d];
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
  }
#pragma unroll
  for (int m = 0; m < NMAT; m++) {
    float v = tot[m][0];
#pragma unroll
    for (int a = 1; a < TERMS; a++) v += tot[m][a];
    if (g < TOK) red[wave][m][g][n] = v;
  }
  __syncthreads();
  if ((int)threadIdx.x < tok * 16) {
    const int t = threadIdx.x >> 4, r = rt * 16 + n;
    float v[NMAT];
#pragma unroll
    for (int m = 0; m < NMAT; m++) {
      v[m] = 0.f;
      for (int w = 0; w < waves; w++) v[m] += red[w][m][t][n];
    }
    if (r < P.rows) int4_store<KIND, NMAT>(P, e, ok, KIND == I4_LINEAR ? t : item, r, v);
  }
}

// A few rows to an expert. A work-group takes `rb` row tiles of an expert, one after another; its
// waves take the tiles of K in turn, KT of them at a time, whose activations (and, as
// they do not change with the weight row, their sums for each group) stay in registers, so that
// only weights move: the next row tile's are loaded as this one's are used up. The waves' sums
// meet in LDS (two buffers, so one barrier to a row tile) and are added in the order of the waves.
// NR: output registers in use, so a tile of operand A holds 4 NR / TERMS rows.
template <int GP, bool ZEROS, int TERMS, int NR, int KIND, int KT>
__device__ __forceinline__ void int4_few(const Int4Params& P, float* red, int e, int first, int count, const int32_t* perm,
                                         bool ok, int rt0, int rt1) {
  constexpr int NMAT = KIND == I4_GATE_UP ? 2 : 1, TPQ = NR / TERMS, TOK = 4 * TPQ;
  constexpr int RED = FEW_WAVES * NMAT * TOK * 16;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ktiles = int4_ktiles(P.cols), rounds = (ktiles + FEW_WAVES * KT - 1) / (FEW_WAVES * KT);
  // this lane's row of operand A: token `ai` of the tile, term `aterm`
  const int ai = (n & 3) / TERMS + (n >> 2) * TPQ, aterm = (n & 3) % TERMS;

  for (int m0 = 0; m0 < count; m0 += TOK) {
    const int here = min(TOK, count - m0);
    const bool a_on = (n & 3) < NR && ai < here;
    size_t arow = 0;
    if (a_on) {
      arow = perm ? perm[m0 + ai] : first + m0 + ai;
      if constexpr (KIND == I4_GATE_UP) arow /= P.top_k;
    }
    const uint16_t* ap = P.act + arow * P.pitch + aterm * P.term + 8 * g;
    u32x4 wv[KT][NMAT], xv[KT][4];
    Side<GP, ZEROS, NMAT> side[KT];
    f32x4_t sx[KT][GP];
    auto load = [&](int rt, int round, int i) {
      const int kt = min((round * KT + i) * FEW_WAVES + wave, ktiles - 1);
      int4_load(P, e, (size_t)rt * ktiles + kt, lane, wv[i], side[i]);
    };
    if (ok) {
#pragma unroll
      for (int i = 0; i < KT; i++) load(rt0, 0, i);
    }
    int buf = 0;
    for (int rt = rt0; rt < rt1; rt++, buf ^= 1) {
      float tot[NMAT][NR];
#pragma unroll
      for (int m = 0; m < NMAT; m++)
#pragma unroll
        for (int r = 0; r < NR; r++) tot[m][r] = 0.f;
      if (ok) {
        for (int round = 0; round < rounds; round++) {
          if (rt == rt0 || rounds > 1) {
#pragma unroll
            for (int i = 0; i < KT; i++) {
              const int k0 = ((round * KT + i) * FEW_WAVES + wave) * 128;
#pragma unroll
              for (int j = 0; j < 4; j++) {  // zeros past the end, and so for tiles past it
                xv[i][j] = u32x4{0u, 0u, 0u, 0u};
                if (a_on && k0 + 32 * j < P.cols) xv[i][j] = ld16(ap + k0 + 32 * j);
              }
            }
#pragma unroll
            for (int i = 0; i < KT; i++)
#pragma unroll
              for (int q = 0; q < GP; q++) {
                f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = q * (4 / GP); j < (q + 1) * (4 / GP); j++) v = mfma(xv[i][j], ones(), v);
                sx[i][q] = v;
              }
          }
#pragma unroll
          for (int i = 0; i < KT; i++) {
            if ((round * KT + i) * FEW_WAVES + wave < ktiles) {
#pragma unroll
              for (int q = 0; q < GP; q++)
#pragma unroll
                for (int m = 0; m < NMAT; m++) {
                  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                  for (int j = q * (4 / GP); j < (q + 1) * (4 / GP); j++) acc = mfma(xv[i][j], int4_operand(wv[i][m][j]), acc);
                  const float s = int4_scale(side[i], m, q), c = int4_offset(side[i], m, q);
#pragma unroll
                  for (int r = 0; r < NR; r++) tot[m][r] = __builtin_fmaf(s, __builtin_fmaf(-c, sx[i][q][r], acc[r]), tot[m][r]);
                  hold(tot[m][NR - 1], acc, sx[i][q]);
                }
            }
            if (round + 1 < rounds) load(rt, round + 1, i);
            else if (rt + 1 < rt1) load(rt + 1, 0, i);
          }
        }
      }
      float* rd = red + buf * RED;
#pragma unroll
      for (int m = 0; m < NMAT; m++)
#pragma unroll
        for (int i = 0; i < TPQ; i++) {
          float v = tot[m][i * TERMS];
#pragma unroll
          for (int a = 1; a < TERMS; a++) v += tot[m][i * TERMS + a];
          rd[((wave * NMAT + m) * TOK + g * TPQ + i) * 16 + n] = v;
        }
      __syncthreads();
      const int t = threadIdx.x >> 4, r = rt * 16 + n;
      if (t < here) {
        float v[NMAT];
#pragma unroll
        for (int m = 0; m < NMAT; m++) {
          v[m] = 0.f;
#pragma unroll
          for (int w = 0; w < FEW_WAVES; w++) v[m] += rd[((w * NMAT + m) * TOK + t) * 16 + n];
        }
        if (r < P.rows) int4_store<KIND, NMAT>(P, e, ok, perm ? perm[m0 + t] : first + m0 + t, r, v);
      }
    }
    __syncthreads();  // the buffers are free again
  }
}

template <int GP, bool ZEROS, int KIND, int KT>
__global__ __launch_bounds__(64 * FEW_WAVES, 2) void k_int4_few(Int4Params P, int rb) {
  __shared__ float red[2 * FEW_WAVES * (KIND == I4_GATE_UP ? 2 : 1) * 16 * 16];
  const int rt0 = blockIdx.x * rb, rt1 = min(rt0 + rb, int4_rtiles(P.rows)), item = blockIdx.y;
  int e = P.expert, first = item * 16, count = min(16, P.T - first);
  const int32_t* perm = nullptr;
  bool ok = true;
  if constexpr (KIND != I4_LINEAR) {
    if (item >= P.route.n_slots()[0]) return;
    e = P.route.slots()[item];
    const int p0 = P.route.offsets()[e];
    count = P.route.offsets()[e + 1] - p0;
    perm = P.route.perm() + p0;
    first = 0;
    ok = e < P.n_experts;  // ids out of range have set the error bit when they were sorted
  }
  if constexpr (KIND == I4_DOWN_PART) {
    int4_few<GP, ZEROS, 3, 3, KIND, KT>(P, red, e, first, count, perm, ok, rt0, rt1);
  } else if (count <= 4) {
    int4_few<GP, ZEROS, 1, 1, KIND, KT>(P, red, e, first, count, perm, ok, rt0, rt1);
  } else if (count <= 8 || KIND == I4_GATE_UP) {  // two matrices and sixteen rows do not fit the registers
    int4_few<GP, ZEROS, 1, 2, KIND, KT>(P, red, e, first, count, perm, ok, rt0, rt1);
  } else if constexpr (KIND != I4_GATE_UP) {
    int4_few<GP, ZEROS, 1, 4, KIND, KT>(P, red, e, first, count, perm, ok, rt0, rt1);
  }
}

// LDS of k_int4_one's rows; more than this and the other kernel takes them.
constexpr size_t ONE_LDS = 96 << 10;
size_t one_lds(int rows, int cols) { return 16 + (size_t)rows * (int4_ktiles(cols) * 256 + 16); }

template <int GP, int TERMS, int KIND, int DEPTH>
hipError_t one(const Int4Params& p, int items, int rows, hipStream_t s, const LaunchEvents* ev) {
  const int steps = int4_ktiles(p.cols) * (KIND == I4_DOWN_SUM ? p.top_k : 1);
  const dim3 g((unsigned)int4_rtiles(p.rows), (unsigned)items), b(64 * (steps < FEW_WAVES ? steps : FEW_WAVES));
  const unsigned lds = (unsigned)one_lds(rows, p.cols);
  auto go = [&](auto k) {
    if (ev) hipExtLaunchKernelGGL(k, g, b, lds, s, ev->start, ev->stop, 0, p);
    else hipLaunchKernelGGL(k, g, b, lds, s, p);
    return hipGetLastError();
  };
  return int4_zeros(p.fmt) ? go(k_int4_one<GP, true, TERMS, KIND, DEPTH>) : go(k_int4_one<GP, false, TERMS, KIND, DEPTH>);
}

// Row tiles of a work-group: few enough that every CU has two of them, at most 16.
#ifndef MOEQ_I4_FEW_WGS
#define MOEQ_I4_FEW_WGS 768
#endif
template <int GP, int KIND>
hipError_t few(const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  const long rt = int4_rtiles(p.rows);
  const int rb = (int)std::min(16l, std::max(1l, rt * items / MOEQ_I4_FEW_WGS));
  const dim3 g((unsigned)((rt + rb - 1) / rb), (unsigned)items), b(64 * FEW_WAVES);
  const int kt = (int4_ktiles(p.cols) + FEW_WAVES - 1) / FEW_WAVES;
  auto go = [&](auto k) {
    if (ev) hipExtLaunchKernelGGL(k, g, b, 0, s, ev->start, ev->stop, 0, p, rb);
    else hipLaunchKernelGGL(k, g, b, 0, s, p, rb);
    return hipGetLastError();
  };
  auto by_k = [&](auto z) {
    constexpr bool Z = decltype(z)::value;
    if (kt <= 1) return go(k_int4_few<GP, Z, KIND, 1>);
    if (kt <= 2) return go(k_int4_few<GP, Z, KIND, 2>);
    return go(k_int4_few<GP, Z, KIND, 4>);
  };
  return int4_zeros(p.fmt) ? by_k(std::true_type()) : by_k(std::false_type());
}

template <int GP>
hipError_t few_kind(int kind, const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  switch (kind) {
    case I4_LINEAR:
      if (p.T <= 4 && one_lds(p.T, p.cols) <= ONE_LDS) return one<GP, 1, I4_LINEAR, 4>(p, 1, p.T, s, ev);
      return few<GP, I4_LINEAR>(p, (p.T + 15) / 16, s, ev);
    case I4_GATE_UP:
      return p.grouped ? few<GP, I4_GATE_UP>(p, items, s, ev) : one<GP, 1, I4_GATE_UP, 4>(p, items, 1, s, ev);
    case I4_DOWN_SUM: return one<GP, 3, I4_DOWN_SUM, 12>(p, items, 3 * p.top_k, s, ev);
    case I4_DOWN_PART: return few<GP, I4_DOWN_PART>(p, items, s, ev);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool int4_one_fits(int kind, int top_k, int cols) {
  return one_lds(kind == I4_DOWN_SUM ? 3 * top_k : 1, cols) <= ONE_LDS;
}

hipError_t launch_int4_few(int kind, const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  if (!is_int4(p.fmt) || p.T < 1 || items < 1 || items > 65535 || p.rows < 1 || p.rows > INT4_MAX_ROWS || p.cols < 32 ||
      p.cols > INT4_MAX_COLS || p.cols % int4_group(p.fmt) || p.pitch % 8 || p.term % 8)
    return hipErrorInvalidValue;
  if ((kind == I4_DOWN_SUM || (kind == I4_GATE_UP && !p.grouped)) && !int4_one_fits(kind, p.top_k, p.cols))
    return hipErrorInvalidValue;
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
    hipLaunchKernelGGL(k_int4_pack, dim3((unsigned)((tiles + 3) / 4), m), dim3(256), 0, s, group, c, sc, (int)scales_bf16,
                       zeros ? zeros + (size_t)e0 * per : nullptr, rows, cols, data + e0 * db, out_scales + e0 * sb, db, sb,
                       int4_zeros_at(fmt, rows, cols), (const uint32_t*)scale2 + e0);
  }
  hipLaunchKernelGGL(k_int4_scale2, dim3((n + 255) / 256), dim3(256), 0, s, scale2, n);
  return hipGetLastError();
}

hipError_t launch_dequant_int4(int fmt, const WeightRef& w, int rows, int cols, int expert, float* out, hipStream_t s) {
  const size_t n = (size_t)rows * (cols / 8);
  hipLaunchKernelGGL(k_int4_dequant, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, int4_group(fmt),
                     w.data + (size_t)expert * w.estride, w.scales + (size_t)expert * w.sestride, int4_zeros_at(fmt, rows, cols),
                     int4_zeros(fmt), w.scale2 + expert, rows, cols, out);
  return hipGetLastError();
}

}  // namespace moeq
