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
constexpr int FEW_DEPTH = 4;  // tiles of 128 columns whose loads a wave has in flight

// A work-group: 16 weight rows (of the gate and of the up matrix for NMAT = 2), all of K, whose
// tiles its waves take in turn; their sums meet in LDS and are added in the order of the waves.
// GP: groups per 128 columns. TERMS: bf16 terms of an activation. NR: output registers in use,
// so a tile holds 4 NR / TERMS tokens.
template <int GP, int TERMS, int NR, int KIND>
__global__ __launch_bounds__(64 * FEW_WAVES) void k_int4_few(Int4Params P) {
  constexpr int NMAT = KIND == I4_GATE_UP ? 2 : 1, TPQ = NR / TERMS, TOK = 4 * TPQ;
  __shared__ float red[FEW_WAVES][NMAT][TOK][16];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int rt = blockIdx.x, item = blockIdx.y, ktiles = int4_ktiles(P.cols);

  // The rows of this work-group's activations: `count` of them, in tiles of TOK.
  int e = 0, first = 0, count = 1;
  const int32_t* perm = nullptr;
  bool ok = true;
  if constexpr (KIND == I4_LINEAR) {
    e = P.expert;
    first = item * TOK;
    count = min(TOK, P.T - first);
  } else if constexpr (KIND != I4_DOWN_SUM) {
    if (P.grouped) {
      if (item >= P.route.n_slots()[0]) return;
      e = P.route.slots()[item];
      const int p0 = P.route.offsets()[e];
      count = P.route.offsets()[e + 1] - p0;
      perm = P.route.perm() + p0;
    } else {
      e = P.ids[item];
      first = item;
    }
    ok = e >= 0 && e < P.n_experts;
    if (!ok && rt == 0 && threadIdx.x == 0) atomicOr(P.err, 1u);
  }
  const int steps = KIND == I4_DOWN_SUM ? P.top_k * ktiles : ktiles;

  // this lane's row of operand A: token `ai` of the tile, term `at`
  const int ai = (n & 3) / TERMS + (n >> 2) * TPQ, aterm = (n & 3) % TERMS;
  const size_t tiles_at = (size_t)rt * ktiles;

  for (int m0 = 0; m0 < count; m0 += TOK) {
    const int here = min(TOK, count - m0);
    float tot[NMAT][NR];
#pragma unroll
    for (int m = 0; m < NMAT; m++)
#pragma unroll
      for (int r = 0; r < NR; r++) tot[m][r] = 0.f;
    const bool a_on = (n & 3) < NR && ai < here;
    size_t arow = 0;
    if (a_on) {
      if constexpr (KIND == I4_LINEAR) arow = first + ai;
      else if constexpr (KIND == I4_DOWN_SUM) arow = (size_t)item * P.top_k;
      else if constexpr (KIND == I4_GATE_UP) arow = (perm ? perm[m0 + ai] : first) / P.top_k;
      else arow = perm ? perm[m0 + ai] : first;
    }
    const uint16_t* ap = P.act + arow * P.pitch + aterm * P.term + 8 * g;

    if (ok) {
      for (int u0 = wave; u0 < steps; u0 += waves * FEW_DEPTH) {
        u32x4 wv[FEW_DEPTH][NMAT], xv[FEW_DEPTH][4];
        u32x2 sv[FEW_DEPTH][NMAT];
        uint32_t zv[FEW_DEPTH][NMAT];
        float fac[FEW_DEPTH];
        bool live[FEW_DEPTH];
#pragma unroll
        for (int d = 0; d < FEW_DEPTH; d++) {
          const int u = min(u0 + d * waves, steps - 1);
          const int kt = KIND == I4_DOWN_SUM ? u % ktiles : u;
          int ee = e;
          fac[d] = 1.f;
          live[d] = u0 + d * waves < steps;
          const uint16_t* a = ap;
          if constexpr (KIND == I4_DOWN_SUM) {
            const int k = u / ktiles;
            ee = P.ids[(size_t)item * P.top_k + k];
            const bool good = ee >= 0 && ee < P.n_experts;
            if (!good && rt == 0 && lane == 0 && kt == 0) atomicOr(P.err, 1u);
            ee = good ? ee : 0;
            live[d] = live[d] && good;
            fac[d] = P.rw[(size_t)item * P.top_k + k] * P.w[0].scale2[ee];
            a += k * P.pitch;
          }
          const size_t tile = tiles_at + kt;
#pragma unroll
          for (int m = 0; m < NMAT; m++) {
            wv[d][m] = ld16(P.w[m].data + (size_t)ee * P.w[m].estride + tile * 1024 + 16 * lane);
            const uint8_t* sp = P.w[m].scales + (size_t)ee * P.w[m].sestride;
            const size_t at = tile * 16 * GP + n * GP;
            if constexpr (GP == 1) sv[d][m][0] = *reinterpret_cast<const uint16_t*>(sp + 2 * at);
            else if constexpr (GP == 2) sv[d][m][0] = *reinterpret_cast<const uint32_t*>(sp + 2 * at);
            else sv[d][m] = *reinterpret_cast<const u32x2*>(sp + 2 * at);
            zv[d][m] = 0x08080808u;
            if (int4_zeros(P.fmt)) {
              const uint8_t* zp = sp + int4_zeros_at(P.fmt, P.rows, P.cols) + at;
              if constexpr (GP == 1) zv[d][m] = *zp;
              else if constexpr (GP == 2) zv[d][m] = *reinterpret_cast<const uint16_t*>(zp);
              else zv[d][m] = *reinterpret_cast<const uint32_t*>(zp);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; j++) {
            xv[d][j] = u32x4{0u, 0u, 0u, 0u};
            if (a_on && kt * 128 + 32 * j < P.cols) xv[d][j] = ld16(a + kt * 128 + 32 * j);
          }
        }
#pragma unroll
        for (int d = 0; d < FEW_DEPTH; d++) {
          if (!live[d]) continue;
          f32x4_t acc[NMAT], sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int m = 0; m < NMAT; m++) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const bf16x8_t x = __builtin_bit_cast(bf16x8_t, xv[d][j]);
            sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                x, __builtin_bit_cast(bf16x8_t, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}), sx, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < NMAT; m++) {
              const uint32_t w = wv[d][m][j];
              const u32x4 q = {((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                               ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u};
              acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, __builtin_bit_cast(bf16x8_t, q), acc[m], 0, 0, 0);
            }
            if ((j + 1) % (4 / GP) == 0) {  // a group's end
              const int gi = j * GP / 4;
#pragma unroll
              for (int m = 0; m < NMAT; m++) {
                const float s = half_bits_f32(sv[d][m][gi / 2] >> (16 * (gi & 1))) * fac[d];
                const float c = 16.0f + (float)(zv[d][m] >> (8 * gi) & 255u);
#pragma unroll
                for (int r = 0; r < NR; r++) tot[m][r] = __builtin_fmaf(s, __builtin_fmaf(-c, sx[r], acc[m][r]), tot[m][r]);
                acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
              }
              sx = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < NMAT; m++)
#pragma unroll
      for (int i = 0; i < TPQ; i++) {
        float v = tot[m][i * TERMS];
#pragma unroll
        for (int a = 1; a < TERMS; a++) v += tot[m][i * TERMS + a];
        red[wave][m][g * TPQ + i][n] = v;
      }
    __syncthreads();
    for (int o = threadIdx.x; o < here * 16; o += blockDim.x) {
      const int t = o >> 4, r = rt * 16 + (o & 15);
      float v[NMAT];
#pragma unroll
      for (int m = 0; m < NMAT; m++) {
        v[m] = 0.f;
        for (int w = 0; w < waves; w++) v[m] += red[w][m][t][o & 15];
      }
      if (r >= P.rows) continue;
      if constexpr (KIND == I4_LINEAR) {
        const size_t at = (size_t)(first + t) * P.rows + r;
        float f = v[0] * P.w[0].scale2[e];
        if (P.bias) f += P.bias[r];
        if (P.out_bf16) ((uint16_t*)P.y)[at] = (uint16_t)f32_bf16_rne_nan(f);
        else ((float*)P.y)[at] = f;
      } else if constexpr (KIND == I4_GATE_UP) {
        const size_t pair = perm ? perm[m0 + t] : first;
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
        ((float*)P.y)[(size_t)item * P.rows + r] = v[0];
      } else {
        const size_t pair = perm ? perm[m0 + t] : first;
        ((float*)P.y)[pair * P.rows + r] = ok ? v[0] * P.w[0].scale2[e] * P.rw[pair] : 0.f;
      }
    }
    __syncthreads();
  }
}

template <int GP, int TERMS, int NR, int KIND>
hipError_t few(const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  const int steps = int4_ktiles(p.cols) * (KIND == I4_DOWN_SUM ? p.top_k : 1);
  const dim3 g((unsigned)int4_rtiles(p.rows), (unsigned)items), b(64 * (steps < FEW_WAVES ? steps : FEW_WAVES));
  if (ev) hipExtLaunchKernelGGL((k_int4_few<GP, TERMS, NR, KIND>), g, b, 0, s, ev->start, ev->stop, 0, p);
  else hipLaunchKernelGGL((k_int4_few<GP, TERMS, NR, KIND>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int GP>
hipError_t few_kind(int kind, const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  // Tokens of a tile: as many as one item can hold.
  const int rows = kind == I4_LINEAR ? p.T : p.grouped ? p.T : 1;
  switch (kind) {
    case I4_LINEAR: {
      if (rows <= 4) return few<GP, 1, 1, I4_LINEAR>(p, 1, s, ev);
      if (rows <= 8) return few<GP, 1, 2, I4_LINEAR>(p, 1, s, ev);
      Int4Params q = p;
      for (long t0 = 0; t0 < p.T; t0 += 16L * 65535) {  // grid rows
        const int n = (int)(p.T - t0 < 16L * 65535 ? p.T - t0 : 16L * 65535);
        q.T = n;
        q.act = p.act + (size_t)t0 * p.pitch;
        q.y = (uint8_t*)p.y + (size_t)t0 * p.rows * (p.out_bf16 ? 2 : 4);
        const hipError_t e = few<GP, 1, 4, I4_LINEAR>(q, (n + 15) / 16, s, ev);
        if (e != hipSuccess) return e;
      }
      return hipSuccess;
    }
    case I4_GATE_UP:
      if (rows <= 4) return few<GP, 1, 1, I4_GATE_UP>(p, items, s, ev);
      if (rows <= 8) return few<GP, 1, 2, I4_GATE_UP>(p, items, s, ev);
      return few<GP, 1, 4, I4_GATE_UP>(p, items, s, ev);
    case I4_DOWN_SUM: return few<GP, 3, 3, I4_DOWN_SUM>(p, items, s, ev);
    case I4_DOWN_PART: return few<GP, 3, 3, I4_DOWN_PART>(p, items, s, ev);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_int4_few(int kind, const Int4Params& p, int items, hipStream_t s, const LaunchEvents* ev) {
  if (!is_int4(p.fmt) || p.T < 1 || items < 1 || items > 65535 || p.rows < 1 || p.rows > INT4_MAX_ROWS || p.cols < 32 ||
      p.cols > INT4_MAX_COLS || p.cols % int4_group(p.fmt) || p.pitch % 8 || p.term % 8)
    return hipErrorInvalidValue;
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
