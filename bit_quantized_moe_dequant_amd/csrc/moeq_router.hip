// The router: logits, scores, the top-k experts of every token and their weights.
//
//   z_te = sum_h W_eh x_th            bf16 x bf16, fp64 sums
//   s_te = softmax_e(z) | sigmoid(z) | sqrt(log(1 + e^z))
//   ids  = the top_k largest s + bias (fp64), ties to the lowest id
//   w    = s[ids] (/ their sum) * scale
//
// Everything up to the weights is held in fp64.
// The choice of experts is discontinuous: fp32 logits carry an error of about 1e-6 that
// depends on the order of summation, so two correct fp32 routers disagree on a near tie
// and a token's output jumps. A product of two bf16 values is exact in fp64 and the vector
// unit issues fp64 FMAs at the fp32 rate here, so the exactness costs the conversions only.
#include "moeq_grid.h"
#include "moeq_router.h"
#include "moeq_router_bound.h"
#include "moeq_tiled.h"

namespace moeq {

namespace {

template <bool GROUPS>
__global__ __launch_bounds__(512) void k_router_few(RouterParams P) {
  router_few<GROUPS>(P, blockIdx.x, blockIdx.y);
}

// All logits in fp64, on the fp64 matrix instruction, whose operands are converted once for
// sixteen rows: v_mfma_f64_16x16x4, lane l: operand A's row l % 16 and B's row l % 16 at
// K = l / 16; output register r: A's row l / 16 + 4 r times B's row l % 16. Which K a lane's
// values stand for is free as long as both operands agree, so a lane takes whole 16-byte
// chunks of its rows. A work-group has 16 tokens and 16 experts; its waves take runs of 128
// bytes of K in turn, and their sums are added in the order of the waves. 2048 tokens, 4096 x
// 256: 85 us, 50 TFLOP/s (one FMA chain per token and expert on the vector unit, its operands
// converted for each: 235); the fp64 matrix rate bounds it, at 78.6 a floor of 55.
constexpr int RL_WAVES = 8;
typedef double f64x4 __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(64 * RL_WAVES) void k_router_logits(RouterParams P) {
  __shared__ double part[RL_WAVES][16][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const int chunks = P.hidden / 8;
  const uint16_t* x = P.x + (size_t)min(t0 + n, P.T - 1) * P.hidden;
  const uint16_t* w = P.w + (size_t)min(e0 + n, P.n_experts - 1) * P.hidden;
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
  for (int c0 = 8 * wave; c0 < chunks; c0 += 8 * RL_WAVES) {
    u32x4 xv[2], wv[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int c = c0 + 4 * i + g, in = min(c, chunks - 1);
      xv[i] = ld16(x + 8 * (size_t)in);
      wv[i] = ld16(w + 8 * (size_t)in);
      if (c >= chunks) xv[i] = wv[i] = u32x4{0u, 0u, 0u, 0u};  // both: 0 times an infinity of the last chunk
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)u2f(xv[i][j] << 16), (double)u2f(wv[i][j] << 16), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)u2f(xv[i][j] & 0xFFFF0000u), (double)u2f(wv[i][j] & 0xFFFF0000u),
                                                   acc, 0, 0, 0);
      }
  }
#pragma unroll
  for (int r = 0; r < 4; r++) part[wave][g + 4 * r][n] = acc[r];
  __syncthreads();
  const int tk = threadIdx.x >> 4, e = e0 + (threadIdx.x & 15);
  if (threadIdx.x < 256 && t0 + tk < P.T && e < P.n_experts) {
    double z = part[0][tk][threadIdx.x & 15];
#pragma unroll
    for (int v = 1; v < RL_WAVES; v++) z += part[v][tk][threadIdx.x & 15];
    P.logits[(size_t)(t0 + tk) * P.n_experts + e] = P.scoring == SCORE_SOFTMAX ? z : score_of(P.scoring, z);
  }
}

template <bool GROUPS>
__global__ __launch_bounds__(256) void k_router_choose(RouterParams P) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= P.T) return;
  if (P.n_experts <= 256) choose<4, false, GROUPS>(P, t, lane);
  else if (P.n_experts <= 512) choose<8, false, GROUPS>(P, t, lane);
  else choose<16, false, GROUPS>(P, t, lane);
}

// ---------------------------------------------------------------- many tokens
// All E logits of a token in fp64 cost E H FMAs at the fp64 rate, and the choice needs only a
// few of them exactly. So:
//
//   1. approximate logits on the bf16 matrix instruction, whose fp32 sums are added up in
//      fp64 every RM_FLUSH steps (k_router_mm);
//   2. one wave per token (k_router_pick): with |approximate - exact| <= d_e, the key at
//      z_e + d_e is an upper bound of the expert's exact key. The K experts with the
//      largest bounds get exact logits; then, while some other expert's bound reaches the
//      K-th exact key, the one with the largest bound does too. What is left cannot be
//      chosen. (Each costs 1 to 2 us, one after another: experts whose logits are equal, not
//      known from the norms and more than a few would be slow.)
//
// Groups: between 1. and 2. the same bounds and lower ones give every group's merit from above and
// below; while that leaves the kept groups open, an exact logit at a time closes it. Experts of
// other groups then drop out. 2048 tokens, 4096 x 256 in 8
// groups: k_router_pick 44 us.
//
// The bound d_e = router_unit() |W_e| |x| + 2^-100: moeq_router_bound.h.
//
// Measured at 2048 tokens, 4096 x 256, 6 of them: 38 us (13 and 26) against 92 with all logits
// in fp64 (k_router_logits 85); what bounds it is the vector unit's fp64 work and the chain of
// choices in k_router_pick. Up to ROUTER_FEW_T tokens the one-launch form is faster (64 tokens
// 24.0 against 26.1 us; 128 tokens 38.0 against 26.7).
constexpr int RM_E = 64, RM_T = 64;  // experts and tokens of a tile

__global__ __launch_bounds__(256) void k_router_mm(RouterParams P, int z_count, int z_bytes, int tiles) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int)blockIdx.x >= tiles * z_count) {  // |W_e|, one expert to a wave
    const int e = ((int)blockIdx.x - tiles * z_count) * 4 + wave;
    if (e >= P.n_experts) return;
    double q = 0.0;
    for (int c = lane; c < P.hidden / 8; c += 64) {
      const u32x4 v = ld16(P.w + (size_t)e * P.hidden + 8 * (size_t)c);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const double lo = (double)u2f(v[j] << 16), hi = (double)u2f(v[j] & 0xFFFF0000u);
        q = __builtin_fma(lo, lo, __builtin_fma(hi, hi, q));
      }
    }
    q = wave_sum(q);
    if (lane == 0) P.norms[e] = sqrt(q);
    return;
  }
  __shared__ __attribute__((aligned(16))) uint8_t lds[tiled_lds<2, 2, 1, 1, 4, 128>()];
  const int z = blockIdx.x / tiles;
  int be, bt;
  tile_of(blockIdx.x % tiles, (P.n_experts + RM_E - 1) / RM_E, (P.T + RM_T - 1) / RM_T, be, bt);
  const int e0 = be * RM_E, t0 = bt * RM_T, pitch = 2 * P.hidden;
  f32x16 acc[1][1];
  double sum[16];
#pragma unroll
  for (int r = 0; r < 16; r++) sum[r] = 0.0;
  auto flush = [&](int s) {
    if (s % RM_FLUSH == RM_FLUSH - 1) {
#pragma unroll
      for (int r = 0; r < 16; r++) {
        sum[r] += (double)acc[0][0][r];
        acc[0][0][r] = 0.f;
      }
    }
  };
  tiled_product<MmaBf16, 2, 2, 1, 1, 4, 128, 4, 1>(
      reinterpret_cast<const int8_t*>(P.w) + (size_t)e0 * pitch + z * z_bytes, P.n_experts - e0,
      reinterpret_cast<const int8_t*>(P.x) + (size_t)t0 * pitch + z * z_bytes, P.T - t0, pitch,
      min(z_bytes, pitch - z * z_bytes), lds, acc, flush);
  flush(RM_FLUSH - 1);
  const int wm = wave & 1, wn = wave >> 1, n = lane & 31, g = lane >> 5;
  const int t = t0 + 32 * wn + n;
  if (t < P.T) {
    float* out = P.approx + ((size_t)z * P.T + t) * P.n_experts;
#pragma unroll
    for (int r = 0; r < 16; r++) {
      const int e = e0 + 32 * wm + (r & 3) + 8 * (r >> 2) + 4 * g;
      if (e < P.n_experts) out[e] = (float)sum[r];
    }
  }
}

// A number not below the score of any logit that is not above v, from the fast fp32
// functions: 2^-17 and |v| 2^-22 of it cover their errors (an ulp each, and the scaling of
// the exponential's argument), 1e-18 what underflows.
__device__ __forceinline__ float score_above(int scoring, float v) {
  v = v + __builtin_fabsf(v) * 0x1p-23f;  // the rounding of v itself
  const float slack = 0x1p-17f + __builtin_fminf(__builtin_fabsf(v), 1e6f) * 0x1p-22f;
  if (scoring == SCORE_SIGMOID) {
    const float p = __fdividef(1.0f, 1.0f + __expf(-v));
    return __builtin_fminf(p + p * slack + 1e-18f, 1.0f);
  }
  const float e = __expf(-__builtin_fabsf(v));
  // log(1 + e) <= e - e^2 / 2 + e^3 / 3, close where e is small and the logarithm of 1 + e is not
  const float l = e < 0.015625f ? e * (1.0f - e * (0.5f - e * 0.33333334f)) : __logf(1.0f + e);
  const float p = __builtin_fmaxf(v, 0.f) + l;
  return __builtin_sqrtf(p + 2.0f * p * slack) + 1e-18f;
}

// The other end: a number not above the score of any logit that is not below v.
__device__ __forceinline__ float score_below(int scoring, float v) {
  v = v - __builtin_fabsf(v) * 0x1p-23f;
  const float slack = 0x1p-17f + __builtin_fminf(__builtin_fabsf(v), 1e6f) * 0x1p-22f;
  if (scoring == SCORE_SIGMOID) {
    const float p = __fdividef(1.0f, 1.0f + __expf(-v));
    return __builtin_fmaxf(p - p * slack - 1e-18f, 0.f);
  }
  const float e = __expf(-__builtin_fabsf(v));
  const float l = e < 0.015625f ? e * (1.0f - e * (0.5f - e * 0.33333334f)) : __logf(1.0f + e);
  const float p = __builtin_fmaxf(v, 0.f) + l;
  return __builtin_fmaxf(__builtin_sqrtf(__builtin_fmaxf(p - 2.0f * p * slack, 0.f)) - 1e-18f, 0.f);
}

// The lane that holds the largest (value, then lowest id) and that value; by every lane.
__device__ __forceinline__ int lane_of_max(uint64_t v, uint32_t id, uint64_t& top) {
  const uint32_t mh = wave_max((uint32_t)(v >> 32));
  bool in = (uint32_t)(v >> 32) == mh;
  const uint32_t ml = wave_max(in ? (uint32_t)v : 0u);
  in = in && (uint32_t)v == ml;
  uint64_t who = __ballot(in);
  if (__popcll(who) > 1) {
    const uint32_t mi = wave_max(in ? ~id : 0u);
    in = in && ~id == mi;
    who = __ballot(in);
  }
  top = ((uint64_t)mh << 32) | ml;
  return __ffsll((long long)who) - 1;
}

constexpr int RP_SEG = 4096;  // values of a token held at a time (64 to a lane)

// Two waves to a SIMD at least: left free, the compiler hoists conversions and constants
// until a SIMD holds one.
template <int N, bool GROUPS>
__global__ __launch_bounds__(256, 2) void k_router_pick(RouterParams P, int z_count) {
  __shared__ double ends[GROUPS ? 4 : 1][2][GROUPS ? 64 * N : 1];  // GROUPS: a wave's keys, from above and from below
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * 4 + wave;
  if (t >= P.T) return;
  const uint16_t* x = P.x + (size_t)t * P.hidden;
  const int chunks = P.hidden / 8, E = P.n_experts, K = P.top_k;
  const int segs = (chunks + RP_SEG / 8 - 1) / (RP_SEG / 8);

  u32x4 xv[RP_SEG / 512];
  auto load = [&](const uint16_t* row, int seg, u32x4 (&v)[RP_SEG / 512]) {  // chunks past the end are zeros
#pragma unroll
    for (int i = 0; i < RP_SEG / 512; i++) {
      const int c = seg * (RP_SEG / 8) + lane + 64 * i;
      v[i] = ld16(row + 8 * (size_t)min(c, chunks - 1));
      if (c >= chunks) v[i] = u32x4{0u, 0u, 0u, 0u};
    }
  };
  auto dot = [&](const u32x4 (&p)[RP_SEG / 512], const u32x4 (&q)[RP_SEG / 512]) {  // this lane's part
    double a[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < RP_SEG / 512; i++) {
      u32x4 u = q[i];
      // the compiler would convert the token's values once for all rows and hold 128 registers of them
      asm volatile("" : "+v"(u));
#pragma unroll
      for (int j = 0; j < 4; j++) {
        a[j] = __builtin_fma((double)u2f(p[i][j] << 16), (double)u2f(u[j] << 16), a[j]);
        a[j] = __builtin_fma((double)u2f(p[i][j] & 0xFFFF0000u), (double)u2f(u[j] & 0xFFFF0000u), a[j]);
      }
    }
    return (a[0] + a[1]) + (a[2] + a[3]);
  };
  auto logit = [&](int e) {  // exact, by every lane
    double a = 0.0;
    for (int s = 0; s < segs; s++) {
      u32x4 wv[RP_SEG / 512];
      load(P.w + (size_t)e * P.hidden, s, wv);
      if (segs > 1) load(x, s, xv);
      a += dot(wv, xv);
    }
    return wave_sum(a);
  };

  double z[N];
  uint64_t bound[N];  // upper bounds; 0: chosen or past the end
  const bool soft = P.scoring == SCORE_SOFTMAX;  // (without a bias here) ordered by the logit
  auto next = [&](int& e, uint64_t& top) {  // the largest bound left, without taking it
    uint64_t b = bound[0];
    uint32_t at = 0;
#pragma unroll
    for (int i = 1; i < N; i++)
      if (bound[i] > b) {
        b = bound[i];
        at = i;
      }
    const int src = lane_of_max(b, lane + 64 * at, top);
    e = src + 64 * __builtin_amdgcn_readlane((int)at, src);
  };
  auto take = [&](int e) {
#pragma unroll
    for (int i = 0; i < N; i++)
      if (lane + 64 * i == e) bound[i] = 0;
  };
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int e = lane + 64 * i;
    z[i] = -__builtin_inf();
    if (e < E) {
      double v = 0.0;
      for (int k = 0; k < z_count; k++) v += (double)P.approx[((size_t)k * P.T + t) * E + e];
      z[i] = v;
    }
  }
  // |x|, rounded up: in fp32 where its squares neither overflow nor vanish there
  float q = 0.f;
  for (int s = segs - 1; s >= 0; s--) {
    load(x, s, xv);
#pragma unroll
    for (int i = 0; i < RP_SEG / 512; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float lo = u2f(xv[i][j] << 16), hi = u2f(xv[i][j] & 0xFFFF0000u);
        q = __builtin_fmaf(lo, lo, __builtin_fmaf(hi, hi, q));
      }
  }
  double nx = wave_sum((double)q) * 1.001;  // at most 2 H / 64 + 1 roundings of 2^-24
  if (!(nx > 1e-30 && nx < 1e38)) {
    nx = 0.0;
    for (int s = segs - 1; s >= 0; s--) {
      load(x, s, xv);
      nx += dot(xv, xv);
    }
    nx = wave_sum(nx);
  }
  nx = sqrt(nx);
  auto score = [&](double v) { return soft ? v : score_of(P.scoring, v); };
  uint32_t known = 0;   // experts whose logit the norms tell
  bool spoilt = false;  // one of them NaN
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int e = lane + 64 * i;
    bound[i] = 0;
    if (e < E) {
      const double size = P.norms[e] * nx;
      double k = z[i] + (router_unit() * size + 0x1p-100);
      if (!soft) k = (double)score_above(P.scoring, (float)k);
      if (P.bias) k += (double)P.bias[e];
      if constexpr (GROUPS) {  // never a softmax
        double l = (double)score_below(P.scoring, (float)(z[i] - (router_unit() * size + 0x1p-100)));
        if (P.bias) l += (double)P.bias[e];
        const bool open = !(__builtin_fabs(z[i]) < __builtin_inf() && k == k && l == l);
        const bool out = P.bias && P.bias[e] != P.bias[e];
        ends[wave][0][e] = out ? -__builtin_inf() : open ? __builtin_inf() : k;
        ends[wave][1][e] = out || open ? -__builtin_inf() : l;
      }
      // nothing is known of a sum that left fp32's range: its exact logit is needed
      bound[i] = __builtin_fabs(z[i]) < __builtin_inf() && k == k ? order_of(k) : ~0ull;
      if (P.bias && P.bias[e] != P.bias[e]) bound[i] = order_of(-__builtin_inf());
      if (!(size > 0.0)) {
        z[i] = size;
        known |= 1u << i;
        spoilt |= size != size;
      }
    }
  }
  // Where the token or the expert is all zeros the logit is 0, and NaN where one of them holds a
  // NaN or an infinity meets nothing but zeros: the product of the norms says which, and the
  // key itself is the bound. Bounds above it would have every expert's exact logit taken for a
  // token of padding (256 tokens, a third of them zeros, 2048 x 256: 419 against 28 us).
  if (__ballot(known != 0)) {
    const double s0 = score(0.0);
#pragma unroll
    for (int i = 0; i < N; i++)
      if (known >> i & 1) {
        const double s = z[i] == 0.0 ? s0 : z[i];
        const double k = P.bias ? s + (double)P.bias[lane + 64 * i] : s;
        bound[i] = order_of(k);
        if constexpr (GROUPS) ends[wave][0][lane + 64 * i] = ends[wave][1][lane + 64 * i] = k == k ? k : -__builtin_inf();
      }
  }
  if constexpr (GROUPS) {
    const int size = E / P.n_groups, gl = group_lanes(P.n_groups), q = lane / gl;
    const bool top2 = P.group_top2 && size > 1;
    double* up = ends[wave][0];
    double* down = ends[wave][1];
    uint64_t kept;
    for (;;) {  // each time around one more expert's ends meet, until the groups are told apart
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // what other lanes wrote
      double a[2] = {-__builtin_inf(), -__builtin_inf()}, b[2] = {-__builtin_inf(), -__builtin_inf()};
      double most = -__builtin_inf();  // of this lane's experts whose ends lie apart the highest
      int at = -1;
      if (q < P.n_groups)
        for (int i = lane % gl; i < size; i += gl) {
          const int e = q * size + i;
          const double v[2] = {up[e], down[e]};
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const double low = a[h] < v[h] ? a[h] : v[h];
            a[h] = a[h] > v[h] ? a[h] : v[h];
            b[h] = b[h] > low ? b[h] : low;
          }
          if (v[0] > v[1] && (at < 0 || v[0] > most)) {
            most = v[0];
            at = e;
          }
        }
      const uint64_t above = group_merit(a[0], b[0], gl, top2), below = group_merit(a[1], b[1], gl, top2);
      int maybe = 0, surely = 0;  // groups that may come before this one, and that must
      for (int o = 0; o < P.n_groups; o++) {
        const uint64_t oa = read_lane(above, o * gl), ob = read_lane(below, o * gl);
        if (o == q) continue;
        maybe += o < q ? oa >= below : oa > below;
        surely += o < q ? ob >= above : ob > above;
      }
      kept = __ballot(q < P.n_groups && lane % gl == 0 && maybe < P.top_groups);
      const bool open = q < P.n_groups && maybe >= P.top_groups && surely < P.top_groups;
      if (__ballot(open) == 0) break;
      // the highest such expert of a group whose merit is not known: an undecided group's, else any's
      uint64_t from = __ballot(open && above > below && at >= 0);
      if (from == 0) from = __ballot(above > below && at >= 0);
      if (from == 0) break;  // not reached: merits that are known tell the groups apart
      uint64_t top;
      const bool in = from >> lane & 1;
      const int e = __builtin_amdgcn_readlane(at, lane_of_max(in ? order_of(most) : 0ull, in ? (uint32_t)at : 0xFFFFFFFFu, top));
      const double s = score(logit(e)), k = P.bias ? s + (double)P.bias[e] : s;
      if (lane == 0) up[e] = down[e] = k == k ? k : -__builtin_inf();
    }
#pragma unroll
    for (int i = 0; i < N; i++)
      if (!(kept >> ((lane + 64 * i) / size * gl & 63) & 1)) bound[i] = 0;
  }
  const bool mine = lane < K;  // lane k < K: an expert of the best K so far, its exact logit and key
  int id = 0;
  double zk = 0.0;
  for (int k = 0; k < K; k++) {
    int e;
    uint64_t top;
    next(e, top);
    take(e);
    if (lane == k) id = e;
  }
  if (segs == 1) {  // the next expert's row is on its way while one is multiplied
    u32x4 wv[2][RP_SEG / 512];
    load(P.w + (size_t)__builtin_amdgcn_readlane(id, 0) * P.hidden, 0, wv[0]);
    for (int k = 0; k < K; k += 2) {
      load(P.w + (size_t)__builtin_amdgcn_readlane(id, min(k + 1, K - 1)) * P.hidden, 0, wv[1]);
      const double v0 = wave_sum(dot(wv[0], xv));
      if (lane == k) zk = v0;
      load(P.w + (size_t)__builtin_amdgcn_readlane(id, min(k + 2, K - 1)) * P.hidden, 0, wv[0]);
      const double v1 = wave_sum(dot(wv[1], xv));
      if (lane == k + 1) zk = v1;
    }
  } else {
    for (int k = 0; k < K; k++) {
      const double v = logit(__builtin_amdgcn_readlane(id, k));
      if (lane == k) zk = v;
    }
  }
  double sk = score(zk);
  uint64_t key = 0;
  if (mine) key = order_of(P.bias ? sk + (double)P.bias[id] : sk);
  bool nan = __ballot((mine && zk != zk) || spoilt) != 0;
  for (;;) {
    int e;
    uint64_t top, low;
    // the lowest of the K: the smallest key, of equal ones the highest id
    const int worst = lane_of_max(mine ? ~key : 0ull, mine ? ~(uint32_t)id : 0xFFFFFFFFu, low);
    low = ~low;
    next(e, top);
    // e has the lowest id of the largest bounds left: a key that is no more than equal to the
    // worst's loses to it behind its id
    if (top == 0 || top < low || (top == low && e > __builtin_amdgcn_readlane(id, worst))) break;
    take(e);
    const double v = logit(e);
    const double s = score(v);
    const uint64_t kv = order_of(P.bias ? s + (double)P.bias[e] : s);
    nan |= v != v;
    if (kv > low || (kv == low && e < __builtin_amdgcn_readlane(id, worst))) {
      if (lane == worst) {
        id = e;
        zk = v;
        sk = s;
        key = kv;
      }
    }
  }

  // Normalised over the K, so the denominator over all experts cancels: but for a NaN logit
  // in it, chosen or not, which leaves no number.
  if (soft) {
    double top = mine ? zk : -__builtin_inf();
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double v = __shfl_xor(top, o, 64);
      top = v > top ? v : top;
    }
    sk = nan ? __builtin_nan("") : exp(zk - top);
  }
  int rank = 0;
  for (int k = 0; k < K; k++) {
    const uint64_t ok = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, k) |
                        ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), k) << 32);
    rank += ok > key || (ok == key && __builtin_amdgcn_readlane(id, k) < id);
  }
  double sum = 0.0;
  for (int r = 0; r < K; r++) sum += read_lane(sk, __ffsll((long long)__ballot(mine && rank == r)) - 1);
  if (mine) {
    P.ids[(size_t)t * K + rank] = id;
    double w = sk;
    if (P.normalize) w = sum == 0.0 ? 0.0 : w / sum;
    P.rw[(size_t)t * K + rank] = (float)(w * (double)P.scale);
  }
}

// Parts of K: enough work-groups for every CU, no part under 512 bytes.
int mm_split(const RouterParams& p, long tiles) {
  int z = 1;
  while (z < ROUTER_MM_Z && tiles * z < 256 && p.hidden / (2 * z) >= 256) z *= 2;
  return z;
}

}  // namespace

bool router_few_fits(int T) { return T <= ROUTER_FEW_T; }

hipError_t launch_router(const RouterParams& p, hipStream_t s) {
  if (p.T < 1 || p.n_experts < 1 || p.n_experts > 1024 || p.top_k < 1 || p.top_k > 16 || p.top_k > p.n_experts ||
      p.hidden < 8 || p.hidden % 8)
    return hipErrorInvalidValue;
  const bool groups = p.n_groups > 1;
  if (groups && (p.n_groups > 64 || p.n_experts % p.n_groups || p.top_groups < 1 || p.top_groups > p.n_groups))
    return hipErrorInvalidValue;
  if (router_few_fits(p.T)) {
    const dim3 g((unsigned)((p.n_experts + RF_EXPERTS - 1) / RF_EXPERTS), (unsigned)((p.T + RF_TOK - 1) / RF_TOK));
    if (groups) hipLaunchKernelGGL(k_router_few<true>, g, dim3(512), 0, s, p);
    else hipLaunchKernelGGL(k_router_few<false>, g, dim3(512), 0, s, p);
    return hipGetLastError();
  }
  // The denominator of a softmax takes all logits, and fp32 ones would be off by up to
  // 274 x 2^-23 |W_e| |x| each. It cancels where the K weights are normalised, unless a bias makes
  // the choice depend on it.
  // With groups a softmax's merits are sums of e^(z - max), over that denominator where there is a
  // bias (without one it drops out of their comparison); the ends below bound no such sums, so all
  // its logits are taken in fp64. And with groups the keys' ends and the undecided groups' exact
  // logits cost more, so that few logits are sooner all taken in fp64. us, bounds |
  // fp64, experts in 8 groups: 512 tokens x 4096 x 256 47 | 33, 1024 49 | 54, 1536 59 | 75, 2048 57 | 95;
  // 2048 x 4096 x 64 45 | 34; 512 x 4096 x 1024 79 | 105; 1024 x 8192 x 512 90 | 180.
  const bool many = (double)p.T * p.n_experts * p.hidden >= 0x1p30;
  if (groups ? many && p.scoring != SCORE_SOFTMAX : p.scoring != SCORE_SOFTMAX || (p.normalize && !p.bias)) {
    for (long t0 = 0; t0 < p.T; t0 += ROUTER_TOKENS) {
      RouterParams q = p;
      q.T = (int)(p.T - t0 < ROUTER_TOKENS ? p.T - t0 : ROUTER_TOKENS);
      q.x += (size_t)t0 * p.hidden;
      q.ids += (size_t)t0 * p.top_k;
      q.rw += (size_t)t0 * p.top_k;
      const int tiles = (q.n_experts + RM_E - 1) / RM_E * ((q.T + RM_T - 1) / RM_T);
      const int z = mm_split(q, tiles);
      const int z_bytes = (2 * q.hidden / z + 127) / 128 * 128;
      hipLaunchKernelGGL(k_router_mm, dim3((unsigned)(tiles * z + (q.n_experts + 3) / 4)), dim3(256), 0, s, q, z, z_bytes, tiles);
      const dim3 g((unsigned)((q.T + 3) / 4)), b(256);
      auto pick = [&](auto n) {
        if (groups) hipLaunchKernelGGL((k_router_pick<decltype(n)::value, true>), g, b, 0, s, q, z);
        else hipLaunchKernelGGL((k_router_pick<decltype(n)::value, false>), g, b, 0, s, q, z);
      };
      if (q.n_experts <= 256) pick(Count<4>{});
      else if (q.n_experts <= 512) pick(Count<8>{});
      else pick(Count<16>{});
    }
    return hipGetLastError();
  }
  for (long t0 = 0; t0 < p.T; t0 += 1 << 19) {  // grid rows
    RouterParams q = p;
    q.T = (int)(p.T - t0 < (1 << 19) ? p.T - t0 : 1 << 19);
    q.x += (size_t)t0 * p.hidden;
    q.logits += (size_t)t0 * p.n_experts;
    q.ids += (size_t)t0 * p.top_k;
    q.rw += (size_t)t0 * p.top_k;
    const dim3 g((unsigned)((p.n_experts + 15) / 16), (unsigned)((q.T + 15) / 16));
    hipLaunchKernelGGL(k_router_logits, g, dim3(64 * RL_WAVES), 0, s, q);
    const dim3 c((unsigned)((q.T + 3) / 4));
    if (groups) hipLaunchKernelGGL(k_router_choose<true>, c, dim3(256), 0, s, q);
    else hipLaunchKernelGGL(k_router_choose<false>, c, dim3(256), 0, s, q);
  }
  return hipGetLastError();
}

}  // namespace moeq
