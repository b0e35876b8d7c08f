// Device side of the router, shared by its own kernels and the whole layer's first launch.
// What it computes, and why in fp64: moeq_router.hip.
#pragma once
#include "moeq_device.h"
#include "moeq_kernels.h"
#include "moeq_wave.h"

namespace moeq {

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {  // v + the lane that CTRL names (0 outside the rows)
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane) |
                                        ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane) << 32));
}

// The sum over the wave (all lanes active), as wave_max gathers its maximum.
__device__ __forceinline__ double wave_sum(double v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  v = dpp_add<0x143, 0xC>(v);
  return read_lane(v, 63);
}

// Scores that need no other expert's logit.
__device__ __forceinline__ double score_of(int scoring, double z) {
  if (scoring == SCORE_SIGMOID) return 1.0 / (1.0 + exp(-z));
  return sqrt((z > 0.0 ? z : z < 0.0 ? 0.0 : z) + log1p(exp(-__builtin_fabs(z))));
}

// Doubles that other work-groups of the same launch wrote or will read: past the L2s of
// the XCDs, which are not kept coherent inside a launch.
__device__ __forceinline__ void put_agent(double* p, double v) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get_agent(const double* p) {
  return __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// A number as an unsigned integer of the same order; a NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint64_t order_of(double k) {
  k = k == k ? k + 0.0 : -__builtin_inf();
  const uint64_t b = __builtin_bit_cast(uint64_t, k);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// Lanes to a group of experts: the largest power of two that leaves every group its own.
__device__ __forceinline__ int group_lanes(int n_groups) { return 1 << (31 - __builtin_clz(64 / n_groups)); }

// The merit of a group, as an integer of its order, from the two largest biased scores of its
// parts, which lie in lanes gl q .. gl q + gl - 1 for group q (gl = group_lanes(); a NaN as -inf);
// in each of these lanes. Lanes past the last group take part with numbers that nobody counts.
__device__ __forceinline__ uint64_t group_merit(double a, double b, int gl, bool top2) {
  for (int o = 1; o < gl; o <<= 1) {
    const double c = __shfl_xor(a, o, 64), d = __shfl_xor(b, o, 64);
    const double low = a < c ? a : c;
    a = a > c ? a : c;
    b = b > d ? b : d;
    b = b > low ? b : low;
  }
  return order_of(top2 && b > -__builtin_inf() ? a + b : top2 ? -__builtin_inf() : a);
}
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane) |
         ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32);
}

// Which groups of experts a wave's token keeps: bit gl q of the result for group q.
__device__ __forceinline__ uint64_t keep_groups(double a, double b, int n_groups, int top_groups, bool top2, int lane) {
  const int gl = group_lanes(n_groups), q = lane / gl;
  const uint64_t mine = group_merit(a, b, gl, top2);
  int rank = 0;
  for (int o = 0; o < n_groups; o++) {
    const uint64_t v = read_lane(mine, o * gl);
    rank += v > mine || (v == mine && o < q);
  }
  return __ballot(q < n_groups && lane % gl == 0 && rank < top_groups);
}

// The choice of one token's experts by one wave; lane l holds experts l, l + 64, ... P.logits
// has logits for a softmax, scores for the other rules (SCORED: written by other work-groups of
// this launch). GROUPS: inside the best groups of experts only.
template <int N, bool SCORED, bool GROUPS = false>
__device__ __forceinline__ void choose(const RouterParams& P, int t, int lane) {
  const double* z = P.logits + (size_t)t * P.n_experts;
  double s[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    s[i] = -__builtin_inf();
    if (lane + 64 * i < P.n_experts) s[i] = SCORED ? get_agent(z + lane + 64 * i) : z[lane + 64 * i];
  }
  // Keys as integers in the order of the numbers: a NaN counts as -inf, -0 as 0, and an
  // expert that is taken or past the end is 0, below every number. A softmax without a bias
  // orders by the logits.
  uint32_t hi[N], lo[N];
  auto keys = [&](const double (&v)[N], bool biased) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = lane + 64 * i;
      double k = v[i];
      if (biased && e < P.n_experts) k += (double)P.bias[e];
      k = k == k ? k + 0.0 : -__builtin_inf();
      uint64_t b = __builtin_bit_cast(uint64_t, k);
      b ^= (uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull;
      if (e >= P.n_experts) b = 0;
      hi[i] = (uint32_t)(b >> 32);
      lo[i] = (uint32_t)b;
    }
  };
  double m = -__builtin_inf(), denom = 1.0;
  if (P.scoring == SCORE_SOFTMAX) {
    if (!P.bias) keys(s, false);
#pragma unroll
    for (int i = 0; i < N; i++) m = s[i] > m ? s[i] : m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double v = __shfl_xor(m, o, 64);
      m = v > m ? v : m;
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < N; i++) {
      s[i] = lane + 64 * i < P.n_experts ? exp(s[i] - m) : 0.0;
      sum += s[i];
    }
    denom = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < N; i++) s[i] /= denom;
    if (P.bias) keys(s, true);
  } else {
    keys(s, P.bias != nullptr);
  }
  if constexpr (GROUPS) {
    // The scores once more, group by group: a group's experts do not lie in one lane's registers.
    const int size = P.n_experts / P.n_groups, gl = group_lanes(P.n_groups), q = lane / gl;
    double a = -__builtin_inf(), b = -__builtin_inf();
    if (q < P.n_groups)
      for (int i = lane % gl; i < size; i += gl) {
        const int e = q * size + i;
        double v = SCORED ? get_agent(z + e) : z[e];
        if (P.scoring == SCORE_SOFTMAX) v = exp(v - m) / denom;
        if (P.bias) v += (double)P.bias[e];
        v = v == v ? v : -__builtin_inf();
        const double low = a < v ? a : v;
        a = a > v ? a : v;
        b = b > low ? b : low;
      }
    const uint64_t kept = keep_groups(a, b, P.n_groups, P.top_groups, P.group_top2 && size > 1, lane);
#pragma unroll
    for (int i = 0; i < N; i++)
      if (!(kept >> ((lane + 64 * i) / size * gl & 63) & 1)) hi[i] = lo[i] = 0;
  }
  double mine = 0.0, sum = 0.0;
  for (int k = 0; k < P.top_k; k++) {
    uint32_t bh = hi[0], bl = lo[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < N; i++)
      if (hi[i] > bh || (hi[i] == bh && lo[i] > bl)) {
        bh = hi[i];
        bl = lo[i];
        at = i;
      }
    // the lanes whose best is the largest; of several equal ones the lowest expert
    bool in = bh == wave_max(bh);
    uint64_t who = __ballot(in);
    if (__popcll(who) > 1) {
      const uint32_t ml = wave_max(in ? bl : 0u);  // by every lane: the exchange reads them all
      in = in && bl == ml;
      who = __ballot(in);
      if (__popcll(who) > 1) {
        const uint32_t id = ~(uint32_t)(lane + 64 * at);
        const uint32_t mi = wave_max(in ? id : 0u);
        in = in && id == mi;
        who = __ballot(in);
      }
    }
    const int src = __ffsll((long long)who) - 1;
    const int i0 = __builtin_amdgcn_readlane(at, src);
    double sc = 0.0;
#pragma unroll
    for (int i = 0; i < N; i++)
      if (i == i0) {  // uniform
        sc = s[i];
        if (lane == src) hi[i] = lo[i] = 0;
      }
    sc = read_lane(sc, src);
    sum += sc;
    if (lane == k) {
      mine = sc;
      P.ids[(size_t)t * P.top_k + k] = src + 64 * i0;
    }
  }
  if (lane < P.top_k) {
    if (P.normalize) mine = sum == 0.0 ? 0.0 : mine / sum;
    P.rw[(size_t)t * P.top_k + lane] = (float)(mine * (double)P.scale);
  }
}

// A few tokens in one launch. A work-group of eight waves takes RF_EXPERTS experts (two
// waves to a row, its 16-byte chunks in turn) for up to RF_TOK tokens, turns its logits
// into scores and counts itself in; the last to arrive for the tokens makes their choice.
constexpr int RF_EXPERTS = 4, RF_TOK = 8, RF_DEPTH = 4;

template <bool GROUPS>
__device__ __forceinline__ void router_few(const RouterParams& P, int block, int group) {
  __shared__ double part[8][RF_TOK];
  __shared__ int is_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = group * RF_TOK, tn = min(RF_TOK, P.T - t0);
  const int e = min(block * RF_EXPERTS + wave / 2, P.n_experts - 1);
  const uint16_t* w = P.w + (size_t)e * P.hidden;
  const uint16_t* x = P.x + (size_t)t0 * P.hidden;
  const int chunks = P.hidden / 8;
  double acc[RF_TOK];
#pragma unroll
  for (int t = 0; t < RF_TOK; t++) acc[t] = 0.0;
  for (int c0 = lane + 64 * (wave & 1); c0 < chunks; c0 += 128 * RF_DEPTH) {
    u32x4 wv[RF_DEPTH];
#pragma unroll
    for (int i = 0; i < RF_DEPTH; i++) {
      wv[i] = ld16(w + 8 * (size_t)min(c0 + 128 * i, chunks - 1));
      if (c0 + 128 * i >= chunks) wv[i] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int t = 0; t < RF_TOK; t++) {
      if (t < tn) {
        u32x4 xv[RF_DEPTH];
#pragma unroll
        for (int i = 0; i < RF_DEPTH; i++) {
          xv[i] = ld16(x + (size_t)t * P.hidden + 8 * (size_t)min(c0 + 128 * i, chunks - 1));
          if (c0 + 128 * i >= chunks) xv[i] = u32x4{0u, 0u, 0u, 0u};  // 0 times an infinity of the last chunk
        }
#pragma unroll
        for (int i = 0; i < RF_DEPTH; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            acc[t] = __builtin_fma((double)u2f(wv[i][j] << 16), (double)u2f(xv[i][j] << 16), acc[t]);
            acc[t] = __builtin_fma((double)u2f(wv[i][j] & 0xFFFF0000u), (double)u2f(xv[i][j] & 0xFFFF0000u), acc[t]);
          }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < RF_TOK; t++)
    if (t < tn) {
      const double v = wave_sum(acc[t]);
      if (lane == 0) part[wave][t] = v;
    }
  __syncthreads();
  const int j = threadIdx.x / RF_TOK, t = threadIdx.x % RF_TOK;
  if (j < RF_EXPERTS && t < tn && block * RF_EXPERTS + j < P.n_experts) {
    const double z = part[2 * j][t] + part[2 * j + 1][t];
    put_agent(P.logits + (size_t)(t0 + t) * P.n_experts + block * RF_EXPERTS + j,
              P.scoring == SCORE_SOFTMAX ? z : score_of(P.scoring, z));
  }
  static_assert(RF_EXPERTS * RF_TOK <= 64, "the scores are the first wave's");
  if (wave == 0) {
    // The stores above are acknowledged from where every XCD reads them before the count.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (lane == 0) {
      const int blocks = (P.n_experts + RF_EXPERTS - 1) / RF_EXPERTS;
      const uint32_t before = __hip_atomic_fetch_add(P.count + group, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      is_last = before == (uint32_t)blocks - 1;
      if (is_last) __hip_atomic_store(P.count + group, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next launch
    }
  }
  __syncthreads();
  if (is_last && wave < tn) {
    if (P.n_experts <= 256) choose<4, true, GROUPS>(P, t0 + wave, lane);
    else if (P.n_experts <= 512) choose<8, true, GROUPS>(P, t0 + wave, lane);
    else choose<16, true, GROUPS>(P, t0 + wave, lane);
  }
}

}  // namespace moeq
