// The router: logits, scores, the top-k experts of every token and their weights.
//
//   z_te = sum_h W_eh x_th            bf16 x bf16, fp64 sums
//   s_te = softmax_e(z) | sigmoid(z) | sqrt(log(1 + e^z))
//   ids  = the top_k largest s + bias (fp64), ties to the lowest id
//   w    = s[ids] (/ their sum) * scale
//
// Everything up to the weights is held in fp64. The choice of experts is discontinuous:
// fp32 logits carry an error of about 1e-6 that depends on the order of summation, so
// two correct fp32 routers disagree on a near tie and a token's output jumps. A product
// of two bf16 values is exact in fp64 and the vector unit issues fp64 FMAs at the fp32
// rate here, so the exactness costs the conversions only.
#include "moeq_device.h"
#include "moeq_kernels.h"

namespace moeq {

namespace {

constexpr int R_WAVES = 4;  // experts per work-group, one per wave
constexpr int R_TOK = 8;    // tokens per work-group

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Lane l takes the 16-byte chunks l, l + 64, ... of the expert's row.
__global__ __launch_bounds__(64 * R_WAVES) void k_router_logits(RouterParams P) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * R_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.y * R_TOK, tn = min(R_TOK, P.T - t0);
  if (e >= P.n_experts) return;
  const uint16_t* w = P.w + (size_t)e * P.hidden;
  const uint16_t* x = P.x + (size_t)t0 * P.hidden;
  double acc[R_TOK];
#pragma unroll
  for (int t = 0; t < R_TOK; t++) acc[t] = 0.0;
  for (int c = lane; c < P.hidden / 8; c += 64) {
    const u32x4 wv = ld16(w + 8 * c);
    double wd[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      wd[2 * i] = (double)u2f(wv[i] << 16);
      wd[2 * i + 1] = (double)u2f(wv[i] & 0xFFFF0000u);
    }
#pragma unroll
    for (int t = 0; t < R_TOK; t++) {
      if (t < tn) {
        const u32x4 xv = ld16(x + (size_t)t * P.hidden + 8 * c);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          acc[t] = __builtin_fma(wd[2 * i], (double)u2f(xv[i] << 16), acc[t]);
          acc[t] = __builtin_fma(wd[2 * i + 1], (double)u2f(xv[i] & 0xFFFF0000u), acc[t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < R_TOK; t++)
    if (t < tn) {
      const double z = wave_sum(acc[t]);
      if (lane == 0) P.logits[(size_t)(t0 + t) * P.n_experts + e] = z;
    }
}

// One wave per token; lane l holds experts l, l + 64, ...
template <int N>
__device__ void choose(const RouterParams& P, int t, int lane) {
  const double* z = P.logits + (size_t)t * P.n_experts;
  double s[N], key[N];
#pragma unroll
  for (int i = 0; i < N; i++) s[i] = lane + 64 * i < P.n_experts ? z[lane + 64 * i] : -__builtin_inf();
  if (P.scoring == SCORE_SOFTMAX) {
    double m = -__builtin_inf();
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
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < N; i++) s[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const double v = s[i];
      if (P.scoring == SCORE_SIGMOID) s[i] = 1.0 / (1.0 + exp(-v));
      else s[i] = sqrt((v > 0.0 ? v : v < 0.0 ? 0.0 : v) + log1p(exp(-__builtin_fabs(v))));
    }
  }
  // A key that is NaN counts below every number, an expert past the end below that.
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int e = lane + 64 * i;
    const double k = e < P.n_experts && P.bias ? s[i] + (double)P.bias[e] : s[i];
    key[i] = k == k ? k : -__builtin_inf();
  }
  uint32_t taken = 0;  // of this lane's experts
  double ws = 0.0, sum = 0.0;
  for (int k = 0; k < P.top_k; k++) {
    double best = 0.0;
    int id = 1 << 30;  // none
#pragma unroll
    for (int i = 0; i < N; i++)
      if (lane + 64 * i < P.n_experts && !((taken >> i) & 1) && (id == (1 << 30) || key[i] > best)) {
        best = key[i];
        id = lane + 64 * i;
      }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double ob = __shfl_xor(best, o, 64);
      const int oi = __shfl_xor(id, o, 64);
      if (oi != (1 << 30) && (id == (1 << 30) || ob > best || (ob == best && oi < id))) {
        best = ob;
        id = oi;
      }
    }
    double sc = 0.0;
#pragma unroll
    for (int i = 0; i < N; i++)
      if (lane + 64 * i == id) {
        taken |= 1u << i;
        sc = s[i];
      }
    sc = __shfl(sc, id & 63, 64);
    sum += sc;
    if (lane == k) {
      ws = sc;
      P.ids[(size_t)t * P.top_k + k] = id;
    }
  }
  if (lane < P.top_k) {
    double w = ws;
    if (P.normalize) w = sum == 0.0 ? 0.0 : w / sum;
    P.rw[(size_t)t * P.top_k + lane] = (float)(w * (double)P.scale);
  }
}

__global__ __launch_bounds__(256) void k_router_choose(RouterParams P) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= P.T) return;
  if (P.n_experts <= 256) choose<4>(P, t, lane);
  else choose<16>(P, t, lane);
}

}  // namespace

hipError_t launch_router(const RouterParams& p, hipStream_t s) {
  if (p.T < 1 || p.n_experts < 1 || p.n_experts > 1024 || p.top_k < 1 || p.top_k > 16 || p.top_k > p.n_experts ||
      p.hidden < 8 || p.hidden % 8)
    return hipErrorInvalidValue;
  for (int t0 = 0; t0 < p.T; t0 += 65535 * R_TOK) {  // grid rows
    RouterParams q = p;
    q.T = p.T - t0 < 65535 * R_TOK ? p.T - t0 : 65535 * R_TOK;
    q.x += (size_t)t0 * p.hidden;
    q.logits += (size_t)t0 * p.n_experts;
    q.ids += (size_t)t0 * p.top_k;
    q.rw += (size_t)t0 * p.top_k;
    const dim3 g((unsigned)((p.n_experts + R_WAVES - 1) / R_WAVES), (unsigned)((q.T + R_TOK - 1) / R_TOK));
    hipLaunchKernelGGL(k_router_logits, g, dim3(64 * R_WAVES), 0, s, q);
    hipLaunchKernelGGL(k_router_choose, dim3((unsigned)((q.T + 3) / 4)), dim3(256), 0, s, q);
  }
  return hipGetLastError();
}

}  // namespace moeq
