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
#include "moeq_router.h"

namespace moeq {

namespace {

__global__ __launch_bounds__(512) void k_router_few(RouterParams P) { router_few(P, blockIdx.x, blockIdx.y); }

constexpr int R_WAVES = 4;  // experts per work-group, one per wave
constexpr int R_TOK = 8;    // tokens per work-group

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

__global__ __launch_bounds__(256) void k_router_choose(RouterParams P) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= P.T) return;
  if (P.n_experts <= 256) choose<4, false>(P, t, lane);
  else choose<16, false>(P, t, lane);
}

}  // namespace

bool router_few_fits(int T) { return T <= ROUTER_FEW_T; }

hipError_t launch_router(const RouterParams& p, hipStream_t s) {
  if (p.T < 1 || p.n_experts < 1 || p.n_experts > 1024 || p.top_k < 1 || p.top_k > 16 || p.top_k > p.n_experts ||
      p.hidden < 8 || p.hidden % 8)
    return hipErrorInvalidValue;
  if (router_few_fits(p.T)) {
    const dim3 g((unsigned)((p.n_experts + RF_EXPERTS - 1) / RF_EXPERTS), (unsigned)((p.T + RF_TOK - 1) / RF_TOK));
    hipLaunchKernelGGL(k_router_few, g, dim3(512), 0, s, p);
    return hipGetLastError();
  }
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
