// The whole MoE layer for a few tokens, in three launches:
//
//   1. router | shared gate/up   the router's 2 MB of weights leave most of the chip idle
//                                while its choice is made; the shared expert needs no choice
//   2. routed gate/up | shared down   (moeq_gu_mx4.hip)
//   3. routed down, route-weighted sum, shared output added, bf16
//
// so that no launch waits for a memory stream that another could have filled. The bytes of
// each: 2 + 16.8 MB, 53.7 T + 8.4 MB, 26.7 T MB for MXFP4 experts of 4096 x 2048 and an INT8
// shared expert of the same size.
#include "moeq_int8.h"
#include "moeq_router.h"

namespace moeq {

namespace {

// The first work-groups are the router's, so that its chain (logits, count, choice) starts
// with the launch.
template <int TPW, int CPL>
__global__ __launch_bounds__(512) void k_moe_front(RouterParams R, Int8Params G) {
  const int nb = (R.n_experts + RF_EXPERTS - 1) / RF_EXPERTS, nr = nb * ((R.T + RF_TOK - 1) / RF_TOK);
  const int b = blockIdx.x;
  if (b < nr) router_few(R, b % nb, b / nb);
  else int8_few<2, TPW, CPL, 8, 0>(G, b - nr);
}

}  // namespace

bool moe_front_fits(int T, int hidden) { return few_bf16_fits(T, hidden) && router_few_fits(T); }

hipError_t launch_moe_front(const RouterParams& r, const Int8Params& g0, hipStream_t s) {
  if (!moe_front_fits(r.T, r.hidden) || g0.T != r.T || g0.cols != r.hidden) return hipErrorInvalidValue;
  Int8Params p = g0;
  const FewPlan f = few_plan(p.T, p.cols, 8);
  p.wpt = f.wpt;
  const int nb = (r.n_experts + RF_EXPERTS - 1) / RF_EXPERTS * ((r.T + RF_TOK - 1) / RF_TOK);
  const dim3 g((unsigned)(nb + (p.rows + 15) / 16)), b(512);
  if (f.tpw == 1 && f.cpl <= 1) hipLaunchKernelGGL((k_moe_front<1, 1>), g, b, 0, s, r, p);
  else if (f.tpw == 1 && f.cpl <= 4) hipLaunchKernelGGL((k_moe_front<1, 4>), g, b, 0, s, r, p);
  else if (f.tpw == 1) hipLaunchKernelGGL((k_moe_front<1, 16>), g, b, 0, s, r, p);
  else if (f.cpl <= 2) hipLaunchKernelGGL((k_moe_front<2, 2>), g, b, 0, s, r, p);
  else hipLaunchKernelGGL((k_moe_front<2, 8>), g, b, 0, s, r, p);
  return hipGetLastError();
}

bool down1_final_fits(int fmt, const Down1Params& p) {
  if ((uintptr_t)p.h % 16) return false;
  if (fmt == FMT_MXFP4) return down1_mx4_fits(p.rows, p.cols, p.top_k) && (uintptr_t)p.w.scales % 16 == 0 && p.w.sestride % 16 == 0;
  return fmt == FMT_Q2_K && down1_q2k_fits(p.rows, p.cols, p.top_k);
}

hipError_t launch_down1_final(int fmt, const Down1Params& p, hipStream_t s) {
  if (!down1_final_fits(fmt, p)) return hipErrorInvalidValue;
  return fmt == FMT_MXFP4 ? launch_down1_mx4_final(p, s) : launch_down1_q2k_final(p, s);
}

}  // namespace moeq
