// The tiled INT4 linear with the scales in the weights (moeq_int4_tiled.h), for bf16 outputs.
#include "moeq_int4_tiled.h"

#ifndef I4_SC
#define I4_SC 8, 1, 2, 8
#endif
namespace moeq {

hipError_t launch_int4_scaled(const Int4Rows& p, long blocks, hipStream_t s) {
  switch (int4_group(p.fmt)) {
    case 32: return tiled<I4_LINEAR, 4, true, I4_SC>(p, blocks, s);
    case 64: return tiled<I4_LINEAR, 2, true, I4_SC>(p, blocks, s);
    default: return tiled<I4_LINEAR, 1, true, I4_SC>(p, blocks, s);
  }
}

}  // namespace moeq
