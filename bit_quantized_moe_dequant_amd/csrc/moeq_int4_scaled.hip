// The tiled INT4 linear with the scales in the weights (moeq_int4_tiled.h), for bf16 outputs.
#include "moeq_int4_tiled.h"

namespace moeq {

hipError_t launch_int4_scaled(const Int4Rows& p, hipStream_t s) {
  switch (int4_group(p.fmt)) {
    case 32: return linear<4, true, 8, 1, 2, 8>(p, s);
    case 64: return linear<2, true, 8, 1, 2, 8>(p, s);
    default: return linear<1, true, 8, 1, 2, 8>(p, s);
  }
}

}  // namespace moeq
