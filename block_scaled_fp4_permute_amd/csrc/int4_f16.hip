// Products with INT4 weights on float16 activations.
#include "int4_gemv.h"

namespace nvfp4 {

hipError_t launch_int4_gemv_f16(const Int4Params& p, int group, int gated, int out32, hipStream_t stream) {
  return i4_launch_type<true>(p, group, gated, out32, stream);
}

}  // namespace nvfp4
