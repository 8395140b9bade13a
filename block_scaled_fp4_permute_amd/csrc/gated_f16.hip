// The grouped products of the 16-bit expert FFN on float16 operands.
#include "skinny_gemm.h"

namespace nvfp4 {

hipError_t launch_tile_gemm_f16(const TileParams& p, int layout, int epilogue, hipStream_t stream) {
  return tg_launch16<TG_F16>(p, layout, epilogue, stream);
}

}  // namespace nvfp4
