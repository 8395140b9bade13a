// The grouped products of the 16-bit expert FFN on bfloat16 operands.
#include "skinny_gemm.h"

namespace nvfp4 {

hipError_t launch_tile_gemm_bf16(const TileParams& p, int layout, int epilogue, hipStream_t stream) {
  return tg_launch16<TG_BF16>(p, layout, epilogue, stream);
}

}  // namespace nvfp4
