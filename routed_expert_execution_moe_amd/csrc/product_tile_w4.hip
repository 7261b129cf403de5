// Tile products of bf16 rows, MXFP4 weights.
#include "product_tile.h"

namespace moert {

hipError_t launch_tile_w4(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s) {
  return launch_tile<MOE_BF16, MOE_MXFP4>(a, glu, v, s);
}

}  // namespace moert
