// Tile products of MXFP4 rows and weights.
#include "product_tile.h"

namespace moert {

hipError_t launch_tile_mx(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s) {
  return launch_tile<MOE_MXFP4, MOE_MXFP4>(a, glu, v, s);
}

}  // namespace moert
