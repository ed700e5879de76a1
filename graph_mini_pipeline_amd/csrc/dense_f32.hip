// The products of the dense layers for fp32 operands, forward.
#include "dense.hpp"

namespace gnnmb {

hipError_t launch_product_f32(ProductArgs a, int tile, bool pair, int load, hipStream_t s) {
    return launch_product<float>(a, tile, pair, load, s);
}

}  // namespace gnnmb
