// The products of the dense layers for bf16 operands, forward.
#include "dense.hpp"

namespace gnnmb {

hipError_t launch_product_bf16(ProductArgs a, int tile, bool pair, int load, hipStream_t s) {
    return launch_product<bf16>(a, tile, pair, load, s);
}

}  // namespace gnnmb
