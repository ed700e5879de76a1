// The products of the dense layers for bf16 operands, backward.
#include "dense.hpp"

namespace gnnmb {

hipError_t launch_gradients_bf16(ProductArgs w, ProductArgs x, const ColumnArgs &c, int tile, int load, hipStream_t s) {
    return launch_gradients<bf16>(w, x, c, tile, load, s);
}

}  // namespace gnnmb
