// The products of the dense layers for fp32 operands, backward.
#include "dense.hpp"

namespace gnnmb {

hipError_t launch_gradients_f32(ProductArgs w, ProductArgs x, const ColumnArgs &c, int tile, int load, hipStream_t s) {
    return launch_gradients<float>(w, x, c, tile, load, s);
}

}  // namespace gnnmb
