// The products of the dense layers for fp32 operands.
#include "dense.hpp"

namespace gnnmb {

hipError_t launch_product_f32(ProductArgs a, const ProductPlan &p, hipStream_t s) {
    if (p.form == kGradX) return launch_form<float, kGradX, false>(a, p, s);
    if (p.form == kGradW) return launch_form<float, kGradW, false>(a, p, s);
    return p.pair ? launch_form<float, kForward, true>(a, p, s) : launch_form<float, kForward, false>(a, p, s);
}

}  // namespace gnnmb
