// The products of the dense layers for bf16 operands.
#include "dense.hpp"

namespace gnnmb {

hipError_t launch_product_bf16(ProductArgs a, const ProductPlan &p, hipStream_t s) {
    if (p.form == kGradX) return launch_form<bf16, kGradX, false>(a, p, s);
    if (p.form == kGradW) return launch_form<bf16, kGradW, false>(a, p, s);
    return p.pair ? launch_form<bf16, kForward, true>(a, p, s) : launch_form<bf16, kForward, false>(a, p, s);
}

}  // namespace gnnmb
