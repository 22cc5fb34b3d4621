// product.hip -- the experts' product in 16 bits and the weights' gradient.
#include "product_call.h"

namespace hr {
namespace {

template <class E>
hr_status product_impl(const hr_experts_product_args *q, hr_stream_t stream) {
    if (q == nullptr || q->x_scales != nullptr || q->w_scales != nullptr) return HR_ERR_INVALID_ARG;
    ProductArgs a{};
    bool any = false;
    const hr_status st = product_check<2>(q, a, any);
    if (st != HR_OK || a.rows == 0) return st;
    return launch_product<E, E>(a, q->transposed != 0, any, stream);
}

template <class E>
hr_status product_grad_impl(const hr_experts_product_grad_args *q, hr_stream_t stream) {
    ProductArgs a{};
    bool any = false;
    const hr_status st = product_grad_check(q, a, any);
    if (st != HR_OK) return st;
    return q->dw_f32 ? launch_product_grad<E, float>(a, any, stream) : launch_product_grad<E, E>(a, any, stream);
}

}  // namespace
}  // namespace hr

extern "C" {

hr_status hr_experts_product_f16(const hr_experts_product_args *args, hr_stream_t stream) {
    return hr::product_impl<hr::F16>(args, stream);
}
hr_status hr_experts_product_bf16(const hr_experts_product_args *args, hr_stream_t stream) {
    return hr::product_impl<hr::BF16>(args, stream);
}
hr_status hr_experts_product_grad_f16(const hr_experts_product_grad_args *args, hr_stream_t stream) {
    return hr::product_grad_impl<hr::F16>(args, stream);
}
hr_status hr_experts_product_grad_bf16(const hr_experts_product_grad_args *args, hr_stream_t stream) {
    return hr::product_grad_impl<hr::BF16>(args, stream);
}

}  // extern "C"
