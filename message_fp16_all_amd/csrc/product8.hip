// product8.hip -- the experts' product of e4m3 values with scales.
#include "product_call.h"

namespace hr {
namespace {

template <class O>
hr_status product8_impl(const hr_experts_product_args *q, hr_stream_t stream) {
    ProductArgs a{};
    bool any = false;
    const hr_status st = product_check<1>(q, a, any);
    if (st != HR_OK || a.rows == 0) return st;
    return launch_product<E4M3, O>(a, q->transposed != 0, any, stream);
}

}  // namespace
}  // namespace hr

extern "C" {

hr_status hr_experts_product_e4m3_f16(const hr_experts_product_args *args, hr_stream_t stream) {
    return hr::product8_impl<hr::F16>(args, stream);
}
hr_status hr_experts_product_e4m3_bf16(const hr_experts_product_args *args, hr_stream_t stream) {
    return hr::product8_impl<hr::BF16>(args, stream);
}

}  // extern "C"
