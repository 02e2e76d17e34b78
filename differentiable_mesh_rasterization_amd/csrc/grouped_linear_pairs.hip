// The backward pass of the linear layers from an upstream gradient that is a
// pair of bfloat16 arrays, as the gated layers' is (a file of its own so that
// it compiles beside the others).
#include "grouped_linear.h"

namespace dmr {

hipError_t launch_grouped_linear_backward_pairs(const GroupedLinearArgs& a) {
    switch (a.dtype) {
        case DMR_FLOAT16:
            return a.weight_low ? launch_backward<__bf16, __bf16, _Float16, 3>(a) : launch_backward<__bf16, _Float16, _Float16, 3>(a);
        case DMR_BFLOAT16: return launch_backward<__bf16, __bf16, __bf16, 2>(a);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace dmr
