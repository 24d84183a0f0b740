// attention_step_bf16.hip -- the row-by-row kernels of linear attention for this io type.
#include "attention_step.hpp"

namespace attention {

hipError_t step_bf16(const Params& p, bool packed, hipStream_t stream) {
    return packed ? launch_step<__bf16, true>(p, stream) : launch_step<__bf16, false>(p, stream);
}

}  // namespace attention
