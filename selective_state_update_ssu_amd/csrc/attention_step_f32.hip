// attention_step_f32.hip -- the row-by-row kernels of linear attention for this io type.
#include "attention_step.hpp"

namespace attention {

hipError_t step_f32(const Params& p, bool packed, hipStream_t stream) {
    return packed ? launch_step<float, true>(p, stream) : launch_step<float, false>(p, stream);
}

}  // namespace attention
