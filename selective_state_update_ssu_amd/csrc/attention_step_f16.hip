// attention_step_f16.hip -- the row-by-row kernels of linear attention for this io type.
#include "attention_step.hpp"

namespace attention {

hipError_t step_f16(const Params& p, bool packed, hipStream_t stream) {
    return packed ? launch_step<_Float16, true>(p, stream) : launch_step<_Float16, false>(p, stream);
}

}  // namespace attention
