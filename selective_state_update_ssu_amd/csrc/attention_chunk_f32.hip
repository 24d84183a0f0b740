// attention_chunk_f32.hip -- the chunked kernels of linear attention for this io type.
#include "attention_chunk.hpp"

namespace attention {

hipError_t chunk_f32(Params p, hipStream_t stream) { return launch_chunks<float>(p, stream); }

}  // namespace attention
