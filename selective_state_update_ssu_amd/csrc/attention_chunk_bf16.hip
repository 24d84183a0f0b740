// attention_chunk_bf16.hip -- the chunked kernels of linear attention for this io type.
#include "attention_chunk.hpp"

namespace attention {

hipError_t chunk_bf16(Params p, hipStream_t stream) { return launch_chunks<__bf16>(p, stream); }

}  // namespace attention
