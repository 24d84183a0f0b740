// Selective scan kernels for bf16 io.
#include "layer_scan.hpp"

namespace layer {

hipError_t scan_varlen_bf16(const ScanParams& p, int dstate, hipStream_t stream) {
    return launch_scan_varlen<__bf16>(p, dstate, stream);
}

hipError_t scan_update_bf16(const ScanParams& p, int dstate, hipStream_t stream) {
    return launch_scan_update<__bf16>(p, dstate, stream);
}

}  // namespace layer
