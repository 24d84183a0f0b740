// Selective scan kernels for f32 io.
#include "layer_scan.hpp"

namespace layer {

hipError_t scan_varlen_f32(const ScanParams& p, int dstate, hipStream_t stream) {
    return launch_scan_varlen<float>(p, dstate, stream);
}

hipError_t scan_update_f32(const ScanParams& p, int dstate, hipStream_t stream) {
    return launch_scan_update<float>(p, dstate, stream);
}

}  // namespace layer
