// Selective scan kernels for f16 io.
#include "layer_scan.hpp"

namespace layer {

hipError_t scan_varlen_f16(const ScanParams& p, int dstate, hipStream_t stream) {
    return launch_scan_varlen<_Float16>(p, dstate, stream);
}

hipError_t scan_update_f16(const ScanParams& p, int dstate, hipStream_t stream) {
    return launch_scan_update<_Float16>(p, dstate, stream);
}

}  // namespace layer
