// Kernel launchers of the RMS norm, the 8-bit and the grouped operators that do
// nothing, for the host-side sanitizer build (no device is used).
#include "layers.hpp"

namespace muon {
int rms_backward_blocks(int64_t rows, int64_t, int) { return rows ? 8 : 0; }
hipError_t launch_rms_forward(const RmsForward&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_rms_backward(const RmsBackward&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_rms_sums(const RmsSums&, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize(const Quantize&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize_weight(const QuantizeWeight&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_scaled(const ScaledArgs&, TileKind, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_grouped(const GroupedArgs&, TileKind, bool, bool, int, unsigned, hipStream_t) { return hipSuccess; }
hipError_t launch_grouped_weight(const GroupedArgs&, TileKind, bool, int, int, unsigned, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_grouped_join(const GroupedArgs&, int, hipStream_t) { return hipSuccess; }
}  // namespace muon
