// Kernel launchers of the layer operators that do nothing, for the host-side
// sanitizer build (no device is used).
#include "layers.hpp"

namespace muon {
hipError_t launch_gemm(const GemmArgs&, int, bool, bool, bool, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_gemm_join(const GemmArgs&, int, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_skinny(const SkinnyArgs&, bool, int, hipStream_t) { return hipSuccess; }
hipError_t launch_pack(const PackArgs*, int, hipStream_t) { return hipSuccess; }
int norm_backward_blocks(int64_t, int64_t, int) { return 8; }
hipError_t launch_norm_forward(const NormForward&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_backward(const NormBackward&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_sums(const NormSums&, hipStream_t) { return hipSuccess; }
}  // namespace muon
