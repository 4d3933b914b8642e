// ssd_selective_f32.cu -- the selective scan's kernels for f32 elements.
#include "selective_scan.cuh"

namespace ssd {

cudaError_t launch_selective_f32(const SelParams &p, cudaStream_t stream) { return launch_selective_t<float>(p, stream); }

}  // namespace ssd
