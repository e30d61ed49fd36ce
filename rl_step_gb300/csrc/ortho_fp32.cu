// Orthogonal updates of fp32 matrices.
#include "ortho_kernel.cuh"

namespace mlk {

cudaError_t launch_ortho_fp32(std::vector<OrthoEntry>& e, const OrthoCoeffs& co, int num_sms, cudaStream_t s) {
    return launch_ortho_t<float>(e, co, num_sms, s);
}

}  // namespace mlk
