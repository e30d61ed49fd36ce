// Orthogonal updates of bf16 matrices.
#include "ortho_kernel.cuh"

namespace mlk {

cudaError_t launch_ortho_bf16(std::vector<OrthoEntry>& e, const OrthoCoeffs& co, int num_sms, cudaStream_t s) {
    return launch_ortho_t<bf16>(e, co, num_sms, s);
}

}  // namespace mlk
