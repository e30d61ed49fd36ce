// Updates made orthogonal (ortho.cu): what its files share.
#pragma once

#include <vector>

#include "internal.h"

namespace mlk {

struct OrthoEntry {
    const void* src;
    void* dst;
    int n;                                   // longer side
    int16_t r;                               // shorter side
    int8_t tall;                             // rows are the longer side
    int8_t vec;                              // 4 elements side by side can be read and written at once
};
struct OrthoCoeffs {
    float a, b, c, eps;
    int steps;
};

// Queues the matrices of e (none of them empty), which it sorts.
cudaError_t launch_ortho_fp32(std::vector<OrthoEntry>& e, const OrthoCoeffs& co, int num_sms, cudaStream_t s);
cudaError_t launch_ortho_bf16(std::vector<OrthoEntry>& e, const OrthoCoeffs& co, int num_sms, cudaStream_t s);

}  // namespace mlk
