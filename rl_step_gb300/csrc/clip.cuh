// Gradient norms over many tensors and clipping (clip.cu): the launches that
// mlora_clip_grads and the handles' clipped optimizer steps share.
#pragma once

#include "internal.h"

namespace mlk {

// Elements of one work chunk: one block's share of a tensor.
constexpr int CLIP_CHUNK = 16384;

// One tensor (or one adapter's contiguous gradient) of a launch.  Chunks are
// numbered over all tensors of the call, tensors in group order, so that a
// group's chunks are the range [g0, g1).
struct ClipEntry {
    const void* src;
    void* dst;
    int64_t size;
    int chunk0;            // number of the tensor's first chunk
    int g0, g1;
    int group;
};

inline int64_t clip_chunks(int64_t size) { return (size + CLIP_CHUNK - 1) / CLIP_CHUNK; }

// part[chunk] = sum of squares of the chunk (fp64 value).  `mask` (may be null):
// only the groups g with mask[g] != 0 are read, the others' chunks get 0.
template <typename T>
cudaError_t launch_clip_norm(const ClipEntry* entries, int n, double* part, const int* mask, cudaStream_t s,
                             int64_t* launches);

}  // namespace mlk
