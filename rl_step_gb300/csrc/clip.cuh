// Gradient norms over many tensors and clipping (clip.cu): the launches that
// mlora_clip_grads and the handles' clipped optimizer steps share.
#pragma once

#include "internal.h"

namespace mlk {

// Elements of one work chunk: one block's share of a tensor.
constexpr int CLIP_CHUNK = 8192;

// A sum of squares v 2^e (e = 0 but where v would leave fp32's safe range).
struct ClipSum {
    float v;
    int e;
};

// One tensor (or one adapter's contiguous gradient) of a launch, tensors in
// group order.  Chunks to scale and sums of squares (per_sum chunks each) are
// numbered over all tensors of the call: a group's sums are the range [g0, g1).
struct ClipEntry {
    const void* src;
    void* dst;
    int64_t size;
    int group;
    int chunk0, sum0;      // numbers of the tensor's first chunk and first sum
    int per_sum;
    int g0, g1;
    int first;             // the group's first tensor
};
constexpr int CLIP_SUMS = 512;             // sums that a large group is cut into, about

inline int64_t clip_chunks(int64_t size) { return (size + CLIP_CHUNK - 1) / CLIP_CHUNK; }
inline int clip_sums(const ClipEntry& e) { return (int)((clip_chunks(e.size) + e.per_sum - 1) / e.per_sum); }
// Numbers the chunks and sums of entries in group order (src, dst, size > 0 and
// group are set); returns the groups.
int clip_number(ClipEntry* e, int n);

// part[sum] for fp32 tensors.  mask (may be null): only the groups g with
// mask[g] != 0 are read, the others' sums are 0.
cudaError_t launch_clip_norm(const ClipEntry* entries, int n, ClipSum* part, const int* mask, cudaStream_t s,
                             int64_t* launches);

// The handles' clipped optimizer steps: adapter a's gradient is the fp32 range
// [off[a], off[a+1]) of G (off: host).  factor[a], norms[a] (may be null): the
// factor that clips it and its norm, for the adapters with mask[a] != 0; 1 and 0
// for the others.  part: clip_adapter_sums(off, n_ad) sums.
int64_t clip_adapter_sums(const int64_t* off, int n_ad);
cudaError_t launch_clip_adapters(const float* G, const int64_t* off, int n_ad, const int* mask, ClipSum* part,
                                 float max_norm, float* factor, float* norms, cudaStream_t s, int64_t* launches);

}  // namespace mlk
