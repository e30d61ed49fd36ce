// The norm of the gradients of each group of tensors, and clipping:
//     n_g = sqrt(sum over the group's tensors of x^2)
//     x <- x * (max_norm / n_g)   where n_g > max_norm.
// Pass 1 sums squares per chunk of 16,384 elements: a thread adds at most 64
// squares in fp32, the block adds its threads' sums in fp64 in a fixed order.
// Pass 2's blocks add their group's chunk sums, again in a fixed order, and
// scale their chunk.  No atomics: results repeat bit for bit.
#include "clip.cuh"
#include "kv_common.cuh"

namespace mlk {

namespace {

constexpr int CT = 256;                      // threads of a block

// Tensors of one launch, passed by value: no table in device memory, so
// nothing of the caller's is kept and a captured launch holds its own copy.
template <int N>
struct ClipTab {
    int n;                                   // entries
    int base;                                // number of the launch's first chunk
    ClipEntry e[N];
};

template <int N>
__device__ __forceinline__ const ClipEntry& clip_find(const ClipTab<N>& t, int chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].chunk0 <= chunk) lo = mid; else hi = mid - 1;
    }
    return t.e[lo];
}

// sum over the block in a fixed order; every thread returns it
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[CT / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < CT / 32; ++w) v += part[w];
    return v;
}
__device__ __forceinline__ float block_max(float v) {
    __shared__ float part[CT / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < CT / 32; ++w) v = fmaxf(v, part[w]);
    return v;
}

// f(value) for each of this thread's elements of p[0 .. n)
template <typename T, typename F>
__device__ __forceinline__ void each(const T* p, int n, F f) {
    int i = 0;
    if ((reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0) {
        for (i = threadIdx.x * 4; i + 3 < n; i += CT * 4) {
            float x[4];
            load4_f(p + i, x);
            f(x[0]); f(x[1]); f(x[2]); f(x[3]);
        }
        i = n / 4 * 4 + threadIdx.x;
    } else {
        i = threadIdx.x;
    }
    for (; i < n; i += CT) f(to_f(p[i]));
}

template <typename T, int N>
__global__ void __launch_bounds__(CT) clip_norm_kernel(const __grid_constant__ ClipTab<N> t, double* part,
                                                       const int* __restrict__ mask) {
    const int chunk = t.base + blockIdx.x;
    const ClipEntry& e = clip_find(t, chunk);
    if (mask && !mask[e.group]) {
        if (threadIdx.x == 0) part[chunk] = 0.0;
        return;
    }
    const int64_t at = (int64_t)(chunk - e.chunk0) * CLIP_CHUNK;
    const T* p = static_cast<const T*>(e.src) + at;
    const int n = e.size - at < CLIP_CHUNK ? (int)(e.size - at) : CLIP_CHUNK;
    float s = 0.f;
    each(p, n, [&](float x) { s = fmaf(x, x, s); });
    double sum = block_sum((double)s);
    // squares beyond fp32's range, or below its smallest normal values: again,
    // relative to the largest magnitude (2^E, so that the scaling is exact)
    if (!(sum < 1e37 && sum > 1e-25)) {
        float m = 0.f;
        bool bad = false;
        each(p, n, [&](float x) {
            const float y = fabsf(x);
            m = fmaxf(m, y);
            bad |= !(y <= FLT_MAX);
        });
        m = block_max(m);
        if (__syncthreads_or(bad)) {
            // an infinity or NaN: their sum says which
            double v = 0.0;
            each(p, n, [&](float x) { v += fabsf(x) <= FLT_MAX ? 0.0 : (double)fabsf(x); });
            sum = block_sum(v);
        } else if (m > 0.f) {
            int E;
            frexpf(m, &E);
            float q = 0.f;
            // in two steps: 2^-E itself can lie outside fp32
            const float f1 = ldexpf(1.f, -E / 2), f2 = ldexpf(1.f, -E - (-E / 2));
            each(p, n, [&](float x) { const float y = x * f1 * f2; q = fmaf(y, y, q); });
            sum = ldexp(block_sum((double)q), 2 * E);
        } else {
            sum = 0.0;
        }
    }
    if (threadIdx.x == 0) part[chunk] = sum;
}

// the group's norm from its chunk sums; every thread returns it
__device__ __forceinline__ double group_norm(const double* part, int g0, int g1) {
    double v = 0.0;
    for (int i = g0 + threadIdx.x; i < g1; i += CT) v += part[i];
    return sqrt(block_sum(v));
}

// the factor of a norm; 1 for a norm that is not finite: such a gradient is
// the caller's to skip, and scaling it would hide it
__device__ __forceinline__ float clip_factor(double norm, float max_norm) {
    return norm > (double)max_norm && norm <= DBL_MAX ? (float)((double)max_norm / norm) : 1.f;
}

template <typename T, int N>
__global__ void __launch_bounds__(CT) clip_scale_kernel(const __grid_constant__ ClipTab<N> t, const double* part,
                                                        float max_norm, float* norms) {
    const int chunk = t.base + blockIdx.x;
    const ClipEntry& e = clip_find(t, chunk);
    const double norm = group_norm(part, e.g0, e.g1);
    if (norms && chunk == e.g0 && threadIdx.x == 0) norms[e.group] = (float)norm;
    const float f = clip_factor(norm, max_norm);
    const int64_t at = (int64_t)(chunk - e.chunk0) * CLIP_CHUNK;
    const T* p = static_cast<const T*>(e.src) + at;
    T* o = static_cast<T*>(e.dst) + at;
    if (f == 1.f && p == o) return;
    const int n = e.size - at < CLIP_CHUNK ? (int)(e.size - at) : CLIP_CHUNK;
    int i = threadIdx.x;
    if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & (4 * sizeof(T) - 1)) == 0) {
        for (i = threadIdx.x * 4; i + 3 < n; i += CT * 4) {
            float x[4];
            load4_f(p + i, x);
            const float y[4] = {x[0] * f, x[1] * f, x[2] * f, x[3] * f};
            store4_f(o + i, y);
        }
        i = n / 4 * 4 + threadIdx.x;
    }
    for (; i < n; i += CT) o[i] = from_f<T>(to_f(p[i]) * f);
}

// calls f(tab, chunks) for the entries in tables of at most N
template <int N, typename F>
cudaError_t by_tables(const ClipEntry* entries, int n, F f) {
    ClipTab<N> t;
    for (int i = 0; i < n; i += N) {
        t.n = n - i < N ? n - i : N;
        for (int j = 0; j < t.n; ++j) t.e[j] = entries[i + j];
        t.base = t.e[0].chunk0;
        const ClipEntry& l = t.e[t.n - 1];
        const int chunks = l.chunk0 + (int)clip_chunks(l.size) - t.base;
        if (chunks > 0) f(t, chunks);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

constexpr int TAB_SMALL = 64, TAB_LARGE = 512;   // 3 KB and 25 KB of kernel parameters (at most 32 KB)

template <typename T>
cudaError_t launch_clip_norm(const ClipEntry* entries, int n, double* part, const int* mask, cudaStream_t s,
                             int64_t* launches) {
    if (n <= TAB_SMALL)
        return by_tables<TAB_SMALL>(entries, n, [&](const ClipTab<TAB_SMALL>& t, int chunks) {
            clip_norm_kernel<T, TAB_SMALL><<<chunks, CT, 0, s>>>(t, part, mask);
            if (launches) ++*launches;
        });
    return by_tables<TAB_LARGE>(entries, n, [&](const ClipTab<TAB_LARGE>& t, int chunks) {
        clip_norm_kernel<T, TAB_LARGE><<<chunks, CT, 0, s>>>(t, part, mask);
        if (launches) ++*launches;
    });
}
template cudaError_t launch_clip_norm<float>(const ClipEntry*, int, double*, const int*, cudaStream_t, int64_t*);

template <typename T>
static cudaError_t launch_clip_scale(const ClipEntry* entries, int n, const double* part, float max_norm, float* norms,
                                     cudaStream_t s) {
    if (n <= TAB_SMALL)
        return by_tables<TAB_SMALL>(entries, n, [&](const ClipTab<TAB_SMALL>& t, int chunks) {
            clip_scale_kernel<T, TAB_SMALL><<<chunks, CT, 0, s>>>(t, part, max_norm, norms);
        });
    return by_tables<TAB_LARGE>(entries, n, [&](const ClipTab<TAB_LARGE>& t, int chunks) {
        clip_scale_kernel<T, TAB_LARGE><<<chunks, CT, 0, s>>>(t, part, max_norm, norms);
    });
}

}  // namespace mlk

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------
#include <algorithm>
#include <new>
#include <vector>

using namespace mlk;

namespace {

// Checks the set; its chunks in *chunks.
int clip_check(const mlora_grad_set* g, int64_t* chunks) {
    if (!g) return kv_fail(MLORA_E_ARG, "NULL gradient set");
    if (g->n_tensors < 0 || g->n_groups < 1)
        return kv_fail(MLORA_E_ARG, "bad gradient set (%d tensors, %d groups)", g->n_tensors, g->n_groups);
    if (g->dtype != MLORA_BF16 && g->dtype != MLORA_FP32) return kv_fail(MLORA_E_ARG, "unknown dtype %d", g->dtype);
    if (g->n_tensors > 0 && (!g->grads || !g->sizes)) return kv_fail(MLORA_E_ARG, "NULL tensor or size array");
    const uintptr_t es = g->dtype == MLORA_BF16 ? 2 : 4;
    int64_t total = 0;
    for (int i = 0; i < g->n_tensors; ++i) {
        if (g->sizes[i] < 0 || g->sizes[i] > (INT64_C(1) << 44))
            return kv_fail(MLORA_E_ARG, "tensor %d: size %lld", i, (long long)g->sizes[i]);
        const void* o = g->out ? g->out[i] : g->grads[i];
        if (g->sizes[i] > 0 && (!g->grads[i] || !o)) return kv_fail(MLORA_E_ARG, "tensor %d is NULL", i);
        if ((reinterpret_cast<uintptr_t>(g->grads[i]) | reinterpret_cast<uintptr_t>(o)) % es)
            return kv_fail(MLORA_E_ARG, "tensor %d is not aligned to its elements", i);
        if (g->groups && (g->groups[i] < 0 || g->groups[i] >= g->n_groups))
            return kv_fail(MLORA_E_ARG, "tensor %d: group %d outside 0..%d", i, g->groups[i], g->n_groups - 1);
        total += clip_chunks(g->sizes[i]);
    }
    if (total > INT32_MAX) return kv_fail(MLORA_E_ARG, "too many elements for one call");
    *chunks = total;
    return MLORA_OK;
}

}  // namespace

extern "C" int64_t mlora_clip_grads_workspace(const mlora_grad_set* g) {
    int64_t chunks = 0;
    if (clip_check(g, &chunks)) return 0;
    return (chunks > 0 ? chunks : 1) * (int64_t)sizeof(double);
}

extern "C" int mlora_clip_grads(const mlora_grad_set* g, float max_norm, float* norms_out, void* workspace,
                                int64_t workspace_bytes, void* stream) try {
    int64_t chunks = 0;
    const int rc = clip_check(g, &chunks);
    if (rc) return rc;
    if (!(max_norm >= 0.f)) return kv_fail(MLORA_E_ARG, "max_norm must be >= 0 (infinity: norms only)");
    if (chunks > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 7) ||
                       workspace_bytes < chunks * (int64_t)sizeof(double)))
        return kv_fail(MLORA_E_ARG, "the workspace must be 8-byte aligned and hold %lld bytes",
                       (long long)(chunks * sizeof(double)));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // tensors in group order; empty ones have nothing to add
    std::vector<ClipEntry> e;
    e.reserve(g->n_tensors);
    for (int i = 0; i < g->n_tensors; ++i) {
        if (g->sizes[i] == 0) continue;
        ClipEntry x;
        x.src = g->grads[i];
        x.dst = g->out ? g->out[i] : const_cast<void*>(g->grads[i]);
        x.size = g->sizes[i];
        x.chunk0 = x.g0 = x.g1 = 0;
        x.group = g->groups ? g->groups[i] : 0;
        e.push_back(x);
    }
    std::stable_sort(e.begin(), e.end(), [](const ClipEntry& a, const ClipEntry& b) { return a.group < b.group; });
    int at = 0, groups = 0;
    for (size_t i = 0; i < e.size();) {
        size_t j = i;
        const int g0 = at;
        for (; j < e.size() && e[j].group == e[i].group; ++j) {
            e[j].chunk0 = at;
            at += (int)clip_chunks(e[j].size);
        }
        for (size_t k = i; k < j; ++k) { e[k].g0 = g0; e[k].g1 = at; }
        ++groups;
        i = j;
    }
    cudaError_t err = cudaSuccess;
    if (norms_out && groups < g->n_groups)       // groups without elements
        err = cudaMemsetAsync(norms_out, 0, sizeof(float) * g->n_groups, s);
    double* part = static_cast<double*>(workspace);
    const int n = (int)e.size();
    if (err == cudaSuccess && n)
        err = g->dtype == MLORA_BF16 ? launch_clip_norm<bf16>(e.data(), n, part, nullptr, s, nullptr)
                                     : launch_clip_norm<float>(e.data(), n, part, nullptr, s, nullptr);
    if (err == cudaSuccess && n)
        err = g->dtype == MLORA_BF16 ? launch_clip_scale<bf16>(e.data(), n, part, max_norm, norms_out, s)
                                     : launch_clip_scale<float>(e.data(), n, part, max_norm, norms_out, s);
    if (err != cudaSuccess) return kv_fail(MLORA_E_CUDA, "clipping: %s", cudaGetErrorString(err));
    return MLORA_OK;
} catch (const std::bad_alloc&) {
    return kv_fail(MLORA_E_NOMEM, "no host memory for the tensor table");
}
