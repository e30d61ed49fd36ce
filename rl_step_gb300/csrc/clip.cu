// The norm of the gradients of each group of tensors, and clipping:
//     n_g = sqrt(sum over the group's tensors of x^2)
//     x <- x * (max_norm / n_g)   where n_g > max_norm.
//
// What bounds it: bytes.  Every element is read for the norm and, the norm
// known, read again and written; the floor is one read and one write, which
// needs the second read to come from L2 (129 MB).
//  * Groups are taken in batches of at most CLIP_BATCH bytes; a launch scales one
//    batch and reads the next for its norms, so a batch is scaled from L2.
//  * A block takes a chunk of 8,192 elements, held in registers from its first
//    load on; for the norms of a large group several, so that a group has about
//    512 sums whatever its size.  Launches overlap (programmatic dependent
//    launch): a block loads its chunk before it waits for the launch before.
//  * fp64 is scarce here (two operations a clock on an SM; a block's reduction in
//    fp64 took longer than its 32 KB): a thread adds at most 32 squares in fp32
//    and its chunks' sums with their rounding errors (a compensated sum), a block
//    its threads' sums and every scaling block its group's sums in fp32 trees.
//    All terms are positive: at most 33 + 2 + 8 + (sums of a group / 256 + 1) + 8
//    roundings of 2^-24 on the square.  Sums outside 1e-25 .. 1e30 carry a power
//    of two of their own and are joined in fp64, as those that are not finite are.
//    No atomics, a fixed order: results repeat bit for bit.
// (One resident kernel that counted arrivals a chunk instead took 981 us on the 32
// adapters of the 8B widths, 39 MB each, two whole passes 670 us, this 474 us, 77 %
// of the copy rate by the floor's bytes; one adapter 37, 37 and 20.6 us.  Of the 474,
// about 100 are lines that left L2 before they were scaled: a launch read 76 MB
// from HBM, 39 of them for the first time, until the scaling loads said that they
// are the last ones and began with the newest lines; 61 MB since.)
#include <algorithm>
#include <cfloat>
#include <new>
#include <vector>

#include "clip.cuh"
#include "kv_common.cuh"

namespace mlk {

namespace {

constexpr int CT = 256;                      // threads of a block

// The tensors of one launch, passed by value: no table in device memory, so
// nothing of the caller's is kept and a captured launch holds its own copy.  The
// first blocks add squares up, the others scale.
template <int N>
struct ClipTab {
    int n_scale, n_norm;                     // entries: those to scale, then those whose norm is wanted
    int scale0, scale_chunks;                // first chunk and chunks to scale
    int norm0;                               // first sum
    ClipEntry e[N];
};

// the entry of a chunk (of a sum) among e[0 .. n): `first` is the entries' first number
__device__ __forceinline__ const ClipEntry& clip_find(const ClipEntry* e, int n, int chunk, int ClipEntry::* first) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (e[mid].*first <= chunk) lo = mid; else hi = mid - 1;
    }
    return e[lo];
}

// s += x, with what the additions before it lost
__device__ __forceinline__ void add_to(float& s, float& lost, float x) {
    const float y = x - lost, z = s + y;
    lost = (z - s) - y;
    s = z;
}

__device__ __forceinline__ int chunk_len(const ClipEntry& e, int64_t at) {
    return e.size - at < CLIP_CHUNK ? (int)(e.size - at) : CLIP_CHUNK;
}

// sum over the block in a fixed order; every thread returns it
template <typename V>
__device__ __forceinline__ V block_sum(V v) {
    __shared__ V part[CT / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (part[0] + part[1]) + (part[2] + part[3]);
    return v + ((part[4] + part[5]) + (part[6] + part[7]));
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

// 16 bytes of elements as floats
__device__ __forceinline__ void unpack16(uint4 w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack16(uint4 w, float (&v)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 pack16(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
template <typename T> constexpr int PER16 = 16 / (int)sizeof(T);
template <typename T> constexpr int VECS = CLIP_CHUNK / CT / PER16<T>;     // of a thread in a whole chunk
__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A block's chunk p[0 .. n) in its threads' registers; elements that 16-byte
// accesses cannot reach (ends, odd pointers) are read where they are used.
template <typename T>
struct Chunk {
    uint4 w[VECS<T>];
    const T* p;
    int n, nv;                               // elements, 16-byte pieces
    // AGAIN: a later launch reads it once more, from L2; else this is that last time, and its lines may go first
    template <bool AGAIN>
    __device__ __forceinline__ void load(const T* p_, int n_) {
        p = p_;
        n = n_;
        nv = aligned16(p) ? n / PER16<T> : 0;
#pragma unroll
        for (int k = 0; k < VECS<T>; ++k)
            if ((int)threadIdx.x + CT * k < nv) {
                const uint4* q = reinterpret_cast<const uint4*>(p) + threadIdx.x + CT * k;
                w[k] = AGAIN ? __ldcg(q) : __ldcs(q);
            }
    }
    // this thread's squares
    __device__ __forceinline__ float sum() const {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < VECS<T>; ++k)
            if ((int)threadIdx.x + CT * k < nv) {
                float v[PER16<T>];
                unpack16(w[k], v);
#pragma unroll
                for (int e = 0; e < PER16<T>; ++e) s = fmaf(v[e], v[e], s);
            }
        for (int i = nv * PER16<T> + threadIdx.x; i < n; i += CT) s = fmaf(to_f(p[i]), to_f(p[i]), s);
        return s;
    }
    __device__ __forceinline__ void scale(T* o, float f) const {
        if (nv == 0 || aligned16(o)) {
#pragma unroll
            for (int k = 0; k < VECS<T>; ++k)
                if ((int)threadIdx.x + CT * k < nv) {
                    float v[PER16<T>];
                    unpack16(w[k], v);
#pragma unroll
                    for (int e = 0; e < PER16<T>; ++e) v[e] *= f;
                    __stcs(reinterpret_cast<uint4*>(o) + threadIdx.x + CT * k, pack16(v));
                }
            for (int i = nv * PER16<T> + threadIdx.x; i < n; i += CT) o[i] = from_f<T>(to_f(p[i]) * f);
        } else {
            for (int i = threadIdx.x; i < n; i += CT) o[i] = from_f<T>(to_f(p[i]) * f);
        }
    }
};

// The sum of squares of p[0 .. n) where it leaves what fp32 adds safely:
// relative to the largest magnitude (2^E, so that the scaling is exact).
template <typename T>
__device__ __noinline__ ClipSum sum_scaled(const T* p, int64_t n) {
    float m = 0.f;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < n; i += CT) {
        const float y = fabsf(to_f(p[i]));
        m = fmaxf(m, y);
        bad |= !(y <= FLT_MAX);
    }
    m = block_max(m);
    if (__syncthreads_or(bad)) {
        // an infinity or NaN: their sum says which
        float v = 0.f;
        for (int64_t i = threadIdx.x; i < n; i += CT) {
            const float y = fabsf(to_f(p[i]));
            v += y <= FLT_MAX ? 0.f : y;
        }
        return ClipSum{block_sum(v), 0};
    }
    if (m == 0.f) return ClipSum{0.f, 0};
    int E;
    frexpf(m, &E);
    // in two steps: 2^-E itself can lie outside fp32
    const float f1 = ldexpf(1.f, -E / 2), f2 = ldexpf(1.f, -E - (-E / 2));
    float q = 0.f, lost = 0.f;
    for (int64_t i = threadIdx.x; i < n; i += CT) {
        const float y = to_f(p[i]) * f1 * f2;
        add_to(q, lost, y * y);
    }
    return ClipSum{block_sum(q), 2 * E};
}

// the group's norm from its sums; every thread returns it
__device__ __forceinline__ double group_norm(const ClipSum* part, int g0, int g1) {
    float s = 0.f, lost = 0.f;
    bool apart = false;
    for (int i = g0 + threadIdx.x; i < g1; i += CT) {
        const ClipSum x = part[i];
        add_to(s, lost, x.v);
        apart |= x.e != 0 || !(x.v <= FLT_MAX);     // (a compensated sum makes an infinity NaN)
    }
    if (!__syncthreads_or(apart)) return (double)sqrtf(block_sum(s));
    double v = 0.0;
    for (int i = g0 + threadIdx.x; i < g1; i += CT) v += ldexp((double)part[i].v, part[i].e);
    return sqrt(block_sum(v));
}

// the factor of a norm; 1 for a norm that is not finite: such a gradient is
// the caller's to skip, and scaling it would hide it
__device__ __forceinline__ float clip_factor(double norm, float max_norm) {
    return norm > (double)max_norm && norm <= DBL_MAX ? (float)((double)max_norm / norm) : 1.f;
}

// mask (may be null): only the groups g with mask[g] != 0 are added up, the
// others' chunks get 0.
template <typename T, int N>
__global__ void __launch_bounds__(CT, 4) clip_kernel(const __grid_constant__ ClipTab<N> t, ClipSum* part,
                                                     const int* __restrict__ mask, float max_norm, float* norms) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the blocks that add up come first: they read from HBM while those that scale wait for the launch before
    const int adding = gridDim.x - t.scale_chunks;
    const bool scale = (int)blockIdx.x >= adding;
    // the last chunks that were read are scaled first: they are the likeliest to be in L2
    const int chunk = scale ? t.scale0 + (int)(gridDim.x - 1 - blockIdx.x) : t.norm0 + blockIdx.x;
    const ClipEntry& e = scale ? clip_find(t.e, t.n_scale, chunk, &ClipEntry::chunk0)
                               : clip_find(t.e + t.n_scale, t.n_norm, chunk, &ClipEntry::sum0);
    const int64_t at = (int64_t)(scale ? chunk - e.chunk0 : (chunk - e.sum0) * e.per_sum) * CLIP_CHUNK;
    const T* p = static_cast<const T*>(e.src) + at;
    T* o = static_cast<T*>(e.dst) + at;
    const bool wanted = scale || !mask || mask[e.group];
    Chunk<T> x;
    if (scale) x.template load<false>(p, chunk_len(e, at));
    else x.template load<true>(p, wanted ? chunk_len(e, at) : 0);
    // every block waits before it writes, so that a launch's end means the end of all before it
    if (scale) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        __shared__ float s_f;
        const double norm = group_norm(part, e.g0, e.g1);
        if (threadIdx.x == 0) {
            if (norms && chunk == e.chunk0 && e.first) norms[e.group] = (float)norm;
            s_f = clip_factor(norm, max_norm);
        }
        __syncthreads();
        if (s_f != 1.f || p != o) x.scale(o, s_f);
    } else {
        float s = x.sum(), lost = 0.f;
        int64_t n = x.n;
        for (int k = 1; k < e.per_sum && wanted && at + (int64_t)k * CLIP_CHUNK < e.size; ++k) {
            x.template load<true>(p + (int64_t)k * CLIP_CHUNK, chunk_len(e, at + (int64_t)k * CLIP_CHUNK));
            n += x.n;
            add_to(s, lost, x.sum());
        }
        ClipSum sum{block_sum(s), 0};
        if (!(sum.v < 1e30f && sum.v > 1e-25f)) sum = sum_scaled(p, n);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (threadIdx.x == 0) part[chunk] = sum;
    }
}

template <typename T, int N>
cudaError_t launch_tab(const ClipEntry* scale, int n_scale, const ClipEntry* norm, int n_norm, ClipSum* part,
                       const int* mask, float max_norm, float* norms, bool first, cudaStream_t s) {
    ClipTab<N> t;
    t.n_scale = n_scale;
    t.n_norm = n_norm;
    int chunks[2] = {0, 0};
    const ClipEntry* from[2] = {scale, norm};
    const int n[2] = {n_scale, n_norm};
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < n[i]; ++j) t.e[(i ? n_scale : 0) + j] = from[i][j];
    }
    if (n_scale) chunks[0] = scale[n_scale - 1].chunk0 + (int)clip_chunks(scale[n_scale - 1].size) - scale[0].chunk0;
    if (n_norm) chunks[1] = norm[n_norm - 1].sum0 + clip_sums(norm[n_norm - 1]) - norm[0].sum0;
    t.scale0 = n_scale ? scale[0].chunk0 : 0;
    t.scale_chunks = chunks[0];
    t.norm0 = n_norm ? norm[0].sum0 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(chunks[0] + chunks[1]));
    cfg.blockDim = dim3(CT);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = first ? 0 : 1;                // a call's first launch follows the stream's earlier work entirely
    return cudaLaunchKernelEx(&cfg, clip_kernel<T, N>, t, part, mask, max_norm, norms);
}

constexpr int TAB_SMALL = 64, TAB_LARGE = 576;   // 3.6 KB and 32 KB of kernel parameters (at most 32 KB)

template <typename T>
cudaError_t launch_tables(const ClipEntry* scale, int n_scale, const ClipEntry* norm, int n_norm, ClipSum* part,
                          const int* mask, float max_norm, float* norms, bool& first, cudaStream_t s, int64_t* launches) {
    while (n_scale > 0 || n_norm > 0) {
        int a = n_scale, b = n_norm;
        if (a + b > TAB_LARGE) {
            if (a > TAB_LARGE / 2) a = b < TAB_LARGE / 2 ? TAB_LARGE - b : TAB_LARGE / 2;
            if (b > TAB_LARGE - a) b = TAB_LARGE - a;
        }
        if (a > n_scale) a = n_scale;
        const cudaError_t e = a + b <= TAB_SMALL
                                  ? launch_tab<T, TAB_SMALL>(scale, a, norm, b, part, mask, max_norm, norms, first, s)
                                  : launch_tab<T, TAB_LARGE>(scale, a, norm, b, part, mask, max_norm, norms, first, s);
        if (e != cudaSuccess) return e;
        if (launches) ++*launches;
        first = false;
        scale += a; n_scale -= a;
        norm += b; n_norm -= b;
    }
    return cudaSuccess;
}

// Bytes of a batch (or one larger group): the next batch passes through L2 while
// this one is scaled and written.  96 groups of 10 MB: 468 us with batches of 10
// MB (too many launches), 404 with 20, 393 with 28, 415 with 40.
constexpr int64_t CLIP_BATCH = 28 << 20;

template <typename T>
cudaError_t launch_clip(const ClipEntry* e, int n, ClipSum* part, float max_norm, float* norms, cudaStream_t s) {
    bool first = true;
    int a = 0, b = 0;                                    // the batch to scale: e[a .. b)
    while (a < n || b < n) {
        int k = b;                                       // the next one: e[b .. k), whole groups
        int64_t bytes = 0;
        while (k < n) {
            int j = k;
            int64_t more = 0;
            for (; j < n && e[j].group == e[k].group; ++j) more += e[j].size * (int64_t)sizeof(T);
            if (k > b && bytes + more > CLIP_BATCH) break;
            bytes += more;
            k = j;
        }
        const cudaError_t err = launch_tables<T>(e + a, b - a, e + b, k - b, part, nullptr, max_norm, norms, first, s, nullptr);
        if (err != cudaSuccess) return err;
        a = b;
        b = k;
        if (a == n) break;
    }
    return cudaSuccess;
}

}  // namespace

int clip_number(ClipEntry* e, int n) {
    int chunk = 0, sum = 0, groups = 0;
    for (int i = 0; i < n; ++groups) {
        int j = i;
        int64_t chunks = 0;
        for (; j < n && e[j].group == e[i].group; ++j) chunks += clip_chunks(e[j].size);
        const int g0 = sum;
        for (int k = i; k < j; ++k) {
            e[k].first = k == i;
            e[k].per_sum = (int)((chunks + CLIP_SUMS - 1) / CLIP_SUMS);
            e[k].chunk0 = chunk;
            e[k].sum0 = sum;
            chunk += (int)clip_chunks(e[k].size);
            sum += clip_sums(e[k]);
        }
        for (int k = i; k < j; ++k) { e[k].g0 = g0; e[k].g1 = sum; }
        i = j;
    }
    return groups;
}

cudaError_t launch_clip_norm(const ClipEntry* entries, int n, ClipSum* part, const int* mask, cudaStream_t s,
                             int64_t* launches) {
    bool first = true;
    return launch_tables<float>(nullptr, 0, entries, n, part, mask, 0.f, nullptr, first, s, launches);
}

namespace {

constexpr int MAX_ADAPTERS = 1024;
struct AdapterSums {
    int g[MAX_ADAPTERS + 1];                 // adapter a's sums are [g[a], g[a+1])
};

__global__ void __launch_bounds__(CT) clip_finish_kernel(const __grid_constant__ AdapterSums t, const ClipSum* part,
                                                         const int* __restrict__ mask, float max_norm, float* factor,
                                                         float* norms) {
    const int a = blockIdx.x;
    const double norm = mask[a] ? group_norm(part, t.g[a], t.g[a + 1]) : 0.0;
    if (threadIdx.x == 0) {
        factor[a] = clip_factor(norm, max_norm);
        if (norms) norms[a] = (float)norm;
    }
}

std::vector<ClipEntry> adapter_entries(const float* G, const int64_t* off, int n_ad) {
    std::vector<ClipEntry> e(n_ad);
    for (int a = 0; a < n_ad; ++a) {
        e[a].src = e[a].dst = const_cast<float*>(G) + off[a];
        e[a].size = off[a + 1] - off[a];
        e[a].group = a;
    }
    clip_number(e.data(), n_ad);
    return e;
}

}  // namespace

int64_t clip_adapter_sums(const int64_t* off, int n_ad) { return adapter_entries(nullptr, off, n_ad).back().g1; }

cudaError_t launch_clip_adapters(const float* G, const int64_t* off, int n_ad, const int* mask, ClipSum* part,
                                 float max_norm, float* factor, float* norms, cudaStream_t s, int64_t* launches) {
    const std::vector<ClipEntry> e = adapter_entries(G, off, n_ad);
    const cudaError_t err = launch_clip_norm(e.data(), n_ad, part, mask, s, launches);
    if (err != cudaSuccess) return err;
    AdapterSums t;
    for (int a = 0; a < n_ad; ++a) t.g[a] = e[a].g0;
    t.g[n_ad] = e[n_ad - 1].g1;
    clip_finish_kernel<<<n_ad, CT, 0, s>>>(t, part, mask, max_norm, factor, norms);
    if (launches) ++*launches;
    return cudaGetLastError();
}

}  // namespace mlk

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------
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
    // no more sums than chunks
    return (chunks > 0 ? chunks : 1) * (int64_t)sizeof(ClipSum);
}

extern "C" int mlora_clip_grads(const mlora_grad_set* g, float max_norm, float* norms_out, void* workspace,
                                int64_t workspace_bytes, void* stream) try {
    int64_t chunks = 0;
    const int rc = clip_check(g, &chunks);
    if (rc) return rc;
    if (!(max_norm >= 0.f)) return kv_fail(MLORA_E_ARG, "max_norm must be >= 0 (infinity: norms only)");
    const int64_t need = mlora_clip_grads_workspace(g);
    if (chunks > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 7) || workspace_bytes < need))
        return kv_fail(MLORA_E_ARG, "the workspace must be 8-byte aligned and hold %lld bytes", (long long)need);
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
        x.group = g->groups ? g->groups[i] : 0;
        e.push_back(x);
    }
    std::stable_sort(e.begin(), e.end(), [](const ClipEntry& a, const ClipEntry& b) { return a.group < b.group; });
    const int groups = clip_number(e.data(), (int)e.size());
    cudaError_t err = cudaSuccess;
    if (norms_out && groups < g->n_groups)       // groups without elements
        err = cudaMemsetAsync(norms_out, 0, sizeof(float) * g->n_groups, s);
    ClipSum* part = static_cast<ClipSum*>(workspace);
    const int n = (int)e.size();
    if (err == cudaSuccess && n)
        err = g->dtype == MLORA_BF16 ? launch_clip<bf16>(e.data(), n, part, max_norm, norms_out, s)
                                     : launch_clip<float>(e.data(), n, part, max_norm, norms_out, s);
    if (err != cudaSuccess) return kv_fail(MLORA_E_CUDA, "clipping: %s", cudaGetErrorString(err));
    return MLORA_OK;
} catch (const std::bad_alloc&) {
    return kv_fail(MLORA_E_NOMEM, "no host memory for the tensor table");
}
