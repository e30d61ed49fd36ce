// Writing and reading the 8-bit key/value cache (include/mlora_kv.h): the
// argument checks shared by its entry points, append and read.
#include <stdarg.h>
#include <stdio.h>

#include "kv_common.cuh"

int mlk_report_error(int code, const char* msg);

namespace mlk {

int kv_fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return mlk_report_error(code, buf);
}

int kv_check(const mlora_kv_cache* c, const mlora_kv_seqs* q, int32_t dtype, KvView* out) {
    if (!c || !q) return kv_fail(MLORA_E_ARG, "NULL cache or sequences");
    if (dtype != MLORA_BF16 && dtype != MLORA_FP32) return kv_fail(MLORA_E_ARG, "unknown dtype %d", dtype);
    if (c->head_dim != 64 && c->head_dim != 128)
        return kv_fail(MLORA_E_ARG, "head_dim %d: only 64 and 128 are supported", c->head_dim);
    if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024)
        return kv_fail(MLORA_E_ARG, "bad cache (%d pages, %d key/value heads)", c->n_pages, c->n_kv_heads);
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return kv_fail(MLORA_E_ARG, "NULL cache buffer");
    if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15)
        return kv_fail(MLORA_E_ARG, "cache buffers must be 16-byte aligned");
    if (q->n_seqs < 0 || q->n_seqs > (1 << 24) || q->n_rows < 0 || q->n_rows > INT32_MAX || q->max_pages < 1 || q->max_rows < 0)
        return kv_fail(MLORA_E_ARG, "bad sequences (n_seqs %d, n_rows %lld, max_pages %d, max_rows %d)", q->n_seqs,
                       (long long)q->n_rows, q->max_pages, q->max_rows);
    if (!q->row_off && (q->max_rows != 1 || q->n_rows < q->n_seqs))
        return kv_fail(MLORA_E_ARG, "row_off NULL needs max_rows = 1 and a row for each sequence");
    if (q->n_seqs > 0 && (!q->page_table || !q->kv_len))
        return kv_fail(MLORA_E_ARG, "NULL page table or kv_len");
    KvView v;
    v.k = c->k; v.v = c->v; v.ks = c->k_scale; v.vs = c->v_scale; v.status = c->status;
    v.table = q->page_table; v.kv_len = q->kv_len; v.row_off = q->row_off; v.row_map = nullptr;
    v.n_rows = q->n_rows; v.n_pages = c->n_pages; v.n_kv = c->n_kv_heads; v.n_seqs = q->n_seqs;
    v.max_pages = q->max_pages;
    // no sequence has more rows than there are
    v.max_rows = q->n_rows < q->max_rows ? (int)q->n_rows : q->max_rows;
    *out = v;
    return MLORA_OK;
}

namespace {

// One block handles one (sequence, touched page, key/value head, K or V).
struct KvUnit {
    int s, p, h, is_v;
};
__device__ __forceinline__ KvUnit kv_unit(int64_t u, int pages, int n_kv) {
    KvUnit x;
    x.is_v = (int)(u & 1);
    u >>= 1;
    x.h = (int)(u % n_kv);
    u /= n_kv;
    x.p = (int)(u % pages);
    x.s = (int)(u / pages);
    return x;
}

// ----------------------------------------------------------------------------
// append
// ----------------------------------------------------------------------------
template <int UT>
__device__ __forceinline__ float unit_max(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (UT == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < UT / 32; ++w) v = fmaxf(v, part[w]);
    return v;
}

// x * f, or NaN if x is an infinity (e4m3 has none, and its saturation would make it 448)
__device__ __forceinline__ float scaled(float x, float f) { return fabsf(x) <= FLT_MAX ? x * f : NAN; }

template <typename T, int HD, int UT>
__global__ void __launch_bounds__(UT) kv_append_kernel(const __grid_constant__ KvView c, const T* __restrict__ k,
                                                       int64_t ldk, const T* __restrict__ v, int64_t ldv, int pages) {
    __shared__ float part[UT / 32];
    const KvUnit u = kv_unit(blockIdx.x, pages, c.n_kv);
    SeqRows r;
    if (!kv_seq(c, u.s, INT64_MAX, r)) {
        if (threadIdx.x == 0) raise_status(c.status, ST_RANGE);
        return;
    }
    if (r.len == 0 || r.n == 0) return;
    const int start = r.len - r.n;
    const int page = start / KV_PAGE + u.p;
    if ((int64_t)page * KV_PAGE >= r.len) return;
    const int id = kv_page(c, u.s, page);
    if (id < 0) return;
    const int first = page * KV_PAGE;
    const int a = start > first ? start - first : 0;                      // new tokens [a, b) of the page
    const int b = r.len - first < KV_PAGE ? r.len - first : KV_PAGE;
    const T* src = (u.is_v ? v : k) + u.h * HD;
    const int64_t ld = u.is_v ? ldv : ldk;
    const int64_t row = (int64_t)r.row0 + first - start;                  // row of the page's token 0
    constexpr int W = HD / 4;

    float amax = 0.f;
    for (int i = threadIdx.x; i < (b - a) * W; i += UT) {
        float x[4];
        load4_f(src + kv_row(c, row + a + i / W) * ld + i % W * 4, x);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float m = fabsf(x[q]);
            if (m <= FLT_MAX) amax = fmaxf(amax, m);
        }
    }
    amax = unit_max<UT>(amax, part);
    // amax = 2^E (1 + mantissa): 448 = 1.75 * 2^8
    const uint32_t bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
    if (e < KV_MIN_EXP) e = KV_MIN_EXP;
    float* sc = (u.is_v ? c.vs : c.ks) + (int64_t)id * c.n_kv + u.h;
    int grow = 0;
    if (a > 0) {
        int old = (int)((__float_as_uint(*sc) >> 23) & 255u) - 127;
        old = old < KV_MIN_EXP ? KV_MIN_EXP : (old > KV_MAX_EXP ? KV_MAX_EXP : old);
        if (old >= e) e = old;
        else grow = e - old;
    }
    if (UT > 32) __syncthreads();                                          // every thread has read the old scale
    else __syncwarp();
    if (threadIdx.x == 0) *sc = kv_pow2(e);
    const float f = kv_pow2(-e);
    const float fo = kv_pow2(grow > 60 ? -60 : -grow);                     // 448 * 2^-60 rounds to 0
    uint8_t* tile = (u.is_v ? c.v : c.k) + ((int64_t)id * c.n_kv + u.h) * (KV_PAGE * HD);
    const int lo = grow ? 0 : a;                                           // tokens whose bytes change: [lo, b)
    if (!u.is_v) {
        for (int i = lo * W + threadIdx.x; i < b * W; i += UT) {
            const int j = i / W, d = i % W * 4;
            uint32_t* w = reinterpret_cast<uint32_t*>(tile + kv_byte_k<HD>(j, d));
            float x[4];
            if (j >= a) {
                load4_f(src + kv_row(c, row + j) * ld + d, x);
                *w = float4_to_e4m3x4(scaled(x[0], f), scaled(x[1], f), scaled(x[2], f), scaled(x[3], f));
            } else {
                e4m3x4_to_float4(*w, x);
                *w = float4_to_e4m3x4(x[0] * fo, x[1] * fo, x[2] * fo, x[3] * fo);
            }
        }
    } else {
        // 16 bytes hold 4 dims of 4 tokens
        for (int i = lo / 4 * W + threadIdx.x; i < (b + 3) / 4 * W; i += UT) {
            const int j0 = i / W * 4, d = i % W * 4;
            uint4* w = reinterpret_cast<uint4*>(tile + kv_byte_v<HD>(j0, d));
            uint32_t x4[4] = {0, 0, 0, 0};                                 // per token: its 4 dims
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int j = j0 + t;
                if (j >= a && j < b) {
                    float x[4];
                    load4_f(src + kv_row(c, row + j) * ld + d, x);
                    x4[t] = float4_to_e4m3x4(scaled(x[0], f), scaled(x[1], f), scaled(x[2], f), scaled(x[3], f));
                }
            }
            uint32_t old[4] = {0, 0, 0, 0};                                // per dim: 4 tokens
            if (j0 < a) {
                const uint4 q = *w;
                old[0] = q.x; old[1] = q.y; old[2] = q.z; old[3] = q.w;
                if (grow) {
#pragma unroll
                    for (int q2 = 0; q2 < 4; ++q2) {
                        float x[4];
                        e4m3x4_to_float4(old[q2], x);
                        old[q2] = float4_to_e4m3x4(x[0] * fo, x[1] * fo, x[2] * fo, x[3] * fo);
                    }
                }
            }
            uint32_t o[4];
#pragma unroll
            for (int q2 = 0; q2 < 4; ++q2) {
                o[q2] = 0;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t by = j0 + t < a ? (old[q2] >> (8 * t)) & 255u : (x4[t] >> (8 * q2)) & 255u;
                    o[q2] |= by << (8 * t);
                }
            }
            *w = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ----------------------------------------------------------------------------
// read
// ----------------------------------------------------------------------------
template <typename T, int HD>
__global__ void __launch_bounds__(128) kv_read_kernel(const __grid_constant__ KvView c, T* __restrict__ ko,
                                                      T* __restrict__ vo, int pages) {
    const KvUnit u = kv_unit(blockIdx.x, pages, c.n_kv);
    T* dst = u.is_v ? vo : ko;
    if (!dst) return;
    SeqRows r;
    if (!kv_seq(c, u.s, INT64_MAX, r)) {
        if (threadIdx.x == 0) raise_status(c.status, ST_RANGE);
        return;
    }
    if (r.len == 0 || r.n == 0) return;
    const int start = r.len - r.n;
    const int page = start / KV_PAGE + u.p;
    if ((int64_t)page * KV_PAGE >= r.len) return;
    const int id = kv_page(c, u.s, page);
    if (id < 0) return;
    const int first = page * KV_PAGE;
    const int a = start > first ? start - first : 0;
    const int b = r.len - first < KV_PAGE ? r.len - first : KV_PAGE;
    const int64_t row = (int64_t)r.row0 + first - start;
    const int64_t ld = (int64_t)c.n_kv * HD;
    dst += u.h * HD;
    const float f = (u.is_v ? c.vs : c.ks)[(int64_t)id * c.n_kv + u.h];
    const uint8_t* tile = (u.is_v ? c.v : c.k) + ((int64_t)id * c.n_kv + u.h) * (KV_PAGE * HD);
    constexpr int W = HD / 4;
    if (!u.is_v) {
        for (int i = a * W + threadIdx.x; i < b * W; i += 128) {
            const int j = i / W, d = i % W * 4;
            float x[4];
            e4m3x4_to_float4(*reinterpret_cast<const uint32_t*>(tile + kv_byte_k<HD>(j, d)), x);
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] *= f;
            store4_f(dst + (row + j) * ld + d, x);
        }
    } else {
        for (int i = a / 4 * W + threadIdx.x; i < (b + 3) / 4 * W; i += 128) {
            const int j0 = i / W * 4, d = i % W * 4;
            const uint4 w = *reinterpret_cast<const uint4*>(tile + kv_byte_v<HD>(j0, d));
            float x[4][4];                                                 // [dim][token]
            e4m3x4_to_float4(w.x, x[0]);
            e4m3x4_to_float4(w.y, x[1]);
            e4m3x4_to_float4(w.z, x[2]);
            e4m3x4_to_float4(w.w, x[3]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (j0 + t < a || j0 + t >= b) continue;
                const float y[4] = {x[0][t] * f, x[1][t] * f, x[2][t] * f, x[3][t] * f};
                store4_f(dst + (row + j0 + t) * ld + d, y);
            }
        }
    }
}

// pages that max_rows consecutive positions can touch
inline int touched_pages(int max_rows) { return (max_rows + KV_PAGE - 2) / KV_PAGE + 1; }

// blocks of a launch over (sequence, touched page, head, K or V); -1 if a grid cannot hold them
inline int64_t unit_blocks(const KvView& c, int pages) {
    const int64_t per = (int64_t)pages * c.n_kv * 2;
    return per > INT32_MAX / (c.n_seqs > 0 ? c.n_seqs : 1) ? -1 : per * c.n_seqs;
}

template <typename T, int HD>
void append_t(const KvView& c, const void* k, int64_t ldk, const void* v, int64_t ldv, int pages, int64_t blocks,
              cudaStream_t s) {
    kv_append_kernel<T, HD, 128><<<(unsigned)blocks, 128, 0, s>>>(c, static_cast<const T*>(k), ldk,
                                                                  static_cast<const T*>(v), ldv, pages);
}

template <typename T>
void read_t(const KvView& c, int head_dim, void* k, void* v, int pages, int64_t blocks, cudaStream_t s) {
    if (head_dim == 64)
        kv_read_kernel<T, 64><<<(unsigned)blocks, 128, 0, s>>>(c, static_cast<T*>(k), static_cast<T*>(v), pages);
    else
        kv_read_kernel<T, 128><<<(unsigned)blocks, 128, 0, s>>>(c, static_cast<T*>(k), static_cast<T*>(v), pages);
}

}  // namespace

bool kv_fits(const KvView& c) { return unit_blocks(c, touched_pages(c.max_rows)) >= 0; }

cudaError_t launch_kv_append(const KvView& c, int head_dim, int dtype, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, cudaStream_t s) {
    const int pages = touched_pages(c.max_rows);
    const int64_t blocks = unit_blocks(c, pages);
    if (dtype == MLORA_BF16)
        (head_dim == 64 ? append_t<bf16, 64> : append_t<bf16, 128>)(c, k, ldk, v, ldv, pages, blocks, s);
    else
        (head_dim == 64 ? append_t<float, 64> : append_t<float, 128>)(c, k, ldk, v, ldv, pages, blocks, s);
    return cudaGetLastError();
}

}  // namespace mlk

using namespace mlk;

namespace {
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
}  // namespace

extern "C" int mlora_kv_append(const mlora_kv_cache* c, const mlora_kv_seqs* q, int32_t dtype, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, void* stream) {
    KvView w;
    const int rc = kv_check(c, q, dtype, &w);
    if (rc) return rc;
    if (w.n_seqs == 0 || w.n_rows == 0 || w.max_rows == 0) return MLORA_OK;
    const int64_t row = (int64_t)c->n_kv_heads * c->head_dim;
    const int64_t per16 = dtype == MLORA_BF16 ? 8 : 4;
    if (!k || !v) return kv_fail(MLORA_E_ARG, "NULL keys or values");
    if (k_stride < row || v_stride < row || k_stride % per16 || v_stride % per16 || !aligned16(k) || !aligned16(v))
        return kv_fail(MLORA_E_ARG, "key and value rows must be 16-byte aligned and at least %lld elements apart",
                       (long long)row);
    if (!kv_fits(w))
        return kv_fail(MLORA_E_ARG, "too many sequences, heads and rows for one call");
    const cudaError_t e = launch_kv_append(w, c->head_dim, dtype, k, k_stride, v, v_stride,
                                           reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "append launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}

extern "C" int mlora_kv_read(const mlora_kv_cache* c, const mlora_kv_seqs* q, int32_t dtype, void* k_out,
                             void* v_out, void* stream) {
    KvView w;
    const int rc = kv_check(c, q, dtype, &w);
    if (rc) return rc;
    if (w.n_seqs == 0 || w.n_rows == 0 || w.max_rows == 0 || (!k_out && !v_out)) return MLORA_OK;
    if (!aligned16(k_out) || !aligned16(v_out)) return kv_fail(MLORA_E_ARG, "outputs must be 16-byte aligned");
    const int pages = touched_pages(w.max_rows);
    const int64_t blocks = unit_blocks(w, pages);
    if (!kv_fits(w)) return kv_fail(MLORA_E_ARG, "too many sequences, heads and rows for one call");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == MLORA_BF16) read_t<bf16>(w, c->head_dim, k_out, v_out, pages, blocks, s);
    else read_t<float>(w, c->head_dim, k_out, v_out, pages, blocks, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "read launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}
