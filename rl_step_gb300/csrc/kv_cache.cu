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

int kv_check(const mlora_kv_cache* c, const mlora_kv_seqs* q, int32_t dtype, int64_t max_len, KvView* out) {
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
    v.max_pages = q->max_pages; v.max_len = max_len;
    // no sequence has more rows than there are
    v.max_rows = q->n_rows < q->max_rows ? (int)q->n_rows : q->max_rows;
    *out = v;
    return MLORA_OK;
}

namespace {

// One unit: a (sequence, touched page, key/value head, K or V).  Pages last: the
// page numbers that few sequences have are together at the end, and their blocks
// leave at once (256 single tokens, append and read of their pages: 30.4 us with
// sequences last, 28.7 so).
struct KvUnit {
    int s, p, h, is_v;
};
__device__ __forceinline__ KvUnit kv_unit(int64_t u, int n_seqs, int n_kv) {
    KvUnit x;
    x.is_v = (int)(u & 1);
    u >>= 1;
    x.h = (int)(u % n_kv);
    u /= n_kv;
    x.s = (int)(u % n_seqs);
    x.p = (int)(u / n_seqs);
    return x;
}

// What a thread holds of a page's tile in registers, DIMS = 16 bytes of the rows'
// type: PK pieces of one token's DIMS dims, or PV pieces of four tokens' DIMS dims,
// 128 bytes either way.  Neighbouring threads hold neighbouring dims, so a warp's
// 16-byte loads and stores of rows are whole lines.  A tile takes UT =
// tile_threads() threads, and a warp alone takes the rows of warp_rows() tokens,
// wherever they begin among the groups of four.
template <typename T>
struct Pieces {
    static constexpr int DIMS = 16 / sizeof(T), K = 8, V = 2;
};
template <typename T, int HD>
constexpr int tile_threads() { return KV_PAGE * HD / (Pieces<T>::K * Pieces<T>::DIMS); }
template <typename T, int HD>
constexpr int warp_rows() { return 4 * (Pieces<T>::V * 32 / (HD / Pieces<T>::DIMS) - 1) + 1; }
static_assert(warp_rows<float, 128>() == 5 && warp_rows<float, 64>() == 13 && warp_rows<bf16, 128>() == 13 &&
              warp_rows<bf16, 64>() == 29, "rows whose groups of four fit PV pieces, and so fit PK = 4 PV pieces");

template <typename T>
__device__ __forceinline__ uint4 load16(const T* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// the DIMS elements of 16 bytes as floats
template <typename T>
__device__ __forceinline__ void floats(const uint4& r, float (&x)[Pieces<T>::DIMS]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(w[i]);
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// The larger of m and the magnitudes' bits, as the type's own (two bf16 apart in a
// word); infinities and NaN are larger than every finite value.
template <typename T>
__device__ __forceinline__ uint32_t max_bits(const uint4& r, uint32_t m) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) m = max(m, w[i] & 0x7fffffffu);
        else m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    }
    return m;
}
template <typename T>
__device__ __forceinline__ uint32_t float_bits(uint32_t m) {               // of the largest one
    return sizeof(T) == 4 ? m : max(m << 16, m & 0xffff0000u);
}
// the same over the finite values alone
template <typename T>
__device__ __forceinline__ uint32_t finite_bits(const uint4& r, uint32_t m) {
    float x[Pieces<T>::DIMS];
    floats<T>(r, x);
#pragma unroll
    for (int i = 0; i < Pieces<T>::DIMS; ++i) {
        const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
        if (b < 0x7f800000u) m = max(m, b);
    }
    return m;
}

// Maximum over a unit's threads (UT: a warp or the block).
template <int UT>
__device__ __forceinline__ uint32_t unit_max(uint32_t m, uint32_t* part) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (UT > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < UT / 32; ++w) m = max(m, part[w]);
    }
    return m;
}

// The elements of 16 bytes times f as e4m3 bytes, 4 a word.  all_finite = false:
// infinities become NaN (e4m3 has none, and its saturation would make them 448).
template <typename T>
__device__ __forceinline__ void to_bytes(const uint4& r, float f, bool all_finite, uint32_t (&b)[Pieces<T>::DIMS / 4]) {
    float x[Pieces<T>::DIMS];
    floats<T>(r, x);
    if (!all_finite) {
#pragma unroll
        for (int i = 0; i < Pieces<T>::DIMS; ++i) x[i] = fabsf(x[i]) <= FLT_MAX ? x[i] : NAN;
    }
#pragma unroll
    for (int i = 0; i < Pieces<T>::DIMS / 4; ++i)
        b[i] = float4_to_e4m3x4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
}
// DIMS bytes, times f, as elements
template <typename T>
__device__ __forceinline__ uint4 from_bytes(const uint32_t (&b)[Pieces<T>::DIMS / 4], float f) {
    float x[4];
    e4m3x4_to_float4(b[0], x);
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(x[0] * f), __float_as_uint(x[1] * f), __float_as_uint(x[2] * f),
                          __float_as_uint(x[3] * f));
    } else {
        float y[4];
        e4m3x4_to_float4(b[1], y);
        return make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                          pack_bf16x2(y[0] * f, y[1] * f), pack_bf16x2(y[2] * f, y[3] * f));
    }
}
// stored bytes under a scale 1 / f times as large
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float f) {
    float x[4];
    e4m3x4_to_float4(w, x);
    return float4_to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}
__device__ __forceinline__ uint4 rescaled(uint4 w, float f) {
    return make_uint4(rescaled(w.x, f), rescaled(w.y, f), rescaled(w.z, f), rescaled(w.w, f));
}
// byte b of each of the four words, in their order
__device__ __forceinline__ uint32_t byte_of4(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, int b) {
    const uint32_t sel = b | (4 + b) << 4;
    return __byte_perm(__byte_perm(w0, w1, sel), __byte_perm(w2, w3, sel), 0x5410);
}

// What a unit's threads find of their page: nothing to do, or the tokens [a, b)
// of the page that the call's rows are, the row of token 0, and the page's id.
struct KvPart {
    int id, a, b;
    int64_t row;
};
__device__ __forceinline__ bool kv_part(const KvView& c, const KvUnit& u, bool first_thread, KvPart& t) {
    SeqRows r;
    if (!kv_seq(c, u.s, r)) {
        if (first_thread) raise_status(c.status, ST_RANGE);
        return false;
    }
    if (r.len == 0 || r.n == 0) return false;
    const int start = r.len - r.n;
    const int page = start / KV_PAGE + u.p;
    if ((int64_t)page * KV_PAGE >= r.len) return false;
    t.id = c.table[(int64_t)u.s * c.max_pages + page];
    if (t.id < 0 || t.id >= c.n_pages) {
        if (first_thread) raise_status(c.status, ST_RANGE);
        return false;
    }
    const int first = page * KV_PAGE;
    t.a = start > first ? start - first : 0;
    t.b = r.len - first < KV_PAGE ? r.len - first : KV_PAGE;
    t.row = (int64_t)r.row0 + first - start;
    return true;
}

// ----------------------------------------------------------------------------
// append
// ----------------------------------------------------------------------------
// Bound by memory: each row is read once and each byte written once (2 + 1 bytes an
// element in bf16).  UT threads a unit: a block, or a warp of one of four.  All of
// a thread's loads are in flight together, and the rows wait in registers for the
// maximum, which is taken on the bits (two bf16 values an instruction); the loops
// with tests for infinities run only for a unit that has one.  64 registers a
// thread (bf16): at 96, 28 % of the warps are resident and the kernel takes 99 us
// where it now takes 70 (65,000 prompt tokens of 8 heads of 128: 5.7 TB/s).  A
// second read of the rows in place of registers: 115 us.  256 single tokens: a warp
// a unit 6.3 us, a block of 128 threads a unit 9.
template <typename T, int HD, int UT>
__global__ void __launch_bounds__(UT == 32 ? 128 : UT, (sizeof(T) == 4 ? 768 : 1024) / (UT == 32 ? 128 : UT))
kv_append_kernel(const __grid_constant__ KvView c, const T* __restrict__ k, int64_t ldk, const T* __restrict__ v,
                 int64_t ldv, int units) {
    using P = Pieces<T>;
    constexpr int D = P::DIMS, R = HD / D;                                 // pieces across a head
    __shared__ uint32_t part[UT / 32];
    const int unit = UT == 32 ? blockIdx.x * 4 + threadIdx.x / 32 : blockIdx.x;
    const int tid = threadIdx.x % UT;
    if (unit >= units) return;
    const KvUnit u = kv_unit(unit, c.n_seqs, c.n_kv);
    KvPart t;
    if (!kv_part(c, u, tid == 0, t)) return;
    const int a = t.a, b = t.b;
    const T* src = (u.is_v ? v : k) + u.h * HD;
    const int64_t ld = u.is_v ? ldv : ldk;
    const int g0 = a / 4;                                                  // the first new token's group of four
    float* sc = (u.is_v ? c.vs : c.ks) + (int64_t)t.id * c.n_kv + u.h;
    uint8_t* tile = (u.is_v ? c.v : c.k) + ((int64_t)t.id * c.n_kv + u.h) * (KV_PAGE * HD);
    int old = a > 0 ? (int)((__float_as_uint(*sc) >> 23) & 255u) - 127 : KV_MIN_EXP;
    old = old < KV_MIN_EXP ? KV_MIN_EXP : (old > KV_MAX_EXP ? KV_MAX_EXP : old);

    // piece i of a thread: keys: token a + at / R; values: tokens 4 (g0 + at / R) + 0..3, at = tid + i UT
    uint4 x[P::K];
#pragma unroll
    for (int i = 0; i < P::K; ++i) {
        const int at = tid + (u.is_v ? i / 4 : i) * UT;
        const int j = u.is_v ? (g0 + at / R) * 4 + i % 4 : a + at / R;
        x[i] = make_uint4(0, 0, 0, 0);
        if (j >= a && j < b) x[i] = load16(src + kv_row(c, t.row + j) * ld + at % R * D);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < P::K; ++i) m = max_bits<T>(x[i], m);
    m = unit_max<UT>(float_bits<T>(m), part);
    const bool all_finite = m < 0x7f800000u;
    if (!all_finite) {
        if (UT > 32) __syncthreads();                                      // part[] is free again
        m = 0;
#pragma unroll
        for (int i = 0; i < P::K; ++i) m = finite_bits<T>(x[i], m);
        m = unit_max<UT>(m, part);
    }
    // m = 2^E (1 + mantissa): 448 = 1.75 * 2^8
    int e = (int)(m >> 23) - 127 - 8 + ((m & 0x7fffffu) > 0x600000u);
    if (e < KV_MIN_EXP) e = KV_MIN_EXP;
    int grow = 0;
    if (a > 0) {
        if (old >= e) e = old;
        else grow = e - old;
    }
    if (UT == 32) __syncwarp();                                            // every thread has read the old scale
    if (tid == 0) *sc = kv_pow2(e);
    const float f = kv_pow2(-e);
    const float fo = kv_pow2(grow > 60 ? -60 : -grow);                     // 448 * 2^-60 rounds to 0
    if (!u.is_v) {
        if (grow)
            for (int i = tid; i < a * (HD / 16); i += UT) {
                uint4* w = reinterpret_cast<uint4*>(tile + kv_byte_k<HD>(i / (HD / 16), i % (HD / 16) * 16));
                *w = rescaled(*w, fo);
            }
#pragma unroll
        for (int i = 0; i < P::K; ++i) {
            const int at = tid + i * UT, j = a + at / R;
            if (j >= b) continue;
            uint32_t y[D / 4];
            to_bytes<T>(x[i], f, all_finite, y);
            uint8_t* w = tile + kv_byte_k<HD>(j, at % R * D);
            if constexpr (D == 8) *reinterpret_cast<uint2*>(w) = make_uint2(y[0], y[1]);
            else *reinterpret_cast<uint32_t*>(w) = y[0];
        }
    } else {
        // 16 bytes hold 4 dims of 4 tokens, and 8 dims lie side by side
        if (grow)
            for (int i = tid; i < g0 * (HD / 4); i += UT) {
                uint4* w = reinterpret_cast<uint4*>(tile + kv_byte_v<HD>(i / (HD / 4) * 4, i % (HD / 4) * 4));
                *w = rescaled(*w, fo);
            }
#pragma unroll
        for (int i = 0; i < P::V; ++i) {
            const int at = tid + i * UT, j0 = (g0 + at / R) * 4;
            if (j0 >= b) continue;
            uint32_t y[4][D / 4];
#pragma unroll
            for (int q = 0; q < 4; ++q) to_bytes<T>(x[4 * i + q], f, all_finite, y[q]);
            uint4* w = reinterpret_cast<uint4*>(tile + kv_byte_v<HD>(j0, at % R * D));
            const uint32_t keep = j0 < a ? (1u << 8 * (a - j0)) - 1 : 0;   // older tokens of the first group
#pragma unroll
            for (int q = 0; q < D / 4; ++q) {
                uint32_t o[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) o[z] = byte_of4(y[0][q], y[1][q], y[2][q], y[3][q], z);
                if (keep) {
                    uint4 was = w[q];
                    if (grow) was = rescaled(was, fo);
                    o[0] = (was.x & keep) | (o[0] & ~keep);
                    o[1] = (was.y & keep) | (o[1] & ~keep);
                    o[2] = (was.z & keep) | (o[2] & ~keep);
                    o[3] = (was.w & keep) | (o[3] & ~keep);
                }
                w[q] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

// ----------------------------------------------------------------------------
// read
// ----------------------------------------------------------------------------
// Bound by memory, most of it writes.  A block a unit: a thread's loads are in
// flight together, and each of its stores is 16 bytes beside its neighbours'
// (65,000 tokens of 8 heads of 128 to fp32: 100 us, 6.6 TB/s; with pieces of 32
// bytes a thread, whose stores leave gaps, 130 us).
template <typename T, int HD>
__global__ void __launch_bounds__(tile_threads<T, HD>(), 2048 / tile_threads<T, HD>())
kv_read_kernel(const __grid_constant__ KvView c, T* __restrict__ ko, T* __restrict__ vo) {
    using P = Pieces<T>;
    constexpr int UT = tile_threads<T, HD>(), D = P::DIMS, R = HD / D;
    const KvUnit u = kv_unit(blockIdx.x, c.n_seqs, c.n_kv);
    T* dst = u.is_v ? vo : ko;
    KvPart t;
    if (!dst || !kv_part(c, u, threadIdx.x == 0, t)) return;
    const int64_t ld = (int64_t)c.n_kv * HD;
    dst += u.h * HD;
    const float f = (u.is_v ? c.vs : c.ks)[(int64_t)t.id * c.n_kv + u.h];
    const uint8_t* tile = (u.is_v ? c.v : c.k) + ((int64_t)t.id * c.n_kv + u.h) * (KV_PAGE * HD);
    if (!u.is_v) {
        uint32_t w[P::K][D / 4] = {};
#pragma unroll
        for (int i = 0; i < P::K; ++i) {
            const int at = threadIdx.x + i * UT, j = t.a + at / R;
            if (j >= t.b) continue;
            const uint8_t* p = tile + kv_byte_k<HD>(j, at % R * D);
            if constexpr (D == 8) {
                const uint2 q = *reinterpret_cast<const uint2*>(p);
                w[i][0] = q.x;
                w[i][1] = q.y;
            } else {
                w[i][0] = *reinterpret_cast<const uint32_t*>(p);
            }
        }
#pragma unroll
        for (int i = 0; i < P::K; ++i) {
            const int at = threadIdx.x + i * UT, j = t.a + at / R;
            if (j < t.b) *reinterpret_cast<uint4*>(dst + (t.row + j) * ld + at % R * D) = from_bytes<T>(w[i], f);
        }
    } else {
        const int g0 = t.a / 4;
        uint4 w[P::V][D / 4] = {};
#pragma unroll
        for (int i = 0; i < P::V; ++i) {
            const int at = threadIdx.x + i * UT, j0 = (g0 + at / R) * 4;
            if (j0 >= t.b) continue;
            const uint4* p = reinterpret_cast<const uint4*>(tile + kv_byte_v<HD>(j0, at % R * D));
#pragma unroll
            for (int z = 0; z < D / 4; ++z) w[i][z] = p[z];
        }
#pragma unroll
        for (int i = 0; i < P::V; ++i) {
            const int at = threadIdx.x + i * UT, j0 = (g0 + at / R) * 4;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = j0 + q;
                if (j < t.a || j >= t.b) continue;
                uint32_t y[D / 4];
#pragma unroll
                for (int z = 0; z < D / 4; ++z) y[z] = byte_of4(w[i][z].x, w[i][z].y, w[i][z].z, w[i][z].w, q);
                *reinterpret_cast<uint4*>(dst + (t.row + j) * ld + at % R * D) = from_bytes<T>(y, f);
            }
        }
    }
}

// pages that max_rows consecutive positions can touch
inline int touched_pages(int max_rows) { return (max_rows + KV_PAGE - 2) / KV_PAGE + 1; }

// units of a call; -1 if a grid cannot hold them
inline int64_t call_units(const KvView& c) {
    const int64_t per = (int64_t)touched_pages(c.max_rows) * c.n_kv * 2;
    return per > (INT32_MAX - 3) / (c.n_seqs > 0 ? c.n_seqs : 1) ? -1 : per * c.n_seqs;
}

template <typename T, int HD, int UT>
void append_u(const KvView& c, const void* k, int64_t ldk, const void* v, int64_t ldv, int64_t units,
              cudaStream_t s) {
    constexpr int BLOCK = UT == 32 ? 128 : UT, PER = BLOCK / UT;
    kv_append_kernel<T, HD, UT><<<(unsigned)((units + PER - 1) / PER), BLOCK, 0, s>>>(
        c, static_cast<const T*>(k), ldk, static_cast<const T*>(v), ldv, (int)units);
}

// A warp a unit where its registers hold the rows.
template <typename T, int HD>
void append_t(const KvView& c, const void* k, int64_t ldk, const void* v, int64_t ldv, int64_t units,
              cudaStream_t s) {
    if (c.max_rows <= warp_rows<T, HD>()) append_u<T, HD, 32>(c, k, ldk, v, ldv, units, s);
    else append_u<T, HD, tile_threads<T, HD>()>(c, k, ldk, v, ldv, units, s);
}

template <typename T, int HD>
void read_u(const KvView& c, void* k, void* v, int64_t units, cudaStream_t s) {
    kv_read_kernel<T, HD><<<(unsigned)units, tile_threads<T, HD>(), 0, s>>>(c, static_cast<T*>(k), static_cast<T*>(v));
}
template <typename T>
void read_t(const KvView& c, int head_dim, void* k, void* v, int64_t units, cudaStream_t s) {
    if (head_dim == 64) read_u<T, 64>(c, k, v, units, s);
    else read_u<T, 128>(c, k, v, units, s);
}

}  // namespace

bool kv_fits(const KvView& c) { return call_units(c) >= 0; }

cudaError_t launch_kv_append(const KvView& c, int head_dim, int dtype, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, cudaStream_t s) {
    const int64_t units = call_units(c);
    if (dtype == MLORA_BF16)
        (head_dim == 64 ? append_t<bf16, 64> : append_t<bf16, 128>)(c, k, ldk, v, ldv, units, s);
    else
        (head_dim == 64 ? append_t<float, 64> : append_t<float, 128>)(c, k, ldk, v, ldv, units, s);
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
    const int rc = kv_check(c, q, dtype, INT64_MAX, &w);
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
    const int rc = kv_check(c, q, dtype, INT64_MAX, &w);
    if (rc) return rc;
    if (w.n_seqs == 0 || w.n_rows == 0 || w.max_rows == 0 || (!k_out && !v_out)) return MLORA_OK;
    if (!aligned16(k_out) || !aligned16(v_out)) return kv_fail(MLORA_E_ARG, "outputs must be 16-byte aligned");
    const int64_t units = call_units(w);
    if (!kv_fits(w)) return kv_fail(MLORA_E_ARG, "too many sequences, heads and rows for one call");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == MLORA_BF16) read_t<bf16>(w, c->head_dim, k_out, v_out, units, s);
    else read_t<float>(w, c->head_dim, k_out, v_out, units, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "read launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}
