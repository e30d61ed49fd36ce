// What the operators on the 8-bit key/value cache share (include/mlora_kv.h):
// the device view of a cache and of a call's sequences, the byte order of a
// page, and the checks of what only the device sees.
#pragma once

#include <cfloat>
#include <math.h>

#include "../../include/mlora_kv.h"
#include "internal.h"

namespace mlk {

constexpr int KV_PAGE = MLORA_KV_PAGE;
constexpr int KV_MIN_EXP = MLORA_KV_MIN_EXP;
constexpr int KV_MAX_EXP = 120;        // 448 * 2^120 is above every finite fp32 value

struct KvView {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int* status;
    const int* table;
    const int* kv_len;
    const int* row_off;                // null: one row a sequence
    const int* row_map;                // null, or where row r's data stands in the row arrays
    int64_t n_rows;
    int64_t max_len;                   // a longer sequence is out of range, in every kernel of the call
    int n_pages, n_kv, n_seqs, max_pages, max_rows;
};

// A sequence's rows as the device finds them.
struct SeqRows {
    int len;                           // kv_len
    int n;                             // its rows
    int row0;                          // the first of them
};

// A sequence's length and rows [a, b) against the ranges of the header; where
// they are outside, only row0 and n of r can be used, clipped to the rows that
// exist.
__device__ __forceinline__ bool kv_seq_ok(const KvView& c, int len, int64_t a, int64_t b, SeqRows& r) {
    r.len = len;
    r.row0 = (int)a;
    r.n = (int)(b - a < INT32_MAX ? b - a : INT32_MAX);
    const int64_t cap = (int64_t)c.max_pages * KV_PAGE;
    return len >= 0 && len <= cap && len <= c.max_len && a >= 0 && b >= a && b <= c.n_rows && r.n <= c.max_rows &&
           (r.n <= len || len == 0);
}
// Reads and checks sequence s (no status).
__device__ __forceinline__ bool kv_seq(const KvView& c, int s, SeqRows& r) {
    return kv_seq_ok(c, c.kv_len[s], c.row_off ? c.row_off[s] : s, c.row_off ? c.row_off[s + 1] : (int64_t)s + 1, r);
}

__device__ __forceinline__ int64_t kv_row(const KvView& c, int64_t r) { return c.row_map ? c.row_map[r] : r; }

// Byte of (token j, dim c) inside a (page, head) tile.
template <int HD>
__device__ __host__ __forceinline__ int kv_byte_k(int j, int c) {
    const int s = HD == 128 ? 4 * (j & 1) : 0;
    return j * HD + (((c >> 4) ^ s) << 4) + (c & 15);
}
template <int HD>
__device__ __host__ __forceinline__ int kv_byte_v(int j, int c) {
    return (j >> 2) * 4 * HD + (((c >> 2) ^ (2 * ((j >> 2) & 3))) << 4) + ((c & 3) << 2) + (j & 3);
}

__device__ __forceinline__ float kv_pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Two e4m3 bytes (the low byte first) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
    return h;
}
// lo and hi rounded to e4m3, to nearest even, lo in the low byte; NaN stays
// NaN, magnitudes above 448 become 448.
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
    uint16_t b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(hi), "f"(lo));
    return b;
}
__device__ __forceinline__ uint32_t float4_to_e4m3x4(float a, float b, float c, float d) {
    return (uint32_t)float2_to_e4m3x2(a, b) | (uint32_t)float2_to_e4m3x2(c, d) << 16;
}
__device__ __forceinline__ void e4m3x4_to_float4(uint32_t w, float (&f)[4]) {
    const uint32_t lo = e4m3x2_to_half2((uint16_t)w), hi = e4m3x2_to_half2((uint16_t)(w >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// four consecutive elements (aligned to their size) from floats
__device__ __forceinline__ void store4_f(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4_f(bf16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// Checks the host can make of a cache and a call's sequences; *out is their
// device view, of sequences of at most max_len tokens.  MLORA_OK or an error code
// with its message set.
int kv_check(const mlora_kv_cache* c, const mlora_kv_seqs* q, int32_t dtype, int64_t max_len, KvView* out);
int kv_fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Whether one launch can hold the calls' blocks (append, read).
bool kv_fits(const KvView& c);

// The operators on checked arguments; the transformer's rollouts call them with a row_map.
cudaError_t launch_kv_append(const KvView& c, int head_dim, int dtype, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, cudaStream_t s);
struct KvAttnArgs {
    const void* q;
    void* out;
    float* lse;
    void* workspace;
    int64_t ldq, ldo, workspace_bytes;
    int n_heads;
    float scale;
};
// launches (may be null) counts the kernels
cudaError_t launch_kv_attention(const KvView& c, int head_dim, int dtype, const KvAttnArgs& a, cudaStream_t s,
                                int64_t* launches);

}  // namespace mlk
