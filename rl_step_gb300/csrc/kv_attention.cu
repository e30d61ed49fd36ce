// Attention of a call's newest rows over the 8-bit key/value cache
// (include/mlora_kv.h): for each row and query head, one pass over the cached
// positions with a running maximum and sum,
//     s_i = scale q . k_i,  out = sum_i exp(s_i - lse) v_i,  lse = log sum_i exp(s_i).
#include "kv_common.cuh"

namespace mlk {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// One block per (sequence, row, query head); four warps take every fourth
// position, a lane holds HD / 32 dims; the warps' results are merged at the end.
template <typename T, int HD>
__global__ void __launch_bounds__(128) kv_attn_simple_kernel(const __grid_constant__ KvView c,
                                                             const T* __restrict__ q, int64_t ldq,
                                                             T* __restrict__ out, int64_t ldo,
                                                             float* __restrict__ lse, int64_t max_len, int n_heads,
                                                             float scale) {
    constexpr int D = HD / 32;
    __shared__ float sm[4], sl[4], so[4][HD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t u = blockIdx.x;
    const int head = (int)(u % n_heads);
    u /= n_heads;
    const int i = (int)(u % c.max_rows), s = (int)(u / c.max_rows);
    SeqRows r;
    bool ok = kv_seq(c, s, max_len, r);
    const int64_t r0 = r.row0 < 0 ? 0 : r.row0;
    if (!ok) {
        // rows of a bad sequence that exist get NaN (from the block of its row 0)
        if (i == 0)
            for (int64_t x = r0; x < (int64_t)r.row0 + r.n && x < c.n_rows; ++x) {
                const int64_t y = kv_row(c, x);
                for (int d = threadIdx.x; d < HD; d += 128) out[y * ldo + head * HD + d] = from_f<T>(NAN);
                if (lse && threadIdx.x == 0) lse[y * n_heads + head] = NAN;
            }
        return;
    }
    if (i >= r.n) return;
    const int64_t row = kv_row(c, (int64_t)r.row0 + i);
    const int n = r.len ? r.len - r.n + i + 1 : 0;          // positions this row sees
    const int h = head / (n_heads / c.n_kv);
    float qv[D], o[D], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < D; ++d) {
        qv[d] = to_f(q[row * ldq + head * HD + lane * D + d]) * (scale * LOG2E);
        o[d] = 0.f;
    }
    for (int p = warp; p < n; p += 4) {
        const int id = kv_page(c, s, p / KV_PAGE);
        if (id < 0) { ok = false; continue; }
        const int64_t t = (int64_t)id * c.n_kv + h;
        const uint8_t* kt = c.k + t * (KV_PAGE * HD);
        const uint8_t* vt = c.v + t * (KV_PAGE * HD);
        const int j = p % KV_PAGE;
        float z = 0.f;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            float f[4];
            e4m3x4_to_float4(kt[kv_byte_k<HD>(j, lane * D + d)], f);
            z += qv[d] * f[0];
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
        z *= c.ks[t];
        const float mn = fmaxf(m, z);
        const float a = mn == -INFINITY ? 0.f : mn;
        const float f0 = exp2f(m - a), w = exp2f(z - a), wv = w * c.vs[t];
        l = l * f0 + w;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            float f[4];
            e4m3x4_to_float4(vt[kv_byte_v<HD>(j, lane * D + d)], f);
            o[d] = o[d] * f0 + wv * f[0];
        }
        m = mn;
    }
    if (!ok) l = NAN;
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
    for (int d = 0; d < D; ++d) so[warp][lane * D + d] = o[d];
    __syncthreads();
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const float A = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int w = 0; w < 4; ++w) L += sl[w] * exp2f(sm[w] - A);
    for (int d = threadIdx.x; d < HD; d += 128) {
        float x = 0.f;
        for (int w = 0; w < 4; ++w) x += so[w][d] * exp2f(sm[w] - A);
        out[row * ldo + head * HD + d] = from_f<T>(n ? x / L : 0.f);
    }
    if (lse && threadIdx.x == 0) lse[row * n_heads + head] = n ? (A + log2f(L)) * LN2 : -INFINITY;
}

template <typename T, int HD>
void attn_t(const KvView& c, const KvAttnArgs& a, cudaStream_t s) {
    const int64_t blocks = (int64_t)c.n_seqs * c.max_rows * a.n_heads;
    kv_attn_simple_kernel<T, HD><<<(unsigned)blocks, 128, 0, s>>>(c, static_cast<const T*>(a.q), a.ldq,
                                                                  static_cast<T*>(a.out), a.ldo, a.lse, a.max_len,
                                                                  a.n_heads, a.scale);
}

}  // namespace

cudaError_t launch_kv_attention(const KvView& c, int head_dim, int dtype, const KvAttnArgs& a, cudaStream_t s) {
    if (dtype == MLORA_BF16) (head_dim == 64 ? attn_t<bf16, 64> : attn_t<bf16, 128>)(c, a, s);
    else (head_dim == 64 ? attn_t<float, 64> : attn_t<float, 128>)(c, a, s);
    return cudaGetLastError();
}

}  // namespace mlk

using namespace mlk;

extern "C" int mlora_kv_attention(const mlora_kv_cache* c, const mlora_kv_seqs* q, const mlora_kv_attn* a,
                                  void* stream) {
    if (!a) return kv_fail(MLORA_E_ARG, "NULL attention arguments");
    KvView w;
    const int rc = kv_check(c, q, a->dtype, &w);
    if (rc) return rc;
    if (a->n_heads < 1 || a->n_heads > 65536 || a->n_heads % c->n_kv_heads)
        return kv_fail(MLORA_E_ARG, "n_heads %d must be a positive multiple of n_kv_heads (%d)", a->n_heads,
                       c->n_kv_heads);
    if (!(fabsf(a->scale) <= FLT_MAX)) return kv_fail(MLORA_E_ARG, "scale is not finite");
    if (a->max_len < 0) return kv_fail(MLORA_E_ARG, "max_len %lld < 0", (long long)a->max_len);
    if (w.n_seqs == 0 || w.n_rows == 0 || w.max_rows == 0) return MLORA_OK;
    const int64_t row = (int64_t)a->n_heads * c->head_dim;
    const int64_t per16 = a->dtype == MLORA_BF16 ? 8 : 4;
    if (!a->q || !a->out) return kv_fail(MLORA_E_ARG, "NULL queries or output");
    if (a->q_stride < row || a->out_stride < row || a->q_stride % per16 || a->out_stride % per16 ||
        ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out)) & 15))
        return kv_fail(MLORA_E_ARG, "query and output rows must be 16-byte aligned and at least %lld elements apart",
                       (long long)row);
    if (!a->workspace || (reinterpret_cast<uintptr_t>(a->workspace) & 15) ||
        a->workspace_bytes < MLORA_KV_COUNTER_BYTES)
        return kv_fail(MLORA_E_ARG, "the workspace must be 16-byte aligned and hold at least %d bytes",
                       MLORA_KV_COUNTER_BYTES);
    if ((int64_t)w.max_rows * a->n_heads > INT32_MAX / w.n_seqs)
        return kv_fail(MLORA_E_ARG, "too many sequences, rows and heads for one call");
    KvAttnArgs k;
    k.q = a->q; k.out = a->out; k.lse = a->lse; k.workspace = a->workspace; k.ldq = a->q_stride; k.ldo = a->out_stride;
    k.workspace_bytes = a->workspace_bytes; k.max_len = a->max_len; k.n_heads = a->n_heads; k.scale = a->scale;
    const cudaError_t e = launch_kv_attention(w, c->head_dim, a->dtype, k, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}
