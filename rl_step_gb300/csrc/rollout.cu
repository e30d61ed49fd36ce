// Kernels of the transformer model's rollouts besides the cache operators
// (rollout.cuh): where the rows stand, their sequences' last rows, and the next
// tokens.
#include "rollout.cuh"
#include "sampling.cuh"

namespace mlk {

namespace {

__global__ void __launch_bounds__(256) cached_rows_kernel(KvView c, const int* __restrict__ perm_pad,
                                                          const int* __restrict__ meta, const int* __restrict__ inv,
                                                          int n, int max_rows, int* pos_pad, int* tgt_pad, int* row_map,
                                                          int* status) {
    const int rows = meta[0] * TILE_M;
    const int first = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
    for (int p = first; p < rows; p += step) {
        const int t = perm_pad[p];
        int pos = 0;
        bool live = false;
        if (t >= 0 && c.n_seqs > 0) {
            int s = t;                       // the last sequence whose rows begin at or before t
            bool mine = t < c.n_seqs;
            if (c.row_off) {
                int lo = 0, hi = c.n_seqs - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (c.row_off[mid] <= t) lo = mid; else hi = mid - 1;
                }
                s = lo;
                mine = c.row_off[s] <= t && t < c.row_off[s + 1];
            }
            if (mine) {
                SeqRows q;
                if (!kv_seq(c, s, q)) {
                    raise_status(status, ST_RANGE);
                } else if (q.len > 0) {
                    live = true;
                    pos = q.len - q.n + (t - q.row0);
                }
            }
        }
        pos_pad[p] = pos;
        if (!live) tgt_pad[p] = -1;
    }
    for (int t = first; t < n; t += step) row_map[t] = inv[t] >= 0 ? inv[t] : max_rows - 1;
}

__global__ void __launch_bounds__(128) last_rows_kernel(KvView c, const int* __restrict__ inv,
                                                        const int* __restrict__ tgt_pad, const bf16* __restrict__ xf,
                                                        int d, bf16* __restrict__ x, int* perm, int* tgt, int* meta) {
    const int s = blockIdx.x;
    int row = -1;
    SeqRows q;
    if (s < c.n_seqs && kv_seq(c, s, q) && q.len > 0 && q.n > 0) {
        row = inv[q.row0 + q.n - 1];
        if (row >= 0 && tgt_pad[row] < 0) row = -1;
    }
    if (threadIdx.x == 0) {
        perm[s] = row >= 0 ? s : -1;
        tgt[s] = row >= 0 ? 0 : -1;
        if (s == 0) meta[0] = gridDim.x / TILE_M;
    }
    for (int i = threadIdx.x * 8; i < d; i += blockDim.x * 8)
        *reinterpret_cast<uint4*>(x + (int64_t)s * d + i) =
            row >= 0 ? *reinterpret_cast<const uint4*>(xf + (int64_t)row * d + i) : make_uint4(0, 0, 0, 0);
}

// One block a row.  Every warp finds the tile (the same one: the partials are
// few), forms 32 of its 256 logits, eight dot products at a time so that their
// loads overlap, and warp 0 picks the column.  Reads 512 d bytes of Wout a row,
// against 2 V d for all rows together in the LM head before it.
constexpr int SAMPLE_TILE = 256;
__global__ void __launch_bounds__(256) tf_sample_kernel(const float* __restrict__ part, int n_nt, int part_ld,
                                                        const float* __restrict__ lse_row, const int* __restrict__ perm,
                                                        const bf16* __restrict__ x, const bf16* __restrict__ Wout, int d,
                                                        int V, const float* __restrict__ uniforms, int* next_out,
                                                        float* logprob_out, int* status) {
    __shared__ float z[SAMPLE_TILE];
    const int s = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float u = uniforms[s], lse = lse_row[s];
    const bool ok_u = u >= 0.f && u < 1.f;
    if (!ok_u || perm[s] < 0 || !(fabsf(lse) <= FLT_MAX)) {
        if (threadIdx.x == 0) {
            if (!ok_u) raise_status(status, ST_RANGE);
            next_out[s] = -1;
            logprob_out[s] = __int_as_float(0x7fc00000);
        }
        return;
    }
    float before;
    const int c0 = sample_tile(part + (int64_t)s * part_ld, n_nt, lse, u, lane, before) * SAMPLE_TILE;
    const bf16* xr = x + (int64_t)s * d;
    constexpr int COLS = 8;
    for (int j0 = warp * 32; j0 < warp * 32 + 32; j0 += COLS) {
        float acc[COLS] = {};
        for (int i = lane * 8; i < d; i += 256) {
            float xv[8];
            const uint4 xw = *reinterpret_cast<const uint4*>(xr + i);
            const uint32_t xs[4] = {xw.x, xw.y, xw.z, xw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&xs[e]));
                xv[2 * e] = f.x;
                xv[2 * e + 1] = f.y;
            }
            uint4 w[COLS];
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                w[j] = *reinterpret_cast<const uint4*>(Wout + (int64_t)min(c0 + j0 + j, V - 1) * d + i);
#pragma unroll
            for (int j = 0; j < COLS; ++j) {
                const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e]));
                    acc[j] = fmaf(xv[2 * e], f.x, acc[j]);
                    acc[j] = fmaf(xv[2 * e + 1], f.y, acc[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < COLS; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
            if (lane == 0) z[j0 + j] = acc[j];
        }
    }
    __syncthreads();
    if (warp) return;
    const int pick = sample_column(z, c0, SAMPLE_TILE, V, lse, u, before, lane);
    if (lane == 0) {
        next_out[s] = pick;
        logprob_out[s] = z[pick - c0] - lse;
    }
}

}  // namespace

void launch_tf_cached_rows(const KvView& c, const int* perm_pad, const int* meta, const int* inv, int n,
                           int max_rows, int* pos_pad, int* tgt_pad, int* row_map, int* status, cudaStream_t s) {
    int blocks = (max_rows + 255) / 256;
    if (blocks > 4096) blocks = 4096;
    cached_rows_kernel<<<blocks, 256, 0, s>>>(c, perm_pad, meta, inv, n, max_rows, pos_pad, tgt_pad, row_map,
                                              status);
}

void launch_tf_last_rows(const KvView& c, const int* inv, const int* tgt_pad, const bf16* xf, int d,
                         bf16* x, int* perm, int* tgt, int* meta, cudaStream_t s) {
    const int rows = (c.n_seqs + TILE_M - 1) / TILE_M * TILE_M;
    last_rows_kernel<<<rows, 128, 0, s>>>(c, inv, tgt_pad, xf, d, x, perm, tgt, meta);
}

void launch_tf_sample(const float* part, int n_nt, int part_ld, const float* lse, const int* perm, const bf16* x,
                      const bf16* Wout, int d, int V, const float* uniforms, int n, int* next_out, float* logprob_out,
                      int* status, cudaStream_t s) {
    tf_sample_kernel<<<n, 256, 0, s>>>(part, n_nt, part_ld, lse, perm, x, Wout, d, V, uniforms, next_out, logprob_out,
                                       status);
}

}  // namespace mlk
