// Page tables of the paged cache built on the GPU (include/mlora_kv.h): sequences
// grow by new tokens, whose pages come from a pool's free list, and are cut back,
// which gives pages to it.
//
// What bounds it: latency.  A call moves kilobytes; the floor is a launch and a
// chain of a few dependent reads.  So one block does a call's prefix sums and moves
// its pages, and writes the rows' positions, sequences and slots as well where they
// are few; more rows go to a second launch over all SMs.  256 sequences cut by up to three
// tokens and grown by four: 10 us for both calls; 51 of up to 2,048 tokens given back and
// as many grown: 18 us.
//
// The free list is a stack.  Growing takes pages from its top in the order of the
// sequences and of their pages; cutting back walks both the other way round, so
// that it undoes a growth exactly, and a page's place does not depend on timing.
#include <algorithm>

#include "kv_common.cuh"

namespace mlk {

namespace {

constexpr int ST_NO_PAGES = 4;
constexpr int PT = 1024;                     // most threads
// Sequences of a thread in a pass: SEQS = 1, or 4 where the block has no thread for each (4,043 sequences
// cut and grown: 21 us, 51 with one; 256: 10 us with one, 13 with four).

struct PoolView {
    int* free_pages;
    int* n_free;
    int* owner;
    int* status;
    int n_pages;
};
struct GrowView {
    int* table;
    int* kv_len;
    const int* n_new;
    int* row_off;
    int* positions;
    int* seqs;
    int64_t* slots;
    int64_t n_rows;
    int64_t max_len;                         // what a table's row and kv_len hold
    int n_seqs, max_pages;
};

__device__ __forceinline__ int pages_of(int64_t len) { return (int)((len + KV_PAGE - 1) / KV_PAGE); }

struct Two {
    int64_t a, b;
};
// inclusive prefix sums over the block; *total: of all threads
__device__ __forceinline__ Two block_scan(Two v, Two* total) {
    __shared__ Two part[PT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, v.a, o), b = __shfl_up_sync(0xffffffffu, v.b, o);
        if (lane >= o) v.a += a, v.b += b;
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    // every warp adds up the warps' sums
    Two w = lane < warps ? part[lane] : Two{0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, w.a, o), b = __shfl_up_sync(0xffffffffu, w.b, o);
        if (lane >= o) w.a += a, w.b += b;
    }
    total->a = __shfl_sync(0xffffffffu, w.a, 31);
    total->b = __shfl_sync(0xffffffffu, w.b, 31);
    const int64_t a = __shfl_sync(0xffffffffu, w.a, (warp + 31) & 31), b = __shfl_sync(0xffffffffu, w.b, (warp + 31) & 31);
    if (warp > 0) v.a += a, v.b += b;
    return v;
}

// how many threads before this one have `have`; *total: of the block
__device__ __forceinline__ int block_rank(bool have, int* total) {
    __shared__ int part[PT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t m = __ballot_sync(0xffffffffu, have);
    __syncthreads();
    if (lane == 0) part[warp] = __popc(m);
    __syncthreads();
    const int w = lane < warps ? part[lane] : 0;
    *total = __reduce_add_sync(0xffffffffu, w);
    return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + __popc(m & ((1u << lane) - 1));
}

// the last of first[0 .. n) that is not above x; first[0] <= x
template <typename I>
__device__ __forceinline__ int find(const I* first, int n, int64_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Row r's position, sequence and slot from the lengths and tables as they are after the growth.
__device__ __forceinline__ void write_row(const PoolView& p, const GrowView& g, int64_t r, int64_t total) {
    int pos = -1, s = -1;
    int64_t slot = -1;
    if (r < total) {
        s = find(g.row_off, g.n_seqs, r);
        pos = g.kv_len[s] - (g.row_off[s + 1] - (int)r);
        const int id = g.table[(int64_t)s * g.max_pages + pos / KV_PAGE];
        if (id >= 0) slot = (int64_t)id * KV_PAGE + pos % KV_PAGE;      // (else the list had no page there: raised)
    }
    if (g.positions) g.positions[r] = pos;
    if (g.seqs) g.seqs[r] = s;
    if (g.slots) g.slots[r] = slot;
}

template <int SEQS>
__global__ void __launch_bounds__(PT) reserve_kernel(const __grid_constant__ PoolView p, const __grid_constant__ GrowView g,
                                                     int rows_here) {
    __shared__ int s_first[PT * SEQS];        // new pages before a sequence's own, of this pass (at most the free ones)
    __shared__ int s_have[PT * SEQS];
    const int tid = threadIdx.x, nt = blockDim.x;
    int avail = *p.n_free;
    const bool pool_ok = avail >= 0 && avail <= p.n_pages;
    if (!pool_ok) {
        if (tid == 0) raise_status(p.status, ST_RANGE);
        avail = 0;
    }
    Two want{0, 0}, got{0, 0};                // pages and rows so far: asked for, and served
    for (int base = 0; base < g.n_seqs; base += nt * SEQS) {
        const int s0 = base + tid * SEQS;
        int len[SEQS], add[SEQS], have[SEQS];
        bool ok[SEQS], served[SEQS];
#pragma unroll
        for (int i = 0; i < SEQS; ++i) {
            len[i] = s0 + i < g.n_seqs ? g.kv_len[s0 + i] : 0;
            add[i] = s0 + i < g.n_seqs ? g.n_new[s0 + i] : 0;
        }
        Two mine[SEQS], sum{0, 0};
        int last[SEQS];                       // the page that the first new row goes into,
        bool inside[SEQS];                    // where that page has rows already
#pragma unroll
        for (int i = 0; i < SEQS; ++i) {
            ok[i] = len[i] >= 0 && add[i] >= 0 && (int64_t)len[i] + add[i] <= g.max_len;
            have[i] = ok[i] ? pages_of(len[i]) : 0;
            mine[i] = Two{ok[i] ? pages_of((int64_t)len[i] + add[i]) - have[i] : 0, ok[i] ? add[i] : 0};
            sum.a += mine[i].a, sum.b += mine[i].b;
            inside[i] = mine[i].b > 0 && len[i] % KV_PAGE > 0;
            last[i] = inside[i] ? g.table[(int64_t)(s0 + i) * g.max_pages + len[i] / KV_PAGE] : -1;
        }
        Two all;
        Two upto = block_scan(sum, &all);
        upto.a += want.a - sum.a, upto.b += want.b - sum.b;
#pragma unroll
        for (int i = 0; i < SEQS; ++i) last[i] = last[i] >= 0 && last[i] < p.n_pages ? p.owner[last[i]] : -1;     // whose it is
        Two take{0, 0};
#pragma unroll
        for (int i = 0; i < SEQS; ++i) {
            // A sequence is served if the pages and rows asked for up to it are there; what needs none always is.
            upto.a += mine[i].a, upto.b += mine[i].b;
            const bool pages_ok = mine[i].a == 0 || upto.a <= avail, rows_ok = mine[i].b == 0 || upto.b <= g.n_rows;
            // rows inside a page that is another's, or nobody's, would overwrite what its owner has or gets there
            const bool own = !inside[i] || last[i] == s0 + i;
            served[i] = ok[i] && pages_ok && rows_ok && own;
            if (!served[i]) raise_status(p.status, !ok[i] || !rows_ok || !own ? ST_RANGE : ST_NO_PAGES);
            else take.a += mine[i].a, take.b += mine[i].b;
        }
        Two taken;
        Two before = block_scan(take, &taken);
        before.a -= take.a, before.b -= take.b;
#pragma unroll
        for (int i = 0; i < SEQS; ++i) {
            s_first[tid * SEQS + i] = (int)before.a;
            s_have[tid * SEQS + i] = have[i];
            if (s0 + i < g.n_seqs) {
                g.row_off[s0 + i] = (int)(got.b + before.b);
                if (served[i] && add[i]) g.kv_len[s0 + i] = len[i] + add[i];
            }
            if (served[i]) before.a += mine[i].a, before.b += mine[i].b;
        }
        __syncthreads();
        for (int64_t j = tid; j < taken.a; j += nt) {
            // the last sequence that begins at or before page j: those behind it that take none begin later
            const int q = find(s_first, nt * SEQS, j);
            const int id = p.free_pages[avail - 1 - (got.a + j)];
            const bool good = id >= 0 && id < p.n_pages;
            if (good) p.owner[id] = base + q;
            else raise_status(p.status, ST_RANGE);
            g.table[(int64_t)(base + q) * g.max_pages + s_have[q] + (j - s_first[q])] = good ? id : -1;
        }
        want.a += all.a, want.b += all.b;
        got.a += taken.a, got.b += taken.b;
        __syncthreads();
    }
    if (tid == 0) {
        g.row_off[g.n_seqs] = (int)got.b;
        if (pool_ok) *p.n_free = (int)(avail - got.a);
    }
    if (!rows_here) return;
    __syncthreads();
    for (int64_t r = tid; r < g.n_rows; r += nt) write_row(p, g, r, got.b);
}

__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ PoolView p,
                                                     const __grid_constant__ GrowView g) {
    const int64_t total = g.row_off[g.n_seqs], step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < g.n_rows; r += step) write_row(p, g, r, total);
}

// Sequences and their pages from the last to the first; a page goes to the list if
// the row of the table owns it.
template <int SEQS>
__global__ void __launch_bounds__(PT) release_kernel(const __grid_constant__ PoolView p, int* table, int* kv_len,
                                                     const int* __restrict__ keep, int n_seqs, int max_pages) {
    __shared__ int64_t s_first[PT * SEQS];    // (pages that many rows share count for each of them)
    const int tid = threadIdx.x, nt = blockDim.x;
    int64_t top = *p.n_free;
    if (top < 0 || top > p.n_pages) {
        if (tid == 0) raise_status(p.status, ST_RANGE);
        return;                               // (the whole block: all read the same number)
    }
    for (int base = 0; base < n_seqs; base += nt * SEQS) {
        const int s0 = n_seqs - 1 - (base + tid * SEQS);                // and downwards
        int len[SEQS], left[SEQS];
#pragma unroll
        for (int i = 0; i < SEQS; ++i) {
            len[i] = s0 - i >= 0 ? kv_len[s0 - i] : 0;
            left[i] = s0 - i >= 0 && keep ? keep[s0 - i] : 0;
        }
        int64_t count[SEQS], sum = 0;
#pragma unroll
        for (int i = 0; i < SEQS; ++i) {
            const bool ok = len[i] >= 0 && len[i] <= (int64_t)max_pages * KV_PAGE && left[i] >= 0;
            if (!ok) raise_status(p.status, ST_RANGE);
            if (!ok || left[i] > len[i]) left[i] = len[i];
            count[i] = pages_of(len[i]) - pages_of(left[i]);
            sum += count[i];
        }
        Two all;
        int64_t at = block_scan(Two{sum, 0}, &all).a - sum;
#pragma unroll
        for (int i = 0; i < SEQS; ++i) {
            s_first[tid * SEQS + i] = at;
            at += count[i];
        }
        __syncthreads();
        for (int64_t j0 = 0; j0 < all.a; j0 += nt) {
            const int64_t j = j0 + tid;
            int id = -1;
            bool mine_too = false;
            if (j < all.a) {
                const int q = find(s_first, nt * SEQS, j), seq = n_seqs - 1 - (base + q);
                int* entry = table + (int64_t)seq * max_pages + pages_of(kv_len[seq]) - 1 - (j - s_first[q]);
                id = *entry;
                *entry = -1;
                if (id < 0 || id >= p.n_pages) raise_status(p.status, ST_RANGE);
                else mine_too = atomicCAS(p.owner + id, seq, -1) == seq;
            }
            int n = 0;
            const int64_t to = top + block_rank(mine_too, &n);
            if (mine_too) {
                if (to < p.n_pages) p.free_pages[to] = id;
                else raise_status(p.status, ST_RANGE);
            }
            top = top + n < p.n_pages ? top + n : p.n_pages;
        }
        __syncthreads();                      // the lengths until here are the old ones
#pragma unroll
        for (int i = 0; i < SEQS; ++i)
            if (left[i] != len[i]) kv_len[s0 - i] = left[i];
    }
    if (tid == 0) *p.n_free = (int)top;
}

int pool_check(const mlora_kv_pool* p, const int32_t* table, const int32_t* kv_len, int n_seqs, int max_pages, PoolView* v) {
    if (!p) return kv_fail(MLORA_E_ARG, "NULL pool");
    if (p->n_pages < 1) return kv_fail(MLORA_E_ARG, "a pool of %d pages", p->n_pages);
    if (!p->free_pages || !p->n_free || !p->owner) return kv_fail(MLORA_E_ARG, "NULL pool arrays");
    if (n_seqs < 0 || n_seqs > INT32_MAX - 8 * PT) return kv_fail(MLORA_E_ARG, "%d sequences", n_seqs);
    if (max_pages < 1) return kv_fail(MLORA_E_ARG, "page tables of %d pages", max_pages);
    if (n_seqs > 0 && (!table || !kv_len)) return kv_fail(MLORA_E_ARG, "NULL page table or lengths");
    *v = PoolView{p->free_pages, p->n_free, p->owner, p->status, p->n_pages};
    return MLORA_OK;
}

// threads of the one block
int block_for(int64_t n) { return n <= 256 ? 256 : n <= 512 ? 512 : PT; }

}  // namespace

}  // namespace mlk

using namespace mlk;

extern "C" int mlora_kv_reserve(const mlora_kv_pool* p, const mlora_kv_growth* q, void* stream) {
    if (!q) return kv_fail(MLORA_E_ARG, "NULL growth");
    PoolView v;
    const int rc = pool_check(p, q->page_table, q->kv_len, q->n_seqs, q->max_pages, &v);
    if (rc) return rc;
    if (q->n_rows < 0 || q->n_rows > INT32_MAX) return kv_fail(MLORA_E_ARG, "%lld rows", (long long)q->n_rows);
    if (!q->row_off || (q->n_seqs > 0 && !q->n_new)) return kv_fail(MLORA_E_ARG, "NULL numbers of new rows or row offsets");
    const GrowView g{q->page_table, q->kv_len, q->n_new, q->row_off, q->positions, q->seqs, q->slots, q->n_rows,
                     q->max_pages < INT32_MAX / KV_PAGE ? (int64_t)q->max_pages * KV_PAGE : INT32_MAX, q->n_seqs, q->max_pages};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool rows = q->n_rows > 0 && (q->positions || q->seqs || q->slots);
    const bool apart = rows && q->n_rows > 2 * PT;
    const int block = block_for(std::max(q->n_seqs, (int)(rows && !apart ? q->n_rows : 0)));
    (q->n_seqs <= PT ? reserve_kernel<1> : reserve_kernel<4>)<<<1, block, 0, s>>>(v, g, rows && !apart);
    if (apart) {
        const int64_t blocks = (q->n_rows + 255) / 256;
        rows_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(v, g);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "reserve launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}

extern "C" int mlora_kv_release(const mlora_kv_pool* p, int32_t* page_table, int32_t* kv_len, const int32_t* keep,
                                int32_t n_seqs, int32_t max_pages, void* stream) {
    PoolView v;
    const int rc = pool_check(p, page_table, kv_len, n_seqs, max_pages, &v);
    if (rc) return rc;
    if (n_seqs == 0) return MLORA_OK;
    (n_seqs <= PT ? release_kernel<1> : release_kernel<4>)<<<1, block_for(n_seqs), 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        v, page_table, kv_len, keep, n_seqs, max_pages);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "release launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}
