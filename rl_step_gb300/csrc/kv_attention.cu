// Attention of a call's newest rows over the 8-bit key/value cache
// (include/mlora_kv.h): for each row and query head, one pass over the cached
// positions with a running maximum and sum,
//     s_i = scale q . k_i,  out = sum_i exp(s_i - lse) v_i,  lse = log sum_i exp(s_i).
//
// What bounds it.  Few rows a sequence: every cached byte is read once and used
// for rows x group products, far below the tensor cores' rate, so the cache's
// bytes over the HBM rate are the floor.  The design streams pages and keeps
// the arithmetic beside the stream cheap:
//  * A work item is up to 8 NT RG (row, head of the group) pairs of a sequence
//    against one key/value head, over a run of pages.  Blocks are persistent and
//    take items from a counter; a producer warp copies each (page, head) tile of
//    K and V -- contiguous 8 KB at head_dim 128 -- into a ring of stages with
//    cp.async.bulk and runs ahead into the next item (its length, table, queries
//    and first pages) while the consumer warps finish the current one.
//  * The products are mma.sync m16n8k16 (fp16 operands, fp32 sums) with the
//    cache's bytes as the 16-row operand and the pairs as the 8 columns:
//    S^T = K q^T (16 tokens x 8 pairs), O^T += V^T P^T (16 dims x 8 pairs).  An
//    e4m3 byte is exactly an fp16 value and two bytes convert in one
//    instruction; 8 columns fit the few pairs of a decode step (with the pairs
//    as 16 rows it took twice the products, exponentials and registers), where
//    a 128-row tcgen05 tile would be at most a sixteenth full and would want
//    the converted tile written back to shared memory first.  The page's byte
//    order (mlora_kv.h) puts each thread's fragment bytes side by side, and one
//    8 x 8 transposition turns the score tile into the second product's operand.
//  * q enters as fp16 relative to its row's largest magnitude (a power of two,
//    folded into the scale): exact for bf16 down to 2^-17 of that magnitude.
//    On fp32 the 8 columns are 4 pairs, each with its high and its low fp16
//    part (2^-22): both products come out of one instruction, in one thread.
//  * The page's value scale 2^ev goes into the exponent of the probability,
//    p' = exp2(s log2 e + ev - m') with m' the running maximum of s log2 e + ev,
//    so pages of any scale add into one accumulator, the largest p' v8 sets the
//    precision, and l += p' 2^-ev is what the definition sums.  m' follows the
//    scores only when one passes it by 2^3 (the sums are then rescaled); p' is
//    held at 2^12 times its value, so that it stays within fp16 and its rounding
//    relative (2^-11) down to 2^-26 of the reference (absolute 2^-37 of it
//    below that); on fp32 it is split like q.
//  * Warps of a row group take different halves of a page and, with one or two
//    row groups, every other page, 32 tokens at a step; each has a running maximum and sum of its own, joined at the
//    item's end, so nothing but the ring's barriers is shared in the loop.
//  * Long sequences are cut into runs of pages (flash-style split); an item
//    leaves its rows' unnormalised sums, maximum and sum in the workspace, and
//    the last item of the sequence and head to arrive joins them in order of
//    the runs, so the result does not depend on who was last.
#include <atomic>
#include <type_traits>

#include "kv_common.cuh"
#include "tc_ptx.cuh"

namespace mlk {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr int P_SHIFT = 12;                 // p' is held at 2^12 times its value,
constexpr float M_SLACK = 3.f;              // against a reference at most 2^3 below the largest: p' <= 2^15
// Runs of pages of a split (see attn_t).
constexpr int KV_LONG_RUN = 64, KV_SHORT_RUN = 2, KV_ITEMS_BLOCK = 1;
// The workspace's counters: the next item, finished blocks, then one for each unit.
constexpr int CTR_NEXT = 0, CTR_DONE = 1, CTR_UNITS = 16;

struct AttnCall {
    const void* q;
    void* out;
    float* lse;
    int* counters;
    float* part;
    int64_t ldq, ldo, max_len;
    int n_heads, group;
    int items;                              // units * splits
    int tiles;                              // row tiles of a (sequence, key/value head)
    int splits, chunk;                      // runs of `chunk` pages
    int prow;                               // rows of a partial result
    int64_t slot;                           // its floats: the rows' sums, maxima and sums of p
    float qk;                               // scale * log2 e
};

// What the producer tells the consumers about an item.
struct Item {
    int index;                              // -1: no more
    int s, h;
    int row0;                               // the sequence's first row
    int pair0, pairs;                       // first pair of the tile, pairs in it
    int before;                             // positions before the sequence's rows
    int page0, np;                          // the run
    int unit, nsplit;
};

template <typename T, int HD, int NT, int RG>
struct AttnShape {
    static constexpr bool FOLD = sizeof(T) == 4;            // a pair takes two columns: its high and its low part
    static constexpr int PR = (FOLD ? 4 : 8) * NT;          // pairs of a row group
    static constexpr int ROWS = PR * RG;
    static constexpr int PG = RG == 1 ? 2 : 1;              // pages in work at once
    static constexpr int WG = 2 * PG;                       // warps of a row group: page parity x half of the page
    static constexpr int NW = RG * WG;                      // consumer warps
    static constexpr int THREADS = 32 * NW + 32;
    static constexpr int TILE = KV_PAGE * HD;               // bytes of a K or V tile
    static constexpr int STAGE = 2 * TILE;
    static constexpr int STAGES = (NT == 1 ? 4 : 6) * (128 / HD);
    static constexpr int BLOCKS_SM = NW > 4 ? 1 : (NT == 1 ? 3 : 2);
    static constexpr int JOIN_WG = 2048 * PG;               // joining space of a row group, bytes
    // ring, raw queries, joining space, per-warp statistics, barriers,
    // exponents, items, flags
    static constexpr int QRAW = STAGES * STAGE;
    static constexpr int JOIN = QRAW + ROWS * HD * (int)sizeof(T);
    static constexpr int STAT = JOIN + RG * JOIN_WG;
    static constexpr int BAR = STAT + 8 * WG * ROWS;
    static constexpr int EXPS = BAR + 16 * STAGES + 64;
    static constexpr int ITEMS = EXPS + 8 * STAGES;
    static constexpr int FLAGS = ITEMS + 2 * 64;
    static constexpr int SMEM = FLAGS + 16;
    static_assert(sizeof(Item) <= 64, "item slots");
    static_assert(BAR % 16 == 0 && QRAW % 16 == 0, "alignment");
    static_assert(STAGES % PG == 0, "a stage belongs to one page parity: its phases are all waited for by the same warps");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// what rounding (a, b) to fp16 left
__device__ __forceinline__ uint32_t half2_rest(float a, float b, uint32_t hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return half2_bits(a - f.x, b - f.y);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ int scale_exp(float s) {
    const int e = (int)((__float_as_uint(s) >> 23) & 255u) - 127;
    return e < KV_MIN_EXP ? KV_MIN_EXP : (e > KV_MAX_EXP ? KV_MAX_EXP : e);
}
// the 8 x 8 matrix of 16-bit values that a warp holds (row g, columns 2 t and 2 t + 1), transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// a value as its fp16 rounding (low half) and the fp16 rounding of the rest
__device__ __forceinline__ uint32_t high_low(float v) {
    const __half h = __float2half_rn(v);
    const __half2 r = __halves2half2(h, __float2half_rn(v - __half2float(h)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
constexpr int EV_BAD = 1 << 20;              // in place of an exponent: a bad page in the run
// 2^e with e clamped to the normal range
__device__ __forceinline__ float pow2_clamped(int e) { return kv_pow2(e < -126 ? -126 : (e > 127 ? 127 : e)); }

// 16 consecutive elements
__device__ __forceinline__ void load16_f(const float* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
    }
}
__device__ __forceinline__ void load16_f(const bf16* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 w = reinterpret_cast<const uint4*>(p)[i];
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[e]));
            v[8 * i + 2 * e] = f.x;
            v[8 * i + 2 * e + 1] = f.y;
        }
    }
}

template <typename T, int HD, int NT, int RG>
__global__ void __launch_bounds__(AttnShape<T, HD, NT, RG>::THREADS, AttnShape<T, HD, NT, RG>::BLOCKS_SM)
    kv_attn_kernel(const __grid_constant__ KvView c, const __grid_constant__ AttnCall a) {
    using S = AttnShape<T, HD, NT, RG>;
    constexpr bool FOLD = S::FOLD;
    constexpr int E = FOLD ? 1 : 2;                         // pairs of a thread in an 8-column tile
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = tcx::smem_u32(smem);
    int* exps = reinterpret_cast<int*>(smem + S::EXPS);     // per stage: K's and V's exponent
    float* st_m = reinterpret_cast<float*>(smem + S::STAT); // [WG][ROWS]
    float* st_l = st_m + S::WG * S::ROWS;
    Item* items = reinterpret_cast<Item*>(smem + S::ITEMS);
    volatile int* flags = reinterpret_cast<volatile int*>(smem + S::FLAGS);   // abort, -, last, -
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full = [&](int i) { return sbase + S::BAR + 16 * i; };
    auto empty = [&](int i) { return sbase + S::BAR + 16 * i + 8; };
    auto item_full = [&](int i) { return sbase + S::BAR + 16 * S::STAGES + 8 * i; };
    auto item_empty = [&](int i) { return sbase + S::BAR + 16 * S::STAGES + 16 + 8 * i; };
    const uint32_t q_full = sbase + S::BAR + 16 * S::STAGES + 32, q_empty = q_full + 8;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            tcx::mbar_init(full(i), 1);
            tcx::mbar_init(empty(i), S::NW / S::PG);
        }
        for (int i = 0; i < 2; ++i) {
            tcx::mbar_init(item_full(i), 1);
            tcx::mbar_init(item_empty(i), S::NW);
        }
        tcx::mbar_init(q_full, 1);
        tcx::mbar_init(q_empty, S::NW);
        flags[0] = flags[1] = flags[2] = flags[3] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    if (warp == S::NW) {
        // ---- producer
        const T* q = static_cast<const T*>(a.q);
        T* out = static_cast<T*>(a.out);
        // a bounded wait of lane 0 that the warp follows
        auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
            int ok = 1;
            if (lane == 0 && !tcx::mbar_wait(bar, parity, flags)) {
                ok = 0;
                raise_status(c.status, ST_TIMEOUT);
                flags[0] = 1;
            }
            return __shfl_sync(0xffffffffu, ok, 0) != 0;
        };
        Item x = {};                                        // the same in every lane
        // lane i: the next 32 pages' tiles and exponents, asked for a batch ahead
        int64_t at = 0;
        int ek = 0, ev = 0;
        // (no branch: the vote and the loads are every lane's)
        auto load_batch = [&](int i0) {
            const int mine = i0 + lane;
            const int64_t entry = (int64_t)x.s * c.max_pages + x.page0 + (mine < x.np ? mine : 0);
            const int id = c.table[entry];
            const bool good = id >= 0 && id < c.n_pages;
            const unsigned bad = __ballot_sync(0xffffffffu, !good);
            at = (int64_t)(good ? id : 0) * c.n_kv + x.h;   // a page that exists stands in; the rows become NaN
            ek = scale_exp(c.ks[at]);
            ev = bad != 0 ? EV_BAD : scale_exp(c.vs[at]);
            if (bad != 0 && lane == 0) raise_status(c.status, ST_RANGE);
            __syncwarp();
        };
        int after = 0;                                      // lane 0: the counter's answer for the item after the next
        auto ask = [&]() {
            if (lane == 0) after = atomicAdd(a.counters + CTR_NEXT, 1);
            __syncwarp();
        };
        // From item `index` on, the first one with work; empty and bad sequences' rows are written on the way.
        auto find = [&](int index) {
            for (;; ) {
                if ((unsigned)index >= (unsigned)a.items) { // (whatever stands in the workspace)
                    x.index = -1;
                    return;
                }
                const int split = index % a.splits;
                x.index = index;
                x.unit = index / a.splits;
                const int tile = x.unit % a.tiles;
                x.h = x.unit / a.tiles % c.n_kv;
                x.s = x.unit / a.tiles / c.n_kv;
                x.page0 = split * a.chunk;
                SeqRows r;
                const bool ok = kv_seq(c, x.s, a.max_len, r);
                if (!ok || r.len == 0) {
                    // rows without positions: zero (or NaN: a bad sequence), by one item of each head
                    if (split == 0 && tile == 0) {
                        const float v = ok ? 0.f : NAN;
                        const int64_t r1 = (int64_t)r.row0 + r.n < c.n_rows ? (int64_t)r.row0 + r.n : c.n_rows;
                        for (int64_t y = r.row0 < 0 ? 0 : r.row0; y < r1; ++y) {
                            const int64_t z = kv_row(c, y);
                            for (int d = lane; d < a.group * HD; d += 32)
                                out[z * a.ldo + (int64_t)x.h * a.group * HD + d] = from_f<T>(v);
                            for (int d = lane; a.lse && d < a.group; d += 32)
                                a.lse[z * a.n_heads + x.h * a.group + d] = ok ? -INFINITY : NAN;
                        }
                    }
                } else {
                    x.pair0 = tile * S::ROWS;
                    x.pairs = r.n * a.group - x.pair0;
                    if (x.pairs > S::ROWS) x.pairs = S::ROWS;
                    if (x.pairs > 0) {
                        x.row0 = r.row0;
                        x.before = r.len - r.n;
                        // positions that the tile's last row sees
                        const int lim = x.before + (x.pair0 + x.pairs - 1) / a.group + 1;
                        const int pages = (lim + KV_PAGE - 1) / KV_PAGE;
                        x.nsplit = (pages + a.chunk - 1) / a.chunk;
                        x.np = pages - x.page0 < a.chunk ? pages - x.page0 : a.chunk;
                        if (x.np > 0) return;
                    }
                }
                index = gridDim.x + __shfl_sync(0xffffffffu, after, 0);
                ask();
            }
        };
        ask();
        find(blockIdx.x);
        if (x.index >= 0) load_batch(0);
        int cnt = 0, n_item = 0;                            // pages and items so far
        bool go = true;
        while (go) {
            const int slot = n_item & 1;
            if (n_item >= 2 && !wait(item_empty(slot), (n_item / 2 - 1) & 1)) break;
            if (lane == 0) {
                items[slot] = x;
                tcx::mbar_arrive(item_full(slot));
            }
            if (x.index < 0) break;
            // the queries: the pairs of a token are contiguous
            if (n_item >= 1 && !wait(q_empty, (n_item - 1) & 1)) break;
            if (lane == 0) tcx::mbar_expect_tx(q_full, x.pairs * HD * (int)sizeof(T));
            __syncwarp();
            for (int tok = x.pair0 / a.group + lane; tok * a.group < x.pair0 + x.pairs; tok += 32) {
                const int p0 = tok * a.group > x.pair0 ? tok * a.group : x.pair0;
                const int p1 = (tok + 1) * a.group < x.pair0 + x.pairs ? (tok + 1) * a.group : x.pair0 + x.pairs;
                bulk_load(sbase + S::QRAW + (p0 - x.pair0) * HD * (int)sizeof(T),
                          q + kv_row(c, (int64_t)x.row0 + tok) * a.ldq + ((int64_t)x.h * a.group + p0 - tok * a.group) * HD,
                          (p1 - p0) * HD * (int)sizeof(T), q_full);
            }
            const int lim = x.before + (x.pair0 + x.pairs - 1) / a.group + 1;
            const int np = x.np, page0 = x.page0;
            for (int i0 = 0; i0 < np && go; i0 += 32) {
                const int64_t at_now = at;
                const int ek_now = ek, ev_now = ev;
                const int n = np - i0 < 32 ? np - i0 : 32;
                for (int i = 0; i < n; ++i) {
                    const int stage = cnt % S::STAGES;
                    const int64_t tile_at = __shfl_sync(0xffffffffu, at_now, i);
                    const int k_ = __shfl_sync(0xffffffffu, ek_now, i), v_ = __shfl_sync(0xffffffffu, ev_now, i);
                    if (cnt >= S::STAGES && !wait(empty(stage), (cnt / S::STAGES - 1) & 1)) {
                        go = false;
                        break;
                    }
                    if (lane == 0) {
                        const int left = lim - (page0 + i0 + i) * KV_PAGE;      // tokens of the page that count
                        const int tok = left < KV_PAGE ? left : KV_PAGE;
                        const uint32_t kb = tok * HD, vb = (tok + 3) / 4 * 4 * HD;
                        exps[2 * stage] = k_;
                        exps[2 * stage + 1] = v_;
                        tcx::mbar_expect_tx(full(stage), kb + vb);
                        bulk_load(sbase + stage * S::STAGE, c.k + tile_at * S::TILE, kb, full(stage));
                        bulk_load(sbase + stage * S::STAGE + S::TILE, c.v + tile_at * S::TILE, vb, full(stage));
                    }
                    ++cnt;
                    // the ring is full, or the batch's pages are on their way: look for what comes next
                    if (i + 1 == (n < S::STAGES ? n : S::STAGES)) {
                        if (i0 + 32 < np) {
                            load_batch(i0 + 32);
                        } else {
                            const int next = gridDim.x + __shfl_sync(0xffffffffu, after, 0);
                            ask();
                            find(next);
                            if (x.index >= 0) load_batch(0);
                        }
                    }
                }
            }
            ++n_item;
        }
        // the counter's last answer is here before the block counts as finished
        asm volatile("" ::"r"(after));
        __threadfence();
    } else {
        const int g = lane >> 2, t = lane & 3;
        const int rg = warp / S::WG, wg = warp % S::WG;     // row group, place in it
        const int half = wg & 1, pg = wg >> 1;              // half of a page, page parity
        // barriers of the consumers; any(): whether one of them says so, the same in all
        auto sync_all = [&]() {
            __syncwarp();
            asm volatile("bar.sync 1, %0;" ::"n"(32 * S::NW) : "memory");
        };
        auto any = [&](bool y) {
            uint32_t r;
            __syncwarp();
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\t"
                "selp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"((uint32_t)y), "n"(32 * S::NW)
                : "memory");
            return r != 0;
        };
        // every lane's wait, or none's: the warp stays together
        auto await = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, tcx::mbar_wait(bar, parity, flags));
        };
        auto gave_up = [&]() {
            if (lane == 0) {
                raise_status(c.status, ST_TIMEOUT);
                flags[0] = 1;
            }
        };
        // this thread's bytes inside a page: keys 16 t .. of token 4 (g / 2) + g % 2
        // (dims 0.. and 64..), values 4 g .. of token quad t
        const uint32_t k_at[2] = {(uint32_t)kv_byte_k<HD>(32 * half + 4 * (g >> 1) + (g & 1), 16 * t),
                                  (uint32_t)kv_byte_k<HD>(32 * half + 4 * (g >> 1) + (g & 1), HD - 64 + 16 * t)};
        const uint32_t v_at = S::TILE + (8 * half + t) * 4 * HD + ((g ^ (2 * t)) << 4);
        T* out = static_cast<T*>(a.out);
        int cnt = 0;                                        // pages so far
        for (int n_item = 0;; ++n_item) {
            // a wait that gives up ends the loop in every consumer at the next any()
            bool go = await(item_full(n_item & 1), (n_item / 2) & 1);
            if (!go) gave_up();
            if (any(!go)) break;
            const Item& x = items[n_item & 1];
            if (x.index < 0) break;
            const int np = x.np, page0 = x.page0;
            const int lim_lo = x.before + x.pair0 / a.group + 1;                        // positions that the tile's first row sees
            const int lim_hi = x.before + (x.pair0 + x.pairs - 1) / a.group + 1;        // .. and its last
            // q's fragments: columns g of the tiles.  A thread's dims at K step
            // (y, i) are 64 y + 16 t + 4 i + 0..3, the four bytes of a word of the
            // key tile.
            if (go) go = await(q_full, n_item & 1);
            if (!go) gave_up();
            uint32_t qb[NT][HD / 16][2];
            float o[HD / 16][NT][4];
            float m[NT][E], l[NT][E], qf[NT][E];            // qf: scale * log2 e, or NaN where q is not finite
            int qe[NT][E], limit[NT][E];                    // exponent of the row's largest |q|; positions it sees
            bool bad = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = rg * S::PR + (FOLD ? 4 * n + (g >> 1) : 8 * n + g);
                const bool live = row < x.pairs;
                const T* src = reinterpret_cast<const T*>(smem + S::QRAW) + row * HD + 16 * t;
                float v[HD / 64][16];
                float big = 0.f;
                bool fin = true;
#pragma unroll
                for (int y = 0; y < HD / 64; ++y) {
                    if (live) {
                        load16_f(src + 64 * y, v[y]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[y][i] = 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        big = fmaxf(big, fabsf(v[y][i]));
                        fin &= fabsf(v[y][i]) <= FLT_MAX;
                    }
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const unsigned nf = __ballot_sync(0xffffffffu, !fin);
                int ex = 0;
                if (big > 0.f && big <= FLT_MAX) frexpf(big, &ex);
                const float f = (nf >> (lane & 28)) & 15u ? NAN : a.qk;
                // 2^-ex in two steps: it can lie outside fp32
                const float f1 = kv_pow2(-ex / 2), f2 = kv_pow2(-ex - (-ex / 2));
#pragma unroll
                for (int y = 0; y < HD / 64; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const float u = v[y][4 * i + 2 * z] * f1 * f2, w = v[y][4 * i + 2 * z + 1] * f1 * f2;
                            const uint32_t hi = half2_bits(u, w);
                            qb[n][4 * y + i][z] = FOLD && (g & 1) ? half2_rest(u, w, hi) : hi;
                        }
                // this thread's scores are those of columns 2 t and 2 t + 1
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int from = 4 * (2 * t + e);
                    const int r2 = rg * S::PR + (FOLD ? 4 * n + t : 8 * n + 2 * t + e);
                    qe[n][e] = __shfl_sync(0xffffffffu, ex, from);
                    qf[n][e] = __shfl_sync(0xffffffffu, f, from);
                    limit[n][e] = r2 < x.pairs ? x.before + (x.pair0 + r2) / a.group + 1 : 0;
                    m[n][e] = -INFINITY;
                    l[n][e] = 0.f;
                }
            }
            __syncwarp();
            if (lane == 0) tcx::mbar_arrive(q_empty);
#pragma unroll
            for (int j = 0; j < HD / 16; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;

            for (int it = S::PG == 2 ? (cnt ^ pg) & 1 : 0; it < np; it += S::PG) {
                const int stage = (cnt + it) % S::STAGES;
                if (!await(full(stage), ((cnt + it) / S::STAGES) & 1)) {
                    go = false;
                    gave_up();
                    break;
                }
                const int ek = exps[2 * stage];
                int ev = exps[2 * stage + 1];
                if (ev == EV_BAD) { bad = true; ev = 0; }
                const uint32_t kt = sbase + stage * S::STAGE;
                const int p0 = (page0 + it) * KV_PAGE + 32 * half;      // the first of this warp's 32 positions
                float fk[NT][E];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < E; ++e) fk[n][e] = qf[n][e] * pow2_clamped(qe[n][e] + ek);
                const float fev = (float)ev, inv_vs = kv_pow2(-ev);
                // EDGE: some row does not see all 32 positions
                auto step = [&](auto edge) {
                    constexpr bool EDGE = decltype(edge)::value;
                    // S^T = K q^T, 16 tokens a tile u: row r < 8 is token 4 (r / 2) + r % 2, row r + 8 the one 2 behind it
                    float z[2][NT][4];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int n = 0; n < NT; ++n) z[u][n][0] = z[u][n][1] = z[u][n][2] = z[u][n][3] = 0.f;
#pragma unroll
                    for (int y = 0; y < HD / 64; ++y) {
                        uint32_t w[2][2][4];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint4 v = lds128(kt + k_at[y] + (16 * u + 2 * j) * HD);
                                w[u][j][0] = v.x; w[u][j][1] = v.y; w[u][j][2] = v.z; w[u][j][3] = v.w;
                            }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint32_t ka[4] = {e4m3x2_to_half2((uint16_t)w[u][0][i]), e4m3x2_to_half2((uint16_t)w[u][1][i]),
                                                        e4m3x2_to_half2((uint16_t)(w[u][0][i] >> 16)),
                                                        e4m3x2_to_half2((uint16_t)(w[u][1][i] >> 16))};
#pragma unroll
                                for (int n = 0; n < NT; ++n) mma16816(z[u][n], ka, qb[n][4 * y + i][0], qb[n][4 * y + i][1]);
                            }
                    }
                    // scores in units of log2, with the value scale's exponent; this thread's largest
                    const int pos = p0 + 4 * (g >> 1) + (g & 1);
                    float mx[NT][E];
                    bool up = false;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int e = 0; e < E; ++e) mx[n][e] = -INFINITY;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if (FOLD) {
                                z[u][n][0] += z[u][n][1];
                                z[u][n][2] += z[u][n][3];
                            }
#pragma unroll
                            for (int k = 0; k < 4; k += 3 - E) {
                                const int e = k & (E - 1);
                                float s2 = fmaf(z[u][n][k], fk[n][e], fev);
                                if (EDGE && pos + 16 * u + (k & 2) >= limit[n][e]) s2 = -INFINITY;
                                mx[n][e] = fmaxf(mx[n][e], s2);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < E; ++e) up |= mx[n][e] > m[n][e] + M_SLACK;
                    }
                    // the reference moves only when a score passes it by 2^M_SLACK: then p' stays below fp16's range
                    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                float v = mx[n][e];
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                                v = fmaxf(v, m[n][e]);
                                const float f = v == -INFINITY ? 1.f : ex2(m[n][e] - v);
                                m[n][e] = v;
                                l[n][e] *= f;
#pragma unroll
                                for (int j = 0; j < HD / 16; ++j) {
                                    o[j][n][e] *= f;
                                    o[j][n][2 + e] *= f;
                                    if (FOLD) {
                                        o[j][n][1] *= f;
                                        o[j][n][3] *= f;
                                    }
                                }
                            }
                    }
                    uint32_t p[2][NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float off[E], add[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            off[e] = fev + P_SHIFT - (m[n][e] == -INFINITY ? 0.f : m[n][e]);
                            add[e] = 0.f;
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
#pragma unroll
                            for (int k = 0; k < 4; k += 3 - E) {
                                const int e = k & (E - 1);
                                float e2 = fmaf(z[u][n][k], fk[n][e], off[e]);
                                if (EDGE && pos + 16 * u + (k & 2) >= limit[n][e]) e2 = -INFINITY;
                                z[u][n][k] = ex2(e2);
                                add[e] += z[u][n][k];
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                p[u][n][j] = transpose8x8(FOLD ? high_low(z[u][n][2 * j]) : half2_bits(z[u][n][2 * j], z[u][n][2 * j + 1]));
                        }
#pragma unroll
                        for (int e = 0; e < E; ++e) l[n][e] = fmaf(add[e], inv_vs, l[n][e]);
                    }
                    // O^T += V^T P^T: rows g and g + 8 of tile 2 y + e are dims 32 y + 4 g + e and the one 2 behind it
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        // bytes of tokens behind the end can be anything, NaN among them: 0 stands in.  A NaN
                        // among the newest tokens' values must not reach the rows before it through 0 * NaN
                        // either: the product takes 0 for it, and the rows that do see it are found by a
                        // second product.
                        const int first = p0 + 16 * u + 4 * t;  // of this thread's four tokens
                        const int valid = lim_hi - first;
                        const uint32_t keep = valid >= 4 ? 0xffffffffu : (valid <= 0 ? 0u : (1u << (8 * valid)) - 1u);
#pragma unroll
                        for (int y = 0; y < HD / 32; ++y) {
                            const uint4 v = lds128(kt + v_at + 16 * u * HD + 128 * y);
                            uint32_t w[4] = {v.x, v.y, v.z, v.w};
                            if (EDGE) {
                                uint32_t nan[4], some = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    w[e] &= keep;
                                    nan[e] = __vcmpeq4(w[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    w[e] &= ~nan[e];
                                    nan[e] &= 0x38383838u;      // 1.0
                                    some |= nan[e];
                                }
                                if (__any_sync(0xffffffffu, some != 0)) {
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        // 1.0 where column g's row sees tokens 0, 1 and 2, 3 of the quad
                                        const int r2 = rg * S::PR + (FOLD ? 4 * n + (g >> 1) : 8 * n + g);
                                        const int left = (r2 < x.pairs ? x.before + (x.pair0 + r2) / a.group + 1 : 0) - first;
                                        const uint32_t see0 = (left > 0 ? 0x3c00u : 0u) | (left > 1 ? 0x3c000000u : 0u);
                                        const uint32_t see1 = (left > 2 ? 0x3c00u : 0u) | (left > 3 ? 0x3c000000u : 0u);
#pragma unroll
                                        for (int e = 0; e < 2; ++e) {
                                            const uint32_t na[4] = {e4m3x2_to_half2((uint16_t)nan[e]), e4m3x2_to_half2((uint16_t)nan[e + 2]),
                                                                    e4m3x2_to_half2((uint16_t)(nan[e] >> 16)),
                                                                    e4m3x2_to_half2((uint16_t)(nan[e + 2] >> 16))};
                                            float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                            mma16816(hit, na, see0, see1);
#pragma unroll
                                            for (int k = 0; k < 4; ++k)
                                                if (hit[k] > 0.f) o[2 * y + e][n][k] = NAN;
                                        }
                                    }
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t va[4] = {e4m3x2_to_half2((uint16_t)w[e]), e4m3x2_to_half2((uint16_t)w[e + 2]),
                                                        e4m3x2_to_half2((uint16_t)(w[e] >> 16)),
                                                        e4m3x2_to_half2((uint16_t)(w[e + 2] >> 16))};
#pragma unroll
                                for (int n = 0; n < NT; ++n) mma16816(o[2 * y + e][n], va, p[u][n][0], p[u][n][1]);
                            }
                        }
                    }
                };
                if (p0 + 32 <= lim_lo) step(std::false_type{});
                else if (p0 < lim_hi) step(std::true_type{});
                __syncwarp();
                if (lane == 0) tcx::mbar_arrive(empty(stage));
            }
            cnt += np;
            // ---- join the row group's warps
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float v = l[n][e];
                    v += __shfl_xor_sync(0xffffffffu, v, 4);
                    v += __shfl_xor_sync(0xffffffffu, v, 8);
                    v += __shfl_xor_sync(0xffffffffu, v, 16);
                    if (g == 0) {
                        const int row = rg * S::PR + (FOLD ? 4 * n + t : 8 * n + 2 * t + e);
                        st_m[wg * S::ROWS + row] = m[n][e];
                        st_l[wg * S::ROWS + row] = bad ? NAN : v;
                    }
                }
                if (FOLD) {
#pragma unroll
                    for (int j = 0; j < HD / 16; ++j) {
                        o[j][n][0] += o[j][n][1];
                        o[j][n][2] += o[j][n][3];
                    }
                }
            }
            if (any(!go)) break;
            float mm[NT][E], ll[NT][E];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int row = rg * S::PR + (FOLD ? 4 * n + t : 8 * n + 2 * t + e);
                    mm[n][e] = -INFINITY;
                    ll[n][e] = 0.f;
#pragma unroll
                    for (int w = 0; w < S::WG; ++w) mm[n][e] = fmaxf(mm[n][e], st_m[w * S::ROWS + row]);
#pragma unroll
                    for (int w = 0; w < S::WG; ++w) {
                        const float mw = st_m[w * S::ROWS + row];       // 1: 0 or NaN stands there
                        ll[n][e] += st_l[w * S::ROWS + row] * (mw == -INFINITY ? 1.f : ex2(mw - mm[n][e]));
                    }
                    const float f = m[n][e] == -INFINITY ? 1.f : ex2(m[n][e] - mm[n][e]);
#pragma unroll
                    for (int j = 0; j < HD / 16; ++j) {
                        o[j][n][e] *= f;
                        o[j][n][2 + e] *= f;
                    }
                }
            // pairwise, in a fixed order: odd pages into even ones, then second halves into first ones,
            // a part of the dims at a time through the joining space
            float* jn = reinterpret_cast<float*>(smem + S::JOIN + rg * S::JOIN_WG);
            auto join = [&](auto givers, bool gives, bool takes, int place) {
                constexpr int PER = 2 * E * NT * 32;                                    // floats of o[j] in a warp
                constexpr int FIT = S::JOIN_WG / 4 / decltype(givers)::value / PER;     // o[j] at a time
                constexpr int STEP = FIT < HD / 16 ? FIT : HD / 16;
                static_assert(STEP >= 1 && HD / 16 % STEP == 0, "whole steps");
                float* at = jn + place * (STEP * PER) + lane;
#pragma unroll
                for (int j0 = 0; j0 < HD / 16; j0 += STEP) {
                    if (gives) {
#pragma unroll
                        for (int j = 0; j < STEP; ++j)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int k = 0; k < 4; k += 3 - E) {
                                    *at = o[j0 + j][n][k];
                                    at += 32;
                                }
                        at -= STEP * PER;
                    }
                    sync_all();
                    if (takes) {
#pragma unroll
                        for (int j = 0; j < STEP; ++j)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int k = 0; k < 4; k += 3 - E) {
                                    o[j0 + j][n][k] += *at;
                                    at += 32;
                                }
                        at -= STEP * PER;
                    }
                    sync_all();
                }
            };
            if (S::PG == 2) join(std::integral_constant<int, 2>{}, pg == 1, pg == 0, half);
            join(std::integral_constant<int, 1>{}, wg == 1, wg == 0, 0);
            const int nsplit = x.nsplit, unit = x.unit;
            float* part = a.part + (int64_t)x.index * a.slot;
            if (wg == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int row = rg * S::PR + (FOLD ? 4 * n + t : 8 * n + 2 * t + e);
                        if (row >= x.pairs) continue;
                        const float inv = nsplit > 1 ? 1.f : 1.f / ll[n][e];
                        const int pair = x.pair0 + row;
                        const int64_t yr = kv_row(c, (int64_t)x.row0 + pair / a.group);
                        const int head = x.h * a.group + pair % a.group;
#pragma unroll
                        for (int y = 0; y < HD / 32; ++y) {
                            const float w[4] = {o[2 * y][n][e] * inv, o[2 * y + 1][n][e] * inv, o[2 * y][n][2 + e] * inv,
                                                o[2 * y + 1][n][2 + e] * inv};
                            if (nsplit > 1) store4_f(part + row * HD + 32 * y + 4 * g, w);
                            else store4_f(out + yr * a.ldo + (int64_t)head * HD + 32 * y + 4 * g, w);
                        }
                        if (g != 0) continue;
                        if (nsplit > 1) {
                            part[a.prow * HD + row] = mm[n][e];
                            part[a.prow * (HD + 1) + row] = ll[n][e];
                        } else if (a.lse) {
                            a.lse[yr * a.n_heads + head] = ((mm[n][e] == -INFINITY ? 0.f : mm[n][e]) - P_SHIFT + log2f(ll[n][e])) * LN2;
                        }
                    }
            }
            if (nsplit > 1) {
                // ---- the last item of the unit to arrive joins its runs
                sync_all();
                if (threadIdx.x == 0) {
                    __threadfence();
                    const int arrived = atomicAdd(a.counters + CTR_UNITS + unit, 1);
                    flags[2] = arrived == nsplit - 1;
                    if (arrived == nsplit - 1) a.counters[CTR_UNITS + unit] = 0;    // as the next call finds it
                    __threadfence();
                }
                sync_all();
                if (flags[2]) {
                    const float* p0 = a.part + (int64_t)unit * a.splits * a.slot;
                    for (int i = threadIdx.x; i < x.pairs * (HD / 4); i += 32 * S::NW) {
                        const int row = i / (HD / 4), d = i % (HD / 4) * 4;
                        float M = -INFINITY;
                        for (int k = 0; k < nsplit; ++k) M = fmaxf(M, __ldcg(p0 + k * a.slot + a.prow * HD + row));
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        float L = 0.f;
#pragma unroll 8
                        for (int k = 0; k < nsplit; ++k) {
                            const float* pk = p0 + k * a.slot;
                            const float mw = __ldcg(pk + a.prow * HD + row);
                            const float f = mw == -INFINITY ? 1.f : ex2(mw - M);    // 1: 0 or NaN stands there
                            const float4 u = __ldcg(reinterpret_cast<const float4*>(pk + row * HD + d));
                            L = fmaf(__ldcg(pk + a.prow * (HD + 1) + row), f, L);
                            v.x = fmaf(u.x, f, v.x); v.y = fmaf(u.y, f, v.y); v.z = fmaf(u.z, f, v.z); v.w = fmaf(u.w, f, v.w);
                        }
                        const int pair = x.pair0 + row;
                        const int64_t yr = kv_row(c, (int64_t)x.row0 + pair / a.group);
                        const int head = x.h * a.group + pair % a.group;
                        const float inv = 1.f / L;
                        const float w[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
                        store4_f(out + yr * a.ldo + (int64_t)head * HD + d, w);
                        if (d == 0 && a.lse)
                            a.lse[yr * a.n_heads + head] = ((M == -INFINITY ? 0.f : M) - P_SHIFT + log2f(L)) * LN2;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tcx::mbar_arrive(item_empty(n_item & 1));
        }
    }
    __syncthreads();
    if (flags[0]) {
        // a wait gave up: let copies that may still be in flight land before the
        // block's memory goes to another (again bounded); nothing more is written
        if (threadIdx.x == 0) {
            const uint64_t t0 = tcx::globaltimer();
            while (tcx::globaltimer() - t0 < 2000000) {}
        }
        return;
    }
    // the last block to finish leaves the item counter as it found it
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(a.counters + CTR_DONE, 1) == (int)gridDim.x - 1) {
            a.counters[CTR_NEXT] = 0;
            a.counters[CTR_DONE] = 0;
        }
    }
}

constexpr int MAX_UNITS_SPLIT = MLORA_KV_COUNTER_BYTES / 4 - CTR_UNITS;   // a counter for each unit

template <typename T, int HD, int NT, int RG>
cudaError_t attn_t(const KvView& c, const KvAttnArgs& a, cudaStream_t s) {
    using S = AttnShape<T, HD, NT, RG>;
    // once a device: its SMs, and the kernel's shared memory (the attribute stays with the function)
    static std::atomic<int> sms[64];
    int dev = 0, n_sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) n_sms = sms[dev].load(std::memory_order_relaxed);
    if (n_sms == 0) {
        e = cudaFuncSetAttribute(kv_attn_kernel<T, HD, NT, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < 64) sms[dev].store(n_sms, std::memory_order_relaxed);
    }
    AttnCall k;
    k.q = a.q; k.out = a.out; k.lse = a.lse; k.ldq = a.ldq; k.ldo = a.ldo; k.max_len = a.max_len;
    k.counters = static_cast<int*>(a.workspace);
    k.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + MLORA_KV_COUNTER_BYTES);
    k.n_heads = a.n_heads; k.group = a.n_heads / c.n_kv;
    k.qk = a.scale * LOG2E;
    const int64_t pairs = (int64_t)c.max_rows * k.group;
    const int64_t tiles = (pairs + S::ROWS - 1) / S::ROWS;
    k.prow = (int)(pairs < S::ROWS ? pairs : S::ROWS);
    k.slot = ((int64_t)k.prow * (HD + 2) + 3) / 4 * 4;      // 16-byte aligned
    const int64_t units = tiles * c.n_kv * c.n_seqs;
    const int64_t cap = (int64_t)c.max_pages * KV_PAGE;
    const int64_t longest = a.max_len < cap ? a.max_len : cap;
    const int64_t pages = longest > 0 ? (longest + KV_PAGE - 1) / KV_PAGE : 1;
    // Runs of pages: short enough that every resident block has one and that a
    // long sequence is no tail of the launch, long enough that an item's start
    // and the join stay small beside it.
    const int64_t blocks = (int64_t)n_sms * S::BLOCKS_SM;
    int64_t chunk = pages;
    if (units <= MAX_UNITS_SPLIT) {
        const int64_t per_unit = (KV_ITEMS_BLOCK * blocks + units - 1) / units;
        chunk = (pages + per_unit - 1) / per_unit;
        if (chunk > KV_LONG_RUN) chunk = KV_LONG_RUN;
        if (chunk < KV_SHORT_RUN) chunk = KV_SHORT_RUN;
        const int64_t slots = (a.workspace_bytes - MLORA_KV_COUNTER_BYTES) / (k.slot * 4);
        const int64_t most = slots / units;                 // runs of a unit that the workspace holds
        if (most < 2) chunk = pages;
        else if ((pages + chunk - 1) / chunk > most) chunk = (pages + most - 1) / most;
    }
    k.tiles = (int)tiles;
    k.chunk = (int)(chunk < pages ? chunk : pages);
    k.splits = (int)((pages + k.chunk - 1) / k.chunk);
    const int64_t items = units * k.splits;
    if (items > (1 << 30)) return cudaErrorInvalidConfiguration;
    k.items = (int)items;
    kv_attn_kernel<T, HD, NT, RG><<<(unsigned)(items < blocks ? items : blocks), S::THREADS, S::SMEM, s>>>(c, k);
    return cudaGetLastError();
}

// One column tile (8 pairs; 4 on fp32) where a sequence's pairs fit it, then two;
// more row groups share each page tile (its reads and its place in shared
// memory) where a sequence has more.
template <typename T, int HD>
cudaError_t attn_rows(const KvView& c, const KvAttnArgs& a, cudaStream_t s) {
    constexpr int PR = AttnShape<T, HD, 1, 1>::PR;
    const int64_t pairs = (int64_t)c.max_rows * (a.n_heads / c.n_kv);
    if (pairs <= PR) return attn_t<T, HD, 1, 1>(c, a, s);
    if (pairs <= 2 * PR) return attn_t<T, HD, 1, 2>(c, a, s);
    if (pairs <= 4 * PR) return attn_t<T, HD, 2, 2>(c, a, s);
    return attn_t<T, HD, 2, 4>(c, a, s);
}

}  // namespace

cudaError_t launch_kv_attention(const KvView& c, int head_dim, int dtype, const KvAttnArgs& a, cudaStream_t s) {
    if (dtype == MLORA_BF16) return head_dim == 64 ? attn_rows<bf16, 64>(c, a, s) : attn_rows<bf16, 128>(c, a, s);
    return head_dim == 64 ? attn_rows<float, 64>(c, a, s) : attn_rows<float, 128>(c, a, s);
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
