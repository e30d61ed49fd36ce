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
//    against one key/value head, over a run of pages.  Blocks are persistent:
//    the pages of all items are one line that is cut into equal shares, one a
//    block, whatever the sequences' lengths.  A producer warp copies each (page,
//    head) tile of K and V -- contiguous 8 KB at head_dim 128 -- into a ring of
//    stages with cp.async.bulk and runs ahead into the next item (its table,
//    scales, queries and first pages) while the consumer warps finish this one.
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
//    part (2^-22, or 2^-36 of the row's largest magnitude): both products come
//    out of one instruction, in one thread.  Low parts are held at 2^11 times
//    their value: unscaled, fp16's smallest step cut them off at 2^-25 of the
//    largest, 2^-15 of a value that is itself 2^-10 of it.
//  * p = exp2(s log2 e - m) with m a running maximum of s log2 e that follows the
//    scores only when one passes it by 2^3 (the sums are then rescaled).  p is held
//    at 2^12 times its value, so that it stays within fp16 and its rounding
//    relative (2^-11) down to 2^-26 of the reference (absolute 2^-37 of it below
//    that); on fp32 it is split like q.
//  * The page's value scale 2^ev: a warp's accumulators are in units of 2^unit, and
//    p' = p 2^(ev - unit) where that is within 2^-3 .. 1 (the factor goes into the
//    exponent, l += p' 2^(unit - ev), and the bounds on p's rounding are 2^3
//    higher).  At any other page the unit becomes 2^ev and the accumulators,
//    fp32 with room for it, are multiplied by the difference: so each dim keeps its
//    precision beside pages whose scale another dim has made large, and l has every
//    p whatever its page's scale.  (With the whole scale in p', p' left fp16's range
//    for the sake of other pages, and the sums of values that are all zero, with
//    ev = -100, left fp32's; it took 31.6 us where this takes 33.0 on 41 sequences
//    of 0 to 3001 tokens, 16 heads of 64, fp32, and 115.5 where this takes 116.5 on
//    256 of 512 to 2048, 8 heads of 128.  Units found by the producer for 32 pages
//    at once: 33.0 and 117.3.)  A page below 2^-64 of the largest so far adds to l
//    alone: below that the accumulators' range could end.
//  * Warps of a row group take different halves of a page and, where a single row
//    group has two pages in work, every other page, 32 tokens at a step; each has
//    a running maximum and sum of its own, joined at the item's end, so nothing
//    but the ring's barriers is shared in the loop.
//  * A share's ends cut sequences: such an item leaves its rows' unnormalised
//    sums, maximum and sum in the workspace, and a second small kernel joins the
//    parts in order.  (Runs of a fixed length taken from a counter left a tail or
//    ended too often: 94 us at best for 32 sequences of 1023 to 8191 tokens, 4
//    rows each, which equal shares serve in 62; joined by the last item to
//    arrive, a run's end cost its block about 6 us of fences and atomics.  Warps
//    that each stream a share of their own hide the ends of items better but
//    end 84 to 125 us after the start where blocks' shares end together.)
#include <atomic>
#include <type_traits>

#include "kv_common.cuh"
#include "tc_ptx.cuh"

namespace mlk {

namespace {

constexpr double LOG2E = 1.4426950408889634;
constexpr float LN2 = 0.6931471805599453f;
constexpr int P_SHIFT = 12;                 // p' is held at 2^12 times its value,
constexpr float M_SLACK = 3.f;              // against a reference at most 2^3 below the largest: p' <= 2^15
constexpr float LOW = 2048.f;               // low parts of fp32 values: rest of at most 2^-11 of a high part <= 2^15
constexpr int V_FOLD = 3;                   // value scales of 2^-V_FOLD to 1 of the accumulators' unit go into p'
constexpr int V_GAP = 64;                   // pages below 2^-V_GAP of the largest so far count as zero values: 2^31 terms
                                            // p' v8 < 2^24 times 2^V_GAP stay within fp32
constexpr int V_GONE = -60;                 // what such a page folds: p' <= 2^-45 is 0 in fp16, and so is its low part
// Places: no block gets fewer.  One sequence of 1000 tokens, 8 heads of 128: 9.8 us at 1, 10.8 at 2, 11.1 at 4; one
// of 4000, 1 head: 10.2, 9.7, 9.9 (replayed graphs); long ones have more places than blocks.
constexpr int KV_SHORT_RUN = 2;
// What a unit's start and end cost, in pages.  41 sequences of 0 to 3001 tokens,
// 16 heads of 64, fp32: 62.4 us at 0, 37.4 at 2, 33.3 at 4 to 6, 34.3 at 8; 256
// sequences of 512 to 2048, 8 heads of 128: 124.2, 120.0, 117.8 to 117.3, 117.0; 64 of
// 4097 to 32767: 363 at 0, 357 to 359 from 2 on.
constexpr int KV_START = 5;
// Pages: sequences up to this are not cut.  Uncut, and cut at 4 or less: 256 sequences of 64 to 512 tokens, 8 heads
// of 128, 60.8 and 68.4 us, 64 of them 18.7 and 20.5, 3 of 21 to 299, 2 heads, 9.3 and 10.3; but 8 of 300 to 512, 8
// heads, 15.9 and 11.2.  At 16, 8 sequences of 600 to 1000 take 20.7 us in place of 12.4 (replayed graphs).
constexpr int KV_WHOLE = 8;

// A cut unit, left in the workspace by the block that begins it.
struct Cut {
    int blocks;                             // blocks that share it, from this one on (0: this block begins none)
    int row0, pair0, pairs, h;
};

struct AttnCall {
    const void* q;
    void* out;
    float* lse;
    Cut* cuts;                              // one a block; null: sequences are not cut
    float* part;                            // two partial results a block
    int64_t ldq, ldo;
    int n_heads, group;
    int prow;                               // rows of a partial result
    int64_t slot;                           // its floats: the rows' sums, maxima, sums of p and units
    float qk;                               // scale * log2 e = qk 2^qk_exp, 1/2 <= |qk| < 1
    int qk_exp;
};

// What the producer tells the consumers about an item.
struct Item {
    int s, h;                               // s < 0: no more
    int row0;                               // the sequence's first row
    int pair0, pairs;                       // first pair of the tile, pairs in it
    int before;                             // positions before the sequence's rows
    int page0, np;                          // the run
    int slot;                               // its partial result's place, or -1: the whole unit
};

template <typename T, int HD, int NT, int RG, int PG_>
struct AttnShape {
    static constexpr bool FOLD = sizeof(T) == 4;            // a pair takes two columns: its high and its low part
    static constexpr int PR = (FOLD ? 4 : 8) * NT;          // pairs of a row group
    static constexpr int ROWS = PR * RG;
    static constexpr int PG = PG_;                          // pages in work at once
    static constexpr int WG = 2 * PG;                       // warps of a row group: page parity x half of the page
    static constexpr int NW = RG * WG;                      // consumer warps
    static constexpr int THREADS = 32 * NW + 32;
    static constexpr int TILE = KV_PAGE * HD;               // bytes of a K or V tile
    static constexpr int STAGE = 2 * TILE;
    // small tiles leave room for a fourth block (41 sequences of 0 to 3001 tokens, 16 heads of 64, fp32: 37 us
    // with three of 8 stages, 33 with four of 6, 36 with five of 4)
    static constexpr bool FOUR = HD == 64 && NT == 1 && RG == 1;
    static constexpr bool SLIM = NW == 2;                   // two consumer warps: four blocks of three stages
    static constexpr int STAGES = FOUR ? 6 : SLIM ? 3 : (NT == 1 ? 4 : 6) * (128 / HD);
    static constexpr int BLOCKS_SM = FOUR || SLIM ? 4 : (NW > 4 ? 1 : 3);
    static constexpr int JOIN_WG = 2048 * PG;               // joining space of a row group, bytes
    // ring, raw queries, joining space, per-warp statistics and units,
    // barriers, exponents, items, flags
    static constexpr int QRAW = STAGES * STAGE;
    static constexpr int JOIN = QRAW + ROWS * HD * (int)sizeof(T);
    static constexpr int STAT = JOIN + RG * JOIN_WG;
    static constexpr int UNIT = STAT + 8 * WG * ROWS;
    static constexpr int BAR = UNIT + (4 * NW + 15) / 16 * 16;
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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    // not volatile: a function of its operands, free to move between the loads and conversions
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// LOW times what rounding (a, b) to fp16 left
__device__ __forceinline__ uint32_t half2_rest(float a, float b, uint32_t hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return half2_bits((a - f.x) * LOW, (b - f.y) * LOW);
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
// a value as its fp16 rounding (low half) and the fp16 rounding of LOW times the rest
__device__ __forceinline__ uint32_t high_low(float v) {
    const __half h = __float2half_rn(v);
    const __half2 r = __halves2half2(h, __float2half_rn((v - __half2float(h)) * LOW));
    return *reinterpret_cast<const uint32_t*>(&r);
}
constexpr int UNIT_NONE = -(1 << 20);        // no page yet
constexpr int EV_BAD = 1 << 20;              // in place of an exponent: a bad page in the run
// x 2^e for |x| < 1: q, the keys' scale and the caller's can lie on both sides of fp32's range and make up for
// one another, so their exponents are added before one factor is formed (|e| beyond 252 is 0 or an infinity)
__device__ __forceinline__ float times_pow2(float x, int e) {
    e = e < -252 ? -252 : (e > 252 ? 252 : e);
    return x * kv_pow2(e >> 1) * kv_pow2(e - (e >> 1));
}
// 2^e for e <= 127, 0 where that is below the normal range
__device__ __forceinline__ float pow2_or_0(int e) { return e < -126 ? 0.f : kv_pow2(e); }

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

template <typename T, int HD, int NT, int RG, int PG_>
__global__ void __launch_bounds__(AttnShape<T, HD, NT, RG, PG_>::THREADS, AttnShape<T, HD, NT, RG, PG_>::BLOCKS_SM)
    kv_attn_kernel(const __grid_constant__ KvView c, const __grid_constant__ AttnCall a) {
    using S = AttnShape<T, HD, NT, RG, PG_>;
    constexpr bool FOLD = S::FOLD;
    constexpr int E = FOLD ? 1 : 2;                         // pairs of a thread in an 8-column tile
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = tcx::smem_u32(smem);
    int* exps = reinterpret_cast<int*>(smem + S::EXPS);     // per stage: K's and V's exponent
    float* st_m = reinterpret_cast<float*>(smem + S::STAT); // [WG][ROWS]
    float* st_l = st_m + S::WG * S::ROWS;
    int* st_u = reinterpret_cast<int*>(smem + S::UNIT);     // [NW]
    Item* items = reinterpret_cast<Item*>(smem + S::ITEMS);
    volatile int* flags = reinterpret_cast<volatile int*>(smem + S::FLAGS);   // [0]: a wait gave up
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
        flags[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // the join's blocks may be set up while this kernel runs; they wait for its end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == S::NW) {
        // ---- producer
        const T* q = static_cast<const T*>(a.q);
        T* out = static_cast<T*>(a.out);
        // The block's share.  All units -- sequence by sequence, then key/value head,
        // row tile -- are one line of `total` places, KV_START for a unit's start and
        // one for each page, cut into equal shares; every block adds the sequences
        // up for itself, a lane `per` of them.
        auto weight = [&](const SeqRows& r) -> int64_t {
            return r.len > 0 ? (int64_t)((r.len + KV_PAGE - 1) / KV_PAGE + KV_START) * ((r.n * a.group + S::ROWS - 1) / S::ROWS) * c.n_kv : 0;
        };
        const int per = (c.n_seqs + 31) / 32, s0 = lane * per;
        // a warp's lanes hold the lengths and rows of 32 sequences, from s_base on
        int s_base = 0;
        int l_len = 0;
        int64_t l_a = 0, l_b = 0;
        auto lengths = [&]() {
            const int s = s_base + lane < c.n_seqs ? s_base + lane : c.n_seqs - 1;
            l_len = c.kv_len[s];
            l_a = c.row_off ? c.row_off[s] : s;
            l_b = c.row_off ? c.row_off[s + 1] : (int64_t)s + 1;
        };
        lengths();
        int64_t mine = 0;
        if (per == 1) {
            SeqRows r;
            const bool ok = kv_seq_ok(c, l_len, l_a, l_b, r);
            mine = ok && lane < c.n_seqs ? weight(r) : 0;
        } else {
#pragma unroll 4
            for (int i = 0; i < per; ++i) {
                SeqRows r;
                const int s = s0 + i < c.n_seqs ? s0 + i : c.n_seqs - 1;
                const bool ok = kv_seq(c, s, r);
                mine += ok && s0 + i < c.n_seqs ? weight(r) : 0;
            }
        }
        int64_t upto = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, x);
            upto += lane >= x ? y : 0;
        }
        const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
        int64_t shares = a.cuts ? (total + KV_SHORT_RUN - 1) / KV_SHORT_RUN : total;
        if (shares > gridDim.x) shares = gridDim.x;
        const bool busy = (int)blockIdx.x < shares;
        const int64_t lo = busy ? (int64_t)blockIdx.x * total / shares : 0, hi = busy ? ((int64_t)blockIdx.x + 1) * total / shares : 0;
        // the lane whose sequences hold place lo; next() goes on from its first one
        const unsigned holds = __ballot_sync(0xffffffffu, upto - mine <= lo && lo < upto);
        const int from = holds ? __ffs(holds) - 1 : 0;
        const int64_t before = __shfl_sync(0xffffffffu, upto - mine, from);
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
        // the items of the share, in order
        int64_t pos = lo, rem = lo - before;                // place in the line, and from the first of s_now's on
        int s_now = from * per;
        if (a.cuts && lane == 0) a.cuts[blockIdx.x].blocks = 0;
        auto next = [&](Item& x) {
            x.s = -1;
            while (pos < hi && s_now < c.n_seqs) {
                if (s_now - s_base >= 32) {
                    s_base = s_now;
                    lengths();
                }
                SeqRows r;
                const int len = __shfl_sync(0xffffffffu, l_len, s_now - s_base);
                const int64_t row_a = __shfl_sync(0xffffffffu, l_a, s_now - s_base);
                const int64_t row_b = __shfl_sync(0xffffffffu, l_b, s_now - s_base);
                const int64_t w = kv_seq_ok(c, len, row_a, row_b, r) ? weight(r) : 0;
                if (rem >= w) {                             // behind the sequence
                    rem -= w;
                    ++s_now;
                    continue;
                }
                const int pages = (len + KV_PAGE - 1) / KV_PAGE, tiles = (r.n * a.group + S::ROWS - 1) / S::ROWS;
                const int size = pages + KV_START;
                const int unit = (int)(rem / size), off = (int)(rem % size);
                int step = size - off;                      // places of the unit from here on
                if (a.cuts) {
                    if (step > hi - pos) step = (int)(hi - pos);
                }
                pos += step;
                rem += step;
                const int page0 = off > KV_START ? off - KV_START : 0, np = off + step - KV_START - page0;
                // nothing but a start; or not cut: the unit is the block's where its line begins
                if (np <= 0 || (!a.cuts && off > 0)) continue;
                const int tile = unit % tiles;
                x.s = s_now;
                x.h = unit / tiles;
                x.row0 = r.row0;
                x.pair0 = tile * S::ROWS;
                x.pairs = r.n * a.group - x.pair0 < S::ROWS ? r.n * a.group - x.pair0 : S::ROWS;
                x.before = r.len - r.n;
                x.page0 = page0;
                x.np = np;
                x.slot = -1;
                if (page0 > 0) {
                    x.slot = 2 * blockIdx.x;
                } else if (np < pages) {
                    x.slot = 2 * blockIdx.x + 1;
                    if (lane == 0) {
                        const int64_t end = pos - step + size - off;    // the share of place p is ((p + 1) shares - 1) / total
                        a.cuts[blockIdx.x] = Cut{(int)((end * shares - 1) / total) - (int)blockIdx.x + 1, x.row0, x.pair0, x.pairs, x.h};
                    }
                    __syncwarp();
                }
                return;
            }
        };
        // lane i: page id of x's page i0 + i
        auto page_id = [&](const Item& x, int i0) -> int {
            const int i = i0 + lane < x.np ? i0 + lane : i0;
            return c.table[(int64_t)x.s * c.max_pages + x.page0 + i];
        };
        // lane i: tile and scales of a page, from its id.  No branch: the vote and the loads are every lane's, and
        // nothing waits for the loads here.
        int64_t at = 0;
        float ks = 0.f, vs = 0.f;
        unsigned bad = 0;
        auto load_batch = [&](const Item& x, int id) {
            const bool good = id >= 0 && id < c.n_pages;
            bad = __ballot_sync(0xffffffffu, !good);
            at = (int64_t)(good ? id : 0) * c.n_kv + x.h;   // a page that exists stands in; the rows become NaN
            ks = c.ks[at];
            vs = c.vs[at];
            if (bad != 0 && lane == 0) raise_status(c.status, ST_RANGE);
            __syncwarp();
        };
        // an item's queries: the pairs of a token are contiguous
        auto queries = [&](const Item& x) {
            if (lane == 0) tcx::mbar_expect_tx(q_full, x.pairs * HD * (int)sizeof(T));
            __syncwarp();
            for (int tok = x.pair0 / a.group + lane; tok * a.group < x.pair0 + x.pairs; tok += 32) {
                const int p0 = tok * a.group > x.pair0 ? tok * a.group : x.pair0;
                const int p1 = (tok + 1) * a.group < x.pair0 + x.pairs ? (tok + 1) * a.group : x.pair0 + x.pairs;
                bulk_load(sbase + S::QRAW + (p0 - x.pair0) * HD * (int)sizeof(T),
                          q + kv_row(c, (int64_t)x.row0 + tok) * a.ldq + ((int64_t)x.h * a.group + p0 - tok * a.group) * HD,
                          (p1 - p0) * HD * (int)sizeof(T), q_full);
            }
            __syncwarp();
        };
        if (s_now >= 32) {
            s_base = s_now;
            lengths();
        }
        Item x = {}, y = {};                                // the same in every lane: the current item and the next
        int y_id = 0;                                       // the next one's page ids, asked for an item ahead
        next(x);
        if (x.s >= 0) {
            // (the pages come behind all of this: asked for here, they delayed the small loads, 29 us against 31 on 8
            // sequences of 4096 to 8192 tokens)
            const int id = page_id(x, 0);
            queries(x);
            load_batch(x, id);
            next(y);
            if (y.s >= 0) y_id = page_id(y, 0);
        }
        int cnt = 0, n_item = 0;                            // pages and items so far
        bool go = true;
        while (go) {
            const int slot = n_item & 1;
            if (n_item >= 2 && !wait(item_empty(slot), (n_item / 2 - 1) & 1)) break;
            if (lane == 0) {
                items[slot] = x;
                tcx::mbar_arrive(item_full(slot));
            }
            if (x.s < 0) break;
            if (n_item >= 1) {
                if (!wait(q_empty, (n_item - 1) & 1)) break;
                queries(x);
            }
            const int lim = x.before + (x.pair0 + x.pairs - 1) / a.group + 1;
            const int np = x.np, page0 = x.page0;
            for (int i0 = 0; i0 < np && go; i0 += 32) {
                const int64_t at_now = at;
                const int ek_now = scale_exp(ks), ev_now = bad != 0 ? EV_BAD : scale_exp(vs);
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
                        const int tok = left < KV_PAGE ? (left > 0 ? left : 0) : KV_PAGE;       // (a tile's last pages may lie behind its rows)
                        const uint32_t kb = tok * HD, vb = (tok + 3) / 4 * 4 * HD;
                        exps[2 * stage] = k_;
                        exps[2 * stage + 1] = v_;
                        tcx::mbar_expect_tx(full(stage), kb + vb);
                        if (tok > 0) {
                            bulk_load(sbase + stage * S::STAGE, c.k + tile_at * S::TILE, kb, full(stage));
                            bulk_load(sbase + stage * S::STAGE + S::TILE, c.v + tile_at * S::TILE, vb, full(stage));
                        }
                    }
                    ++cnt;
                    // the ring is full, or the batch's pages are on their way: look for what comes next
                    if (i + 1 == (n < S::STAGES ? n : S::STAGES)) {
                        if (i0 + 32 < np) {
                            load_batch(x, page_id(x, i0 + 32));
                        } else {
                            x = y;
                            const int id = y_id;
                            if (x.s >= 0) {
                                next(y);
                                if (y.s >= 0) y_id = page_id(y, 0);
                                load_batch(x, id);
                            }
                        }
                    }
                }
            }
            ++n_item;
        }
        // rows without positions, shared out over the blocks: zero (or NaN: a bad sequence)
        for (int s = blockIdx.x; s < c.n_seqs; s += gridDim.x) {
            SeqRows r;
            const bool ok = kv_seq(c, s, r);
            if (!ok) raise_status(c.status, ST_RANGE);
            if (ok && r.len > 0) continue;
            const int64_t r1 = (int64_t)r.row0 + r.n < c.n_rows ? (int64_t)r.row0 + r.n : c.n_rows;
            for (int64_t i = r.row0 < 0 ? 0 : r.row0; i < r1; ++i) {
                const int64_t z = kv_row(c, i);
                for (int d = lane; d < a.n_heads * HD; d += 32) out[z * a.ldo + d] = from_f<T>(ok ? 0.f : NAN);
                for (int d = lane; a.lse && d < a.n_heads; d += 32) a.lse[z * a.n_heads + d] = ok ? -INFINITY : NAN;
            }
        }
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
            // a wait that gives up ends the loop in every consumer at the item's any()
            bool go = await(item_full(n_item & 1), (n_item / 2) & 1);
            if (!go) gave_up();
            const Item& x = items[n_item & 1];
            const bool end = go && x.s < 0;
            if (!go || end) {
                any(!go);
                break;
            }
            const int np = x.np, page0 = x.page0;
            const int lim_lo = x.before + x.pair0 / a.group + 1;                        // positions that the tile's first row sees
            const int lim_hi = x.before + (x.pair0 + x.pairs - 1) / a.group + 1;        // .. and its last
            // q's fragments: columns g of the tiles.  A thread's dims at K step
            // (y, i) are 64 y + 16 t + 4 i + 0..3, the four bytes of a word of the
            // key tile.
            go = await(q_full, n_item & 1);
            if (!go) gave_up();
            uint32_t qb[NT][HD / 16][2];
            float o[HD / 16][NT][4];
            float m[NT][E], l[NT][E], qf[NT][E];            // qf: qk, NaN where q is not finite, 0 where it is 0
            int qe[NT][E], limit[NT][E];                    // exponent of the row's largest |q| and of qk; positions it sees
            int unit = UNIT_NONE, top = UNIT_NONE;          // o is in units of 2^unit; largest value scale so far
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
                const float f = (nf >> (lane & 28)) & 15u ? NAN : (big > 0.f ? a.qk : 0.f);
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
                    qe[n][e] = __shfl_sync(0xffffffffu, ex, from) + a.qk_exp;
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

            for (int it = S::PG == 2 ? (cnt ^ pg) & 1 : 0; go && it < np; it += S::PG) {
                const int stage = (cnt + it) % S::STAGES;
                if (!await(full(stage), ((cnt + it) / S::STAGES) & 1)) {
                    go = false;
                    gave_up();
                    break;
                }
                const int ek = exps[2 * stage];
                int ev = exps[2 * stage + 1];
                if (ev == EV_BAD) { bad = true; ev = 0; }
                const uint8_t* kt = smem + stage * S::STAGE;
                const int p0 = (page0 + it) * KV_PAGE + 32 * half;      // the first of this warp's 32 positions
                float fk[NT][E];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < E; ++e) fk[n][e] = times_pow2(qf[n][e], qe[n][e] + ek);
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
                                const uint4 v = *reinterpret_cast<const uint4*>(kt + k_at[y] + (16 * u + 2 * j) * HD);
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
                    // scores in units of log2; this thread's largest
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
                                z[u][n][0] = fmaf(z[u][n][1], 1.f / LOW, z[u][n][0]);
                                z[u][n][2] = fmaf(z[u][n][3], 1.f / LOW, z[u][n][2]);
                            }
#pragma unroll
                            for (int k = 0; k < 4; k += 3 - E) {
                                const int e = k & (E - 1);
                                float s2 = z[u][n][k] * fk[n][e];
                                if (EDGE && pos + 16 * u + (k & 2) >= limit[n][e]) s2 = -INFINITY;
                                mx[n][e] = fmaxf(mx[n][e], s2);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < E; ++e) up |= mx[n][e] > m[n][e] + M_SLACK;
                    }
                    // the reference moves only when a score passes it by 2^M_SLACK: then p' stays below fp16's range;
                    // the unit only when the page's scale does not fold into p' (and not before the products, which
                    // would wait for that scale)
                    int fold = ev - unit;
                    const bool off_unit = (unsigned)(fold + V_FOLD) > (unsigned)V_FOLD;
                    if (__any_sync(0xffffffffu, up || off_unit)) {
                        float fm = 1.f;
                        if (off_unit) {
                            if (ev >= top - V_GAP) {
                                top = max(top, ev);
                                fm = pow2_or_0(unit - ev);
                                unit = ev;
                                fold = 0;
                            } else {
                                fold = V_GONE;
                            }
                        }
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
                                const float fo = f * fm;
#pragma unroll
                                for (int j = 0; j < HD / 16; ++j) {
                                    o[j][n][e] *= fo;
                                    o[j][n][2 + e] *= fo;
                                    if (FOLD) {
                                        o[j][n][1] *= fo;
                                        o[j][n][3] *= fo;
                                    }
                                }
                            }
                    }
                    const float shift = (float)(P_SHIFT + fold), unfold = kv_pow2(-fold);
                    uint32_t p[2][NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float off[E], add[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            off[e] = shift - (m[n][e] == -INFINITY ? 0.f : m[n][e]);
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
                        for (int e = 0; e < E; ++e) l[n][e] = fmaf(add[e], unfold, l[n][e]);
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
                            const uint4 v = *reinterpret_cast<const uint4*>(kt + v_at + 16 * u * HD + 128 * y);
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
                        o[j][n][0] = fmaf(o[j][n][1], 1.f / LOW, o[j][n][0]);
                        o[j][n][2] = fmaf(o[j][n][3], 1.f / LOW, o[j][n][2]);
                    }
                }
            }
            if (lane == 0) st_u[warp] = unit;
            if (any(!go)) break;
            int uu = KV_MIN_EXP;                            // the row group's unit: the largest
#pragma unroll
            for (int w = 0; w < S::WG; ++w) uu = max(uu, st_u[rg * S::WG + w]);
            const float fu = pow2_or_0(unit - uu);
            float mm[NT][E], ll[NT][E];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int row = rg * S::PR + (FOLD ? 4 * n + t : 8 * n + 2 * t + e);
                    float mw[S::WG], lw[S::WG];
                    mm[n][e] = -INFINITY;
#pragma unroll
                    for (int w = 0; w < S::WG; ++w) {
                        mw[w] = st_m[w * S::ROWS + row];
                        lw[w] = st_l[w * S::ROWS + row];
                        mm[n][e] = fmaxf(mm[n][e], mw[w]);
                    }
#pragma unroll
                    for (int w = 0; w < S::WG; ++w) lw[w] *= mw[w] == -INFINITY ? 1.f : ex2(mw[w] - mm[n][e]);   // 1: 0 or NaN
                    // the same whichever page parity came first
                    ll[n][e] = S::WG == 4 ? (lw[0] + lw[2 % S::WG]) + (lw[1] + lw[3 % S::WG]) : lw[0] + lw[1];
                    const float f = fu * (m[n][e] == -INFINITY ? 1.f : ex2(m[n][e] - mm[n][e]));
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
            const int slot = x.slot;                        // >= 0: a part of a unit
            float* part = a.part + (int64_t)slot * a.slot;
            if (wg == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int row = rg * S::PR + (FOLD ? 4 * n + t : 8 * n + 2 * t + e);
                        if (row >= x.pairs) continue;
                        const float inv = slot >= 0 ? 1.f : 1.f / ll[n][e], back = slot >= 0 ? 1.f : kv_pow2(uu);
                        const int pair = x.pair0 + row;
                        const int64_t yr = kv_row(c, (int64_t)x.row0 + pair / a.group);
                        const int head = x.h * a.group + pair % a.group;
#pragma unroll
                        for (int y = 0; y < HD / 32; ++y) {
                            const float w[4] = {o[2 * y][n][e] * inv * back, o[2 * y + 1][n][e] * inv * back,
                                                o[2 * y][n][2 + e] * inv * back, o[2 * y + 1][n][2 + e] * inv * back};
                            if (slot >= 0) store4_f(part + row * HD + 32 * y + 4 * g, w);
                            else store4_f(out + yr * a.ldo + (int64_t)head * HD + 32 * y + 4 * g, w);
                        }
                        if (g != 0) continue;
                        if (slot >= 0) {
                            part[a.prow * HD + row] = mm[n][e];
                            part[a.prow * (HD + 1) + row] = ll[n][e];
                            part[a.prow * (HD + 2) + row] = (float)uu;
                        } else if (a.lse) {
                            a.lse[yr * a.n_heads + head] = ((mm[n][e] == -INFINITY ? 0.f : mm[n][e]) - P_SHIFT + log2f(ll[n][e])) * LN2;
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
        // block's memory goes to another (again bounded)
        if (threadIdx.x == 0) {
            const uint64_t t0 = tcx::globaltimer();
            while (tcx::globaltimer() - t0 < 2000000) {}
        }
    }
}

// ----------------------------------------------------------------------------
// Joins the parts of cut units, in order: the block that begins one left its
// description.  W warps take a pair's parts in turn, lane i HD / 32 dims, and are
// then added in order; a block holds 8 / W pairs.
// ----------------------------------------------------------------------------
template <typename T, int HD, int W>
__global__ void __launch_bounds__(256) kv_join_kernel(const __grid_constant__ KvView c,
                                                      const __grid_constant__ AttnCall a, int total) {
    constexpr int D = HD / 32;
    __shared__ float sm[8], sl[8], so[8][HD];
    __shared__ int su[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at = blockIdx.x * (8 / W) + warp / W;         // (block of the attention kernel, pair)
    const int from = at / a.prow, row = at % a.prow;
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the attention kernel's results are visible from here on
    Cut u = {};
    if (at < total) u = a.cuts[from];
    const bool work = u.blocks > 0 && row < u.pairs;
    auto part = [&](int k) { return a.part + (int64_t)(k == 0 ? 2 * from + 1 : 2 * (from + k)) * a.slot; };
    // the running maximum M, sum l and sums o (in units of 2^U) of the warp's parts; JB parts' loads in flight
    constexpr int JB = 4;
    float M = -INFINITY, l = 0.f, o[D];
    int U = KV_MIN_EXP;
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] = 0.f;
    auto add = [&](float m, float lm, int unit, const float (&x)[D]) {
        const float v = fmaxf(M, m);
        const float fo = M == -INFINITY ? 1.f : ex2(M - v), fn = m == -INFINITY ? 1.f : ex2(m - v);   // 1: 0 or NaN stands there
        const int w = max(U, unit);
        const float po = fo * pow2_or_0(U - w), pn = fn * pow2_or_0(unit - w);
        l = l * fo + lm * fn;
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = o[d] * po + x[d] * pn;
        M = v;
        U = w;
    };
    if (work)
        for (int k0 = warp % W; k0 < u.blocks; k0 += JB * W) {
            float m[JB], lm[JB], un[JB], x[JB][D];
#pragma unroll
            for (int i = 0; i < JB; ++i) {
                const float* pk = part(k0 + i * W < u.blocks ? k0 + i * W : k0);
                m[i] = pk[a.prow * HD + row];
                lm[i] = pk[a.prow * (HD + 1) + row];
                un[i] = pk[a.prow * (HD + 2) + row];
#pragma unroll
                for (int d = 0; d < D; ++d) x[i][d] = pk[row * HD + lane + 32 * d];
            }
#pragma unroll
            for (int i = 0; i < JB; ++i)
                if (k0 + i * W < u.blocks) add(m[i], lm[i], (int)un[i], x[i]);
        }
    if (W > 1) {
        if (lane == 0) {
            sm[warp] = M;
            sl[warp] = l;
            su[warp] = U;
        }
#pragma unroll
        for (int d = 0; d < D; ++d) so[warp][lane + 32 * d] = o[d];
        __syncthreads();
        if (warp % W != 0) return;
#pragma unroll
        for (int w = 1; w < W; ++w) {
            float x[D];
#pragma unroll
            for (int d = 0; d < D; ++d) x[d] = so[warp + w][lane + 32 * d];
            add(sm[warp + w], sl[warp + w], su[warp + w], x);
        }
    }
    if (!work) return;
    const int pair = u.pair0 + row;
    const int64_t y = kv_row(c, (int64_t)u.row0 + pair / a.group);
    const int head = u.h * a.group + pair % a.group;
#pragma unroll
    for (int d = 0; d < D; ++d) static_cast<T*>(a.out)[y * a.ldo + (int64_t)head * HD + lane + 32 * d] = from_f<T>(o[d] / l * kv_pow2(U));
    if (lane == 0 && a.lse) a.lse[y * a.n_heads + head] = ((M == -INFINITY ? 0.f : M) - P_SHIFT + log2f(l)) * LN2;
}

template <typename T, int HD, int NT, int RG, int PG_>
cudaError_t attn_t(const KvView& c, const KvAttnArgs& a, cudaStream_t s, int64_t* launches) {
    using S = AttnShape<T, HD, NT, RG, PG_>;
    // once a device: its SMs, and the kernel's shared memory (the attribute stays with the function)
    static std::atomic<int> sms[64];
    int dev = 0, n_sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) n_sms = sms[dev].load(std::memory_order_relaxed);
    if (n_sms == 0) {
        e = cudaFuncSetAttribute(kv_attn_kernel<T, HD, NT, RG, PG_>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kv_attn_kernel<T, HD, NT, RG, PG_>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < 64) sms[dev].store(n_sms, std::memory_order_relaxed);
    }
    AttnCall k;
    k.q = a.q; k.out = a.out; k.lse = a.lse; k.ldq = a.ldq; k.ldo = a.ldo;
    k.n_heads = a.n_heads; k.group = a.n_heads / c.n_kv;
    k.qk = (float)frexp((double)a.scale * LOG2E, &k.qk_exp);
    const int64_t pairs = (int64_t)c.max_rows * k.group;
    k.prow = (int)(pairs < S::ROWS ? pairs : S::ROWS);
    k.slot = ((int64_t)k.prow * (HD + 3) + 3) / 4 * 4;      // 16-byte aligned
    const int64_t units = (pairs + S::ROWS - 1) / S::ROWS * c.n_kv * c.n_seqs;
    const int64_t cap = (int64_t)c.max_pages * KV_PAGE;
    const int64_t longest = c.max_len < cap ? c.max_len : cap;
    const int64_t pages = longest > 0 ? (longest + KV_PAGE - 1) / KV_PAGE : 1;
    // The blocks' equal shares cut sequences anywhere; a share's two ends leave
    // partial results.  Short sequences and small workspaces: whole units only.
    const int64_t most = (int64_t)n_sms * S::BLOCKS_SM;
    int64_t blocks = (units * pages + KV_SHORT_RUN - 1) / KV_SHORT_RUN;
    if (blocks > most) blocks = most;
    const bool cut = pages > KV_WHOLE && a.workspace &&
                     a.workspace_bytes >= blocks * (2 * k.slot * (int64_t)sizeof(float) + (int64_t)sizeof(Cut));
    if (!cut) blocks = units < most ? units : most;
    k.part = static_cast<float*>(a.workspace);
    k.cuts = cut ? reinterpret_cast<Cut*>(k.part + blocks * 2 * k.slot) : nullptr;
    kv_attn_kernel<T, HD, NT, RG, PG_><<<(unsigned)blocks, S::THREADS, S::SMEM, s>>>(c, k);
    e = cudaGetLastError();
    if (launches) *launches += cut ? 2 : 1;
    if (e != cudaSuccess || !cut) return e;
    // the join waits on the device for the attention kernel's end: only its launch overlaps it
    const int total = (int)(blocks * k.prow);
    const bool many = blocks / units > 8;                   // parts of a unit: 8 warps a pair, or one
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(many ? total : (total + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, many ? kv_join_kernel<T, HD, 8> : kv_join_kernel<T, HD, 1>, c, k, total);
}

// One column tile (8 pairs; 4 on fp32) where a sequence's pairs fit it.  More row
// groups share each page tile (its reads and its place in shared memory) where a
// sequence has more: two of a tile, or, where that pads little, four of two tiles,
// which convert each byte for twice the columns (32 sequences of 1023 to 8191
// tokens, 8 heads of 128: 36 pairs 181 us in tiles of 64, 132 in tiles of 16; 64
// pairs 184 and 202; 72 pairs 337 and 247; 8 prompts of 2000 rows 2.09 and 2.25 ms;
// fp32, 32 and 8: 231 and 209, 304 and 359, 443 and 402, 3.58 and 4.09 ms).  A single
// row group has two pages in work; or, heads of 128 and many units, one page and
// more blocks, which hide the ends of units better (256 sequences of 512 to 2048
// tokens, 2048 units: 122 us against 118; of 64 to 512: 75 against 64; one of 130,001,
// 8 units: 54.0 against 55.8; heads of 64, 656 units: 31.7 against 40.6; where units
// are twice as long, 64 sequences of 1000 to 4001 and 16 heads, 109 against 113).
// That choice looks at the whole batch, so it is made only where the workspace lets
// results depend on it.  The tile follows the call's largest row count: a prompt of
// 2000 rows beside 255 single tokens takes 694 us, the two in calls of their own 300
// and 117.
constexpr int64_t KV_MANY = 600;
template <typename T, int HD>
cudaError_t attn_rows(const KvView& c, const KvAttnArgs& a, cudaStream_t s, int64_t* launches) {
    constexpr int PR = AttnShape<T, HD, 1, 1, 2>::PR;
    const int64_t pairs = (int64_t)c.max_rows * (a.n_heads / c.n_kv);
    if (pairs <= PR) {
        if constexpr (HD == 128)
            if (a.workspace && a.workspace_bytes >= MLORA_KV_WORKSPACE_BYTES && (int64_t)c.n_seqs * c.n_kv >= KV_MANY)
                return attn_t<T, HD, 1, 1, 1>(c, a, s, launches);
        return attn_t<T, HD, 1, 1, 2>(c, a, s, launches);
    }
    // in columns, a padded one of the larger tile at 8 / 9 of the smaller one's cost
    const int64_t small = (pairs + 2 * PR - 1) / (2 * PR) * 2 * PR, large = (pairs + 8 * PR - 1) / (8 * PR) * 8 * PR;
    return 8 * large <= 9 * small ? attn_t<T, HD, 2, 4, 1>(c, a, s, launches) : attn_t<T, HD, 1, 2, 1>(c, a, s, launches);
}

}  // namespace

cudaError_t launch_kv_attention(const KvView& c, int head_dim, int dtype, const KvAttnArgs& a, cudaStream_t s,
                                int64_t* launches) {
    if (dtype == MLORA_BF16) return (head_dim == 64 ? attn_rows<bf16, 64> : attn_rows<bf16, 128>)(c, a, s, launches);
    return (head_dim == 64 ? attn_rows<float, 64> : attn_rows<float, 128>)(c, a, s, launches);
}

}  // namespace mlk

using namespace mlk;

namespace {

// Whether a row that the call writes holds a part of a row that it may still
// read: n rows of `row` bytes, sq and so >= row bytes apart.  The queries
// themselves as the output are no such case.
bool rows_clash(uintptr_t q, int64_t sq, uintptr_t o, int64_t so, int64_t row, int64_t n) {
    if (q == o && (sq == so || n == 1)) return false;
    if (o >= q + (n - 1) * sq + row || q >= o + (n - 1) * so + row) return false;
    if (sq == so) {                                         // columns of one buffer: side by side or not
        const int64_t d = (int64_t)((o > q ? o - q : q - o) % (uintptr_t)so);
        return d < row || so - d < row;
    }
    for (int64_t i = 0; i < n; ++i) {                       // the output rows that begin just before and behind row i
        const int64_t at = (int64_t)(q - o) + i * sq;
        const int64_t j = at >= 0 ? at / so : -1;
        if (j >= 0 && j < n && at - j * so < row) return true;
        if (j + 1 < n && (j + 1) * so - at < row) return true;
    }
    return false;
}

}  // namespace

extern "C" int mlora_kv_attention(const mlora_kv_cache* c, const mlora_kv_seqs* q, const mlora_kv_attn* a,
                                  void* stream) {
    if (!a) return kv_fail(MLORA_E_ARG, "NULL attention arguments");
    KvView w;
    const int rc = kv_check(c, q, a->dtype, a->max_len, &w);
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
    const int64_t es = 16 / per16, furthest = INT64_MAX / 16 / w.n_rows;
    if (a->q_stride > furthest || a->out_stride > furthest)
        return kv_fail(MLORA_E_ARG, "query or output rows are further apart than memory reaches");
    if (rows_clash(reinterpret_cast<uintptr_t>(a->q), a->q_stride * es, reinterpret_cast<uintptr_t>(a->out),
                   a->out_stride * es, row * es, w.n_rows))
        return kv_fail(MLORA_E_ARG, "the output's rows overlap queries (out may be q, with its stride, or lie apart)");
    if ((reinterpret_cast<uintptr_t>(a->workspace) & 15) || a->workspace_bytes < 0)
        return kv_fail(MLORA_E_ARG, "the workspace must be 16-byte aligned");
    if ((int64_t)w.max_rows * a->n_heads > INT32_MAX / w.n_seqs)
        return kv_fail(MLORA_E_ARG, "too many sequences, rows and heads for one call");
    KvAttnArgs k;
    k.q = a->q; k.out = a->out; k.lse = a->lse; k.workspace = a->workspace; k.ldq = a->q_stride; k.ldo = a->out_stride;
    k.workspace_bytes = a->workspace_bytes; k.n_heads = a->n_heads; k.scale = a->scale;
    const cudaError_t e = launch_kv_attention(w, c->head_dim, a->dtype, k, reinterpret_cast<cudaStream_t>(stream), nullptr);
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}
