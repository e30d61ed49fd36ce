// Attention of a call's newest rows over the 8-bit key/value cache
// (include/mlora_kv.h): for each row and query head, one pass over the cached
// positions with a running maximum and sum,
//     s_i = scale q . k_i,  out = sum_i exp(s_i - lse) v_i,  lse = log sum_i exp(s_i).
//
// What bounds it.  Few rows a sequence: every cached byte is read once and used
// for rows x group products, far below the tensor cores' rate, so the cache's
// bytes over the HBM rate are the floor.  The design streams pages and keeps
// the arithmetic beside the stream cheap:
//  * One block handles 16 RG of a sequence's (row, head of the group) pairs
//    against one key/value head, over a run of pages.  A producer warp copies
//    each (page, head) tile of K and V -- contiguous 8 KB at head_dim 128 --
//    into a ring of stages with cp.async.bulk.
//  * The pairs are the 16 rows of mma.sync m16n8k16 (fp16 operands, fp32 sums):
//    an e4m3 byte is exactly an fp16 value, two bytes convert in one
//    instruction, and M = 16 fits the few rows of a decode step, where a
//    128-row tcgen05 tile would be at most an eighth full and would want the
//    converted tile written back to shared memory first.  The page's byte
//    order (mlora_kv.h) puts each thread's fragment bytes side by side.
//  * q enters as fp16 relative to its row's largest magnitude (a power of two,
//    folded into the scale): exact for bf16 down to 2^-17 of that magnitude,
//    and as a high and a low part (2^-22) on fp32.
//  * The page's value scale 2^ev goes into the exponent of the probability,
//    p' = exp2(s log2 e + ev - m') with m' the running maximum of s log2 e + ev,
//    so pages of any scale add into one accumulator, the largest p' v8 sets the
//    precision, and l += p' 2^-ev is what the definition sums.  m' follows the
//    scores only when one passes it by 2^3 (the sums are then rescaled); p' is
//    held at 2^12 times its value, so that it stays within fp16 and its rounding
//    relative (2^-11) down to 2^-26 of the reference (absolute 2^-37 of it
//    below that); on fp32 it is split like q.
//  * Warps of a block take different halves of a page and, with one or two row
//    groups, every other page, 32 tokens at a step (four independent chains of
//    products); each has a running maximum and sum of its own, joined at the
//    end, so nothing but the ring's barriers is shared in the loop.
//  * Long sequences are cut into runs of pages (flash-style split); a block
//    leaves its rows' unnormalised sums, maximum and sum in the workspace, and
//    the last block of the sequence and head to arrive joins them in order of
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
constexpr int KV_SPLIT_BLOCKS = 456;
constexpr int KV_LONG_RUN = 16, KV_SHORT_RUN = 2;

struct AttnCall {
    const void* q;
    void* out;
    float* lse;
    int* counters;
    float* part;
    int64_t ldq, ldo, max_len;
    int n_heads, group;
    int tiles;                              // blocks' row tiles of a (sequence, key/value head)
    int splits, chunk;                      // runs of `chunk` pages
    int prow;                               // rows of a partial result
    int64_t slot;                           // its floats: the rows' sums, maxima and sums of p
    float qk;                               // scale * log2 e
};

template <typename T, int HD, int RG>
struct AttnShape {
    static constexpr int NP = sizeof(T) == 4 ? 2 : 1;       // fp16 parts of q and of p
    static constexpr int PG = RG == 4 ? 1 : 2;              // pages in work at once
    static constexpr int WG = 2 * PG;                       // warps of a row group: page parity x half of the page
    static constexpr int NW = RG * WG;                      // consumer warps
    static constexpr int THREADS = 32 * NW + 32;
    static constexpr int TILE = KV_PAGE * HD;               // bytes of a K or V tile
    static constexpr int STAGE = 2 * TILE;
    static constexpr int STAGES = HD == 128 ? 4 : 6;
    static constexpr int ROWS = 16 * RG;
    static constexpr int BLOCKS_SM = RG == 1 ? 3 : 1;
    // ring, then q's fragments, barriers (16 B each stage), exponents, per-warp statistics, flags
    static constexpr int QFRAG = STAGES * STAGE;
    static constexpr int BAR = QFRAG + RG * NP * (HD / 16) * 32 * 16;
    static constexpr int EXPS = BAR + 16 * STAGES;
    static constexpr int STAT = EXPS + 8 * STAGES;
    static constexpr int FLAGS = STAT + 2 * 4 * WG * ROWS;
    static constexpr int SMEM = FLAGS + 16;
    static_assert(WG * ROWS * HD * 4 <= QFRAG, "the joined sums reuse the ring");
    static_assert(STAGES % PG == 0, "a stage keeps its page parity");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
                 : "memory");
}
// expected bytes without an arrival
__device__ __forceinline__ void mbar_expect_only(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
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

template <typename T, int HD, int RG>
__global__ void __launch_bounds__(AttnShape<T, HD, RG>::THREADS, AttnShape<T, HD, RG>::BLOCKS_SM)
    kv_attn_kernel(const __grid_constant__ KvView c, const __grid_constant__ AttnCall a) {
    using S = AttnShape<T, HD, RG>;
    constexpr int NP = S::NP;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = tcx::smem_u32(smem);
    int* exps = reinterpret_cast<int*>(smem + S::EXPS);     // per stage: K's and V's exponent
    float* st_m = reinterpret_cast<float*>(smem + S::STAT);
    float* st_l = st_m + S::WG * S::ROWS;
    volatile int* flags = reinterpret_cast<volatile int*>(smem + S::FLAGS);   // abort, bad page, last, never set
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full = [&](int i) { return sbase + S::BAR + 16 * i; };
    auto empty = [&](int i) { return sbase + S::BAR + 16 * i + 8; };

    const int split = (int)(blockIdx.x % a.splits);
    const int unit = (int)(blockIdx.x / a.splits);          // (sequence, key/value head, row tile)
    const int tile = unit % a.tiles;
    const int h = unit / a.tiles % c.n_kv;
    const int s = unit / a.tiles / c.n_kv;
    const int page0 = split * a.chunk;
    // the producer's first page ids, asked for before the length is known
    int id = -1;
    if (warp == S::NW && lane < a.chunk && page0 + lane < c.max_pages)
        id = c.table[(int64_t)s * c.max_pages + page0 + lane];

    SeqRows r;
    const bool ok = kv_seq(c, s, a.max_len, r);
    const T* q = static_cast<const T*>(a.q);
    T* out = static_cast<T*>(a.out);
    if (!ok || r.len == 0) {
        // rows without positions: zero (or NaN: a bad sequence), from one block of each head
        if (split == 0 && tile == 0) {
            const float v = ok ? 0.f : NAN;
            const int64_t r1 = (int64_t)r.row0 + r.n < c.n_rows ? (int64_t)r.row0 + r.n : c.n_rows;
            for (int64_t x = r.row0 < 0 ? 0 : r.row0; x < r1; ++x) {
                const int64_t y = kv_row(c, x);
                for (int d = threadIdx.x; d < a.group * HD; d += S::THREADS) out[y * a.ldo + h * a.group * HD + d] = from_f<T>(v);
                for (int d = threadIdx.x; a.lse && d < a.group; d += S::THREADS)
                    a.lse[y * a.n_heads + h * a.group + d] = ok ? -INFINITY : NAN;
            }
        }
        return;
    }
    const int pair0 = tile * S::ROWS;                       // first (row, head) pair of the tile
    const int pairs = r.n * a.group;
    if (pair0 >= pairs) return;
    const int before = r.len - r.n;                         // positions before the sequence's rows
    const int pair1 = pair0 + S::ROWS < pairs ? pair0 + S::ROWS : pairs;
    const int lim_lo = before + pair0 / a.group + 1;        // positions that the tile's first row sees
    const int lim_hi = before + (pair1 - 1) / a.group + 1;  // .. and its last
    const int pages = (lim_hi + KV_PAGE - 1) / KV_PAGE;
    const int nsplit = (pages + a.chunk - 1) / a.chunk;
    if (split >= nsplit) return;
    const int np = pages - page0 < a.chunk ? pages - page0 : a.chunk;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            tcx::mbar_init(full(i), 1);
            tcx::mbar_init(empty(i), S::NW / S::PG);
        }
        flags[0] = flags[1] = flags[2] = flags[3] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    float o[HD / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int g = lane >> 2, t = lane & 3;
    const int rg = warp / S::WG, wg = warp % S::WG;         // consumers: row group, place in it
    const int half = wg & 1, pg = wg >> 1;                  // half of a page, page parity
    if (warp == S::NW) {
        // ---- producer
        bool go = true;
        for (int i0 = 0; i0 < np && go; i0 += 32) {
            const int mine = i0 + lane;
            if (i0 > 0 && mine < np) id = c.table[(int64_t)s * c.max_pages + page0 + mine];
            bool good = true;
            if (mine < np && (id < 0 || id >= c.n_pages)) {
                raise_status(c.status, ST_RANGE);
                good = false;
                id = 0;                                     // a page that exists stands in; the rows become NaN
            }
            if (__any_sync(0xffffffffu, !good) && lane == 0) flags[1] = 1;
            const int64_t at = (int64_t)(mine < np ? id : 0) * c.n_kv + h;
            int ek = 0, ev = 0;
            const int n = np - i0 < 32 ? np - i0 : 32;
            bool have = false;
            for (int i = 0; i < n; ++i) {
                const int it = i0 + i, stage = it % S::STAGES;
                const int64_t tile_at = __shfl_sync(0xffffffffu, at, i);
                const int left = lim_hi - (page0 + it) * KV_PAGE;               // tokens of the page that count
                const int tok = left < KV_PAGE ? left : KV_PAGE;
                if (it >= S::STAGES) {
                    if (lane == 0) go = tcx::mbar_wait(empty(stage), (it / S::STAGES - 1) & 1, flags);
                    go = __shfl_sync(0xffffffffu, (int)go, 0);
                    if (!go) {
                        if (lane == 0) {
                            raise_status(c.status, ST_TIMEOUT);
                            flags[0] = 1;
                        }
                        break;
                    }
                }
                if (lane == 0) {
                    const uint32_t kb = tok * HD, vb = (tok + 3) / 4 * 4 * HD;
                    mbar_expect_only(full(stage), kb + vb);
                    bulk_load(sbase + stage * S::STAGE, c.k + tile_at * S::TILE, kb, full(stage));
                    bulk_load(sbase + stage * S::STAGE + S::TILE, c.v + tile_at * S::TILE, vb, full(stage));
                }
                if (!have && (i + 1 == S::STAGES || i + 1 == n)) {
                    // the scales of these pages, read behind the first copies
                    if (mine < np) {
                        ek = scale_exp(c.ks[at]);
                        ev = scale_exp(c.vs[at]);
                    }
                    have = true;
                    for (int j = 0; j <= i; ++j) {
                        const int k_ = __shfl_sync(0xffffffffu, ek, j), v_ = __shfl_sync(0xffffffffu, ev, j);
                        if (lane == 0) {
                            exps[2 * ((i0 + j) % S::STAGES)] = k_;
                            exps[2 * ((i0 + j) % S::STAGES) + 1] = v_;
                            tcx::mbar_arrive(full((i0 + j) % S::STAGES));
                        }
                    }
                } else if (have) {
                    const int k_ = __shfl_sync(0xffffffffu, ek, i), v_ = __shfl_sync(0xffffffffu, ev, i);
                    if (lane == 0) {
                        exps[2 * stage] = k_;
                        exps[2 * stage + 1] = v_;
                        tcx::mbar_arrive(full(stage));
                    }
                }
            }
        }
    } else {
        // ---- consumers: q fragments, written by the group's first warps and read
        // from shared memory at each step (the registers go to the sums).  A
        // thread's dims at K step (y, i) are 64 y + 16 t + 4 i + 0..3, the four
        // bytes of a word of the key tile.
        uint4* qs = reinterpret_cast<uint4*>(smem + S::QFRAG) + rg * NP * (HD / 16) * 32 + lane;
        float qf[2];                                        // scale * log2 e, or NaN where q is not finite
        int qe[2];                                          // exponent of the row's largest magnitude
        int limit[2];                                       // positions the row sees
        {
            uint32_t qa[NP][HD / 16][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int pair = pair0 + rg * 16 + g + 8 * e;
                const bool live = pair < pairs;
                limit[e] = live ? before + pair / a.group + 1 : 0;
                const T* src = live ? q + kv_row(c, (int64_t)r.row0 + pair / a.group) * a.ldq +
                                          ((int64_t)h * a.group + pair % a.group) * HD
                                    : nullptr;
                float x[HD / 64][16];
                float big = 0.f;
                bool fin = true;
#pragma unroll
                for (int y = 0; y < HD / 64; ++y) {
                    if (live) {
                        load16_f(src + 64 * y + 16 * t, x[y]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[y][i] = 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        big = fmaxf(big, fabsf(x[y][i]));
                        fin &= fabsf(x[y][i]) <= FLT_MAX;
                    }
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const unsigned nf = __ballot_sync(0xffffffffu, !fin);
                int ex = 0;
                if (big > 0.f && big <= FLT_MAX) frexpf(big, &ex);
                qe[e] = ex;
                qf[e] = (nf >> (lane & 28)) & 15u ? NAN : a.qk;
                // 2^-ex in two steps: it can lie outside fp32
                const float f1 = kv_pow2(-ex / 2), f2 = kv_pow2(-ex - (-ex / 2));
#pragma unroll
                for (int y = 0; y < HD / 64; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const float u = x[y][4 * i + 2 * z] * f1 * f2, w = x[y][4 * i + 2 * z + 1] * f1 * f2;
                            const uint32_t hi = half2_bits(u, w);
                            qa[0][4 * y + i][2 * z + e] = hi;
                            if (NP == 2) qa[NP - 1][4 * y + i][2 * z + e] = half2_rest(u, w, hi);
                        }
            }
            if (wg == 0) {
#pragma unroll
                for (int n = 0; n < NP; ++n)
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        qs[(n * (HD / 16) + k) * 32] = make_uint4(qa[n][k][0], qa[n][k][1], qa[n][k][2], qa[n][k][3]);
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * S::NW) : "memory");   // the consumers
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[j][x] = 0.f;

        for (int it = pg; it < np; it += S::PG) {
            const int stage = it % S::STAGES;
            if (!tcx::mbar_wait(full(stage), (it / S::STAGES) & 1, flags)) {
                if (lane == 0) {
                    raise_status(c.status, ST_TIMEOUT);
                    flags[0] = 1;
                }
                break;
            }
            const int ek = exps[2 * stage], ev = exps[2 * stage + 1];
            const uint32_t kt = sbase + stage * S::STAGE, vt = kt + S::TILE;
            const int p0 = (page0 + it) * KV_PAGE + 32 * half;      // the first of this warp's 32 positions
            const float fk[2] = {qf[0] * pow2_clamped(qe[0] + ek), qf[1] * pow2_clamped(qe[1] + ek)};
            const float fev = (float)ev, inv_vs = kv_pow2(-ev);
            // EDGE: some row does not see all 32 positions
            auto step = [&](auto edge) {
                constexpr bool EDGE = decltype(edge)::value;
                // S = q K^T, 16 tokens a slice u: column n of key tile j is token 4 (n / 2) + 2 j + n % 2
                float z[2][2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j) z[u][j][0] = z[u][j][1] = z[u][j][2] = z[u][j][3] = 0.f;
#pragma unroll
                for (int y = 0; y < HD / 64; ++y) {
                    uint4 w[2][2];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            w[u][j] = lds128(kt + kv_byte_k<HD>(32 * half + 16 * u + 4 * (g >> 1) + 2 * j + (g & 1),
                                                                64 * y + 16 * t));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t qa[NP][4];
#pragma unroll
                        for (int n = 0; n < NP; ++n) {
                            const uint4 v = qs[(n * (HD / 16) + 4 * y + i) * 32];
                            qa[n][0] = v.x; qa[n][1] = v.y; qa[n][2] = v.z; qa[n][3] = v.w;
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t b = i == 0 ? w[u][j].x : i == 1 ? w[u][j].y : i == 2 ? w[u][j].z : w[u][j].w;
                                const uint32_t b0 = e4m3x2_to_half2((uint16_t)b);
                                const uint32_t b1 = e4m3x2_to_half2((uint16_t)(b >> 16));
#pragma unroll
                                for (int n = 0; n < NP; ++n) mma16816(z[u][j], qa[n], b0, b1);
                            }
                    }
                }
                // scores in units of log2, with the value scale's exponent; this lane's largest
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float s2 = fmaf(z[u][j][x], fk[x >> 1], fev);
                            if (EDGE && p0 + 16 * u + 4 * t + 2 * j + (x & 1) >= limit[x >> 1]) s2 = -INFINITY;
                            mx[x >> 1] = fmaxf(mx[x >> 1], s2);
                        }
                // the reference moves only when a score passes it by 2^M_SLACK: then p' stays below fp16's range
                if (__any_sync(0xffffffffu, mx[0] > m[0] + M_SLACK || mx[1] > m[1] + M_SLACK)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                        mx[e] = fmaxf(mx[e], m[e]);
                        const float f = mx[e] == -INFINITY ? 1.f : ex2(m[e] - mx[e]);
                        m[e] = mx[e];
                        l[e] *= f;
#pragma unroll
                        for (int j = 0; j < HD / 8; ++j) {
                            o[j][2 * e] *= f;
                            o[j][2 * e + 1] *= f;
                        }
                    }
                }
                const float off[2] = {fev + P_SHIFT - (m[0] == -INFINITY ? 0.f : m[0]),
                                      fev + P_SHIFT - (m[1] == -INFINITY ? 0.f : m[1])};
                float add[2] = {0.f, 0.f};
                uint32_t p[2][NP][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float e2 = fmaf(z[u][j][x], fk[x >> 1], off[x >> 1]);
                            if (EDGE && p0 + 16 * u + 4 * t + 2 * j + (x & 1) >= limit[x >> 1]) e2 = -INFINITY;
                            z[u][j][x] = ex2(e2);
                            add[x >> 1] += z[u][j][x];
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t hi = half2_bits(z[u][j][2 * e], z[u][j][2 * e + 1]);
                            p[u][0][2 * j + e] = hi;
                            if (NP == 2) p[u][NP - 1][2 * j + e] = half2_rest(z[u][j][2 * e], z[u][j][2 * e + 1], hi);
                        }
                    }
                l[0] = fmaf(add[0], inv_vs, l[0]);
                l[1] = fmaf(add[1], inv_vs, l[1]);
                // O += P V: dim 32 x + 4 n + e is column n of tile 4 x + e
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // bytes of tokens behind the end can be anything, NaN among them: 0 stands in.  A NaN
                    // among the newest tokens' values must not reach the rows before it through 0 * NaN
                    // either: the product takes 0 for it, and the rows that do see it are found by a
                    // second product.
                    const int first = p0 + 16 * u + 4 * t;  // of this lane's four tokens
                    const int valid = lim_hi - first;
                    const uint32_t keep = valid >= 4 ? 0xffffffffu : (valid <= 0 ? 0u : (1u << (8 * valid)) - 1u);
#pragma unroll
                    for (int x = 0; x < HD / 32; ++x) {
                        const uint4 w = lds128(vt + (8 * half + 4 * u + t) * 4 * HD + (((8 * x + g) ^ (2 * t)) << 4));
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t b = ws[e];
                            if (EDGE) {
                                b &= keep;
                                const uint32_t nan = __vcmpeq4(b & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                if (__any_sync(0xffffffffu, nan != 0)) {
                                    b &= ~nan;
                                    uint32_t see[4];
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {   // 1.0 where row k % 2 sees tokens 2 (k / 2) + 0, 1
                                        const int left = limit[k & 1] - (first + (k & 2));
                                        see[k] = (left > 0 ? 0x3c00u : 0u) | (left > 1 ? 0x3c000000u : 0u);
                                    }
                                    float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma16816(hit, see, e4m3x2_to_half2((uint16_t)(nan & 0x3838u)),   // 0x38 is 1.0
                                             e4m3x2_to_half2((uint16_t)((nan >> 16) & 0x3838u)));
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        if (hit[k] > 0.f) o[4 * x + e][k] = NAN;
                                }
                            }
                            const uint32_t b0 = e4m3x2_to_half2((uint16_t)b);
                            const uint32_t b1 = e4m3x2_to_half2((uint16_t)(b >> 16));
#pragma unroll
                            for (int n = 0; n < NP; ++n) mma16816(o[4 * x + e], p[u][n], b0, b1);
                        }
                    }
                }
            };
            if (p0 + 32 <= lim_lo) step(std::false_type{});
            else if (p0 < lim_hi) step(std::true_type{});
            __syncwarp();
            if (lane == 0) tcx::mbar_arrive(empty(stage));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (t == 0) {
                st_m[wg * S::ROWS + rg * 16 + g + 8 * e] = m[e];
                st_l[wg * S::ROWS + rg * 16 + g + 8 * e] = l[e];
            }
        }
    }
    __syncthreads();                                        // every page is used: the ring's memory is free
    if (flags[0]) {
        // a wait gave up: let the copies that may still be in flight land
        // before the block's memory goes to another (again bounded), write nothing
        if (threadIdx.x == 0)
            for (int i = 0; i < S::STAGES && i < np; ++i) {
                const int last = (np - 1 - i) / S::STAGES * S::STAGES + i;
                tcx::mbar_wait(full(i), (last / S::STAGES) & 1, flags + 3, 1000000);
            }
        return;
    }
    // ---- join the warps of a row group
    float* so = reinterpret_cast<float*>(smem);             // [WG][ROWS][HD]
    if (warp < S::NW) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = rg * 16 + g + 8 * e;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < S::WG; ++w) mm = fmaxf(mm, st_m[w * S::ROWS + row]);
            const float f = m[e] == -INFINITY ? (mm == -INFINITY ? 1.f : 0.f) : ex2(m[e] - mm);
            float* dst = so + (wg * S::ROWS + row) * HD + 8 * t;
#pragma unroll
            for (int x = 0; x < HD / 32; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    *reinterpret_cast<float4*>(dst + 32 * x + 4 * y) =
                        make_float4(o[4 * x][2 * e + y] * f, o[4 * x + 1][2 * e + y] * f, o[4 * x + 2][2 * e + y] * f,
                                    o[4 * x + 3][2 * e + y] * f);
        }
    }
    __syncthreads();
    const int rows = pair1 - pair0;
    float* part = a.part + (int64_t)blockIdx.x * a.slot;
    const bool bad = flags[1] != 0;
    for (int i = threadIdx.x; i < rows * (HD / 4); i += S::THREADS) {
        const int row = i / (HD / 4), d = i % (HD / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < S::WG; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(so + (w * S::ROWS + row) * HD + d);
            v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
            mm = fmaxf(mm, st_m[w * S::ROWS + row]);
        }
#pragma unroll
        for (int w = 0; w < S::WG; ++w) {
            const float mw = st_m[w * S::ROWS + row];
            ll += st_l[w * S::ROWS + row] * (mw == -INFINITY ? 1.f : ex2(mw - mm));
        }
        if (bad) ll = NAN;
        if (nsplit > 1) {
            *reinterpret_cast<float4*>(part + row * HD + d) = v;
            if (d == 0) {
                part[a.prow * HD + row] = mm;
                part[a.prow * (HD + 1) + row] = ll;
            }
        } else {
            const int pair = pair0 + row;
            const int64_t y = kv_row(c, (int64_t)r.row0 + pair / a.group);
            const int head = h * a.group + pair % a.group;
            const float inv = 1.f / ll;
            const float w[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
            store4_f(out + y * a.ldo + (int64_t)head * HD + d, w);
            if (d == 0 && a.lse) a.lse[y * a.n_heads + head] = ((mm == -INFINITY ? 0.f : mm) - P_SHIFT + log2f(ll)) * LN2;
        }
    }
    if (nsplit == 1) return;
    // ---- the last block of the unit to arrive joins its runs
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const int arrived = atomicAdd(a.counters + unit, 1);
        flags[2] = arrived == nsplit - 1;
        if (arrived == nsplit - 1) a.counters[unit] = 0;    // as the next call finds it
        __threadfence();
    }
    __syncthreads();
    if (!flags[2]) return;
    const float* p0 = a.part + (int64_t)unit * a.splits * a.slot;
    for (int i = threadIdx.x; i < rows * (HD / 4); i += S::THREADS) {
        const int row = i / (HD / 4), d = i % (HD / 4) * 4;
        float mm = -INFINITY;
        for (int x = 0; x < nsplit; ++x) mm = fmaxf(mm, __ldcg(p0 + x * a.slot + a.prow * HD + row));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float ll = 0.f;
#pragma unroll 8
        for (int x = 0; x < nsplit; ++x) {
            const float* px = p0 + x * a.slot;
            const float mw = __ldcg(px + a.prow * HD + row);
            const float f = mw == -INFINITY ? 1.f : ex2(mw - mm);   // 1: nothing but 0 or NaN stands there
            const float4 u = __ldcg(reinterpret_cast<const float4*>(px + row * HD + d));
            ll = fmaf(__ldcg(px + a.prow * (HD + 1) + row), f, ll);
            v.x = fmaf(u.x, f, v.x); v.y = fmaf(u.y, f, v.y); v.z = fmaf(u.z, f, v.z); v.w = fmaf(u.w, f, v.w);
        }
        const int pair = pair0 + row;
        const int64_t y = kv_row(c, (int64_t)r.row0 + pair / a.group);
        const int head = h * a.group + pair % a.group;
        const float inv = 1.f / ll;
        const float w[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
        store4_f(out + y * a.ldo + (int64_t)head * HD + d, w);
        if (d == 0 && a.lse) a.lse[y * a.n_heads + head] = ((mm == -INFINITY ? 0.f : mm) - P_SHIFT + log2f(ll)) * LN2;
    }
}

constexpr int MAX_UNITS_SPLIT = MLORA_KV_COUNTER_BYTES / 4;   // a counter for each unit

template <typename T, int HD, int RG>
cudaError_t attn_t(const KvView& c, const KvAttnArgs& a, cudaStream_t s) {
    using S = AttnShape<T, HD, RG>;
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
    // Runs of pages: short enough that the blocks fill the GPU (about BLOCKS_SM
    // on each SM) and that a long sequence is no tail of the launch, long
    // enough that a block's start and the join stay small beside it.
    int64_t chunk = pages;
    if (units <= MAX_UNITS_SPLIT) {
        const int64_t want = (int64_t)KV_SPLIT_BLOCKS;
        const int64_t per_unit = (want + units - 1) / units;
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
    const int64_t blocks = units * k.splits;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    // once a device: the attribute stays with the function
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(kv_attn_kernel<T, HD, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    kv_attn_kernel<T, HD, RG><<<(unsigned)blocks, S::THREADS, S::SMEM, s>>>(c, k);
    return cudaGetLastError();
}

// 16 pairs a block where one row's group fits; more row groups share each page
// tile (its reads and its place in shared memory) where a sequence has more.
template <typename T, int HD>
cudaError_t attn_rows(const KvView& c, const KvAttnArgs& a, cudaStream_t s) {
    const int64_t pairs = (int64_t)c.max_rows * (a.n_heads / c.n_kv);
    if (pairs <= 16) return attn_t<T, HD, 1>(c, a, s);
    if (pairs <= 32) return attn_t<T, HD, 2>(c, a, s);
    return attn_t<T, HD, 4>(c, a, s);
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
