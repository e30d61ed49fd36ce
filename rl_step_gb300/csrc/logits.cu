// Log-probabilities of given tokens with entropy, log-sum-exp and alternatives,
// and their gradient in the logits (include/mlora_logits.h).
//
// What bounds both: bytes.  The forward reads each logit once, the gradient
// reads and writes each once.  8,192 bf16 rows of 151,936 logits: the forward 367 us
// without alternatives, 100 % of the copy rate, 408 with 5 and 421 with 20, whose search
// stops a team's reads; the gradient 652 us, a fifth of the rows zeros (101 %).  Few or
// short rows: the launch and the chain of a row's joins, 8 us for one row of 151,936 (a
// cluster of eight blocks), 4.4 us for 1,024 of 1,000.
//
// Forward.  A team of threads (a warp to a block by the vocabulary, a cluster of blocks
// where the rows are few) takes a row.  In base 2, with c = scale log2 e,
// each thread keeps the maximum m of its x c and
//     s = sum 2^(x c - m),   t = sum 2^(x c - m) (x c - m),
// corrected when m rises, a group of 16 logits at a time; joined over the team
//     lse = (m + log2 s) ln 2,   entropy = (log2 s - t / s) ln 2.
// m is the maximum itself, so the largest term of t is 0 and the entropy of a sure
// row does not come from a difference of large numbers.
// Alternatives without a second pass: a thread leaves each group's largest value
// in shared memory.  The `top` largest groups -- of equal ones the first -- hold all
// alternatives, as a group is 16 ids in a row; they are found from 64-bit keys
// (value, complement of the id), whose order is the order of the results, and only
// their 32 or 64 bytes are read again.
#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>

#include "kv_common.cuh"
#include "logits.cuh"
#include "packed.cuh"

namespace cg = cooperative_groups;

namespace mlk {

namespace {

constexpr int G = 16;                         // logits of a group
constexpr int BT = 256;                       // threads of a block
constexpr int MAX_TOP = MLORA_LOGITS_MAX_TOP;
constexpr int LIST = 96;                      // groups that a team lists
constexpr int FOUND = MAX_TOP * G + 32;       // and logits: MAX_TOP groups of 16 and at most 30 beside them
constexpr float LOWEST = -1e30f;              // a logit below it counts as this one in the quick pass: its products are finite
constexpr float FAR = 1e6f;                   // a maximum this far from 0, in base 2, is for the careful pass
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

typedef unsigned long long u64;

// ---- elementary operations ---------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// a number in the order of the values (-0 as 0); no value maps to 0
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ u64 key64(uint32_t key, uint32_t id) { return (u64)key << 32 | (uint32_t)~id; }
__device__ __forceinline__ uint32_t id_of(u64 key) { return ~(uint32_t)key; }

// 32 bytes, for the last time or not
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// A group's 16 logits as they are loaded.
template <typename T> struct Group;
template <> struct Group<bf16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const bf16* p) { load32(p, w); }
    __device__ __forceinline__ float max() const {
        uint32_t m = max_nan2(max_nan2(max_nan2(w[0], w[1]), max_nan2(w[2], w[3])),
                              max_nan2(max_nan2(w[4], w[5]), max_nan2(w[6], w[7])));
        const float2 f = bf16_pair(m);
        return max_nan(f.x, f.y);
    }
    // pair i, not below LOWEST (the bf16 value above it)
    __device__ __forceinline__ float2 clamped(int i) const { return bf16_pair(max_nan2(w[i], 0xf149f149u)); }
};
template <> struct Group<float> {
    uint32_t w[16];
    __device__ __forceinline__ void load(const float* p) {
        load32(p, reinterpret_cast<uint32_t (&)[8]>(w[0]));
        load32(p + 8, reinterpret_cast<uint32_t (&)[8]>(w[8]));
    }
    __device__ __forceinline__ float max() const {
        float m = max_nan(__uint_as_float(w[0]), __uint_as_float(w[1]));
#pragma unroll
        for (int i = 2; i < 16; ++i) m = max_nan(m, __uint_as_float(w[i]));
        return m;
    }
    __device__ __forceinline__ float2 clamped(int i) const {
        return make_float2(max_nan(__uint_as_float(w[2 * i]), LOWEST), max_nan(__uint_as_float(w[2 * i + 1]), LOWEST));
    }
};

// m, s, t of some of a row's logits (above).  m is at least -FAR, so that tokens that are not
// allowed (-infinity or any number far below) have terms of 0 wherever they stand: as the maximum of the first ids
// that a thread sees they would be what the terms are relative to, and the rounding of their product, 2^-24 of a
// huge number, the exponent.
struct Part {
    float m, s, t;
};
__device__ __forceinline__ Part join(const Part& a, const Part& b) {
    const float m = max_nan(a.m, b.m);
    const float da = a.m - m, db = b.m - m, fa = ex2(da), fb = ex2(db);
    return Part{m, fmaf(a.s, fa, b.s * fb), __fmul_rn(fmaf(a.s, da, a.t), fa) + __fmul_rn(fmaf(b.s, db, b.t), fb)};
}

// What a team shares.
struct TeamShared {
    u64 list[LIST], found[FOUND];
    u64 pick[MAX_TOP];
    Part part[BT / 32];
    u64 tau;
    int n, n_found;
};
// What the blocks of a cluster hand to its first one.
constexpr int MAX_BLOCKS = 8;
struct ClusterShared {
    u64 pick[MAX_BLOCKS * MAX_TOP];
    Part part[MAX_BLOCKS];
};

template <int NT>
__device__ __forceinline__ void team_sync() {
    if (NT == 32) __syncwarp();
    else if (NT == BT) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"((int)(threadIdx.x / NT) + 1), "n"(NT) : "memory");
}

// over the team; every thread returns it, in one fixed order
template <int NT>
__device__ __forceinline__ Part team_join(Part p, TeamShared& sh, int tid) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        Part q;
        q.m = __shfl_xor_sync(0xffffffffu, p.m, o);
        q.s = __shfl_xor_sync(0xffffffffu, p.s, o);
        q.t = __shfl_xor_sync(0xffffffffu, p.t, o);
        // the lower lane's part first on both sides, so that both form the same number
        p = tid & o ? join(q, p) : join(p, q);
    }
    if (NT == 32) return p;
    team_sync<NT>();
    if ((tid & 31) == 0) sh.part[tid >> 5] = p;
    team_sync<NT>();
    p = sh.part[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) p = join(p, sh.part[w]);
    return p;
}

// A block's share of a row: groups of 16 that begin at 32 bytes, and the logits
// before and behind them, which the cluster's first block takes one by one.
template <typename T>
struct Share {
    const T* row;
    const T* first;                          // group 0 of the share
    int id0;                                 // its first id
    int groups;
    int head, tail0, edges;                  // ids [0, head) and [tail0, V); edges = both
    __device__ __forceinline__ int edge_id(int i) const { return i < head ? i : tail0 + i - head; }
};
template <typename T>
__device__ __forceinline__ Share<T> share_of(const T* row, int V, int rank, int blocks) {
    Share<T> s;
    s.row = row;
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 31) / (int)sizeof(T);
    s.head = off ? 32 / (int)sizeof(T) - off : 0;
    if (s.head > V) s.head = V;
    const int all = (V - s.head) / G;
    s.tail0 = s.head + all * G;
    s.edges = rank == 0 ? s.head + V - s.tail0 : 0;
    const int per = (all + blocks - 1) / blocks, a = min(rank * per, all), b = min(a + per, all);
    s.groups = b - a;
    s.id0 = s.head + a * G;
    s.first = row + s.id0;
    return s;
}

// The k largest of the n keys of list into out, in falling order (n may be below
// k); the keys are distinct.
template <int NT>
__device__ __forceinline__ void rank_keys(const u64* list, int n, int k, u64* out, int tid) {
    for (int i = tid; i < n; i += NT) {
        const u64 mine = list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += list[j] > mine;
        if (rank < k) out[rank] = mine;
    }
}

// Appends the keys of the threads that have one, a warp's side by side; all threads of a warp come here.
__device__ __forceinline__ void append(u64* list, int* n, int room, bool have, u64 key) {
    const uint32_t m = __ballot_sync(0xffffffffu, have);
    if (m == 0) return;
    int at = 0;
    if ((threadIdx.x & 31) == 0) at = atomicAdd(n, __popc(m));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << (threadIdx.x & 31)) - 1));
    if (have && at < room) list[at] = key;
}

// For one warp: the k largest of list's n keys into out, in falling order, one after
// the other: each lane knows the largest of its own that is left.
__device__ __noinline__ void pick_one_by_one(const u64* list, int n, int k, u64* out, int lane) {
    u64 mine = 0;
    for (int i = lane; i < n; i += 32) mine = list[i] > mine ? list[i] : mine;
    for (int r = 0; r < k; ++r) {
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
        if (hi == 0) break;                  // none left (no key's upper half is 0)
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0);
        const u64 best = (u64)hi << 32 | lo;
        if (mine == best) {
            out[r] = best;
            mine = 0;
            for (int i = lane; i < n; i += 32) {
                const u64 key = list[i];
                mine = key < best && key > mine ? key : mine;
            }
        }
        __syncwarp();
    }
}

// The share's k largest logits in sh.pick as (value, id) keys in falling order, 0
// where there are none.  gmax: the groups' largest values; best, at: the largest of this
// thread's and its group (-1: none); a thread of a warp's team has two, of its even and its odd groups.
template <typename T, int NT>
__device__ void top_of_share(const Share<T>& r, const T* gmax, const float (&best)[2], const int (&at)[2], int k,
                             TeamShared& sh, int tid) {
    for (int i = tid; i < k; i += NT) sh.pick[i] = 0;
    u64 tau = 0;
    int ng = r.groups;
    const bool all = NT == 32 && ng <= MAX_TOP;          // (few groups: all of them)
    if (tid == 0) sh.n_found = 0;
    if (!all) {
        // 64 first-round keys: two a thread of a warp, or one of NT / 64 threads
        constexpr int MINE = NT == 32 ? 2 : 1, QUAD = NT == 32 ? 1 : NT / 64, KEYS = 64;
        u64 mine[2];
#pragma unroll
        for (int u = 0; u < MINE; ++u) mine[u] = at[u] >= 0 ? key64(key_of(best[u]), at[u]) : 0;
        if (tid == 0) { sh.tau = 1; sh.n = 0; }
#pragma unroll
        for (int o = 1; o < QUAD; o <<= 1) {
            const u64 q = __shfl_xor_sync(0xffffffffu, mine[0], o);
            mine[0] = q > mine[0] ? q : mine[0];
        }
        if (tid % QUAD == 0) {
            sh.list[tid / QUAD] = mine[0];
            if (MINE == 2) sh.list[32 + tid] = mine[1];
        }
        team_sync<NT>();
        // the k-th largest of these keys: at least k groups are not below it.  A quad counts for its key together.
        int rank[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < KEYS / QUAD; ++j) {
            const u64 other = sh.list[j * QUAD + tid % QUAD];
            rank[0] += other > mine[0];
            if (MINE == 2) rank[1] += other > mine[1];
        }
#pragma unroll
        for (int o = 1; o < QUAD; o <<= 1) rank[0] += __shfl_xor_sync(0xffffffffu, rank[0], o);
#pragma unroll
        for (int u = 0; u < MINE; ++u)
            if (rank[u] == k - 1 && mine[u] && tid % QUAD == 0) sh.tau = mine[u];
        team_sync<NT>();
        tau = sh.tau;
        for (int g0 = 0; g0 < r.groups; g0 += NT) {
            const int g = g0 + tid;
            const u64 key = g < r.groups ? key64(key_of(to_f(gmax[g])), g) : 0;
            append(sh.list, &sh.n, LIST, g < r.groups && key >= tau, key);
        }
        team_sync<NT>();
        if (sh.n > LIST) {
            // few threads hold many of the largest groups: the k-th largest key bit by bit
            tau = 0;
            for (int bit = 63; bit >= 0; --bit) {
                const u64 want = tau | (u64)1 << bit;
                team_sync<NT>();
                if (tid == 0) sh.n = 0;
                team_sync<NT>();
                int c = 0;
                for (int g = tid; g < r.groups; g += NT) c += key64(key_of(to_f(gmax[g])), g) >= want;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
                if ((tid & 31) == 0) atomicAdd(&sh.n, c);
                team_sync<NT>();
                if (sh.n >= k) tau = want;
            }
            team_sync<NT>();
            if (tid == 0) sh.n = 0;
            team_sync<NT>();
            for (int g = tid; g < r.groups; g += NT) {
                const u64 key = key64(key_of(to_f(gmax[g])), g);
                if (key >= tau) sh.list[atomicAdd(&sh.n, 1)] = key;      // (k of them)
            }
            team_sync<NT>();
        }
        ng = sh.n;
        if (ng > MAX_TOP) {
            // more than their logits have room for: the k largest alone
            rank_keys<NT>(sh.list, ng, k, sh.pick, tid);
            team_sync<NT>();
            ng = k;
            tau = sh.pick[k - 1];
            u64 mine_too = 0;
            if (NT == 32 || tid < 32) mine_too = tid < k ? sh.pick[tid] : 0;
            team_sync<NT>();
            if (tid < k) { sh.list[tid] = mine_too; sh.pick[tid] = 0; }
            team_sync<NT>();
        }
    }
    team_sync<NT>();
    // their logits that are not below that group's largest, and the edges'
    const uint32_t low = (uint32_t)(tau >> 32);
    const int total = ng * G + r.edges;
#pragma unroll 4
    for (int i0 = 0; i0 < total; i0 += NT) {
        const int i = i0 + tid;
        u64 key = 0;
        if (i < total) {
            const int id = i >= ng * G ? r.edge_id(i - ng * G) : r.id0 + (all ? i : (int)id_of(sh.list[i / G]) * G + i % G);
            const float x = to_f(r.row[id]);
            const uint32_t value = key_of(x);
            if (x > -INFINITY && value >= low) key = key64(value, id);
        }
        append(sh.found, &sh.n_found, FOUND, key != 0, key);
    }
    team_sync<NT>();
    // (a warp's time: n^2 / 32 comparisons, or k rounds of about 25 of them)
    if (NT == 32 && sh.n_found * sh.n_found > 800 * k) pick_one_by_one(sh.found, sh.n_found, k, sh.pick, tid);
    else rank_keys<NT>(sh.found, sh.n_found, k, sh.pick, tid);
    team_sync<NT>();
}

// A row that the quick pass cannot take: NaN, an infinite maximum, or one so far from 0
// that what a product's rounding leaves is not small.  *kind: 1 NaN or +infinity, 2 no
// finite logit; *top: the maximum.
template <typename T, int NT>
__device__ __noinline__ Part careful(const Share<T>& r, float c, TeamShared& sh, int tid, int* kind, float* top) {
    float m = -INFINITY;
    auto each = [&](auto&& f) {
        for (int i = tid; i < r.groups * G; i += NT) f(to_f(r.first[i]));
        for (int i = tid; i < r.edges; i += NT) f(to_f(r.row[r.edge_id(i)]));
    };
    each([&](float x) { m = max_nan(m, x); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    team_sync<NT>();
    if ((tid & 31) == 0) sh.part[tid >> 5].m = m;
    team_sync<NT>();
    m = sh.part[0].m;
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) m = max_nan(m, sh.part[w].m);
    team_sync<NT>();
    *kind = !(m <= FLT_MAX) ? 1 : m == -INFINITY ? 2 : 0;
    *top = m;
    Part p{0.f, 0.f, 0.f};                   // relative to the maximum, whose product with c may leave fp32
    if (*kind) return p;
    each([&](float x) {
        // distances that leave fp32 or its exponents count as none
        const float d = fmaxf((x - m) * c, -200.f), e = ex2(d);
        p.s += e;
        p.t = fmaf(e, d, p.t);
    });
    return team_join<NT>(p, sh, tid);
}


// (by their registers: 64 for bf16, which fit; 80 for fp32, where 48 to 88 bytes spill)
template <typename T> constexpr int blocks_an_sm() { return sizeof(T) == 2 ? 4 : 3; }

template <typename T, int NT, bool CLUSTER>
__global__ void __launch_bounds__(BT, blocks_an_sm<T>())
token_logprobs_kernel(const __grid_constant__ LogitsView v, const __grid_constant__ mlora_token_stats out, int gcap) {
    extern __shared__ __align__(16) unsigned char gmax_all[];
    __shared__ TeamShared shared[BT / NT];
    __shared__ ClusterShared got;            // (the first block's is used)
    const int tid = threadIdx.x % NT, team = threadIdx.x / NT;
    TeamShared& sh = shared[team];
    T* gmax = reinterpret_cast<T*>(gmax_all) + team * gcap;
    int rank = 0, blocks = 1;
    if (CLUSTER) {
        rank = (int)cg::this_cluster().block_rank();
        blocks = (int)cg::this_cluster().num_blocks();
        // the first block's memory may be written once it runs: waited for before that
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    }
    const int k = v.top;
    const float c = v.scale * LOG2E;
    const int64_t row = CLUSTER ? blockIdx.x / blocks : (int64_t)blockIdx.x * (BT / NT) + team;
    int64_t o = row;
    int y = -1;
    bool leave = row >= v.n_rows;            // a whole team, a whole cluster
    if (!leave) {
        y = v.targets ? v.targets[row] : -1;
        if (v.out_row) {
            leave = row + v.row0 >= (int64_t)v.row_tiles[0] * TILE_M || y < 0 || v.out_row[row] < 0;
            if (!leave) o = v.out_row[row];
        } else if (y < -1 || y >= v.V) {
            if (rank == 0 && tid == 0) raise_status(v.status, ST_RANGE);
            y = -1;
        }
    }
    if (leave) {
        if (CLUSTER) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        return;
    }
    const T* x = static_cast<const T*>(v.x) + row * v.ld;
    const Share<T> r = share_of(x, v.V, rank, blocks);

    // the quick pass
    constexpr int UN = 2;                    // groups in work, and as many on their way
    Part p{-FAR, 0.f, 0.f};
    float2 s2 = make_float2(0.f, 0.f), t2 = s2;
    float best[2] = {-INFINITY, -INFINITY};
    int at[2] = {-1, -1};
    const float2 cc = make_float2(c, c);
    Group<T> next[UN];
    auto fetch = [&](int g0) {
#pragma unroll
        for (int u = 0; u < UN; ++u)
            if (g0 + u * NT < r.groups) next[u].load(r.first + (int64_t)(g0 + u * NT) * G);
    };
    fetch(tid);
    for (int g0 = tid; g0 < r.groups; g0 += UN * NT) {
        Group<T> q[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) q[u] = next[u];
        fetch(g0 + UN * NT);
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int g = g0 + u * NT;
            if (g >= r.groups) break;
            const float gm = q[u].max();
            if (k) {
                gmax[g] = from_f<T>(gm);     // (exact)
                const int w = NT == 32 ? u : 0;
                if (gm > best[w] || at[w] < 0) best[w] = gm, at[w] = g;
            }
            const float m = max_nan(p.m, gm * c);
            const float d = p.m - m, f = ex2(d);
            p.m = m;
            // the group's sums apart: 8 and V / (16 threads) additions in a row, not their product
            const float2 mm = make_float2(-m, -m);
            float2 sg = make_float2(0.f, 0.f), tg = sg;
#pragma unroll
            for (int i = 0; i < G / 2; ++i) {
                const float2 a = fma2(q[u].clamped(i), cc, mm);
                const float2 e = make_float2(ex2(a.x), ex2(a.y));
                sg = add2(sg, e);
                tg = fma2(e, a, tg);
            }
            const float2 ff = make_float2(f, f);
            t2 = fma2(fma2(s2, make_float2(d, d), t2), ff, tg);
            s2 = fma2(s2, ff, sg);
        }
    }
    p.s = s2.x + s2.y;
    p.t = t2.x + t2.y;
    for (int i = tid; i < r.edges; i += NT) {
        const float xv = max_nan(to_f(x[r.edge_id(i)]), LOWEST);
        // its term relative to it: what the rounding of its product leaves, up to 2^-24 of it, as in every group
        const float m = max_nan(__fmul_rn(xv, c), -FAR), left = fmaf(xv, c, -m), e = ex2(left);
        p = join(p, Part{m, e, e * left});
    }
    p = team_join<NT>(p, sh, tid);
    // (in a row with NaN what is found is not used)
    if (k) top_of_share<T, NT>(r, gmax, best, at, k, sh, tid);
    if (CLUSTER) {
        // the other blocks hand theirs to the first one and are done
        cg::cluster_group cl = cg::this_cluster();
        ClusterShared& first = *cl.map_shared_rank(&got, 0);
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        for (int i = tid; i < k; i += NT) first.pick[rank * k + i] = sh.pick[i];
        if (tid == 0) first.part[rank] = p;
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        if (rank) return;
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        p = got.part[0];
        for (int b = 1; b < blocks; ++b) p = join(p, got.part[b]);
        if (k) {
            // places without one are all 0 and hold no rank of their own
            if (tid == 0) sh.n_found = 0;
            for (int i = tid; i < k; i += NT) sh.pick[i] = 0;
            __syncthreads();
            for (int i = tid; i < blocks * k; i += NT)
                if (got.pick[i]) sh.found[atomicAdd(&sh.n_found, 1)] = got.pick[i];
            __syncthreads();
            rank_keys<NT>(sh.found, sh.n_found, k, sh.pick, tid);
            __syncthreads();
        }
    }
    int kind = 0;
    float top = 0.f;
    const bool large = !(fabsf(p.m) < FAR);
    if (large) p = careful<T, NT>(share_of(x, v.V, 0, 1), c, sh, tid, &kind, &top);
    const float ls = log2f(p.s);
    auto logprob = [&](float xv) {
        if (large) return fmaf(xv - top, v.scale, -ls * LN2);
        if (xv < LOWEST) return xv * v.scale;            // (its product with c may leave fp32)
        return (fmaf(xv, c, -p.m) - ls) * LN2;           // the product is taken from m before it is rounded, as in the sums
    };
    const float nan = __int_as_float(0x7fc00000);
    for (int i = tid; i < k; i += NT) {
        const u64 key = kind ? 0 : sh.pick[i];
        if (out.top_ids) out.top_ids[o * k + i] = key ? (int)id_of(key) : -1;
        if (out.top_logprobs) {
            out.top_logprobs[o * k + i] = kind == 1 ? nan : key ? logprob(of_key((uint32_t)(key >> 32))) : -INFINITY;
        }
    }
    if (tid == 0) {
        if (out.lse) out.lse[o] = kind == 1 ? nan : kind == 2 ? -INFINITY : large ? fmaf(top, v.scale, ls * LN2) : (p.m + ls) * LN2;
        if (out.entropy) out.entropy[o] = kind == 1 ? nan : kind == 2 ? 0.f : fmaxf((ls - p.t / p.s) * LN2, 0.f);
        if (out.logprobs)
            out.logprobs[o] = y < 0 || kind == 1 ? nan : kind == 2 ? -INFINITY : logprob(to_f(x[y]));
    }
}

// ----------------------------------------------------------------------------
// gradient
// ----------------------------------------------------------------------------
struct GradView {
    LogitsView v;
    mlora_token_grads g;
    void* out;
    int64_t ldo;
};

// dx = p (k0 + k1 a) + what the row's own ids add, a = log2 p.
struct RowGrad {
    float c, lse2, k0, k1;
};
__device__ __forceinline__ float2 grad2(float2 x, const RowGrad& r) {
    float2 a = fma2(x, make_float2(r.c, r.c), make_float2(-r.lse2, -r.lse2));
    a.x = max_nan(a.x, -200.f);
    a.y = max_nan(a.y, -200.f);
    return mul2(make_float2(ex2(a.x), ex2(a.y)), fma2(make_float2(r.k1, r.k1), a, make_float2(r.k0, r.k0)));
}

// What a warp knows of its row: lane l the l-th alternative's id and gradient, every
// lane the target's.
struct RowIds {
    int id, y;
    float d, dy;
    // which of them are such; bit 32: the target
    template <typename F>
    __device__ __forceinline__ u64 which(F&& such) const {
        const u64 m = __ballot_sync(0xffffffffu, such(id));
        return such(y) ? m | (u64)1 << 32 : m;
    }
    __device__ __forceinline__ u64 within(int a, int b) const {
        return which([=](int i) { return i >= a && i < b; });
    }
    // f(id, gradient) for each id of the mask, in one order
    template <typename F>
    __device__ __forceinline__ void each(u64 mask, F&& f) const {
        if (mask >> 32) f(y, dy);
        for (uint32_t m = (uint32_t)mask; m; m &= m - 1) {
            const int l = __ffs(m) - 1;
            f(__shfl_sync(0xffffffffu, id, l), __shfl_sync(0xffffffffu, d, l));
        }
    }
};

// The ids [a, b) of a row one by one (rows that do not lie alike in memory): one load on its way a lane.
// 1,021 bf16 rows of 32,003 in rows of 32,128 with a contiguous output: 158 us, 23 where they lie alike.
template <typename T>
__device__ __forceinline__ void grad_one_by_one(const T* x, T* out, int a, int b, const RowGrad& r, const RowIds& ids,
                                                bool zero, int lane) {
    for (int i0 = a; i0 < b; i0 += 32) {
        const int i = i0 + lane;
        const u64 hit = zero ? 0 : ids.within(i0, min(i0 + 32, b));
        float d = 0.f;
        if (i < b && !zero) d = grad2(make_float2(to_f(x[i]), 0.f), r).x;
        ids.each(hit, [&](int id, float add) { d += id == i ? add : 0.f; });
        if (i < b) out[i] = from_f<T>(d);
    }
}

// A warp works alone: it finds what its row's gradients come to, then takes windows of
// 2 x 32 x 32 bytes of the row, the next one on its way while one is formed.  The
// target's and the alternatives' own gradients are added where a window holds them,
// before the one rounding (barriers between a block's warps cost a third: 1,011 us
// against 653 for 8,192 bf16 rows of 151,936); as each id is read and written by one thread, dlogits may be
// the logits.  WARPS: of a row (1: rows so short that a block takes eight).
template <typename T, int WARPS>
__global__ void __launch_bounds__(BT, WARPS == 1 ? 4 : 3) token_grad_kernel(const __grid_constant__ GradView w) {
    const LogitsView& v = w.v;
    constexpr int ROWS = BT / 32 / WARPS, PER = 32 / (int)sizeof(T);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * ROWS + warp / WARPS;
    if (row >= v.n_rows) return;
    const int V = v.V, k = w.g.d_top ? v.top : 0;
    const int first = blockIdx.y * WARPS + warp % WARPS, step = gridDim.y * WARPS;     // this warp's windows
    const T* x = static_cast<const T*>(v.x) + row * v.ld;
    T* out = static_cast<T*>(w.out) + row * w.ldo;

    const uintptr_t px = reinterpret_cast<uintptr_t>(x) & 31, po = reinterpret_cast<uintptr_t>(out) & 31;
    // 32 bytes at a time between two ends
    const int lead = min((int)((32 - px) % 32 / sizeof(T)), V), vecs = (V - lead) / PER, tail = lead + vecs * PER;
    const int edge = first > 0 ? V : lane < lead ? lane : tail + lane - lead;          // this lane's id of the ends
    constexpr int UN = WARPS == 1 ? 1 : 2, WIN = UN * 32;    // vectors of a window
    uint32_t q[UN][8], next[UN][8];
    auto fetch = [&](int v0, bool wanted) {
#pragma unroll
        for (int u = 0; u < UN; ++u)
            if (v0 + 32 * u + lane < vecs && wanted) load32(x + lead + (int64_t)(v0 + 32 * u + lane) * PER, next[u]);
    };
    float at_edge = 0.f;
    // short rows: all loads at once
    if (WARPS == 1 && px == po) {
        if (edge < V) at_edge = to_f(x[edge]);
        fetch(0, true);
    }
    // every load that the row's factors need at once
    RowIds ids;
    ids.id = lane < k ? w.g.top_ids[row * v.top + lane] : -1;
    ids.y = v.targets && w.g.d_logprobs ? v.targets[row] : -1;
    ids.d = lane < k ? w.g.d_top[row * v.top + lane] : 0.f;
    ids.dy = w.g.d_logprobs ? w.g.d_logprobs[row] : 0.f;
    const float de = w.g.d_entropy ? w.g.d_entropy[row] : 0.f, dl = w.g.d_lse ? w.g.d_lse[row] : 0.f;
    const float lse = w.g.lse[row], entropy = w.g.d_entropy ? w.g.entropy[row] : 0.f;
    const bool bad = ids.id < -1 || ids.id >= V || ids.y < -1 || ids.y >= V;
    if (bad && first == 0) raise_status(v.status, ST_RANGE);
    if (ids.id < 0 || ids.id >= V) ids.id = -1, ids.d = 0.f;
    if (ids.y < 0 || ids.y >= V) ids.y = -1, ids.dy = 0.f;
    const bool zero = __all_sync(0xffffffffu, ids.d == 0.f && ids.dy == 0.f && de == 0.f && dl == 0.f) || lse == -INFINITY;
    float sum = ids.d;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    RowGrad r;
    r.c = v.scale * LOG2E;
    r.lse2 = lse * LOG2E;
    r.k0 = v.scale * (dl - (sum + ids.dy));
    r.k1 = 0.f;
    if (de != 0.f) {
        r.k0 = fmaf(-v.scale * de, entropy, r.k0);
        r.k1 = -v.scale * de * LN2;
    }
    ids.d *= v.scale;
    ids.dy *= v.scale;

    if (px != po) {
        constexpr int SPAN = 256;
        for (int64_t a = (int64_t)first * SPAN; a < V; a += (int64_t)step * SPAN)
            grad_one_by_one(x, out, (int)a, (int)min(a + SPAN, (int64_t)V), r, ids, zero, lane);
        return;
    }
    if (WARPS > 1) {
        if (edge < V && !zero) at_edge = to_f(x[edge]);
        fetch(first * WIN, !zero);
    }
    if (first == 0) {
        const u64 hit = zero ? 0 : ids.which([=](int i) { return i >= 0 && (i < lead || i >= tail); });
        float d = zero ? 0.f : grad2(make_float2(at_edge, 0.f), r).x;
        ids.each(hit, [&](int id, float add) { d += id == edge ? add : 0.f; });
        if (edge < V) out[edge] = from_f<T>(d);
    }
    T* ov = out + lead;
    for (int v0 = first * WIN; v0 < vecs; v0 += step * WIN) {
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) q[u][j] = zero ? 0 : next[u][j];
        fetch(v0 + step * WIN, !zero);
        const int id0 = lead + v0 * PER;
        const u64 hit = zero ? 0 : ids.within(id0, id0 + WIN * PER);
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            float2 d[PER / 2];
#pragma unroll
            for (int j = 0; j < PER / 2; ++j) {
                const float2 xx = sizeof(T) == 2 ? bf16_pair(q[u][j % 8])
                                                 : make_float2(__uint_as_float(q[u][2 * j % 8]), __uint_as_float(q[u][(2 * j + 1) % 8]));
                d[j] = grad2(xx, r);
            }
            if (hit) {
                const int mine = id0 + (32 * u + lane) * PER;
                ids.each(hit, [&](int id, float add) {
#pragma unroll
                    for (int j = 0; j < PER / 2; ++j) {
                        d[j].x += id == mine + 2 * j ? add : 0.f;
                        d[j].y += id == mine + 2 * j + 1 ? add : 0.f;
                    }
                });
            }
            if (!zero) {
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) {
                    if (sizeof(T) == 2) {
                        q[u][j % 8] = pack_bf16x2(d[j].x, d[j].y);
                    } else {
                        q[u][2 * j % 8] = __float_as_uint(d[j].x);
                        q[u][(2 * j + 1) % 8] = __float_as_uint(d[j].y);
                    }
                }
            }
            if (v0 + 32 * u + lane < vecs) store32(ov + (int64_t)(v0 + 32 * u + lane) * PER, q[u]);
        }
    }
}

constexpr int SHORT_V = 4096;                // rows of at most this many logits go to a warp each

template <typename T>
void launch_grad(const GradView& w, int num_sms, cudaStream_t s) {
    const int64_t n = w.v.n_rows;
    if (w.v.V <= SHORT_V) {
        token_grad_kernel<T, 1><<<(unsigned)((n + 7) / 8), BT, 0, s>>>(w);
        return;
    }
    // as many blocks a row as fill the SMs, and as have a window for each warp
    const int64_t most = w.v.V * (int64_t)sizeof(T) / (8 * 2048) + 1, want = (3 * 2 * (int64_t)num_sms + n - 1) / n;
    token_grad_kernel<T, 8><<<dim3((unsigned)n, (unsigned)(want < most ? want : most)), BT, 0, s>>>(w);
}

// ----------------------------------------------------------------------------
// launches
// ----------------------------------------------------------------------------
constexpr int MAX_GROUPS = MLORA_LOGITS_MAX_VOCAB / G / MAX_BLOCKS;

template <typename T, int NT, bool CLUSTER>
cudaError_t launch_rows(const LogitsView& v, const mlora_token_stats& out, int blocks, cudaStream_t s) {
    const int groups = v.V / G, gcap = v.top ? (groups + blocks - 1) / blocks : 0;
    const size_t smem = sizeof(T) * gcap * (BT / NT);
    auto* kern = token_logprobs_kernel<T, NT, CLUSTER>;
    if (smem > 2 * 1024) {
        // one size for all calls: threads that launch at once do not lower each other's
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_GROUPS * 4);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    const int64_t grid = CLUSTER ? v.n_rows * blocks : (v.n_rows + BT / NT - 1) / (BT / NT);
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(BT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = CLUSTER ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, v, out, gcap);
}

// Rows of at most this many logits go to a warp each, to two warps, and to four while the
// groups of a block's teams leave room for four blocks an SM.  8,192 bf16 rows with 20
// alternatives, in us with teams of 32, 64, 128 and 256 threads: 4,000 logits 35, 39, 51, 80;
// 16,000 84, 72, 80, 109; 32,000 142, 116, 117, 141; 151,936 -, 528, 416, 426 (4,096 fp32
// rows: -, -, 428, 383): what a row takes besides its logits is most of it for short ones.
constexpr int WARP_V = 8192, PAIR_V = 24576, QUAD_BYTES = 40 << 10;

template <typename T>
cudaError_t launch_t(const LogitsView& v, const mlora_token_stats& out, int num_sms, cudaStream_t s) {
    // few rows: a cluster of blocks each, no more than give each SM two, with shares of 4,096 logits at least,
    // and groups that fit shared memory (256 fp32 rows of 151,936: 35 us with a block each, 49 with two)
    int blocks = 1;
    while (blocks < MAX_BLOCKS && v.n_rows * blocks <= (int64_t)num_sms && v.V / blocks >= 8192) blocks *= 2;
    while (blocks < MAX_BLOCKS && v.top && v.V / G / blocks > 12000) blocks *= 2;
    if (blocks > 1) return launch_rows<T, BT, true>(v, out, blocks, s);
    int team = v.V <= WARP_V ? 32 : v.V <= PAIR_V ? 64 : 2 * (v.V / G) * (int)sizeof(T) <= QUAD_BYTES ? 128 : BT;
    // too few teams for two blocks an SM: larger ones, of four groups a thread at least
    while (team < BT && v.n_rows * team < 2 * BT * (int64_t)num_sms && v.V >= 4 * G * 2 * team) team *= 2;
    switch (team) {
    case 32: return launch_rows<T, 32, false>(v, out, 1, s);
    case 64: return launch_rows<T, 64, false>(v, out, 1, s);
    case 128: return launch_rows<T, 128, false>(v, out, 1, s);
    default: return launch_rows<T, BT, false>(v, out, 1, s);
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogitsView& x, const mlora_token_stats& out, int num_sms, cudaStream_t s) {
    return x.dtype == MLORA_BF16 ? launch_t<bf16>(x, out, num_sms, s) : launch_t<float>(x, out, num_sms, s);
}

int logits_check(float scale, int32_t top, int32_t vocab) {
    if (vocab < 1 || vocab > MLORA_LOGITS_MAX_VOCAB)
        return kv_fail(MLORA_E_ARG, "a vocabulary of %d, 1 .. %d are possible", vocab, MLORA_LOGITS_MAX_VOCAB);
    if (top < 0 || top > MAX_TOP) return kv_fail(MLORA_E_ARG, "%d alternatives, at most %d", top, MAX_TOP);
    if (!(scale >= 0x1p-20f && scale <= 0x1p20f)) return kv_fail(MLORA_E_ARG, "scale must lie in 2^-20 .. 2^20");
    return MLORA_OK;
}

}  // namespace mlk

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------
using namespace mlk;

namespace {

int view_check(const mlora_logits* x, LogitsView* v) {
    if (!x) return kv_fail(MLORA_E_ARG, "NULL logits");
    const int rc = logits_check(x->scale, x->top, x->vocab);
    if (rc) return rc;
    if (x->dtype != MLORA_BF16 && x->dtype != MLORA_FP32) return kv_fail(MLORA_E_ARG, "unknown dtype %d", x->dtype);
    const int es = x->dtype == MLORA_BF16 ? 2 : 4;
    // (a launch has a block or eight a row)
    if (x->n_rows < 0 || x->n_rows > INT32_MAX / 8) return kv_fail(MLORA_E_ARG, "%lld rows", (long long)x->n_rows);
    if (x->stride < x->vocab || x->stride > INT64_MAX / 4 / (x->n_rows + 1) / es)
        return kv_fail(MLORA_E_ARG, "rows %lld elements apart", (long long)x->stride);
    if (x->n_rows > 0 && !x->logits) return kv_fail(MLORA_E_ARG, "NULL logits");
    if (reinterpret_cast<uintptr_t>(x->logits) % es) return kv_fail(MLORA_E_ARG, "logits are not aligned to their elements");
    *v = LogitsView{};
    v->x = x->logits;
    v->ld = x->stride;
    v->n_rows = x->n_rows;
    v->targets = x->targets;
    v->status = x->status;
    v->scale = x->scale;
    v->V = x->vocab;
    v->dtype = x->dtype;
    v->top = x->top;
    return MLORA_OK;
}

int sm_count(int* n) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "device: %s", cudaGetErrorString(e));
    return MLORA_OK;
}

// Whether n rows of `width` bytes, lda and ldb bytes apart (width at least), share a byte.
bool rows_overlap(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t n, int64_t width) {
    const char *pa = static_cast<const char*>(a), *pb = static_cast<const char*>(b);
    if (pa + (n - 1) * lda + width <= pb || pb + (n - 1) * ldb + width <= pa) return false;
    if (lda == ldb && n > 1) {
        const int64_t d = ((pb - pa) % lda + lda) % lda;
        return d < width || d + width > lda;
    }
    // b's rows between a's: each against the last of a's rows that begins at or before it, and the next one
    for (int64_t i = 0; i < n; ++i) {
        const int64_t at = pb + i * ldb - pa, k = at < 0 ? -1 : at / lda < n ? at / lda : n - 1;
        if ((k >= 0 && at - k * lda < width) || (k + 1 < n && (k + 1) * lda - at < width)) return true;
    }
    return false;
}

}  // namespace

extern "C" int mlora_token_logprobs(const mlora_logits* x, const mlora_token_stats* out, void* stream) {
    LogitsView v;
    int rc = view_check(x, &v);
    if (rc) return rc;
    if (!out) return kv_fail(MLORA_E_ARG, "NULL results");
    if (out->logprobs && !x->targets && x->n_rows > 0) return kv_fail(MLORA_E_ARG, "log-probabilities without targets");
    mlora_token_stats o = *out;
    if (v.top == 0) o.top_ids = nullptr, o.top_logprobs = nullptr;
    if (!o.top_ids && !o.top_logprobs) v.top = 0;
    if (v.n_rows == 0 || !(o.logprobs || o.entropy || o.lse || v.top)) return MLORA_OK;
    int sms = 0;
    if ((rc = sm_count(&sms))) return rc;
    const cudaError_t e = launch_token_logprobs(v, o, sms, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "log-probabilities launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}

extern "C" int mlora_token_logprobs_backward(const mlora_logits* x, const mlora_token_grads* g, void* dlogits,
                                             int64_t out_stride, void* stream) {
    GradView w;
    int rc = view_check(x, &w.v);
    if (rc) return rc;
    if (!g) return kv_fail(MLORA_E_ARG, "NULL gradients");
    const int64_t n = x->n_rows, es = x->dtype == MLORA_BF16 ? 2 : 4;
    if (out_stride < x->vocab || out_stride > INT64_MAX / 4 / (n + 1) / es)
        return kv_fail(MLORA_E_ARG, "output rows %lld elements apart", (long long)out_stride);
    if (n == 0) return MLORA_OK;
    if (!dlogits || reinterpret_cast<uintptr_t>(dlogits) % es)
        return kv_fail(MLORA_E_ARG, "dlogits is NULL or not aligned to its elements");
    if (!g->lse) return kv_fail(MLORA_E_ARG, "NULL lse");
    if (g->d_entropy && !g->entropy) return kv_fail(MLORA_E_ARG, "d_entropy without the entropy");
    if (g->d_logprobs && !x->targets) return kv_fail(MLORA_E_ARG, "d_logprobs without targets");
    if (g->d_top && x->top > 0 && !g->top_ids) return kv_fail(MLORA_E_ARG, "d_top without the ids");
    if (!(dlogits == x->logits && (out_stride == x->stride || n == 1)) &&
        rows_overlap(x->logits, x->stride * es, dlogits, out_stride * es, n, x->vocab * es))
        return kv_fail(MLORA_E_ARG, "dlogits overlaps the logits and is not the logits themselves");
    w.g = *g;
    if (x->top == 0) w.g.d_top = nullptr;
    w.out = dlogits;
    w.ldo = out_stride;
    int sms = 0;
    if ((rc = sm_count(&sms))) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (x->dtype == MLORA_BF16) launch_grad<bf16>(w, sms, s);
    else launch_grad<float>(w, sms, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return kv_fail(MLORA_E_CUDA, "gradient launch: %s", cudaGetErrorString(e));
    return MLORA_OK;
}
