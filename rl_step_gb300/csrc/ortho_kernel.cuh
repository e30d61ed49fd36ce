// The kernel of updates made orthogonal by Newton-Schulz products (mlora_orthogonalize in
// include/mlora.h), compiled for each element type by a file of its own.  It takes
// matrices whose shorter side is at most 64, as LoRA factors' is.  With X [r x n] over
// the shorter side, X_0 = M / (|M| + eps):
//     X <- a X + (b A + c A^2) X,   A = X X^T.
//
// Everything but the long side is r x r: the products with X stay polynomials in A,
//     X_k = P_k X_0,   A_k = P_k A_0 P_k^T,
// so a step costs r^3, and the long side is read for the first A and for the last
// product alone.  In 32 bits that would be too coarse for small singular values: an
// error u of A_0 grows with P^2, a^(2 k) for those.  So A is formed again from P_k X
// after at most STEPS_A_PHASE steps, without storing P_k X: P_k M tile by tile, and
// each tile's products at once.  Five steps are two such phases (2 + 3 steps) and
// three passes over M; its trace gives the norm in the first.
//
// A block, or a cluster of them where the matrices are few, takes a matrix and does all
// of it: no launch, workspace or wait for other matrices is between the passes, and two
// blocks an SM work while the other is at its r x r steps.  Sums meet in a fixed order:
// results repeat.  What bounds it: for many matrices the passes, 1.7, 3.8 and 2.7
// thousand cycles for 16 warps' tiles of 32 x 32 without their fetches (the tensor
// cores' share 1.4, 3.4 and 1.9) and 2.7, 4.3 and 3.4 with them (32 x 4,096, fp32), at 63 %
// of the copy rate for eight adapters of the 8B widths and 75 % for 32, the tensor cores at 41 %:
// M is read three times, 2.7 of them from HBM where 304 matrices exceed L2.  For few matrices the chain of dependent steps: of 17 us for
// one of 32 x 256 the r x r steps take 6, the three passes 4, the sums between them 2.
//
// The products run on mma.sync with fp16 operands and fp32 sums: each factor, scaled
// by a power of two so that nothing exceeds fp16, as two of them (x = hi + lo, three
// products, the fourth is left out; an X that was bf16 needs no lo).  That is 2^-22 of x, or
// 2^-25 of the scaled 1 where lo is below fp16's normal range: 2^-30 of the root mean
// square that a warp's first tile is scaled by in the first pass, 2^-39 of |M| in the others.
// All 24 bits would take a third part and six products; what the two leave in the result is of the
// size of the plain fp32 form's errors (one small fp32 adapter 1.48e-6 beside 1.35e-6, 32 of the
// 8B widths 1.47e-6 beside 4.45e-6).  Fragments of X come from a warp's own tiles in
// shared memory, filled ahead with cp.async; the same fragment is both operands of X X^T,
// and the output fragment of P X becomes both of the next without leaving its thread.  The
// tensor cores cut their sums off (towards 0), so few products are chained, the small
// parts first, and their results are added in fp32.  r is 4 to 64: a 128-row tcgen05 tile
// would hold 2 to 8 matrices and form their cross products for nothing.
#pragma once

#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>

#include "kv_common.cuh"
#include "ortho.cuh"
#include "packed.cuh"

namespace cg = cooperative_groups;

namespace mlk {

namespace {

constexpr int OT = 256;                      // threads of a block
constexpr int OW = OT / 32;
constexpr int STEPS_A_PHASE = 3;
constexpr int MAX_BLOCKS = 8;                // of a cluster

template <int N>
struct OrthoTab {
    OrthoCoeffs co;
    OrthoEntry e[N];
};

// the nearest value of 11 bits (away from 0 between two), infinity near fp32's largest; a NaN may become 0 here: small_steps
// sees it where it comes up
__device__ __forceinline__ float tf32_hi(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }

// d += a b, 16 x 8 x 8 with tf32 operands
__device__ __forceinline__ void mma8(float (&d)[4], const float (&a)[4], float b0, float b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                   "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
// d += a b, 16 x 8 x 16 with pairs of fp16
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_of(float x, float y) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
    return h;
}
// x and y times f (a power of two) as fp16, and what that leaves
__device__ __forceinline__ void split(float x, float y, float f, uint32_t& hi, uint32_t& lo) {
    const float2 v = make_float2(x, y), ff = make_float2(f, f), p = mul2(v, ff);
    hi = half2_of(p.x, p.y);
    const float2 h = __half22float2(__hneg2(*reinterpret_cast<const __half2*>(&hi))), q = fma2(v, ff, h);
    lo = half2_of(q.x, q.y);
}

// Four elements side by side as floats.
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&v)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
}
// Two.
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load2(const bf16* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 4 elements to shared memory, or zeros
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from, bool there) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if (BYTES == 16)                         // (past the first cache, which takes no smaller pieces so)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(there ? BYTES : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at), "l"(from), "n"(BYTES), "r"(there ? BYTES : 0)
                     : "memory");
}

constexpr int TC = 32;                       // columns of a tile

// X of an entry: X(i, k) = M[i][k], or M[k][i] where M is tall; 0 outside.
// Row slots: the fragments' row 8 j + g is row i = 8 j + g of X, or (R / 8) g + j where
// M is tall, so that a thread's rows lie side by side there.
// A tile holds the columns k0 .. k0 + 31 as M has them, [R][32] or tall [32][R], in
// pieces of four elements that are moved inside their row so that the threads' reads
// meet few banks twice.
template <typename T, int R, bool TALL>
struct Matrix {
    static constexpr int TILE = R * TC;      // elements
    const T* src;
    T* dst;
    int n, r;
    bool vec;
    float f;                                 // a power of two that X is taken with
    __device__ __forceinline__ explicit Matrix(const OrthoEntry& e)
        : src(static_cast<const T*>(e.src)), dst(static_cast<T*>(e.dst)), n(e.n), r(e.r), vec(e.vec), f(1.f) {}
    static __device__ __forceinline__ int row_of(int slot) { return TALL ? slot % 8 * (R / 8) + slot / 8 : slot; }
    // the row of X at place q (0 .. 3: 2 t, 2 t + 1, 2 t + 8, 2 t + 9) of the 16 rows s of a product P X
    static __device__ __forceinline__ int k_row(int s, int t, int q) {
        return 16 * s + (TALL ? 4 * t + q : 2 * t + q % 2 + q / 2 * 8);
    }
    // where (row, piece) of a tile lies
    static __device__ __forceinline__ int wide_at(int row, int piece) {
        return row * TC + 4 * (piece ^ (2 * (row >> 1 & 3) ^ 4 * (row & 1)));
    }
    static __device__ __forceinline__ int tall_at(int row, int piece) {
        return row * R + 4 * (piece ^ ((2 * (row >> 2 & 3) ^ 4 * (row & 1)) & (R / 4 - 1)));
    }
    // the tile from column k0 on, for a warp
    __device__ __forceinline__ void fetch(T* tile, int k0, int lane) const {
        if (vec) {
            // Lane l takes piece l % P of the rows l / P, l / P + ROWS, ..; what moves a piece inside its row
            // splits into a part of the lane's and one of the round's.
            constexpr int P = TALL ? R / 4 : TC / 4, ROWS = 32 / P, ROUNDS = R / 4;
            const int p = lane % P, row = lane / P;
            const int64_t ld = TALL ? r : n;
            const T* from = TALL ? src + (int64_t)(k0 + row) * r + 4 * p : src + (int64_t)row * n + k0 + 4 * p;
            const bool piece_in = TALL ? 4 * p < r : k0 + 4 * p < n;
            const int rows = TALL ? n - k0 : r;
#pragma unroll
            for (int q = 0; q < ROUNDS; ++q) {
                const bool in = piece_in && row + ROWS * q < rows;
                const int to = TALL ? tall_at(row + ROWS * q, p) : wide_at(row + ROWS * q, p);
                copy_async<4 * sizeof(T)>(tile + to, in ? from : src, in);
                from += ROWS * ld;
            }
        } else {
            for (int at = lane; at < TILE; at += 32) {
                if (TALL) {
                    const int k = at / R, i = at % R;
                    tile[tall_at(k, i / 4) + i % 4] = k0 + k < n && i < r ? src[(int64_t)(k0 + k) * r + i] : from_f<T>(0.f);
                } else {
                    const int i = at / TC, k = at % TC;
                    tile[wide_at(i, k / 4) + k % 4] = i < r && k0 + k < n ? src[(int64_t)i * n + k0 + k] : from_f<T>(0.f);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

// A warp's tiles of its block's columns, one after the other.  The first one is fetched
// by begin_tiles, long before it is needed; then each(tile, k0) has its tile while the
// next one is on its way.
template <typename T, int R>
struct OrthoShared;
constexpr int STEP = TC * OW;                // columns from a warp's tile to its next one
template <typename T, int R, bool TALL>
__device__ __forceinline__ void begin_tiles(const Matrix<T, R, TALL>& x, OrthoShared<T, R>& sh, int first, int end) {
    const int warp = threadIdx.x >> 5, k0 = first + TC * warp;
    __syncwarp();
    if (k0 < end) x.fetch(sh.ring0[warp], k0, threadIdx.x & 31);
}
template <typename T, int R, bool TALL, typename F>
__device__ __forceinline__ void over_tiles(const Matrix<T, R, TALL>& x, OrthoShared<T, R>& sh, int first, int end, F&& each) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* here = sh.ring0[warp];
    T* other = sh.ring1[warp];
#pragma unroll 1
    for (int k0 = first + TC * warp; k0 < end; k0 += STEP) {
        // (the whole warp has read the tile whose place the next one takes)
        if (k0 + STEP < end) {
            x.fetch(other, k0 + STEP, lane);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        each(here, k0);
        __syncwarp();
        T* const swap = here;
        here = other;
        other = swap;
    }
}

// Tiles of a symmetric product: block row m (16 rows) and 8 columns j, j >= 2 m.
template <int R>
struct Gram {
    static constexpr int M = R / 16, J = R / 8, TILES = M * (M + 1);
    float v[TILES][4];
    static __device__ __forceinline__ constexpr int tile(int m, int j) { return m * J - m * (m - 1) + j - 2 * m; }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[t][e] = 0.f;
    }
    // += x x^T over 16 columns; [j][0 / 1]: row slot 8 j + g, columns 2 t, 2 t + 1 / 2 t + 8, 2 t + 9.
    // EXACT: x has no low part.
    template <bool EXACT>
    __device__ __forceinline__ void add(const uint32_t (&hi)[J][2], const uint32_t (&lo)[J][2]) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j0 = 2 * m; j0 < J; j0 += 2) {
                // two tiles at a time: a product waits for the one before it in its chain
                float d[2][4] = {};
                if (!EXACT) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        mma16(d[j], lo[2 * m][0], lo[2 * m + 1][0], lo[2 * m][1], lo[2 * m + 1][1], hi[j0 + j][0], hi[j0 + j][1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        mma16(d[j], hi[2 * m][0], hi[2 * m + 1][0], hi[2 * m][1], hi[2 * m + 1][1], lo[j0 + j][0], lo[j0 + j][1]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma16(d[j], hi[2 * m][0], hi[2 * m + 1][0], hi[2 * m][1], hi[2 * m + 1][1], hi[j0 + j][0], hi[j0 + j][1]);
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        float* a = &v[tile(m, j0 + j)][e];
                        const float2 sum = add2(make_float2(a[0], a[1]), make_float2(d[j][e], d[j][e + 1]));
                        a[0] = sum.x;
                        a[1] = sum.y;
                    }
                }
            }
    }
};

// Shared memory of a block: r x r matrices of pitch R + 8 (a thread reads two values
// side by side, eight rows at once), P's fragments, the warps' tiles, and in the second
// tiles' place the sums of the warps between the passes.
template <typename T, int R>
struct OrthoShared {
    static constexpr int LD = R + 8, SLOTS = R == 64 ? OW / 2 : OW;
    float A[R * LD], Q[R * LD], W[R * LD], P[R * LD];
    uint4 ph[R / 16][R / 16][32], pl[R / 16][R / 16][32];   // [m][s][lane]
    alignas(16) float red[OW];
    alignas(16) T ring0[OW][R * TC];
    union {
        alignas(16) T ring1[OW][R * TC];
        float part[SLOTS][R * LD];           // [0]: the block's
    };
};

// 16 x 8 of A B at (m, n) for R x R matrices in shared memory; ROWS: B is symmetric, its rows are read.
template <int R, bool ROWS>
__device__ __forceinline__ void small_tile(const float* A, const float* B, int m, int n, float (&sum)[4]) {
    constexpr int LD = R + 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = 0.f;
#pragma unroll
    for (int k = 0; k < R; k += 8) {
        // the places t and t + 4 of the eight are 2 t and 2 t + 1 of both factors
        const float2 u = *reinterpret_cast<const float2*>(A + (m + g) * LD + k + 2 * t);
        const float2 v = *reinterpret_cast<const float2*>(A + (m + g + 8) * LD + k + 2 * t);
        const float2 b = ROWS ? *reinterpret_cast<const float2*>(B + (n + g) * LD + k + 2 * t)
                              : make_float2(B[(k + 2 * t) * LD + n + g], B[(k + 2 * t + 1) * LD + n + g]);
        const float a[4] = {u.x, v.x, u.y, v.y};
        float ah[4], al[4], c[4] = {}, d[4] = {};
#pragma unroll
        for (int e = 0; e < 4; ++e) ah[e] = tf32_hi(a[e]), al[e] = tf32_hi(a[e] - ah[e]);
        const float b0 = tf32_hi(b.x), b1 = tf32_hi(b.y), l0 = tf32_hi(b.x - b0), l1 = tf32_hi(b.y - b1);
        // all four products of the parts, in two short chains
        mma8(c, al, l0, l1);
        mma8(d, ah, l0, l1);
        mma8(c, al, b0, b1);
        mma8(d, ah, b0, b1);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += d[e] + c[e];
    }
}

// Every tile of an R x R product, shared among the warps: each(m, n).
template <int R, typename F>
__device__ __forceinline__ void small_tiles(F&& each) {
#pragma unroll 1
    for (int tile = threadIdx.x >> 5; tile < R / 16 * (R / 8); tile += OW) each(tile / (R / 8) * 16, tile % (R / 8) * 8);
}
template <int R, typename F>
__device__ __forceinline__ void small_store(float* C, int m, int n, F&& value) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = m + g + 8 * h, j = n + 2 * t;
        *reinterpret_cast<float2*>(C + i * (R + 8) + j) = make_float2(value(i, j, 2 * h), value(i, j + 1, 2 * h + 1));
    }
}

// The blocks' sums of a product, in X's row order and times `scale`, in sh.A of every
// block of the cluster.
template <typename T, int R, bool TALL>
__device__ __forceinline__ void gather(Gram<R>& s, const Matrix<T, R, TALL>& x, float scale, OrthoShared<T, R>& sh) {
    constexpr int LD = R + 8, SLOTS = OrthoShared<T, R>::SLOTS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    __syncthreads();                         // (the tiles have been read)
#pragma unroll
    for (int turn = 0; turn < OW / SLOTS; ++turn) {
        // (64 rows: room for half of the warps, the others add to theirs)
        if (warp / SLOTS == turn) {
            float* p = sh.part[warp % SLOTS];
#pragma unroll
            for (int m = 0; m < R / 16; ++m)
#pragma unroll
                for (int j = 2 * m; j < R / 8; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float* v = s.v[Gram<R>::tile(m, j)];
                        float2& q = *reinterpret_cast<float2*>(p + (16 * m + g + h * 8) * LD + 8 * j + 2 * t);
                        if (turn) q = make_float2(q.x + v[2 * h], q.y + v[2 * h + 1]);
                        else q = make_float2(v[2 * h], v[2 * h + 1]);
                    }
        }
        __syncthreads();
    }
    cg::cluster_group cl = cg::this_cluster();
    const int blocks = (int)cl.num_blocks();
    // (the tiles below the diagonal's block row are not there)
    auto place = [](int a, int b) { return a / 16 <= b / 16 ? a * LD + b : b * LD + a; };
    auto of_block = [&](int at) {
        float v = sh.part[0][at];
#pragma unroll
        for (int w = 1; w < SLOTS; ++w) v += sh.part[w][at];
        return v;
    };
    if (blocks == 1) {
        for (int i = threadIdx.x; i < R * R; i += OT)
            sh.A[x.row_of(i / R) * LD + x.row_of(i % R)] = of_block(place(i / R, i % R)) * scale;
        __syncthreads();
        return;
    }
    // each element's sum over the block's warps by one thread, into the first place, which others do not read
    for (int i = threadIdx.x; i < R * R; i += OT)
        if (i / R / 16 <= i % R / 16) sh.part[0][i / R * LD + i % R] = of_block(i / R * LD + i % R);
    cl.sync();
    const float* from[MAX_BLOCKS];
#pragma unroll
    for (int k = 0; k < MAX_BLOCKS; ++k) from[k] = cl.map_shared_rank(&sh, k < blocks ? k : 0)->part[0];
#pragma unroll 4
    for (int i = threadIdx.x; i < R * R; i += OT) {
        const int a = i / R, b = i % R;
        if (a / 16 > b / 16) continue;
        // all blocks' loads at once
        float v[MAX_BLOCKS], sum = 0.f;
#pragma unroll
        for (int k = 0; k < MAX_BLOCKS; ++k) v[k] = k < blocks ? from[k][a * LD + b] : 0.f;
#pragma unroll
        for (int k = 0; k < MAX_BLOCKS; ++k) sum += v[k];
        sum *= scale;
        sh.A[x.row_of(a) * LD + x.row_of(b)] = sum;
        if (a / 16 < b / 16) sh.A[x.row_of(b) * LD + x.row_of(a)] = sum;
    }
    cl.sync();
}

// the largest of the block's values, none of them negative
__device__ __forceinline__ float block_max(float m, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < OW; ++w) m = fmaxf(m, red[w]);
    return m;
}
// 2^e with e such that 2^e m lies in [2^(to - 1), 2^to); m is positive and finite, the
// power is held to 2^+-126
__device__ __forceinline__ float scale_to(float m, int to) {
    int e;
    frexpf(m, &e);
    return ldexpf(1.f, max(-126, min(126, to - e)));
}

// sh.P as fragments for P X, times the power of two that is returned; NaN, all of them and the power, where a
// thread is `bad` or P has left fp32: so are P X, the next A and the result then
template <typename T, int R, bool TALL>
__device__ __forceinline__ float fragments(const Matrix<T, R, TALL>& x, OrthoShared<T, R>& sh, bool bad) {
    constexpr int LD = R + 8;
    float m = 0.f;
    for (int i = threadIdx.x; i < R * R; i += OT) m = fmaxf(m, fabsf(sh.P[i / R * LD + i % R]));
    m = block_max(bad ? INFINITY : m, sh.red);
    const float scale = m > FLT_MAX ? __int_as_float(0x7fc00000) : m > 0.f ? scale_to(m, 14) : 1.f;
    for (int i = threadIdx.x; i < R / 16 * (R / 16) * 32; i += OT) {
        const int lane = i % 32, s = i / 32 % (R / 16), mm = i / 32 / (R / 16), g = lane >> 2, t = lane & 3;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {        // rows g, g + 8, g, g + 8; places 0, 1 and then 2, 3
            const float* p = sh.P + x.row_of(16 * mm + g + e % 2 * 8) * LD;
            split(p[x.k_row(s, t, e / 2 * 2)], p[x.k_row(s, t, e / 2 * 2 + 1)], scale, hi[e], lo[e]);
        }
        sh.ph[mm][s][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        sh.pl[mm][s][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __syncthreads();
    return scale;
}

// Columns 16 h .. 16 h + 15 of a tile of P X: d[m][c][e], row slot 16 m + g + 8 (e / 2), column
// 16 h + 4 t + 2 (e % 2) + c (M wide) or 16 h + 8 c + 2 t + e % 2 (tall).
template <typename T, int R, bool TALL>
__device__ __forceinline__ void times_p(const Matrix<T, R, TALL>& x, const OrthoShared<T, R>& sh, const T* tile, int h,
                                        float (&d)[R / 16][2][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr bool EXACT = sizeof(T) == 2;   // eight bits fit fp16
    constexpr int S = R / 16;
    uint32_t hi[S][2][2], lo[S][2][2];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float v[2][4];                       // [c][place]
        if constexpr (TALL) {
#pragma unroll
            for (int c = 0; c < 2; ++c) load4(tile + Matrix<T, R, TALL>::tall_at(16 * h + 8 * c + g, 4 * s + t), v[c]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 w = load2(tile + Matrix<T, R, TALL>::wide_at(16 * s + 2 * t + q % 2 + q / 2 * 8, 4 * h + g / 2) + 2 * (g % 2));
                v[0][q] = w.x;
                v[1][q] = w.y;
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (EXACT) hi[s][c][e] = half2_of(v[c][2 * e] * x.f, v[c][2 * e + 1] * x.f);
                else split(v[c][2 * e], v[c][2 * e + 1], x.f, hi[s][c][e], lo[s][c][e]);
            }
    }
#pragma unroll
    for (int m = 0; m < R / 16; ++m) {
        uint4 a[S];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[m][c][e] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint4 l = sh.pl[m][s][lane];
            a[s] = sh.ph[m][s][lane];
#pragma unroll
            for (int c = 0; c < 2; ++c) mma16(d[m][c], l.x, l.y, l.z, l.w, hi[s][c][0], hi[s][c][1]);
            if (!EXACT) {
#pragma unroll
                for (int c = 0; c < 2; ++c) mma16(d[m][c], a[s].x, a[s].y, a[s].z, a[s].w, lo[s][c][0], lo[s][c][1]);
            }
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int c = 0; c < 2; ++c) mma16(d[m][c], a[s].x, a[s].y, a[s].z, a[s].w, hi[s][c][0], hi[s][c][1]);
    }
}

// The sums of X X^T over the block's columns.  f: the scale, or 0: each warp's own, from the
// root mean square of its first tile (2^5, which leaves 2^10 for larger elements); then the
// sums are those of M itself.  Where that does not do, they are no numbers, and the caller takes the
// scale from M's largest element: an elementwise read and this pass again.  A first tile of zeros is such a
// case, and one beyond 2^-30 .. 2^30 (1,200 matrices of 32 x 4,096 whose first 32 columns are 0, or whose
// elements are near 1e-10: 680 us instead of 473, all zeros 596).
template <typename T, int R, bool TALL>
__device__ __forceinline__ void gram_of_x(const Matrix<T, R, TALL>& x, OrthoShared<T, R>& sh, float f, int first, int end,
                                          Gram<R>& acc) {
    constexpr int J = R / 8;
    constexpr bool EXACT = sizeof(T) == 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    acc.clear();
    const bool own = f == 0.f && first + TC * warp < end;
    bool sure = true;
    if (own) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        float sq = 0.f;
#pragma unroll
        for (int q = 0; q < R / 4; ++q) {
            float v[4];
            load4(sh.ring0[warp] + 4 * (lane + 32 * q), v);
#pragma unroll
            for (int e = 0; e < 4; ++e) sq = fmaf(v[e], v[e], sq);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        sq *= 1.f / (R * TC);
        sure = sq > 0x1p-60f && sq < 0x1p60f;
        f = sure ? scale_to(sqrtf(sq), 5) : 1.f;
    }
    over_tiles<T, R, TALL>(x, sh, first, end, [&](const T* tile, int) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            uint32_t hi[J][2], lo[J][2];
            auto put = [&](int j, int e, float a, float b) {
                if (EXACT) hi[j][e] = half2_of(a * f, b * f);
                else split(a, b, f, hi[j][e], lo[j][e]);
            };
            if constexpr (TALL) {
                // columns 16 h + 4 t + q, rows J g ..
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = 16 * h + 4 * t + 2 * e;
                    if constexpr (J >= 4) {
#pragma unroll
                        for (int j = 0; j < J; j += 4) {
                            float a[4], b[4];
                            load4(tile + Matrix<T, R, TALL>::tall_at(k, (J * g + j) / 4), a);
                            load4(tile + Matrix<T, R, TALL>::tall_at(k + 1, (J * g + j) / 4), b);
#pragma unroll
                            for (int q = 0; q < 4; ++q) put(j + q, e, a[q], b[q]);
                        }
                    } else {
                        const float2 a = load2(tile + Matrix<T, R, TALL>::tall_at(k, g / 2) + 2 * (g % 2));
                        const float2 b = load2(tile + Matrix<T, R, TALL>::tall_at(k + 1, g / 2) + 2 * (g % 2));
                        put(0, e, a.x, b.x);
                        put(1, e, a.y, b.y);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float v[4];
                    load4(tile + Matrix<T, R, TALL>::wide_at(8 * j + g, 4 * h + t), v);
                    put(j, 0, v[0], v[1]);
                    put(j, 1, v[2], v[3]);
                }
            }
            acc.template add<EXACT>(hi, lo);
        }
    });
    if (own) {
        const float back = sure ? 1.f / (f * f) : __int_as_float(0x7fc00000);
#pragma unroll
        for (int i = 0; i < Gram<R>::TILES; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc.v[i][e] *= back;
    }
}

// The same of P X times `scale`.
template <typename T, int R, bool TALL>
__device__ __forceinline__ void gram_of_px(const Matrix<T, R, TALL>& x, OrthoShared<T, R>& sh, float scale, int first, int end,
                                           Gram<R>& acc) {
    constexpr int J = R / 8;
    acc.clear();
    over_tiles<T, R, TALL>(x, sh, first, end, [&](const T* tile, int) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float d[R / 16][2][4];
            times_p<T, R, TALL>(x, sh, tile, h, d);
            uint32_t hi[J][2], lo[J][2];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    split(d[j / 2][c][j % 2 * 2], d[j / 2][c][j % 2 * 2 + 1], scale, hi[j][c], lo[j][c]);
            acc.template add<false>(hi, lo);
        }
    });
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(bf16* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// dst = P X times `scale`
template <typename T, int R, bool TALL>
__device__ __forceinline__ void write_px(const Matrix<T, R, TALL>& x, OrthoShared<T, R>& sh, float scale, int first, int end) {
    constexpr int J = R / 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    over_tiles<T, R, TALL>(x, sh, first, end, [&](const T* tile, int k0) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float d[R / 16][2][4];
            times_p<T, R, TALL>(x, sh, tile, h, d);
            if constexpr (TALL) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = k0 + 16 * h + 8 * c + 2 * t + e;
                        if (k >= x.n) continue;
                        T* out = x.dst + (int64_t)k * x.r;
                        auto v = [&](int j) { return d[j / 2][c][j % 2 * 2 + e] * scale; };
                        if constexpr (J % 4 == 0) {
#pragma unroll
                            for (int j = 0; j < J; j += 4) {
                                const int i = J * g + j;
                                if (x.vec && i + 4 <= x.r) {
                                    store4(out + i, v(j), v(j + 1), v(j + 2), v(j + 3));
                                } else {
#pragma unroll
                                    for (int q = 0; q < 4; ++q)
                                        if (i + q < x.r) out[i + q] = from_f<T>(v(j + q));
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < J; ++j)
                                if (J * g + j < x.r) out[J * g + j] = from_f<T>(v(j));
                        }
                    }
            } else {
#pragma unroll
                for (int m = 0; m < R / 16; ++m)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int i = 16 * m + 8 * q + g, k = k0 + 16 * h + 4 * t;
                        if (i >= x.r) continue;
                        T* out = x.dst + (int64_t)i * x.n + k;
                        const float v[4] = {d[m][0][2 * q] * scale, d[m][1][2 * q] * scale, d[m][0][2 * q + 1] * scale,
                                            d[m][1][2 * q + 1] * scale};
                        if (x.vec && k + 4 <= x.n) {
                            store4(out, v[0], v[1], v[2], v[3]);
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (k + c < x.n) out[c] = from_f<T>(v[c]);
                        }
                    }
            }
        }
    });
}

// `steps` steps on sh.A and sh.P: P <- Q P with Q = a I + b A + c A^2, and A <- Q A Q
// between them.  All are polynomials in A, which commute and are symmetric but for
// roundings.  Two of the products take a factor by rows for that; A^2 and Q P by columns:
// a transposed P or A there let the roundings grow (a spread of singular values of 100
// was off by 1e-5 of the result's norm instead of 2e-6).  Returns whether this thread has
// stored a number that is not finite: an iteration that leaves fp32 is seen by one of them (Q takes A's numbers
// with b as they are), although the factors' parts need not keep its NaN.
template <typename T, int R>
__device__ __forceinline__ bool small_steps(OrthoShared<T, R>& sh, const OrthoCoeffs& co, int steps) {
    constexpr int LD = R + 8, TILES = R / 16 * (R / 8), MINE = (TILES + OW - 1) / OW;
    const int warp = threadIdx.x >> 5;
    float none = 0.f;                        // NaN from the first infinity or NaN on
    auto seen = [&](float v) {
        none = fmaf(v, 0.f, none);
        return v;
    };
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        small_tiles<R>([&](int m, int n) {
            float d[4];
            small_tile<R, false>(sh.A, sh.A, m, n, d);
            small_store<R>(sh.Q, m, n, [&](int i, int j, int e) {
                return seen(fmaf(co.c, d[e], co.b * sh.A[i * LD + j]) + (i == j ? co.a : 0.f));
            });
        });
        __syncthreads();
        float p[MINE][4];
#pragma unroll
        for (int q = 0; q < MINE; ++q) {
            const int tile = warp + q * OW;
            if (tile < TILES) small_tile<R, false>(sh.Q, sh.P, tile / (R / 8) * 16, tile % (R / 8) * 8, p[q]);
        }
        if (k + 1 < steps) {
            small_tiles<R>([&](int m, int n) {
                float d[4];
                small_tile<R, true>(sh.Q, sh.A, m, n, d);
                small_store<R>(sh.W, m, n, [&](int, int, int e) { return seen(d[e]); });
            });
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < MINE; ++q) {
            const int tile = warp + q * OW;
            if (tile < TILES) small_store<R>(sh.P, tile / (R / 8) * 16, tile % (R / 8) * 8, [&](int, int, int e) { return seen(p[q][e]); });
        }
        if (k + 1 < steps) {
            small_tiles<R>([&](int m, int n) {
                float d[4];
                small_tile<R, true>(sh.W, sh.Q, m, n, d);
                small_store<R>(sh.A, m, n, [&](int, int, int e) { return seen(d[e]); });
            });
        }
        __syncthreads();
    }
    return !(none == 0.f);
}

// All of one matrix, or a block's part of it.
template <typename T, int R, bool TALL>
__device__ __forceinline__ void orthogonal(const OrthoEntry& entry, const OrthoCoeffs& co, OrthoShared<T, R>& sh) {
    constexpr int LD = R + 8;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), blocks = (int)cl.num_blocks(), tid = threadIdx.x;
    Matrix<T, R, TALL> x(entry);
    // the block's columns, in whole tiles
    const int all = (x.n + TC - 1) / TC, per = (all + blocks - 1) / blocks;
    const int first = min(rank * per, all) * TC, end = min(rank * per + per, all) * TC;
    const int64_t size = (int64_t)x.n * x.r;
    Gram<R> acc;
    auto trace = [&]() {
        float s = 0.f;
        for (int i = 0; i < x.r; ++i) s += sh.A[i * LD + i];
        return s;
    };
    begin_tiles<T, R, TALL>(x, sh, first, end);
    gram_of_x<T, R, TALL>(x, sh, 0.f, first, end, acc);
    begin_tiles<T, R, TALL>(x, sh, first, end);
    gather<T, R, TALL>(acc, x, 1.f, sh);
    float sq = trace();
    if (!(sq > 0.f && sq <= FLT_MAX)) {
        // the largest magnitude says
        float m = 0.f;
        bool bad = false;
        for (int64_t i = tid + (int64_t)rank * OT; i < size; i += (int64_t)OT * blocks) {
            const float v = fabsf(to_f(x.src[i]));
            bad |= !(v <= FLT_MAX);
            m = fmaxf(m, v);
        }
        block_max(bad ? INFINITY : m, sh.red);
        cl.sync();
        m = 0.f;
        for (int b = 0; b < blocks; ++b)
            for (int w = 0; w < OW; ++w) m = fmaxf(m, cl.map_shared_rank(&sh, b)->red[w]);
        cl.sync();
        if (m > FLT_MAX) {
            // an infinity or NaN
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            for (int64_t i = tid + (int64_t)rank * OT; i < size; i += (int64_t)OT * blocks)
                x.dst[i] = from_f<T>(__int_as_float(0x7fc00000));
            return;
        }
        sq = 0.f;
        if (m > 0.f) {
            x.f = scale_to(m, 15);
            gram_of_x<T, R, TALL>(x, sh, x.f, first, end, acc);
            begin_tiles<T, R, TALL>(x, sh, first, end);
            gather<T, R, TALL>(acc, x, 1.f, sh);
            sq = trace();
        } else {
            for (int i = tid; i < R * LD; i += OT) sh.A[i] = 0.f;
        }
    }
    // From here on |f M| is below 2^15, and so is every element.  X_0 = inv (f M); a matrix of zeros stays zero.
    float f = sq > 0.f ? x.f * scale_to(sqrtf(sq), 15) : x.f;
    if (!(f >= 0x1p-126f && f <= 0x1p126f)) f = x.f;         // (at the ends of fp32 the largest element's scale stays)
    const float again = f / x.f;
    const float inv = sq > 0.f ? 1.f / (sqrtf(sq) * again + co.eps * f) : 0.f, to_a = inv * again;
    x.f = f;
    __syncthreads();                         // (all have their trace)
    for (int i = tid; i < R * LD; i += OT) {
        sh.A[i] = sh.A[i] * to_a * to_a;
        sh.P[i] = i % LD == i / LD ? inv : 0.f;
    }
    __syncthreads();
    // phases of at most STEPS_A_PHASE steps, the shorter ones first
    int left = co.steps, phases = (left + STEPS_A_PHASE - 1) / STEPS_A_PHASE;
    while (true) {
        const int now = left / phases;
        const bool bad = small_steps<T, R>(sh, co, now);
        left -= now;
        const float p = 1.f / fragments<T, R, TALL>(x, sh, bad);
        if (--phases == 0) {
            write_px<T, R, TALL>(x, sh, p, first, end);
            return;
        }
        // P's elements are below 2^14 and M's columns below 2^15 long, so the product's below 2^32
        constexpr float u = 0x1p-17f;
        gram_of_px<T, R, TALL>(x, sh, u, first, end, acc);
        begin_tiles<T, R, TALL>(x, sh, first, end);
        gather<T, R, TALL>(acc, x, (p / u) * (p / u), sh);
    }
}

template <typename T, int R, int N>
__global__ void __launch_bounds__(OT, R == 64 ? 1 : 2) ortho_kernel(const __grid_constant__ OrthoTab<N> tab) {
    extern __shared__ __align__(16) unsigned char smem[];
    OrthoShared<T, R>& sh = *reinterpret_cast<OrthoShared<T, R>*>(smem);
    const OrthoEntry& e = tab.e[blockIdx.x / cg::this_cluster().num_blocks()];
    if (e.tall) orthogonal<T, R, true>(e, tab.co, sh);
    else orthogonal<T, R, false>(e, tab.co, sh);
}

template <typename T, int R, int N>
cudaError_t launch_n(const OrthoEntry* e, int n, const OrthoCoeffs& co, int blocks, cudaStream_t s) {
    OrthoTab<N> tab;
    tab.co = co;
    std::copy(e, e + n, tab.e);
    auto* kern = ortho_kernel<T, R, N>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(OrthoShared<T, R>));
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n * blocks));
    cfg.blockDim = dim3(OT);
    cfg.dynamicSmemBytes = sizeof(OrthoShared<T, R>);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tab);
}

constexpr int TAB_SMALL = 64, TAB_LARGE = 1300;      // 1.6 KB and 31 KB of kernel parameters

int tile_for(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : 64; }

// Blocks of a cluster for n matrices, the longest of `longest` columns: the first power of two that
// gives each SM at least two (for 56 matrices 448 blocks on 304 places), and no more than have
// 512 columns each, two tiles a warp.  (Two fp32 adapters of the
// 8B widths, 112 matrices: 98 us with clusters of four, 129 of eight, 121 of two; 1,200 of 32 x
// 4,096: 478 us with a block each, 598 with two: a block does the r x r steps of its matrix, so
// more blocks do them more often.)  The blocks decide the order of a matrix's sums, and so do the other matrices of
// a call: one size for each shape would cost a large set two blocks' r x r steps or one adapter its second block.
int blocks_for(int n, int longest, int num_sms) {
    int blocks = 1;
    while (blocks < MAX_BLOCKS && (int64_t)n * blocks < 2 * num_sms && longest / blocks >= 1024) blocks *= 2;
    return blocks;
}

template <typename T, int R>
cudaError_t launch_r(const OrthoEntry* e, int n, const OrthoCoeffs& co, int blocks, cudaStream_t s) {
    for (; n > 0; e += TAB_LARGE, n -= TAB_LARGE) {
        const int k = n < TAB_LARGE ? n : TAB_LARGE;
        const cudaError_t err = k <= TAB_SMALL ? launch_n<T, R, TAB_SMALL>(e, k, co, blocks, s)
                                               : launch_n<T, R, TAB_LARGE>(e, k, co, blocks, s);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t launch_ortho_t(std::vector<OrthoEntry>& e, const OrthoCoeffs& co, int num_sms, cudaStream_t s) {
    // a launch for each size of tile, the longest first: short ones fill the end
    std::stable_sort(e.begin(), e.end(), [](const OrthoEntry& a, const OrthoEntry& b) {
        return tile_for(a.r) != tile_for(b.r) ? tile_for(a.r) > tile_for(b.r) : a.n > b.n;
    });
    for (size_t i = 0; i < e.size();) {
        size_t j = i;
        while (j < e.size() && tile_for(e[j].r) == tile_for(e[i].r)) ++j;
        const int n = (int)(j - i), tile = tile_for(e[i].r), blocks = blocks_for(n, e[i].n, num_sms);
        const cudaError_t err = tile == 16   ? launch_r<T, 16>(&e[i], n, co, blocks, s)
                                : tile == 32 ? launch_r<T, 32>(&e[i], n, co, blocks, s)
                                             : launch_r<T, 64>(&e[i], n, co, blocks, s);
        if (err != cudaSuccess) return err;
        i = j;
    }
    return cudaSuccess;
}

}  // namespace

}  // namespace mlk
