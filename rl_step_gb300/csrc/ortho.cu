// Updates made orthogonal by Newton-Schulz products (mlora_orthogonalize in
// include/mlora.h), for matrices whose shorter side is at most 64, as LoRA
// factors' is.  With X [r x n] over the shorter side, X_0 = M / (|M| + eps):
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
// A cluster of blocks takes a matrix and does all of it, its blocks each a part of
// the long side: the second and third pass find it in L2, and no launch or
// workspace is between them.  Sums meet in a fixed order: results repeat.
//
// The products run on mma.sync with tf32 operands, each fp32 factor as two of them
// (x = hi + lo, hi of 11 bits; three products, at most 2^-20 of the terms off), straight
// from registers: the same fragment of X serves as both operands of X X^T, and the
// output fragment of P X serves as both of the next.  The tensor cores cut their sums off
// (towards 0), so few products are chained, the small parts first, and their results
// are added in fp32 (rounded to nearest): chained over the whole length a 64 x 700
// matrix was off by 8e-6 of its norm where plain fp32 products are by 1e-6.  r is 4 to 64: a 128-row tcgen05
// tile would hold 2 to 8 matrices and form their cross products for nothing.
#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>
#include <new>
#include <vector>

#include "kv_common.cuh"

namespace cg = cooperative_groups;

namespace mlk {

namespace {

constexpr int OT = 256;                      // threads of a block
constexpr int OW = OT / 32;
constexpr int STEPS_A_PHASE = 3;

struct OrthoEntry {
    const void* src;
    void* dst;
    int n;                                   // longer side
    int16_t r;                               // shorter side
    int8_t tall;                             // rows are the longer side
    int8_t vec;                              // 4 elements side by side can be read and written at once
};
struct OrthoCoeffs {
    float a, b, c, eps;
    int steps;
};
template <int N>
struct OrthoTab {
    OrthoCoeffs co;
    OrthoEntry e[N];
};

// the nearest value of 11 bits (away from 0 between two); x is far below fp32's largest
__device__ __forceinline__ float tf32_hi(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }

__device__ __forceinline__ void mma8(float (&d)[4], const float (&a)[4], float b0, float b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                   "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
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

// X of an entry: X(i, k) = M[i][k], or M[k][i] where M is tall; 0 outside.
// Row slots: the fragments' row 8 j + g is row i = 8 j + g of X, or (R / 8) g + j where
// M is tall, so that a thread's rows lie side by side there.
template <typename T, int R>
struct Matrix {
    const T* src;
    T* dst;
    int n, r;
    bool tall, vec;
    float f;                                 // a power of two that X is taken with
    __device__ __forceinline__ explicit Matrix(const OrthoEntry& e)
        : src(static_cast<const T*>(e.src)), dst(static_cast<T*>(e.dst)), n(e.n), r(e.r), tall(e.tall), vec(e.vec), f(1.f) {}
    __device__ __forceinline__ float at(int i, int k) const {
        if (i >= r || k >= n) return 0.f;
        return to_f(src[tall ? (int64_t)k * r + i : (int64_t)i * n + k]) * f;
    }
    // X(i, k .. k + 3)
    __device__ __forceinline__ void along_k(int i, int k, float (&v)[4]) const {
        if (vec && i < r && k + 4 <= n) {
            load4(src + (int64_t)i * n + k, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= f;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = at(i, k + e);
        }
    }
    // X(i .. i + 3, k)
    __device__ __forceinline__ void along_i(int i, int k, float (&v)[4]) const {
        if (vec && i + 4 <= r && k < n) {
            load4(src + (int64_t)k * r + i, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= f;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = at(i + e, k);
        }
    }
    __device__ __forceinline__ int row_of(int slot) const { return tall ? slot % 8 * (R / 8) + slot / 8 : slot; }
    // the row of X at place t (0 .. 3) or t + 4 of the k-step s of a product P X
    __device__ __forceinline__ int k_row(int s, int t, int second) const {
        return tall ? s / 2 * 16 + 4 * t + s % 2 * 2 + second : 8 * s + t + 4 * second;
    }
};

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
    // += x x^T over 8 columns; x[j][0 / 1]: row slot 8 j + g, place t / t + 4.  EXACT: x has no low part.
    template <bool EXACT>
    __device__ __forceinline__ void add(const float (&x)[J][2]) {
        float hi[J][2], lo[J][2];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                hi[j][e] = EXACT ? x[j][e] : tf32_hi(x[j][e]);
                lo[j][e] = x[j][e] - hi[j][e];
            }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const float ah[4] = {hi[2 * m][0], hi[2 * m + 1][0], hi[2 * m][1], hi[2 * m + 1][1]};
            const float al[4] = {lo[2 * m][0], lo[2 * m + 1][0], lo[2 * m][1], lo[2 * m + 1][1]};
#pragma unroll
            for (int j = 2 * m; j < J; ++j) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                if (!EXACT) {
                    mma8(d, al, hi[j][0], hi[j][1]);
                    mma8(d, ah, lo[j][0], lo[j][1]);
                }
                mma8(d, ah, hi[j][0], hi[j][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[tile(m, j)][e] += d[e];
            }
        }
    }
};

// Shared memory of a block: the products, P and A as plain r x r matrices of pitch R + 4, and P's fragments.
template <int R>
struct OrthoShared {
    static constexpr int LD = R + 4;
    float part[4][R * LD];                   // the warps' sums; [0]: the block's
    float A[R * LD], Q[R * LD], B[R * LD], P[R * LD];
    // P's fragments [m][s][lane][4], high and low parts
    float4 ph[R / 16][R / 8][32], pl[R / 16][R / 8][32];
    float red[OW];
};

// C = x A B + y D + z I for R x R matrices in shared memory (D may be null); C is none of them.
template <int R>
__device__ __forceinline__ void small_product(float* C, const float* A, const float* B, float x, const float* D, float y,
                                              float z) {
    constexpr int LD = R + 4, TILES = R / 16 * (R / 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int tile = warp; tile < TILES; tile += OW) {
        const int m = tile / (R / 8) * 16, n = tile % (R / 8) * 8;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < R; k += 8) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            const float a[4] = {A[(m + g) * LD + k + t], A[(m + g + 8) * LD + k + t], A[(m + g) * LD + k + t + 4],
                                A[(m + g + 8) * LD + k + t + 4]};
            const float b[2] = {B[(k + t) * LD + n + g], B[(k + t + 4) * LD + n + g]};
            float ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) ah[e] = tf32_hi(a[e]), al[e] = a[e] - ah[e];
            const float bh[2] = {tf32_hi(b[0]), tf32_hi(b[1])};
            mma8(d, al, bh[0], bh[1]);
            mma8(d, ah, b[0] - bh[0], b[1] - bh[1]);
            mma8(d, ah, bh[0], bh[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += d[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = m + g + e / 2 * 8, j = n + 2 * t + e % 2;
            C[i * LD + j] = x * sum[e] + (D ? y * D[i * LD + j] : 0.f) + (i == j ? z : 0.f);
        }
    }
    __syncthreads();
}

// The blocks' sums of a product, in X's row order, in sh.A of every block of the cluster.
template <typename T, int R>
__device__ __forceinline__ void gather(const Gram<R>& acc, const Matrix<T, R>& x, OrthoShared<R>& sh) {
    constexpr int LD = R + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    Gram<R> s = acc;
    auto each = [&](float* p, bool load) {
#pragma unroll
        for (int m = 0; m < R / 16; ++m)
#pragma unroll
            for (int j = 2 * m; j < R / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float& v = s.v[Gram<R>::tile(m, j)][e];
                    float& q = p[(16 * m + g + e / 2 * 8) * LD + 8 * j + 2 * t + e % 2];
                    if (load) v += q; else q = v;
                }
    };
    // half of the warps hand theirs to the other half
#pragma unroll
    for (int half = OW / 2; half >= 1; half /= 2) {
        if (warp >= half && warp < 2 * half) each(sh.part[warp - half], false);
        __syncthreads();
        if (warp < half) each(sh.part[warp], true);
        __syncthreads();
    }
    if (warp == 0) each(sh.part[0], false);
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    const int blocks = (int)cl.num_blocks();
    for (int i = threadIdx.x; i < R * R; i += OT) {
        int a = i / R, b = i % R;
        // (the tiles below the diagonal's block row are not there)
        const int at = a / 16 <= b / 16 ? a * LD + b : b * LD + a;
        float v = 0.f;
        for (int k = 0; k < blocks; ++k) v += cl.map_shared_rank(&sh, k)->part[0][at];
        sh.A[x.row_of(a) * LD + x.row_of(b)] = v;
    }
    cl.sync();
}

// P as fragments for P X
template <typename T, int R>
__device__ __forceinline__ void fragments(const Matrix<T, R>& x, OrthoShared<R>& sh) {
    constexpr int LD = R + 4;
    for (int i = threadIdx.x; i < R / 16 * (R / 8) * 32; i += OT) {
        const int lane = i % 32, s = i / 32 % (R / 8), m = i / 32 / (R / 8), g = lane >> 2, t = lane & 3;
        float v[4], hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = sh.P[x.row_of(16 * m + g + e % 2 * 8) * LD + x.k_row(s, t, e / 2)];
            hi[e] = tf32_hi(v[e]);
        }
        sh.ph[m][s][lane] = make_float4(hi[0], hi[1], hi[2], hi[3]);
        sh.pl[m][s][lane] = make_float4(v[0] - hi[0], v[1] - hi[1], v[2] - hi[2], v[3] - hi[3]);
    }
    __syncthreads();
}

// A warp's columns [k0, k0 + 32) of P X: d[m][c][e], row slot 16 m + g + 8 (e / 2) and column
// k0 + 4 (2 t + e % 2) + c (M wide) or k0 + 8 c + 2 t + e % 2 (tall).
template <typename T, int R>
__device__ __forceinline__ void times_p(const Matrix<T, R>& x, const OrthoShared<R>& sh, int k0, float (&d)[R / 16][4][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr bool EXACT = sizeof(T) == 2;   // (times a power of two)
#pragma unroll
    for (int m = 0; m < R / 16; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[m][c][e] = 0.f;
#pragma unroll
    for (int s2 = 0; s2 < R / 16; ++s2) {
        // 16 rows of X: b[c][s][place]
        float b[4][2][2];
        if (x.tall) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v[4];
                x.along_i(16 * s2 + 4 * t, k0 + 8 * c + g, v);
                b[c][0][0] = v[0]; b[c][0][1] = v[1]; b[c][1][0] = v[2]; b[c][1][1] = v[3];
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
                x.along_k(16 * s2 + 8 * (q / 2) + 4 * (q % 2) + t, k0 + 4 * g, v);
#pragma unroll
                for (int c = 0; c < 4; ++c) b[c][q / 2][q % 2] = v[c];
            }
        }
        float hi[2][4][2], lo[2][4][2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    hi[s][c][e] = EXACT ? b[c][s][e] : tf32_hi(b[c][s][e]);
                    lo[s][c][e] = b[c][s][e] - hi[s][c][e];
                }
#pragma unroll
        for (int m = 0; m < R / 16; ++m) {
            float z[4][4] = {};
            float ah[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float4 h4 = sh.ph[m][2 * s2 + s][lane], l4 = sh.pl[m][2 * s2 + s][lane];
                const float al[4] = {l4.x, l4.y, l4.z, l4.w};
                ah[s][0] = h4.x; ah[s][1] = h4.y; ah[s][2] = h4.z; ah[s][3] = h4.w;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mma8(z[c], al, hi[s][c][0], hi[s][c][1]);
                    if (!EXACT) mma8(z[c], ah[s], lo[s][c][0], lo[s][c][1]);
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int c = 0; c < 4; ++c) mma8(z[c], ah[s], hi[s][c][0], hi[s][c][1]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[m][c][e] += z[c][e];
        }
    }
}

// The sums of X X^T over the block's columns.
template <typename T, int R>
__device__ __forceinline__ void gram_of_x(const Matrix<T, R>& x, int first, int end, Gram<R>& acc) {
    constexpr int J = R / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    acc.clear();
    for (int k0 = first + 32 * warp; k0 < end; k0 += 32 * OW) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {        // 16 columns: two products of 8
            float u[2][J][2];
            if (x.tall) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = k0 + 16 * h + 8 * s + t + 4 * e;
                        if constexpr (J % 4 == 0) {
#pragma unroll
                            for (int j = 0; j < J; j += 4) {
                                float v[4];
                                x.along_i(J * g + j, k, v);
#pragma unroll
                                for (int q = 0; q < 4; ++q) u[s][j + q][e] = v[q];
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < J; ++j) u[s][j][e] = x.at(J * g + j, k);
                        }
                    }
            } else {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float v[4];
                    x.along_k(8 * j + g, k0 + 16 * h + 4 * t, v);
                    u[0][j][0] = v[0]; u[0][j][1] = v[1]; u[1][j][0] = v[2]; u[1][j][1] = v[3];
                }
            }
            acc.template add<sizeof(T) == 2>(u[0]);
            acc.template add<sizeof(T) == 2>(u[1]);
        }
    }
}

// The same of P X.
template <typename T, int R>
__device__ __forceinline__ void gram_of_px(const Matrix<T, R>& x, const OrthoShared<R>& sh, int first, int end, Gram<R>& acc) {
    constexpr int J = R / 8;
    const int warp = threadIdx.x >> 5;
    acc.clear();
    for (int k0 = first + 32 * warp; k0 < end; k0 += 32 * OW) {
        float d[R / 16][4][4];
        times_p<T, R>(x, sh, k0, d);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float u[J][2];
#pragma unroll
            for (int j = 0; j < J; ++j) u[j][0] = d[j / 2][c][j % 2 * 2], u[j][1] = d[j / 2][c][j % 2 * 2 + 1];
            acc.template add<false>(u);
        }
    }
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(bf16* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// dst = P X
template <typename T, int R>
__device__ __forceinline__ void write_px(const Matrix<T, R>& x, const OrthoShared<R>& sh, int first, int end) {
    constexpr int J = R / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int k0 = first + 32 * warp; k0 < end; k0 += 32 * OW) {
        float d[R / 16][4][4];
        times_p<T, R>(x, sh, k0, d);
        if (x.tall) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = k0 + 8 * c + 2 * t + e;
                    if (k >= x.n) continue;
                    T* out = x.dst + (int64_t)k * x.r;
                    auto v = [&](int j) { return d[j / 2][c][j % 2 * 2 + e]; };
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
                for (int h = 0; h < 2; ++h) {
                    const int i = 16 * m + 8 * h + g;
                    if (i >= x.r) continue;
                    T* out = x.dst + (int64_t)i * x.n;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = k0 + 8 * t + 4 * e;
                        auto v = [&](int c) { return d[m][c][2 * h + e]; };
                        if (x.vec && k + 4 <= x.n) {
                            store4(out + k, v(0), v(1), v(2), v(3));
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (k + c < x.n) out[k + c] = from_f<T>(v(c));
                        }
                    }
                }
        }
    }
}

// `steps` steps on sh.A and sh.P: P <- Q P with Q = a I + b A + c A^2, A <- Q A Q (they commute).
template <int R>
__device__ __forceinline__ void small_steps(OrthoShared<R>& sh, const OrthoCoeffs& co, int steps) {
    constexpr int LD = R + 4;
    auto copy = [&](float* to, const float* from) {
        for (int i = threadIdx.x; i < R * LD; i += OT) to[i] = from[i];
        __syncthreads();
    };
    for (int k = 0; k < steps; ++k) {
        small_product<R>(sh.Q, sh.A, sh.A, co.c, sh.A, co.b, co.a);
        small_product<R>(sh.B, sh.Q, sh.P, 1.f, nullptr, 0.f, 0.f);
        copy(sh.P, sh.B);
        if (k + 1 < steps) {
            small_product<R>(sh.B, sh.Q, sh.A, 1.f, nullptr, 0.f, 0.f);
            small_product<R>(sh.A, sh.B, sh.Q, 1.f, nullptr, 0.f, 0.f);
        }
    }
}

template <typename T, int R, int N>
__global__ void __launch_bounds__(OT) ortho_kernel(const __grid_constant__ OrthoTab<N> tab) {
    constexpr int LD = R + 4;
    extern __shared__ __align__(16) unsigned char smem[];
    OrthoShared<R>& sh = *reinterpret_cast<OrthoShared<R>*>(smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), blocks = (int)cl.num_blocks(), tid = threadIdx.x;
    Matrix<T, R> x(tab.e[blockIdx.x / blocks]);
    // the block's columns, in stretches of 32
    const int all = (x.n + 31) / 32, per = (all + blocks - 1) / blocks;
    const int first = min(rank * per, all) * 32, end = min(rank * per + per, all) * 32;
    Gram<R> acc;
    gram_of_x<T, R>(x, first, end, acc);
    gather<T, R>(acc, x, sh);
    auto trace = [&]() {
        float s = 0.f;
        for (int i = 0; i < x.r; ++i) s += sh.A[i * LD + i];
        return s;
    };
    float sq = trace();
    if (!(sq > 1e-25f && sq < 1e30f)) {
        // squares beyond fp32, or none: X relative to its largest magnitude
        float m = 0.f;
        bool bad = false;
        for (int64_t i = tid + (int64_t)rank * OT; i < (int64_t)x.n * x.r; i += (int64_t)OT * blocks) {
            const float v = fabsf(to_f(x.src[i]));
            bad |= !(v <= FLT_MAX);
            m = fmaxf(m, v);
        }
        if (bad) m = INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((tid & 31) == 0) sh.red[tid >> 5] = m;
        cl.sync();
        for (int b = 0; b < blocks; ++b)
            for (int w = 0; w < OW; ++w) m = fmaxf(m, cl.map_shared_rank(&sh, b)->red[w]);
        cl.sync();
        if (m > FLT_MAX) {
            // an infinity or NaN
            for (int64_t i = tid + (int64_t)rank * OT; i < (int64_t)x.n * x.r; i += (int64_t)OT * blocks)
                x.dst[i] = from_f<T>(__int_as_float(0x7fc00000));
            return;
        }
        if (m > 0.f) {
            int e;
            frexpf(m, &e);
            // X becomes at most 2; a factor that fp32 holds
            x.f = ldexpf(1.f, min(1 - e, 126));
            gram_of_x<T, R>(x, first, end, acc);
            gather<T, R>(acc, x, sh);
            sq = trace();
        }
    }
    // X_0 = inv (f M); its products.  A matrix of zeros stays zero whatever eps.
    const float inv = sq == 0.f ? 0.f : 1.f / (sqrtf(sq) + tab.co.eps * x.f);
    __syncthreads();                         // (all have their trace)
    for (int i = tid; i < R * LD; i += OT) {
        sh.A[i] = sh.A[i] * inv * inv;
        sh.P[i] = i % LD == i / LD ? inv : 0.f;
    }
    __syncthreads();
    // phases of at most STEPS_A_PHASE steps, the shorter ones first
    int left = tab.co.steps, phases = (left + STEPS_A_PHASE - 1) / STEPS_A_PHASE;
    while (true) {
        const int now = left / phases;
        small_steps<R>(sh, tab.co, now);
        left -= now;
        fragments<T, R>(x, sh);
        if (--phases == 0) break;
        gram_of_px<T, R>(x, sh, first, end, acc);
        gather<T, R>(acc, x, sh);
    }
    write_px<T, R>(x, sh, first, end);
}

template <typename T, int R, int N>
cudaError_t launch_n(const OrthoEntry* e, int n, const OrthoCoeffs& co, int blocks, cudaStream_t s) {
    OrthoTab<N> tab;
    tab.co = co;
    std::copy(e, e + n, tab.e);
    auto* kern = ortho_kernel<T, R, N>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(OrthoShared<R>));
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n * blocks));
    cfg.blockDim = dim3(OT);
    cfg.dynamicSmemBytes = sizeof(OrthoShared<R>);
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

template <typename T, int R>
cudaError_t launch_r(const OrthoEntry* e, int n, const OrthoCoeffs& co, cudaStream_t s) {
    for (; n > 0; e += TAB_LARGE, n -= TAB_LARGE) {
        const int k = n < TAB_LARGE ? n : TAB_LARGE, blocks = 4;
        const cudaError_t err = k <= TAB_SMALL ? launch_n<T, R, TAB_SMALL>(e, k, co, blocks, s)
                                               : launch_n<T, R, TAB_LARGE>(e, k, co, blocks, s);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t launch_t(std::vector<OrthoEntry>& e, const OrthoCoeffs& co, cudaStream_t s) {
    // by the tiles' size, the longest first: short ones fill the end
    auto tile = [](const OrthoEntry& x) { return x.r <= 16 ? 16 : x.r <= 32 ? 32 : 64; };
    std::stable_sort(e.begin(), e.end(), [&](const OrthoEntry& a, const OrthoEntry& b) {
        return tile(a) != tile(b) ? tile(a) > tile(b) : a.n > b.n;
    });
    for (size_t i = 0; i < e.size();) {
        size_t j = i;
        while (j < e.size() && tile(e[j]) == tile(e[i])) ++j;
        const int n = (int)(j - i);
        const cudaError_t err = tile(e[i]) == 16   ? launch_r<T, 16>(&e[i], n, co, s)
                                : tile(e[i]) == 32 ? launch_r<T, 32>(&e[i], n, co, s)
                                                   : launch_r<T, 64>(&e[i], n, co, s);
        if (err != cudaSuccess) return err;
        i = j;
    }
    return cudaSuccess;
}

}  // namespace

}  // namespace mlk

// ----------------------------------------------------------------------------
// C ABI
// ----------------------------------------------------------------------------
using namespace mlk;

extern "C" int mlora_orthogonalize(const mlora_matrix_set* m, const mlora_newton_schulz* p, void* stream) try {
    if (!m || !p) return kv_fail(MLORA_E_ARG, "NULL matrices or parameters");
    if (m->n_matrices < 0) return kv_fail(MLORA_E_ARG, "%d matrices", m->n_matrices);
    if (m->dtype != MLORA_BF16 && m->dtype != MLORA_FP32) return kv_fail(MLORA_E_ARG, "unknown dtype %d", m->dtype);
    if (m->n_matrices > 0 && (!m->src || !m->rows || !m->cols)) return kv_fail(MLORA_E_ARG, "NULL matrix or size array");
    if (p->steps < 1 || p->steps > MLORA_ORTHO_MAX_STEPS)
        return kv_fail(MLORA_E_ARG, "%d steps, 1 .. %d are possible", p->steps, MLORA_ORTHO_MAX_STEPS);
    if (!(fabsf(p->a) <= FLT_MAX && fabsf(p->b) <= FLT_MAX && fabsf(p->c) <= FLT_MAX) || !(p->eps > 0.f && p->eps <= FLT_MAX))
        return kv_fail(MLORA_E_ARG, "coefficients must be finite, eps positive");
    const uintptr_t es = m->dtype == MLORA_BF16 ? 2 : 4;
    std::vector<OrthoEntry> e;
    e.reserve(m->n_matrices);
    for (int i = 0; i < m->n_matrices; ++i) {
        const int64_t rows = m->rows[i], cols = m->cols[i];
        if (rows < 0 || cols < 0 || rows > INT32_MAX - 4096 || cols > INT32_MAX - 4096)
            return kv_fail(MLORA_E_ARG, "matrix %d: %lld x %lld", i, (long long)rows, (long long)cols);
        if (rows == 0 || cols == 0) continue;
        const int64_t r = rows < cols ? rows : cols;
        if (r > MLORA_MAX_RANK)
            return kv_fail(MLORA_E_ARG, "matrix %d: %lld x %lld, the shorter side is at most %d", i, (long long)rows,
                           (long long)cols, MLORA_MAX_RANK);
        const void* src = m->src[i];
        void* dst = m->dst ? m->dst[i] : const_cast<void*>(src);
        if (!src || !dst) return kv_fail(MLORA_E_ARG, "matrix %d is NULL", i);
        const uintptr_t both = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst);
        if (both % es) return kv_fail(MLORA_E_ARG, "matrix %d is not aligned to its elements", i);
        OrthoEntry x;
        x.src = src;
        x.dst = dst;
        x.n = (int)(rows < cols ? cols : rows);
        x.r = (int16_t)r;
        x.tall = rows > cols;
        x.vec = both % (4 * es) == 0 && cols % 4 == 0;
        e.push_back(x);
    }
    const OrthoCoeffs co{p->a, p->b, p->c, p->eps, p->steps};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = m->dtype == MLORA_BF16 ? launch_t<bf16>(e, co, s) : launch_t<float>(e, co, s);
    if (err != cudaSuccess) return kv_fail(MLORA_E_CUDA, "orthogonalising: %s", cudaGetErrorString(err));
    return MLORA_OK;
} catch (const std::bad_alloc&) {
    return kv_fail(MLORA_E_NOMEM, "no host memory for the matrix table");
}
