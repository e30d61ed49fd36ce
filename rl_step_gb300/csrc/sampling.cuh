// Inverse-CDF sampling of one row by a warp, in vocabulary order, from the
// log-sum-exp partials of the vocabulary tiles and the logits of one tile.
#pragma once

#include "internal.h"

namespace mlk {

// The tile in which the cumulative sum of exp(prow[j] - lse) passes u, and the
// mass before it.  When rounding leaves the total at or below u: the last tile
// with a non-zero mass and before = -infinity.
__device__ __forceinline__ int sample_tile(const float* __restrict__ prow, int n_nt, float lse, float u, int lane,
                                           float& before) {
    float run = 0.f;          // mass of the tiles before `base`
    int T = -1, last_nz = -1;
    before = 0.f;
    for (int base = 0; base < n_nt && T < 0; base += 32) {
        const int j = base + lane;
        const float m = j < n_nt ? __expf(prow[j] - lse) : 0.f;
        float c = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) c += x;
        }
        const unsigned nz = __ballot_sync(0xffffffffu, m > 0.f);
        if (nz) last_nz = base + 31 - __clz(nz);
        const unsigned pass = __ballot_sync(0xffffffffu, run + c > u);
        if (pass) {
            const int L = __ffs(pass) - 1;
            T = base + L;
            const float cprev = __shfl_sync(0xffffffffu, c - m, L);
            before = run + cprev;
        } else {
            run += __shfl_sync(0xffffffffu, c, 31);
        }
    }
    if (T < 0) {                 // rounding: u at or above the total mass
        T = last_nz >= 0 ? last_nz : 0;
        before = -INFINITY;      // take the tile's last non-zero column
    }
    return T;
}

// The column of the tile [c0, c0 + bn) at which the sum passes u; z: the tile's
// logits, z[0] that of column c0 (bn = 256: 8 columns per lane; bn = 32: 1).
// When rounding leaves the sum at or below u, the last column with a non-zero
// probability.
__device__ __forceinline__ int sample_column(const float* z, int c0, int bn, int V, float lse, float u, float before,
                                             int lane) {
    const int per = bn / 32;
    float pv[8];
    float ls = 0.f;
    for (int e = 0; e < per; ++e) {
        const int v = lane * per + e;
        pv[e] = c0 + v < V ? __expf(z[v] - lse) : 0.f;
        ls += pv[e];
    }
    float c = ls;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += x;
    }
    int pick = -1;
    const unsigned pass = __ballot_sync(0xffffffffu, before + c > u);
    if (pass) {
        const int L = __ffs(pass) - 1;
        if (lane == L) {
            float r = before + (c - ls);
            for (int e = 0; e < per; ++e) {
                r += pv[e];
                if (r > u) { pick = c0 + lane * per + e; break; }
            }
            if (pick < 0) {          // rounding inside the lane's columns
                for (int e = per - 1; e >= 0; --e)
                    if (pv[e] > 0.f) { pick = c0 + lane * per + e; break; }
            }
        }
        pick = __shfl_sync(0xffffffffu, pick, L);
    }
    if (pick < 0) {                  // last non-zero column of the tile
        int mine = -1;
        for (int e = per - 1; e >= 0; --e)
            if (pv[e] > 0.f) { mine = c0 + lane * per + e; break; }
        const unsigned has = __ballot_sync(0xffffffffu, mine >= 0);
        pick = has ? __shfl_sync(0xffffffffu, mine, 31 - __clz(has)) : c0;
    }
    return pick;
}

}  // namespace mlk
