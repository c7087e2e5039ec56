// entmax.cuh -- the exact alpha-entmax threshold of a set of candidates, solved
// by one CTA (shared by the decode paths over bf16 and 4-bit caches).
#pragma once

#include "common.cuh"

namespace ekv {

// The entmax threshold: the root t of sum_c [z_c - t]_+^r = 1 over the
// candidates (every token with weight has z > z_max - 1), which lies in
// [lo, hi] = [z_max - 1, z_max - n^(1-alpha)] where F(t) = sum - 1 decreases.
// Newton's method, for r >= 1 (alpha <= 2) on g(t) = (sum_c [z_c - t]_+^r)^(1/r),
// a norm of (z - t)_+ and so convex (one step when the support's z are equal),
// from the left end; for r < 1 on F, which is then concave, from the right
// end: either way the iterates move to the root monotonically.
// for_each(add, first, stride) calls add(z) on candidates first, first +
// stride, ...  With n candidates, n <= TAU_WARP_MAX, warp 0 runs every pass
// by itself (lane-strided sums, a shuffle butterfly) and hands t to the other
// warps with one barrier at the end.  Otherwise each thread takes a
// NT-strided share and the warps' sums are added in warp order
// (reproducible), one barrier per pass (red is double-buffered).  All NT
// threads call it and return the same t.
constexpr int TAU_WARP_MAX = 256;
template <int NT, class ForEach>
__device__ float entmax_tau(ForEach for_each, int n, float lo, float hi, float zmax, float r, int ri,
                            float (*red)[NT / 32][2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool per_warp = n <= TAU_WARP_MAX;
    const int first = per_warp ? lane : (int)threadIdx.x, stride = per_warp ? 32 : NT;
    const float tol = 1e-7f * fmaxf(1.f, fabsf(zmax));
    const int rim1 = ri >= 2 ? ri - 1 : 0;
    float t = r >= 1.f ? lo : hi;
    for (int it = 0; it < 40 && (!per_warp || warp == 0); ++it) {
        float s0 = 0.f, s1 = 0.f;  // sum x^r, sum x^(r-1) over x = z - t > 0
        auto add = [&](float z) {
            const float x = z - t;
            if (ri == 2) {  // alpha = 3/2: branch-free
                const float y = fmaxf(x, 0.f);
                s0 = fmaf(y, y, s0);
                s1 += y;
            } else if (x > 0.f) {
                const float y = ri == 1 ? 1.f : pos_pow(x, r - 1.f, rim1);
                s0 = fmaf(x, y, s0);
                s1 += y;
            }
        };
        for_each(add, first, stride);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s0 += __shfl_xor_sync(FULL, s0, o);
            s1 += __shfl_xor_sync(FULL, s1, o);
        }
        float S0 = s0, S1 = s1;
        if (!per_warp) {
            if (lane == 0) {
                red[it & 1][warp][0] = s0;
                red[it & 1][warp][1] = s1;
            }
            __syncthreads();
            S0 = 0.f;
            S1 = 0.f;
#pragma unroll
            for (int ww = 0; ww < NT / 32; ++ww) {
                S0 += red[it & 1][ww][0];
                S1 += red[it & 1][ww][1];
            }
        }
        if (!(S1 > 0.f)) break;  // no weight right of t (t at the top already)
        // r >= 1: t' = t + (S0 - S0^(1-1/r)) / S1;  r < 1: t' = t + (S0 - 1) / (r S1)
        float step;
        if (ri == 2) step = (S0 - sqrtf(S0)) / S1;
        else if (ri == 1) step = (S0 - 1.f) / S1;
        else if (r >= 1.f) step = (S0 - powf(S0, 1.f - 1.f / r)) / S1;
        else step = (S0 - 1.f) / (r * S1);
        const float tn = fminf(hi, fmaxf(lo, t + step));
        const bool done = !(fabsf(tn - t) > tol);
        t = tn;
        if (done) break;
    }
    if (per_warp) {
        __syncthreads();  // every warp is past the caller's earlier use of red
        if (threadIdx.x == 0) red[0][0][0] = t;
        __syncthreads();
        t = red[0][0][0];
    }
    return t;
}

// The same root for r < 1, by halving [lo, hi]: a token that comes into the
// support does so with an infinite slope, and Newton's steps may pass the root
// back and forth.  The weight of a token next to the root hangs on more bits
// of z - t than there are (alpha = 10: a weight of 0.1 is z - t = 1e-9, one of
// 0.03 2e-14), but is well determined by the others': tokens between the
// neighbours lo and hi that the halving (in 64 bits) ends with share what those
// above hi leave.
struct EntmaxEdge {
    double lo = 0., hi = 0.;  // sum [z - lo]_+^r >= 1, sum [z - hi]_+^r <= 1
    float rest = 0.f;         // weight of each token in (lo, hi]
    __device__ __forceinline__ float weight(float z, float r) const {
        return (double)z > hi ? powf((float)((double)z - hi), r) : (double)z > lo ? rest : 0.f;
    }
};
template <int NT, class ForEach>
__device__ EntmaxEdge entmax_tau_halving(ForEach for_each, float from, float to, float r, float (*red)[NT / 32][2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    EntmaxEdge e;
    e.lo = from;
    e.hi = to;
    for (int it = 0;; ++it) {
        const double mid = 0.5 * (e.lo + e.hi);
        const bool last = it == 80 || !(mid > e.lo && mid < e.hi);  // neighbours, or both next to 0
        const double t = last ? e.hi : mid;
        float s = 0.f, n = 0.f;
        for_each([&](float z) {
            if ((double)z > t) s += powf((float)((double)z - t), r);
            else if (last && (double)z > e.lo) n += 1.f;
        }, (int)threadIdx.x, NT);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s += __shfl_xor_sync(FULL, s, o);
            n += __shfl_xor_sync(FULL, n, o);
        }
        if (lane == 0) {
            red[it & 1][warp][0] = s;
            red[it & 1][warp][1] = n;
        }
        __syncthreads();
        s = n = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            s += red[it & 1][w][0];
            n += red[it & 1][w][1];
        }
        if (last) {
            e.rest = n > 0.f ? fmaxf(1.f - s, 0.f) / n : 0.f;
            return e;
        }
        if (s >= 1.f) e.lo = mid;
        else e.hi = mid;
    }
}

}  // namespace ekv
