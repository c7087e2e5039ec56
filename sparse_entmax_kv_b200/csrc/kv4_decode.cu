// kv4_decode.cu -- decode attention over the 4-bit cache, and its C entry
// points (include/entmaxkv_kv4.h).
//
// Mathematics.  With k_tj = s_tg c_tj + lo_tg for the coordinates j of group
// g, the score of token t is
//   q.k_t = sum_g [ s_tg sum_{j in g} q_j c_tj  +  lo_tg sum_{j in g} q_j ],
// so the codes themselves are the tensor-core operand: a code in the top
// mantissa bits of a bf16 with exponent 4 is the number 16 + c, exact, made
// by one shift and one mask for two codes; the 16 moves into the offset
// (lo - 16 s).  The products with the bf16 query are exact and are summed in
// fp32.  The values are treated the same way: the weights p_t s_tg (in three
// bf16 parts, 24 bits together) multiply 16 + c, and sum_t p_t (lo_tg - 16
// s_tg) is added at the end.
//
// Every warp owns a run of 16-token tiles of its group's page list and reads
// each tile once for all query heads of the group (heads are the n dimension
// of m16n8k16, tokens or value coordinates the m dimension).
//   softmax  running max, sum and output per head, one partial a CTA, merged
//            by combine_kernel in split order
//   entmax   scan_kernel keeps the tokens whose z can still carry weight
//            (z > running max - 1: no weight exceeds 1) as a list of (z,
//            value row) per warp; tau_kernel, one CTA a head, drops those
//            below the head's max - 1, solves for tau and sums p v over the
//            support
#include <cmath>
#include <cstring>

#include "../../include/entmaxkv_kv4.h"
#include "entmax.cuh"
#include "kv4.cuh"

namespace ekv {

namespace {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = AT_WARPS * 32;
constexpr int AT_SPLIT_CTAS = 148 * 6;  // CTAs the grid aims at
constexpr int AT_MIN_TILES = 4;         // tiles a warp gets at least

struct Kv4DecodeArgs {
    const uint16_t *q;
    const uint8_t *k4, *v4;
    const int *page_table, *seq_lens;
    const int *union_e, *union_blk, *union_cnt;  // null: every page
    float *out, *tau_out;
    float *part;          // [S][B Hq][d + 2] softmax partials
    float *cand_z;        // [B Hq][max_pages P]
    unsigned *cand_row;   // [B Hq][max_pages P]  blk P + slot
    int *seg_n;           // [B Hq][seg_len]
    float *seg_max;       // [B Hq][seg_len]
    int seg_len;          // segments of a head at most (any kv-head range)
    int B, Hq, Hkv, P, max_pages, num_blocks, S;
    int kv0, nk;
    float alpha;
    int r_int;
    int *status;
};

// (16 + code) of code pair p (bits 4p.. of each half of the unrotated word) as
// two bf16: the stored word holds pair 0 at the top of the mantissas already.
template <int p>
__device__ __forceinline__ unsigned codes_bf16(unsigned w) {
    const unsigned x = p == 0 ? w : p == 3 ? __funnelshift_r(w, w, 12) : w >> (4 * p);
    return (x & 0x00780078u) | 0x41804180u;
}

template <int N>
__device__ __forceinline__ void load_words(const unsigned char *src, unsigned (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
        w[0] = v.x;
        w[1] = v.y;
    }
}

// The group's queries as B fragments (lane: head lane / 4), and the sums of
// each coordinate group for the two heads of the lane's accumulator columns.
template <int D>
struct Queries {
    unsigned b[D / 16][2];
    float sum[Kv4<D>::NG][2];
    __device__ __forceinline__ void load(const uint16_t *q, int G) {
        const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
        const unsigned *qw = reinterpret_cast<const unsigned *>(q + (size_t)r * D);
#pragma unroll
        for (int g = 0; g < Kv4<D>::NG; ++g) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int j0 = 64 * g + 16 * c + 8 * i + 4 * h;
                    unsigned *d = b[2 * (2 * g + i) + h];
                    d[0] = r < G ? qw[j0 / 2] : 0u;
                    d[1] = r < G ? qw[j0 / 2 + 1] : 0u;
                    t += (bf16lo(d[0]) + bf16hi(d[0])) + (bf16lo(d[1]) + bf16hi(d[1]));
                }
            t += __shfl_xor_sync(FULL, t, 1);
            t += __shfl_xor_sync(FULL, t, 2);
            sum[g][0] = __shfl_sync(FULL, t, 8 * c);
            sum[g][1] = __shfl_sync(FULL, t, 8 * c + 4);
        }
    }
};

// q.k of the 16 tokens of a tile: z[0], z[1] token lane / 4, heads 2 (lane % 4)
// and + 1; z[2], z[3] token lane / 4 + 8.
template <int D>
__device__ __forceinline__ void tile_scores(const unsigned char *tile, const Queries<D> &Q, float scale, float (&z)[4]) {
    constexpr int NG = Kv4<D>::NG, WPL = Kv4<D>::WPL;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    unsigned w0[WPL], w1[WPL];
    load_words<WPL>(tile + r * (D / 2) + c * (4 * WPL), w0);
    load_words<WPL>(tile + (r + 8) * (D / 2) + c * (4 * WPL), w1);
    const unsigned *pp = reinterpret_cast<const unsigned *>(tile + Kv4<D>::CODES);
    unsigned p0[NG], p1[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        p0[g] = __ldg(pp + r * NG + g);
        p1[g] = __ldg(pp + (r + 8) * NG + g);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) z[v] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 2 * g; i < 2 * g + 2; ++i) {
            mma_bf16_16816(acc, codes_bf16<0>(w0[i]), codes_bf16<0>(w1[i]), codes_bf16<1>(w0[i]),
                           codes_bf16<1>(w1[i]), Q.b[2 * i][0], Q.b[2 * i][1]);
            mma_bf16_16816(acc, codes_bf16<2>(w0[i]), codes_bf16<2>(w1[i]), codes_bf16<3>(w0[i]),
                           codes_bf16<3>(w1[i]), Q.b[2 * i + 1][0], Q.b[2 * i + 1][1]);
        }
        const float s0 = bf16lo(p0[g]), s1 = bf16lo(p1[g]);
        const float o0 = fmaf(-16.f, s0, bf16hi(p0[g])), o1 = fmaf(-16.f, s1, bf16hi(p1[g]));
        z[0] = fmaf(s0, acc[0], fmaf(o0, Q.sum[g][0], z[0]));
        z[1] = fmaf(s0, acc[1], fmaf(o0, Q.sum[g][1], z[1]));
        z[2] = fmaf(s1, acc[2], fmaf(o1, Q.sum[g][0], z[2]));
        z[3] = fmaf(s1, acc[3], fmaf(o1, Q.sum[g][1], z[3]));
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) z[v] *= scale;
}

// The page list of a group and the tiles of one warp of one CTA.
struct Span {
    int b, kvh, bk, U, seq;
    int first, last;  // tiles [first, last) of the list
};

__device__ __forceinline__ Span warp_span(const Kv4DecodeArgs &a, int group, int seg) {
    Span s;
    group_of(group, a.kv0, a.nk, s.b, s.kvh);
    s.bk = s.b * a.Hkv + s.kvh;
    s.seq = seq_len_of(a.seq_lens, s.b, a.P, a.max_pages, a.status);
    s.U = a.union_e ? a.union_cnt[s.bk] : n_pages_of(s.seq, a.P);
    const long long T = (long long)s.U * (a.P / 16);
    const int W = a.S * AT_WARPS;
    s.first = (int)(T * seg / W);
    s.last = (int)(T * (seg + 1) / W);
    return s;
}

// Tile `t` of the list: its page's block (-1: skip), valid tokens and heads.
struct TileAt {
    int blk, t16, nval, mask;
};
__device__ __forceinline__ TileAt tile_at(const Kv4DecodeArgs &a, const Span &s, int t) {
    const int per = a.P / 16;
    const int e = t / per;
    TileAt r;
    r.t16 = t - e * per;
    int page;
    if (a.union_e) {
        const int entry = __ldg(a.union_e + (size_t)s.bk * a.max_pages + e);
        r.blk = __ldg(a.union_blk + (size_t)s.bk * a.max_pages + e);
        page = entry >> 8;
        r.mask = entry & 0xff;
    } else {
        r.blk = __ldg(a.page_table + (size_t)s.b * a.max_pages + e);
        page = e;
        r.mask = 0xff;
        if (r.blk < 0 || r.blk >= a.num_blocks) {
            atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
            r.blk = -1;
        }
    }
    r.nval = max(0, min(16, s.seq - page * a.P - 16 * r.t16));
    if (r.nval == 0) r.blk = -1;
    return r;
}

// -------------------------------------------------------------- softmax

template <int D>
struct __align__(16) SoftmaxShared {
    float o[AT_WARPS][8][D];
    float m[AT_WARPS][8], l[AT_WARPS][8];
};

template <int D>
__global__ void __launch_bounds__(AT_THREADS) kv4_softmax_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    constexpr int NG = Kv4<D>::NG, WPL = Kv4<D>::WPL, MT = D / 16;
    __shared__ SoftmaxShared<D> sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    const int group = blockIdx.x / a.S, split = blockIdx.x % a.S;
    const int G = a.Hq / a.Hkv;
    const Span sp = warp_span(a, group, split * AT_WARPS + warp);
    Queries<D> Q;
    Q.load(a.q + ((size_t)sp.b * a.Hq + sp.kvh * G) * D, G);
    const float scale = 1.4426950408889634f * rsqrtf((float)D);  // z in powers of two

    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][v] = 0.f;
    float off[NG] = {};                     // head r: sum p (lo - 16 s), this lane's tokens
    float m[2] = {-INFINITY, -INFINITY};    // heads 2c, 2c + 1
    float l[2] = {0.f, 0.f};
    for (int t = sp.first; t < sp.last; ++t) {
        const TileAt ta = tile_at(a, sp, t);
        if (ta.blk < 0) continue;
        const size_t at = kv4_tile<D>(ta.blk, a.Hkv, sp.kvh, a.P, ta.t16);
        float z[4];
        tile_scores<D>(a.k4 + at, Q, scale, z);
        const int mask = ta.mask & ((1 << G) - 1);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (r + 8 * (v >> 1) >= ta.nval || !((mask >> (2 * c + (v & 1))) & 1)) z[v] = -INFINITY;
        float corr[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float tm = fmaxf(z[e], z[2 + e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) tm = fmaxf(tm, __shfl_xor_sync(FULL, tm, o));
            const float mn = fmaxf(m[e], tm);
            const float base = mn == -INFINITY ? 0.f : mn;
            corr[e] = exp2f(m[e] - base);
            m[e] = mn;
            z[e] = exp2f(z[e] - base);
            z[2 + e] = exp2f(z[2 + e] - base);
            l[e] = fmaf(l[e], corr[e], z[e] + z[2 + e]);
        }
        if (__any_sync(FULL, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][v] *= corr[v & 1];
            const float c0 = __shfl_sync(FULL, corr[0], r >> 1), c1 = __shfl_sync(FULL, corr[1], r >> 1);
#pragma unroll
            for (int g = 0; g < NG; ++g) off[g] *= (r & 1) ? c1 : c0;
        }
        // weights of head r, tokens 2c, 2c + 1, 2c + 8, 2c + 9
        float p[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int src = 4 * (2 * c + u) + (r >> 1);
            const float x0 = __shfl_sync(FULL, z[0], src), x1 = __shfl_sync(FULL, z[1], src);
            const float y0 = __shfl_sync(FULL, z[2], src), y1 = __shfl_sync(FULL, z[3], src);
            p[u] = (r & 1) ? x1 : x0;
            p[2 + u] = (r & 1) ? y1 : y0;
        }
        const unsigned char *vt = a.v4 + at;
        unsigned w0[WPL], w1[WPL];
        const int piece = (r ^ kv4_vswz<D>(c)) * (4 * WPL);  // pairs c and c + 4 have the same swizzle
        load_words<WPL>(vt + c * D + piece, w0);
        load_words<WPL>(vt + (c + 4) * D + piece, w1);
        const unsigned *vp = reinterpret_cast<const unsigned *>(vt + Kv4<D>::CODES);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int tok = 2 * c + (u & 1) + 8 * (u >> 1);
                // rows behind the sequence, and rows of pages that head r did not
                // select, count as zero whatever they hold
                const unsigned pr = tok < ta.nval && ((mask >> r) & 1) ? __ldg(vp + tok * NG + g) : 0u;
                const float s = bf16lo(pr);
                off[g] = fmaf(p[u], fmaf(-16.f, s, bf16hi(pr)), off[g]);
                x[u] = p[u] * s;
            }
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                const unsigned b0 = (unsigned)f2bf(x[0]) | ((unsigned)f2bf(x[1]) << 16);
                const unsigned b1 = (unsigned)f2bf(x[2]) | ((unsigned)f2bf(x[3]) << 16);
                x[0] -= bf16lo(b0);
                x[1] -= bf16hi(b0);
                x[2] -= bf16lo(b1);
                x[3] -= bf16hi(b1);
#pragma unroll
                for (int i = 2 * g; i < 2 * g + 2; ++i) {
                    mma_bf16_16816(acc[2 * i], codes_bf16<0>(w0[i]), codes_bf16<1>(w0[i]), codes_bf16<0>(w1[i]),
                                   codes_bf16<1>(w1[i]), b0, b1);
                    mma_bf16_16816(acc[2 * i + 1], codes_bf16<2>(w0[i]), codes_bf16<3>(w0[i]), codes_bf16<2>(w1[i]),
                                   codes_bf16<3>(w1[i]), b0, b1);
                }
            }
        }
    }
    // the warp's state: sums over the lanes that share a head
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[e] += __shfl_xor_sync(FULL, l[e], o);
    if (lane < 4)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sh.m[warp][2 * c + e] = m[e];
            sh.l[warp][2 * c + e] = l[e];
        }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        off[g] += __shfl_xor_sync(FULL, off[g], 1);
        off[g] += __shfl_xor_sync(FULL, off[g], 2);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        // tile mt holds coordinates j (row r) and j + 1 (row r + 8)
        const int j = 64 * (mt >> 2) + 8 * r + 4 * ((mt >> 1) & 1) + 2 * (mt & 1);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float o = __shfl_sync(FULL, off[mt >> 2], 4 * (2 * c + (v & 1)));
            sh.o[warp][2 * c + (v & 1)][j + (v >> 1)] = acc[mt][v] + o;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += AT_THREADS) {
        const int g = i / D, j = i % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < AT_WARPS; ++w) M = fmaxf(M, sh.m[w][g]);
        float num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < AT_WARPS; ++w) {
            if (sh.l[w][g] == 0.f) continue;  // no token (NaN scores make it NaN)
            const float f = exp2f(sh.m[w][g] - M);
            num = fmaf(f, sh.o[w][g][j], num);
            den = fmaf(f, sh.l[w][g], den);
        }
        float *o = a.part + ((size_t)split * a.B * a.Hq + sp.b * a.Hq + sp.kvh * G + g) * (D + 2);
        o[2 + j] = num;
        if (j == 0) {
            o[0] = M;
            o[1] = den;
        }
    }
}

// The splits of a head, merged in order.
template <int D>
__global__ void __launch_bounds__(D) kv4_combine_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    const int G = a.Hq / a.Hkv, j = threadIdx.x;
    int b, h;
    head_of(blockIdx.x, a.kv0 * G, a.nk * G, b, h);
    const int bh = b * a.Hq + h;
    const uint16_t qb = a.q[(size_t)bh * D + j];
    const bool fine = __syncthreads_and((qb & 0x7f80u) != 0x7f80u);
    const size_t step = (size_t)a.B * a.Hq * (D + 2);
    const float *p = a.part + (size_t)bh * (D + 2);
    float M = -INFINITY;
    for (int s = 0; s < a.S; ++s) M = fmaxf(M, __ldcg(p + s * step));
    float num = 0.f, den = 0.f;
    for (int s = 0; s < a.S; ++s) {
        const float l = __ldcg(p + s * step + 1);
        if (l == 0.f) continue;
        const float f = exp2f(__ldcg(p + s * step) - M);
        den = fmaf(f, l, den);
        num = fmaf(f, __ldcg(p + s * step + 2 + j), num);
    }
    const float nan = __int_as_float(0x7fc00000);
    if (!fine && j == 0) atomicOr(a.status, ENTMAXKV_STATUS_NONFINITE);
    // den is 0 only without tokens (the largest weight of a split is 1); NaN
    // scores make it NaN
    const bool none = den == 0.f;
    a.out[(size_t)bh * D + j] = !fine ? nan : none ? 0.f : num / den;
    if (j == 0 && a.tau_out) a.tau_out[bh] = !fine || none ? nan : 0.6931471805599453f * (M + log2f(den));
}

// --------------------------------------------------------------- entmax

template <int D>
__global__ void __launch_bounds__(AT_THREADS) kv4_scan_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    const int group = blockIdx.x / a.S, seg = (blockIdx.x % a.S) * AT_WARPS + warp;
    const int G = a.Hq / a.Hkv;
    const Span sp = warp_span(a, group, seg);
    Queries<D> Q;
    const int h0 = sp.b * a.Hq + sp.kvh * G;
    Q.load(a.q + (size_t)h0 * D, G);
    const float scale = (a.alpha - 1.f) * rsqrtf((float)D);
    const size_t row_len = (size_t)a.max_pages * a.P;

    float m[2] = {-INFINITY, -INFINITY};  // heads 2c, 2c + 1: the warp's max so far
    int n[8] = {};                        // candidates of each head
    bool bad[2] = {false, false};         // the lane saw a NaN score
    for (int t = sp.first; t < sp.last; ++t) {
        const TileAt ta = tile_at(a, sp, t);
        if (ta.blk < 0) continue;
        float z[4];
        tile_scores<D>(a.k4 + kv4_tile<D>(ta.blk, a.Hkv, sp.kvh, a.P, ta.t16), Q, scale, z);
        const int mask = ta.mask & ((1 << G) - 1);
        bool any = false;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (r + 8 * (v >> 1) >= ta.nval || !((mask >> (2 * c + (v & 1))) & 1)) z[v] = -INFINITY;
            any |= !(z[v] <= m[v & 1] - 1.f);  // NaN stays a candidate
        }
        if (!__any_sync(FULL, any)) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            bad[e] |= z[e] != z[e] || z[2 + e] != z[2 + e];
            float tm = fmaxf(z[e], z[2 + e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) tm = fmaxf(tm, __shfl_xor_sync(FULL, tm, o));
            m[e] = fmaxf(m[e], tm);
        }
        const unsigned row = (unsigned)ta.blk * a.P + 16 * ta.t16 + r;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            if (h >= G) break;
            const int e = h & 1;
            const bool mine = c == (h >> 1);
            const unsigned lo = __ballot_sync(FULL, mine && !(z[e] <= m[e] - 1.f));
            const unsigned hi = __ballot_sync(FULL, mine && !(z[2 + e] <= m[e] - 1.f));
            if (lo | hi) {
                const size_t at = (h0 + h) * row_len + (size_t)sp.first * 16 + n[h];
                const unsigned below = (1u << lane) - 1u;
                if ((lo >> lane) & 1u) {
                    const size_t k = at + __popc(lo & below);
                    a.cand_z[k] = z[e];
                    a.cand_row[k] = row;
                }
                if ((hi >> lane) & 1u) {
                    const size_t k = at + __popc(lo) + __popc(hi & below);
                    a.cand_z[k] = z[2 + e];
                    a.cand_row[k] = row + 8;
                }
                n[h] += __popc(lo) + __popc(hi);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        float mh = __shfl_sync(FULL, m[h & 1], h >> 1);
        // a NaN stays a candidate: its segment may not be passed over for a low max
        if (__any_sync(FULL, c == (h >> 1) && bad[h & 1])) mh = __int_as_float(0x7fc00000);
        if (h < G && lane == 0) {
            a.seg_n[(size_t)(h0 + h) * a.seg_len + seg] = n[h];
            a.seg_max[(size_t)(h0 + h) * a.seg_len + seg] = mh;
        }
    }
}

constexpr int TK_NT = 256;
constexpr int TK_NW = TK_NT / 32;
constexpr int TK_CAP = 4096;  // candidates held on chip

// One CTA a head: the candidates above the head's max - 1 in list order, their
// threshold, and the sum of p v over the support.
template <int D>
__global__ void __launch_bounds__(TK_NT) kv4_tau_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    constexpr int NG = Kv4<D>::NG;
    extern __shared__ int seg_at[];  // [W + 1] place of each segment's candidates
    __shared__ float cz[TK_CAP];
    __shared__ unsigned crow[TK_CAP];
    __shared__ float o_sh[TK_NW][D];
    __shared__ float red[2][TK_NW][2];
    __shared__ float s_max[TK_NW];
    __shared__ int scan[72];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.Hq / a.Hkv;
    int b, h;
    head_of(blockIdx.x, a.kv0 * G, a.nk * G, b, h);
    const int bh = b * a.Hq + h, kvh = h / G;
    const int W = a.S * AT_WARPS;
    const float nan = __int_as_float(0x7fc00000);
    const uint16_t qb = threadIdx.x < D ? a.q[(size_t)bh * D + threadIdx.x] : (uint16_t)0;
    const bool fine = __syncthreads_and((qb & 0x7f80u) != 0x7f80u);
    if (!fine && threadIdx.x == 0) atomicOr(a.status, ENTMAXKV_STATUS_NONFINITE);

    const int *sn = a.seg_n + (size_t)bh * a.seg_len;
    const float *sm = a.seg_max + (size_t)bh * a.seg_len;
    float zmax = -INFINITY;
    int listed = 0;
    for (int i = threadIdx.x; i < W; i += TK_NT) {
        zmax = fmaxf(zmax, __ldcg(sm + i));
        listed |= __ldcg(sn + i);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) zmax = fmaxf(zmax, __shfl_xor_sync(FULL, zmax, o));
    if (lane == 0) s_max[warp] = zmax;
    const bool some = __syncthreads_or(listed);
    zmax = s_max[0];
#pragma unroll
    for (int w = 1; w < TK_NW; ++w) zmax = fmaxf(zmax, s_max[w]);
    if (!fine || !some || !(fabsf(zmax) < INFINITY)) {
        // no token, a query that is not finite, nothing but NaN scores, or an overflow
        for (int j = threadIdx.x; j < D; j += TK_NT) a.out[(size_t)bh * D + j] = fine && !some ? 0.f : nan;
        if (threadIdx.x == 0 && a.tau_out) a.tau_out[bh] = nan;
        return;
    }

    const float thr = zmax - 1.f;
    const int seq = seq_len_of(a.seq_lens, b, a.P, a.max_pages, nullptr);
    const long long T = (long long)(a.union_e ? a.union_cnt[b * a.Hkv + kvh] : n_pages_of(seq, a.P)) * (a.P / 16);
    const float *zl = a.cand_z + (size_t)bh * a.max_pages * a.P;
    const unsigned *rl = a.cand_row + (size_t)bh * a.max_pages * a.P;
    auto seg_base = [&](int w) { return (size_t)(T * w / W) * 16; };

    // how many of each segment stay, and where they go
    for (int w = warp; w < W; w += TK_NW) {
        const int n = __ldcg(sn + w);
        const float *src = zl + seg_base(w);
        int k = 0;
        if (!(__ldcg(sm + w) <= thr))
            for (int i = lane; i < n; i += 32) k += !(__ldcg(src + i) <= thr);
#pragma unroll
        for (int o = 16; o; o >>= 1) k += __shfl_xor_sync(FULL, k, o);
        if (lane == 0) seg_at[w] = k;
    }
    __syncthreads();
    int nc = 0;
    for (int w0 = 0; w0 < W; w0 += TK_NT) {
        const int w = w0 + threadIdx.x;
        const int k = w < W ? seg_at[w] : 0;
        int tot;
        const int at = block_excl_scan(k, scan, &tot);
        if (w < W) seg_at[w] = nc + at;
        nc += tot;
    }
    if (threadIdx.x == 0) seg_at[W] = nc;
    __syncthreads();
    const bool onchip = nc <= TK_CAP;
    bool bad = false;
    // every kept candidate: f(place, z, row)
    auto each = [&](auto f) {
        for (int w = warp; w < W; w += TK_NW) {
            int at = seg_at[w];
            if (at == seg_at[w + 1]) continue;
            const int n = __ldcg(sn + w);
            const size_t src = seg_base(w);
            for (int i0 = 0; i0 < n; i0 += 32) {
                const float z = i0 + lane < n ? __ldcg(zl + src + i0 + lane) : -INFINITY;
                const bool keep = !(z <= thr);
                const unsigned bal = __ballot_sync(FULL, keep);
                if (keep) f(at + __popc(bal & ((1u << lane) - 1u)), z, src + i0 + lane);
                at += __popc(bal);
            }
        }
    };
    each([&](int at, float z, size_t i) {
        bad |= z != z;
        if (onchip) {
            cz[at] = z;
            crow[at] = __ldcg(rl + i);
        }
    });
    if (__syncthreads_or(bad)) {
        for (int j = threadIdx.x; j < D; j += TK_NT) a.out[(size_t)bh * D + j] = nan;
        if (threadIdx.x == 0 && a.tau_out) a.tau_out[bh] = nan;
        return;
    }
    const float r = 1.f / (a.alpha - 1.f);
    const int ri = a.r_int;
    const float hi = zmax - powf((float)nc, 1.f - a.alpha);
    float tau = thr;
    if (nc > 1 && hi > thr) {
        if (onchip)
            tau = entmax_tau<TK_NT>([&](auto add, int f, int st) { for (int i = f; i < nc; i += st) add(cz[i]); }, nc,
                                    thr, hi, zmax, r, ri, red);
        else  // every thread adds the candidates of its place, pass by pass
            tau = entmax_tau<TK_NT>([&](auto add, int, int) { each([&](int, float z, size_t) { add(z); }); }, nc, thr, hi,
                                    zmax, r, ri, red);
    }
    if (threadIdx.x == 0 && a.tau_out) a.tau_out[bh] = tau;

    // p v over the support.  A value word holds 4 coordinates of both tokens
    // of a pair: one word a lane is a row (d = 128), half a warp a row (64).
    constexpr int LPR = D / 4;        // lanes of a row
    constexpr int RPW = 32 / LPR;     // rows of a warp at a time
    const int ll = lane % LPR, sub = lane / LPR;
    const int piece = ll / Kv4<D>::WPL, wi = ll % Kv4<D>::WPL;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const size_t rec = (size_t)(a.P / 16) * Kv4<D>::TILE;
    auto add_row = [&](float z, unsigned row) {
        const float p = pos_pow(z - tau, r, ri);
        if (!(p > 0.f)) return;
        const unsigned blk = row / (unsigned)a.P;
        const int slot = (int)(row - blk * a.P), t = slot & 15, pair = t >> 1;
        const unsigned char *tile = a.v4 + ((size_t)blk * a.Hkv + kvh) * rec + (size_t)(slot >> 4) * Kv4<D>::TILE;
        // the lane's coordinate block keeps its place: read the word that holds it
        const unsigned w =
            rotr3(__ldg(reinterpret_cast<const unsigned *>(tile) + pair * (D / 4) +
                        (piece ^ kv4_vswz<D>(pair)) * Kv4<D>::WPL + wi)) >>
            (16 * (t & 1));
        const unsigned pr = __ldg(reinterpret_cast<const unsigned *>(tile + Kv4<D>::CODES) + t * NG + (wi >> 1));
        const float s = p * bf16lo(pr), lo = p * bf16hi(pr);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += fmaf(s, (float)((w >> (4 * i)) & 15u), lo);
    };
    if (onchip) {
        for (int i = warp * RPW + sub; i < nc; i += TK_NW * RPW) add_row(cz[i], crow[i]);
    } else {
        for (int w = warp; w < W; w += TK_NW) {
            if (seg_at[w] == seg_at[w + 1]) continue;
            const int n = __ldcg(sn + w);
            const size_t src = seg_base(w);
            for (int i = sub; i < n; i += RPW) {
                const float z = __ldcg(zl + src + i);
                if (z > tau) add_row(z, __ldcg(rl + src + i));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (RPW == 2) acc[i] += __shfl_xor_sync(FULL, acc[i], 16);
    if (sub == 0) {
        const int j = 64 * (wi >> 1) + 8 * piece + 4 * (wi & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) o_sh[warp][j + i] = acc[i];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += TK_NT) {
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < TK_NW; ++w) o += o_sh[w][j];
        a.out[(size_t)bh * D + j] = o;
    }
}

// --------------------------------------------------------------- launch

// Splits a group's page list is cut into.
int splits(const entmaxkv_shape *s, int nk) {
    const long long tiles = (long long)s->max_pages * (s->page_size / 16);
    const long long groups = (long long)s->B * nk;
    long long S = AT_SPLIT_CTAS / groups;
    const long long most = (tiles + AT_WARPS * AT_MIN_TILES - 1) / (AT_WARPS * AT_MIN_TILES);
    if (S > most) S = most;
    return S < 1 ? 1 : (int)S;
}

struct Carve {
    size_t part, cand_z, cand_row, seg_n, seg_max, union_e, union_blk, union_cnt, zmax, counters, total;
};

// The regions hold full-size rows of every head, and as many splits as a call
// on one kv head alone may use, so calls on disjoint kv-head ranges can share
// the workspace.
Carve carve(const entmaxkv_shape *s) {
    Carve c;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off += (bytes + 255) & ~(size_t)255;
        return o;
    };
    const size_t heads = (size_t)s->B * s->Hq, groups = (size_t)s->B * s->Hkv;
    const size_t tokens = heads * s->max_pages * s->page_size;
    const size_t S = splits(s, 1);
    c.part = take(S * heads * (s->d + 2) * 4);
    c.cand_z = take(tokens * 4);
    c.cand_row = take(tokens * 4);
    c.seg_n = take(heads * S * AT_WARPS * 4);
    c.seg_max = take(heads * S * AT_WARPS * 4);
    c.union_e = take(groups * s->max_pages * 4);
    c.union_blk = take(groups * s->max_pages * 4);
    c.union_cnt = take(groups * 4);
    c.zmax = take(heads * 4);
    c.counters = take(groups * 4);
    c.total = off;
    return c;
}

template <int D>
cudaError_t decode_t(const Kv4DecodeArgs &a, cudaStream_t st) {
    const int groups = a.B * a.nk, heads = groups * (a.Hq / a.Hkv);
    cudaError_t e;
    if (a.alpha == 1.f) {
        e = launch_pdl(kv4_softmax_kernel<D>, dim3(groups * a.S), dim3(AT_THREADS), 0, st, a);
        if (e != cudaSuccess) return e;
        return launch_pdl(kv4_combine_kernel<D>, dim3(heads), dim3(D), 0, st, a);
    }
    e = launch_pdl(kv4_scan_kernel<D>, dim3(groups * a.S), dim3(AT_THREADS), 0, st, a);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)(a.S * AT_WARPS + 1) * 4;
    auto k = kv4_tau_kernel<D>;
    if ((e = ensure_smem(reinterpret_cast<const void *>(k), smem)) != cudaSuccess) return e;
    return launch_pdl(k, dim3(heads), dim3(TK_NT), smem, st, a);
}

}  // namespace

}  // namespace ekv

using namespace ekv;

extern "C" {

size_t entmaxkv_kv4_workspace_size(const entmaxkv_shape *s) {
    if (check_shape(s)) return (size_t)-1;
    return carve(s).total;
}

int entmaxkv_kv4_decode(const entmaxkv_shape *s, const void *q, const void *k4, const void *v4,
                        const int32_t *page_table, const int32_t *seq_lens, const int32_t *sel, const int32_t *cnt,
                        float alpha, float *out, float *tau_out, void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    if (!q || !k4 || !v4 || !page_table || !seq_lens || !out || (sel == nullptr) != (cnt == nullptr))
        return ENTMAXKV_ERR_NULL;
    if (!aligned16(q) || !aligned16(k4) || !aligned16(v4)) return ENTMAXKV_ERR_ALIGN;
    if (!std::isfinite(alpha) || !(alpha >= 1.f)) return ENTMAXKV_ERR_ALPHA;
    if (sel && s->max_pages > MAX_SEL_PAGES) return ENTMAXKV_ERR_SHAPE;
    const Carve c = carve(s);
    if (!workspace || ws_bytes < c.total) return ENTMAXKV_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return ENTMAXKV_ERR_ALIGN;
    DevInfo di;
    if ((rc = device_info(&di))) return rc;
    char *w = static_cast<char *>(workspace);
    Kv4DecodeArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.k4 = static_cast<const uint8_t *>(k4);
    a.v4 = static_cast<const uint8_t *>(v4);
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.out = out;
    a.tau_out = tau_out;
    a.part = reinterpret_cast<float *>(w + c.part);
    a.cand_z = reinterpret_cast<float *>(w + c.cand_z);
    a.cand_row = reinterpret_cast<unsigned *>(w + c.cand_row);
    a.seg_n = reinterpret_cast<int *>(w + c.seg_n);
    a.seg_max = reinterpret_cast<float *>(w + c.seg_max);
    a.B = s->B;
    a.Hq = s->Hq;
    a.Hkv = s->Hkv;
    a.P = s->page_size;
    a.max_pages = s->max_pages;
    a.num_blocks = s->num_blocks;
    kv_range(s, &a.kv0, &a.nk);
    a.S = splits(s, a.nk);
    a.seg_len = splits(s, 1) * AT_WARPS;
    a.alpha = alpha;
    a.r_int = alpha > 1.f ? integer_r(alpha) : 0;
    a.status = di.status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (sel) {
        DecodeArgs u;
        std::memset(&u, 0, sizeof(u));
        u.page_table = page_table;
        u.seq_lens = seq_lens;
        u.sel = sel;
        u.cnt = cnt;
        u.B = s->B;
        u.Hq = s->Hq;
        u.Hkv = s->Hkv;
        u.P = s->page_size;
        u.max_pages = s->max_pages;
        u.num_blocks = s->num_blocks;
        u.kv0 = a.kv0;
        u.nk = a.nk;
        u.sel_stride = s->max_pages;
        u.status = di.status;
        u.ws.union_e = reinterpret_cast<int *>(w + c.union_e);
        u.ws.union_blk = reinterpret_cast<int *>(w + c.union_blk);
        u.ws.union_cnt = reinterpret_cast<int *>(w + c.union_cnt);
        u.ws.zmax = reinterpret_cast<int *>(w + c.zmax);
        u.ws.counters = reinterpret_cast<int *>(w + c.counters);
        if (launch_union_list(u, st) != cudaSuccess) return ENTMAXKV_ERR_CUDA;
        a.union_e = u.ws.union_e;
        a.union_blk = u.ws.union_blk;
        a.union_cnt = u.ws.union_cnt;
    }
    const cudaError_t e = s->d == 64 ? decode_t<64>(a, st) : decode_t<128>(a, st);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_ERR_CUDA;
}

}  // extern "C"
