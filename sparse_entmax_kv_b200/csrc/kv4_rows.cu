// kv4_rows.cu -- rows into and out of the 4-bit cache, and the C entry points
// of both (include/entmaxkv_kv4.h).
//
// write: one CTA per (touched page, kv head).  A lane takes 16 neighbouring
// coordinates of a key row and of the value row of the same token, so that a
// 64-coordinate group is four lanes: min and max are packed bf16 operations in
// a lane and two shuffles, and a code costs five instructions (the rounding to
// an integer is an addition of 1.5 2^23, whose low bits are then shifted into
// place by an integer multiply-add).  A value word holds both tokens of a
// pair: the two lanes trade halves, and where only one token is new the other
// half of the word is kept (the lane is the word's only writer).  With
// metadata the page's key tiles are also kept in shared memory, old tokens
// copied in, and 1024 / d threads share the statistics of a coordinate.
// read: the same split, the other way round.
//
// 38.5k rows of 8 heads, d = 128, pages of 64 (12 prompts of 2k to 4k tokens):
// write 51 us without metadata and 79 with it (210 MB: 32 at a copy's rate),
// read 43.  Bound by instructions: the integer pipe is half busy, issue 70 %;
// the statistics are 28 us of the write, 8 of them conversions to fp64.  One
// appended token a sequence (32 x 8 heads) takes 9.5 us cold: three dependent
// loads, the page's old tiles, 64 tokens of statistics.
#include <cmath>

#include "../../include/entmaxkv_kv4.h"
#include "kv4.cuh"

namespace ekv {

namespace {

constexpr int RW_THREADS = 256;
constexpr int RW_WARPS = RW_THREADS / 32;
constexpr float ROUND = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, ties to even

// What one CTA works on: tokens [t0, t1) of logical page `page` of sequence
// b are new, [0, n) hold valid tokens, row0 is the row of token t0.
struct PageJob {
    int b, page, blk, t0, t1, n;
    long long row0;
};

// Page slot -> job.  Sequence b owns the slots from row_start[b] / P + 2 b:
// n_b rows touch at most n_b / P + 2 pages.  False: nothing to do.
template <int P>
__device__ __forceinline__ bool page_job(const Kv4RowArgs &a, int slot, PageJob &j) {
    const bool report = blockIdx.y == 0 && threadIdx.x == 0;
    int b = slot, first = slot, count = 1, idx = 0;
    if (a.row_start) {
        if (slot == 0 && blockIdx.y == 0)  // rows that run backwards may own no slot: the first CTA looks at them all
            for (int i = threadIdx.x; i < a.m.B; i += blockDim.x)
                if (a.row_start[i + 1] < a.row_start[i]) atomicOr(a.m.status, ENTMAXKV_STATUS_BAD_LENGTH);
        // the last sequence whose slots begin at or before this one, 32 tries at a time
        int lo = 0;
        for (int n = a.m.B; n > 1;) {
            const int step = (n + 31) / 32, at = (int)(threadIdx.x & 31) * step;
            const unsigned before = __ballot_sync(FULL, at < n && a.row_start[lo + at] / P + 2 * (lo + at) <= slot);
            const int k = max(0, __popc(before) - 1) * step;
            lo += k;
            n = min(step, n - k);
        }
        b = lo;
        first = a.row_start[b];
        const int end = a.row_start[b + 1];
        if (first < 0 || end < first || end > a.n_rows) {
            if (report) atomicOr(a.m.status, ENTMAXKV_STATUS_BAD_LENGTH);
            return false;
        }
        count = end - first;
        idx = slot - (first / P + 2 * b);
    }
    const int L = a.seq_lens[b];
    if (count == 0 || L <= 0 || idx < 0) {
        if (report && L <= 0 && count > 0 && a.row_start) atomicOr(a.m.status, ENTMAXKV_STATUS_BAD_LENGTH);
        return false;
    }
    if (L > a.m.max_pages * P || count > L) {
        if (report) atomicOr(a.m.status, ENTMAXKV_STATUS_BAD_LENGTH);
        return false;
    }
    const int start = L - count;
    j.b = b;
    j.page = start / P + idx;
    if ((long long)j.page * P >= L) return false;
    j.t0 = idx == 0 ? start - j.page * P : 0;
    j.n = min(P, L - j.page * P);
    j.t1 = j.n;
    j.row0 = (long long)first + (j.page * P + j.t0 - start);
    j.blk = a.page_table[(size_t)b * a.m.max_pages + j.page];
    if (j.blk < 0 || j.blk >= a.m.num_blocks) {
        if (report) atomicOr(a.m.status, ENTMAXKV_STATUS_BAD_PAGE);
        return false;
    }
    return true;
}

// Lanes of a row, and the rows that a warp takes at a time.
template <int D>
constexpr int LPR = D / 16;
template <int D>
constexpr int RPW = 32 / LPR<D>;

__device__ __forceinline__ unsigned min2(unsigned x, unsigned y) {
    unsigned r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ unsigned max2(unsigned x, unsigned y) {
    unsigned r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

struct Row16 {
    unsigned x[8];  // 16 bf16, then their codes' bits
    __device__ __forceinline__ void load(const uint16_t *row) {
        const uint4 a = reinterpret_cast<const uint4 *>(row)[0], b = reinterpret_cast<const uint4 *>(row)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0u;
    }
};

// Codes of the 16 coordinates as c + constants in two words of eight (KEYS:
// coordinate n of a word at bits 16 (n & 1) + 4 (n >> 1); else in two words of
// two quads each, coordinate n of a quad at bits 4 n), and the parameter word
// of the group, which its four lanes return alike.
template <bool KEYS>
__device__ __forceinline__ unsigned quantise(const Row16 &row, unsigned (&w)[2]) {
    unsigned mn = row.x[0], mx = row.x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        mn = min2(mn, row.x[i]);
        mx = max2(mx, row.x[i]);
    }
    // the smallest in the low half, the largest in the high one
    unsigned m = __byte_perm(min2(mn, mn >> 16), max2(mx, mx << 16), 0x7610);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const unsigned y = __shfl_xor_sync(FULL, m, o);
        m = __byte_perm(min2(m, y), max2(m, y), 0x7610);
    }
    const float lo = bf16lo(m);
    const float range = __fsub_rn(bf16hi(m), lo);
    if (!(range < INFINITY)) {  // a NaN (it stays through min and max), an infinity, or an overflow
        w[0] = w[1] = 0u;
        return 0x7fc07fc0u;
    }
    float s = bf16f(f2bf(__fdiv_rn(range, 15.f)));
    if (s < 1.17549435e-38f) s = 0.f;  // 2^-126: below, 1 / s may overflow
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    // s is within 2^-9 of range / 15, so no quotient exceeds 15.04: no clamp
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = 0u;
        unsigned bias = 0u;  // what ROUND's bits add up to
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const unsigned xx = row.x[4 * i + k];
                const float x = h ? bf16hi(xx) : bf16lo(xx);
                const unsigned c = __float_as_uint(__fadd_rn(__fmul_rn(__fsub_rn(x, lo), inv), ROUND));
                const unsigned place = KEYS ? 1u << (16 * h + 4 * k) : 1u << (8 * k + 4 * h);
                w[i] += c * place;
                bias += 0x4b400000u * place;
            }
        w[i] -= bias;
    }
    return (__float_as_uint(s) >> 16) | (m << 16);
}

// bf16 neighbours of x on either side (x itself when it is a bf16 value).
__device__ __forceinline__ uint16_t bf16_down(float x) {
    const unsigned u = __float_as_uint(x);
    if (x != x) return 0x7fc0;
    return (uint16_t)((x < 0.f ? u + 0xffffu : u) >> 16);
}
__device__ __forceinline__ uint16_t bf16_up(float x) {
    const unsigned u = __float_as_uint(x);
    if (x != x) return 0x7fc0;
    return (uint16_t)((x > 0.f ? u + 0xffffu : u) >> 16);
}

__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// The code at bits K .. K + 3 (K <= 16) of w, times 2^K, as a float: 2^23 + c
// 2^K, less 2^23.  big: the bits of 2^23, from a kernel argument, so that mask
// and or are one instruction (see code_f16 of the attention kernels).
template <int K>
__device__ __forceinline__ float code_f32(unsigned w, unsigned big) {
    unsigned x;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w), "n"(15 << K), "r"(big));
    return __uint_as_float(x) - 8388608.f;
}
// The parameters of a row's group: s, s / 16, s / 256 and s / 4096 (exact) and
// lo.  s / 2^K times a code times 2^K is the definition's product.
struct Scales {
    float s[4], lo;
    __device__ __forceinline__ explicit Scales(unsigned pr) {
        s[0] = bf16lo(pr);
        lo = bf16hi(pr);
#pragma unroll
        for (int i = 1; i < 4; ++i) s[i] = s[i - 1] * 0.0625f;
    }
    // Value of the code at bits 4 I of w.
    template <int I>
    __device__ __forceinline__ float at(unsigned w, unsigned big) const {
        return __fmaf_rn(s[I], code_f32<4 * I>(w, big), lo);
    }
};

// The metadata record of a page from its key tiles in shared memory.  A thread
// takes four coordinates (half a word, one pair of parameters a token), so
// 1024 / d threads share them, each every (1024 / d)-th token; their sums are
// added in order.
template <int D>
struct Stats {
    static constexpr int PARTS = 4 * RW_THREADS / D;
    double s1[PARTS][D], s2[PARTS][D];
    float mn[PARTS][D], mx[PARTS][D];
};
template <int D>
__device__ __forceinline__ void build_record(const MetaArgs &m, const unsigned char *image, Stats<D> &sh, int b,
                                             int kvh, int page, int n, unsigned big) {
    constexpr int PARTS = Stats<D>::PARTS;
    {
        const int q = threadIdx.x % (D / 4), part = threadIdx.x / (D / 4);
        const unsigned *words = reinterpret_cast<const unsigned *>(image);
        const int at = kv4_kword<D>(0, q >> 1), pat = Kv4<D>::CODES / 4 + (q >> 4), shift = 8 * (q & 1);
        float mn[4], mx[4];
        double s1[4], s2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mn[i] = INFINITY;
            mx[i] = -INFINITY;
            s1[i] = s2[i] = 0.0;
        }
#pragma unroll 2
        for (int t = part; t < n; t += PARTS) {
            const unsigned *tile = words + (t >> 4) * (Kv4<D>::TILE / 4);
            const unsigned w = tile[at + (t & 15) * (D / 8)] >> shift, pr = tile[pat + (t & 15) * Kv4<D>::NG];
            const float s0 = bf16lo(pr), s1x = s0 * 0.0625f, lo = bf16hi(pr);
            const float v[4] = {__fmaf_rn(s0, code_f32<0>(w, big), lo), __fmaf_rn(s0, code_f32<0>(w >> 16, big), lo),
                                __fmaf_rn(s1x, code_f32<4>(w, big), lo), __fmaf_rn(s1x, code_f32<4>(w >> 16, big), lo)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = v[i];
                mn[i] = min_nan(mn[i], x);
                mx[i] = max_nan(mx[i], x);
                const double xd = (double)x;
                s1[i] = __dadd_rn(s1[i], xd);
                s2[i] = __fma_rn(xd, xd, s2[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sh.s1[part][4 * q + i] = s1[i];
            sh.s2[part][4 * q + i] = s2[i];
            sh.mn[part][4 * q + i] = mn[i];
            sh.mx[part][4 * q + i] = mx[i];
        }
    }
    __syncthreads();
    const int j = threadIdx.x;
    if (j >= D) return;
    double s1 = sh.s1[0][j], s2 = sh.s2[0][j];
    float mn = sh.mn[0][j], mx = sh.mx[0][j];
#pragma unroll
    for (int k = 1; k < PARTS; ++k) {
        s1 = __dadd_rn(s1, sh.s1[k][j]);
        s2 = __dadd_rn(s2, sh.s2[k][j]);
        mn = min_nan(mn, sh.mn[k][j]);
        mx = max_nan(mx, sh.mx[k][j]);
    }
    const double dn = (double)n;
    const double mean = __ddiv_rn(s1, dn);
    double v = __dsub_rn(__ddiv_rn(s2, dn), __dmul_rn(mean, mean));
    if (v < 0.0) v = 0.0;
    const int sl = page % META_TILE;
    const long long T = ((long long)b * m.Hkv + kvh) * m.n_tiles + page / META_TILE;
    const int ch = j / 16, e = j % 16;
    uint8_t *bb = m.meta + T * 128 * D + ch * 2048;
    const int ob = sl * 32 + 16 * ((e >> 3) ^ ((sl >> 2) & 1)) + 2 * (e & 7);
    *reinterpret_cast<uint16_t *>(bb + ob) = bf16_down(mn);
    *reinterpret_cast<uint16_t *>(bb + 1024 + ob) = bf16_up(mx);
    uint8_t *mm = m.meta + m.n_tiles_total * 128 * D + T * 256 * D + ch * 4096;
    const int om = sl * 64 + 16 * ((e >> 2) ^ ((sl >> 1) & 3)) + 4 * (e & 3);
    *reinterpret_cast<float *>(mm + om) = (float)mean;
    *reinterpret_cast<float *>(mm + 2048 + om) = (float)v;
}

template <int D, int P>
__global__ void __launch_bounds__(RW_THREADS) kv4_write_kernel(const __grid_constant__ Kv4RowArgs a) {
    pdl_wait();
    constexpr int NG = Kv4<D>::NG, WPL = Kv4<D>::WPL, TILE = Kv4<D>::TILE, CODES = Kv4<D>::CODES;
    __shared__ __align__(16) unsigned char image[P / 16 * TILE];  // the page's key tiles (with metadata)
    __shared__ Stats<D> stats;
    PageJob j;
    if (!page_job<P>(a, blockIdx.x, j)) return;
    const int kvh = a.m.kv0 + blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *kt = a.k4 + kv4_tile<D>(j.blk, a.m.Hkv, kvh, P, 0);
    unsigned char *vt = a.v4 + kv4_tile<D>(j.blk, a.m.Hkv, kvh, P, 0);
    const bool meta = a.m.meta != nullptr;
    const int l = lane % LPR<D>, g = l >> 2, c = l & 3;  // the lane's coordinates are 16 l .. 16 l + 15
    const uint16_t *kr = a.k_new + (j.row0 - j.t0) * a.stride + (size_t)kvh * D + 16 * l;  // of slot 0
    const uint16_t *vr = a.v_new + (j.row0 - j.t0) * a.stride + (size_t)kvh * D + 16 * l;
    Row16 k, v;
    auto fetch = [&](int t) {
        if (t >= j.t0 && t < j.t1) {
            k.load(kr + t * a.stride);
            v.load(vr + t * a.stride);
        } else {
            k.clear();
            v.clear();
        }
    };
    const int first = j.t0 / RPW<D> + warp;
    fetch(first * RPW<D> + lane / LPR<D>);
    if (meta && j.t0 > 0) {  // the page's old tokens
        for (int i = threadIdx.x; i < (j.t0 + 15) / 16 * TILE / 16; i += RW_THREADS)
            cp_async16(image + 16 * i, kt + 16 * i);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
    }
    for (int q = first; q * RPW<D> < j.t1; q += RW_WARPS) {
        const int t = q * RPW<D> + lane / LPR<D>, u = t & 15, pair = u >> 1;
        const bool mine = t >= j.t0 && t < j.t1, other = (t ^ 1) >= j.t0 && (t ^ 1) < j.t1;
        unsigned kw[2], vw[2];
        const unsigned kp = quantise<true>(k, kw), vp = quantise<false>(v, vw);
        // halves of value words: the even token's lane makes those of coordinates 0 to 7
        const bool odd = t & 1;
        const unsigned keep = odd ? vw[1] : vw[0];
        const unsigned got = __shfl_xor_sync(FULL, odd ? vw[0] : vw[1], LPR<D>);
        const int tile = (t >> 4) * TILE;
        if (mine) {
            const uint2 w = make_uint2(kw[0], kw[1]);
            const int at = tile + 4 * (u * (D / 8) + c * WPL + 2 * g), pat = tile + CODES + 4 * (u * NG + g);
            *reinterpret_cast<uint2 *>(kt + at) = w;
            if (c == 0) {
                *reinterpret_cast<unsigned *>(kt + pat) = kp;
                *reinterpret_cast<unsigned *>(vt + pat) = vp;
            }
            if (meta) {
                *reinterpret_cast<uint2 *>(image + at) = w;
                if (c == 0) *reinterpret_cast<unsigned *>(image + pat) = kp;
            }
        }
        if (mine || other) {
            const unsigned lo = odd ? got : keep, hi = odd ? keep : got;  // of the even and of the odd token
            uint2 w = make_uint2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
            uint2 *to = reinterpret_cast<uint2 *>(
                vt + tile + 4 * (pair * (D / 4) + ((2 * c + odd) ^ kv4_vswz<D>(pair)) * WPL + 2 * g));
            if (!(mine && other)) {  // the other token of the pair keeps its half
                const uint2 old = *to;
                const unsigned mask = mine == odd ? 0xffff0000u : 0x0000ffffu;  // of the new one
                w.x = (w.x & mask) | (old.x & ~mask);
                w.y = (w.y & mask) | (old.y & ~mask);
            }
            *to = w;
        }
        fetch(t + RW_WARPS * RPW<D>);
    }
    if (!meta) return;
    __syncthreads();
    build_record<D>(a.m, image, stats, j.b, kvh, j.page, j.n, a.big);
}

// 16 values to fp32 or bf16.
__device__ __forceinline__ void store16(void *out, long long at, int f32, const float (&x)[16]) {
    if (f32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at);
        unsigned w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <int D, int P>
__global__ void __launch_bounds__(RW_THREADS) kv4_read_kernel(const __grid_constant__ Kv4RowArgs a) {
    pdl_wait();
    constexpr int NG = Kv4<D>::NG, WPL = Kv4<D>::WPL, TILE = Kv4<D>::TILE, CODES = Kv4<D>::CODES;
    PageJob j;
    if (!page_job<P>(a, blockIdx.x, j)) return;
    const int kvh = a.m.kv0 + blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % LPR<D>, g = l >> 2, c = l & 3;
    const size_t page = kv4_tile<D>(j.blk, a.m.Hkv, kvh, P, 0);
    for (int t = j.t0 + warp * RPW<D> + lane / LPR<D>; t < j.t1; t += RW_WARPS * RPW<D>) {
        const int u = t & 15, pair = u >> 1;
        const size_t tile = page + (size_t)(t >> 4) * TILE;
        const unsigned char *kt = a.k4 + tile, *vt = a.v4 + tile;
        const uint2 kw = *reinterpret_cast<const uint2 *>(kt + 4 * (u * (D / 8) + c * WPL + 2 * g));
        const unsigned kp = *reinterpret_cast<const unsigned *>(kt + CODES + 4 * (u * NG + g));
        const unsigned vp = *reinterpret_cast<const unsigned *>(vt + CODES + 4 * (u * NG + g));
        uint2 vw[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            vw[h] = *reinterpret_cast<const uint2 *>(
                vt + 4 * (pair * (D / 4) + ((2 * c + h) ^ kv4_vswz<D>(pair)) * WPL + 2 * g));
        const long long at = (j.row0 + t - j.t0) * a.stride + (long long)kvh * D + 16 * l;
        float x[16];
        const Scales ks(kp), vs(vp);
        auto half = [&](unsigned w, const Scales &sc, float *x, int step) {  // four codes of 16 bits
            x[0] = sc.template at<0>(w, a.big);
            x[step] = sc.template at<1>(w, a.big);
            x[2 * step] = sc.template at<2>(w, a.big);
            x[3 * step] = sc.template at<3>(w, a.big);
        };
        half(kw.x, ks, x, 2);
        half(kw.x >> 16, ks, x + 1, 2);
        half(kw.y, ks, x + 8, 2);
        half(kw.y >> 16, ks, x + 9, 2);
        store16(a.k_out, at, a.f32, x);
        const int sh = 16 * (t & 1);
        half(vw[0].x >> sh, vs, x, 1);
        half(vw[0].y >> sh, vs, x + 4, 1);
        half(vw[1].x >> sh, vs, x + 8, 1);
        half(vw[1].y >> sh, vs, x + 12, 1);
        store16(a.v_out, at, a.f32, x);
    }
}

template <int D, int P>
cudaError_t write_t(const Kv4RowArgs &a, dim3 grid, cudaStream_t st) {
    return launch_pdl(kv4_write_kernel<D, P>, grid, dim3(RW_THREADS), 0, st, a);
}
template <int D, int P>
cudaError_t read_t(const Kv4RowArgs &a, dim3 grid, cudaStream_t st) {
    return launch_pdl(kv4_read_kernel<D, P>, grid, dim3(RW_THREADS), 0, st, a);
}

// Page slots: one a sequence, or n_rows / P + 2 B (see page_job).
dim3 slots(const Kv4RowArgs &a) {
    return dim3(a.row_start ? a.n_rows / a.m.P + 2 * a.m.B : a.m.B, a.m.nk);
}

}  // namespace

#define KV4_DP(FN, a, ...)                                  \
    do {                                                    \
        if ((a).m.d == 64) switch ((a).m.P) {               \
                case 16: return FN<64, 16>(a, __VA_ARGS__);  \
                case 32: return FN<64, 32>(a, __VA_ARGS__);  \
                case 64: return FN<64, 64>(a, __VA_ARGS__);  \
            }                                               \
        else switch ((a).m.P) {                             \
                case 16: return FN<128, 16>(a, __VA_ARGS__); \
                case 32: return FN<128, 32>(a, __VA_ARGS__); \
                case 64: return FN<128, 64>(a, __VA_ARGS__); \
            }                                               \
        return cudaErrorInvalidValue;                       \
    } while (0)

cudaError_t launch_kv4_write(const Kv4RowArgs &a, cudaStream_t st) { KV4_DP(write_t, a, slots(a), st); }
cudaError_t launch_kv4_read(const Kv4RowArgs &a, cudaStream_t st) { KV4_DP(read_t, a, slots(a), st); }

namespace {

// Checks shared by write and read; fills everything but the row pointers.
int fill_rows(const entmaxkv_shape *s, const void *k_rows, const void *v_rows, int64_t row_stride,
              const int32_t *row_start, int32_t n_rows, const int32_t *page_table, const int32_t *seq_lens,
              const void *k4, const void *v4, void *meta, Kv4RowArgs *a) {
    int rc = check_shape(s);
    if (rc) return rc;
    if ((n_rows > 0 && (!k_rows || !v_rows)) || !page_table || !seq_lens || !k4 || !v4) return ENTMAXKV_ERR_NULL;
    if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(k4) || !aligned16(v4) || !aligned16(meta))
        return ENTMAXKV_ERR_ALIGN;
    if (row_stride < (int64_t)s->Hkv * s->d || row_stride % 8) return ENTMAXKV_ERR_SHAPE;
    if (n_rows < 0 || (!row_start && n_rows != s->B)) return ENTMAXKV_ERR_SHAPE;
    if (s->Hkv > 65535) return ENTMAXKV_ERR_SHAPE;
    DevInfo di;
    if ((rc = device_info(&di))) return rc;
    *a = Kv4RowArgs{};
    a->big = 0x4b000000u;
    a->stride = row_stride;
    a->row_start = row_start;
    a->n_rows = n_rows;
    a->page_table = page_table;
    a->seq_lens = seq_lens;
    a->k4 = static_cast<uint8_t *>(const_cast<void *>(k4));
    a->v4 = static_cast<uint8_t *>(const_cast<void *>(v4));
    a->m.meta = static_cast<uint8_t *>(meta);
    a->m.n_tiles = meta_tiles(s->max_pages);
    a->m.n_tiles_total = (long long)s->B * s->Hkv * a->m.n_tiles;
    a->m.B = s->B;
    a->m.Hkv = s->Hkv;
    a->m.d = s->d;
    a->m.P = s->page_size;
    a->m.max_pages = s->max_pages;
    a->m.num_blocks = s->num_blocks;
    kv_range(s, &a->m.kv0, &a->m.nk);
    a->m.status = di.status;
    return ENTMAXKV_OK;
}

}  // namespace

}  // namespace ekv

using namespace ekv;

extern "C" {

size_t entmaxkv_kv4_bytes(const entmaxkv_shape *s) {
    if (check_shape(s)) return 0;
    return (size_t)s->num_blocks * s->Hkv * s->page_size * s->d / 16 * 9;
}

int entmaxkv_kv4_write(const entmaxkv_shape *s, const void *k_new, const void *v_new, int64_t row_stride,
                       const int32_t *row_start, int32_t n_rows, const int32_t *page_table,
                       const int32_t *seq_lens, void *k4, void *v4, void *meta, void *stream) {
    Kv4RowArgs a;
    const int rc =
        fill_rows(s, k_new, v_new, row_stride, row_start, n_rows, page_table, seq_lens, k4, v4, meta, &a);
    if (rc || n_rows == 0) return rc;
    a.k_new = static_cast<const uint16_t *>(k_new);
    a.v_new = static_cast<const uint16_t *>(v_new);
    return launch_kv4_write(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_ERR_CUDA;
}

int entmaxkv_kv4_read(const entmaxkv_shape *s, const void *k4, const void *v4, int64_t row_stride,
                      const int32_t *row_start, int32_t n_rows, const int32_t *page_table, const int32_t *seq_lens,
                      int32_t rows, void *k_out, void *v_out, void *stream) {
    Kv4RowArgs a;
    if (rows != ENTMAXKV_ROWS_BF16 && rows != ENTMAXKV_ROWS_F32) return ENTMAXKV_ERR_POLICY;
    const int rc =
        fill_rows(s, k_out, v_out, row_stride, row_start, n_rows, page_table, seq_lens, k4, v4, nullptr, &a);
    if (rc || n_rows == 0) return rc;
    a.k_out = k_out;
    a.v_out = v_out;
    a.f32 = rows == ENTMAXKV_ROWS_F32;
    return launch_kv4_read(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_ERR_CUDA;
}

}  // extern "C"
