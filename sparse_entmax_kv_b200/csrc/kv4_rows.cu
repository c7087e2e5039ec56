// kv4_rows.cu -- rows into and out of the 4-bit cache, and the C entry points
// of both (include/entmaxkv_kv4.h).
//
// write: one CTA per (touched page, kv head).  A warp takes a token pair: its
// lanes hold 4 (d = 128) or 2 (d = 64) neighbouring coordinates of both rows,
// min and max of a 64-coordinate group come from shuffles, and the codes of a
// word are joined across the lanes that share it.  A value word holds both
// tokens of a pair; when only one of them is new the other's half is kept
// (the warp is the word's only writer).  With metadata the page's dequantised
// keys are kept in shared memory and thread j then walks coordinate j in
// token order, as the bf16 build does.
// read: the same split, the other way round.
#include <cmath>

#include "../../include/entmaxkv_kv4.h"
#include "kv4.cuh"

namespace ekv {

namespace {

constexpr int RW_THREADS = 128;
constexpr int RW_WARPS = RW_THREADS / 32;

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
        int lo = 0, hi = a.m.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.row_start[mid] / P + 2 * mid <= slot) lo = mid;
            else hi = mid - 1;
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

template <int D>
constexpr int CPL = D / 32;  // coordinates of a lane

// The lane's coordinates of a bf16 row.
template <int D>
__device__ __forceinline__ void load_row(const uint16_t *row, float (&x)[CPL<D>]) {
    const int lane = threadIdx.x & 31;
    if constexpr (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2 *>(row + 4 * lane);
        x[0] = bf16lo(w.x);
        x[1] = bf16hi(w.x);
        x[2] = bf16lo(w.y);
        x[3] = bf16hi(w.y);
    } else {
        const unsigned w = *reinterpret_cast<const unsigned *>(row + 2 * lane);
        x[0] = bf16lo(w);
        x[1] = bf16hi(w);
    }
}

// Codes of one row's coordinates held by the warp, and its group's parameters
// (every lane of the group returns them).
template <int D>
__device__ __forceinline__ void quantise(const float (&x)[CPL<D>], unsigned (&c)[CPL<D>], float &s, float &lo) {
    float mn = x[0], mx = x[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < CPL<D>; ++i) {
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
        bad |= !(fabsf(x[i]) < INFINITY);
    }
#pragma unroll
    for (int o = D == 128 ? 8 : 16; o; o >>= 1) {
        mn = fminf(mn, __shfl_xor_sync(FULL, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
    }
    const unsigned bal = __ballot_sync(FULL, bad);
    const int lane = threadIdx.x & 31;
    const unsigned mine = D == 128 ? (lane < 16 ? 0xffffu : 0xffff0000u) : FULL;
    const float range = __fsub_rn(mx, mn);
    if ((bal & mine) || !(range < INFINITY)) {
        s = lo = __int_as_float(0x7fc00000);
#pragma unroll
        for (int i = 0; i < CPL<D>; ++i) c[i] = 0u;
        return;
    }
    lo = mn;
    s = bf16f(f2bf(__fdiv_rn(range, 15.f)));
    if (s < 1.17549435e-38f) s = 0.f;  // 2^-126: below, 1 / s may overflow
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int i = 0; i < CPL<D>; ++i)
        c[i] = (unsigned)fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(x[i], lo), inv)), 0.f), 15.f);
}

// Joins the lane's codes of a key row into its 8-coordinate word (all lanes
// that share the word return it).
template <int D>
__device__ __forceinline__ unsigned join_k(const unsigned (&c)[CPL<D>]) {
    const int lane = threadIdx.x & 31;
    unsigned w;
    if constexpr (D == 128) {
        w = (c[0] | (c[1] << 16) | (c[2] << 4) | (c[3] << 20)) << (8 * (lane & 1));
    } else {
        w = (c[0] | (c[1] << 16)) << (4 * (lane & 3));
        w |= __shfl_xor_sync(FULL, w, 2);
    }
    return w | __shfl_xor_sync(FULL, w, 1);
}
// The 16 bits of a value row's 4-coordinate word.
template <int D>
__device__ __forceinline__ unsigned join_v(const unsigned (&c)[CPL<D>]) {
    if constexpr (D == 128) {
        return c[0] | (c[1] << 4) | (c[2] << 8) | (c[3] << 12);
    } else {
        const unsigned w = (c[0] | (c[1] << 4)) << (8 * (threadIdx.x & 1));
        return w | __shfl_xor_sync(FULL, w, 1);
    }
}
// The lane's codes of token t's key / value from its stored words.
template <int D>
__device__ __forceinline__ void split_k(const unsigned *tile, int t, unsigned (&c)[CPL<D>]) {
    const int lane = threadIdx.x & 31;
    if constexpr (D == 128) {
        const unsigned w = tile[kv4_kword<D>(t, lane >> 1)] >> (8 * (lane & 1));
        c[0] = w & 15;
        c[1] = (w >> 16) & 15;
        c[2] = (w >> 4) & 15;
        c[3] = (w >> 20) & 15;
    } else {
        const unsigned w = tile[kv4_kword<D>(t, lane >> 2)] >> (4 * (lane & 3));
        c[0] = w & 15;
        c[1] = (w >> 16) & 15;
    }
}
template <int D>
__device__ __forceinline__ void split_v(const unsigned *tile, int t, unsigned (&c)[CPL<D>]) {
    const int lane = threadIdx.x & 31;
    const int q4 = D == 128 ? lane : lane >> 1;
    unsigned w = tile[kv4_vword<D>(t >> 1, q4)] >> (16 * (t & 1));
    if constexpr (D == 64) w >>= 8 * (lane & 1);
#pragma unroll
    for (int i = 0; i < CPL<D>; ++i) c[i] = (w >> (4 * i)) & 15;
}

__device__ __forceinline__ unsigned pack_params(float s, float lo) {
    return (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xffff0000u);  // both are bf16 values
}

// Group of the lane's coordinates.
template <int D>
__device__ __forceinline__ int lane_group() {
    return D == 128 ? (int)(threadIdx.x & 31) >> 4 : 0;
}
// One lane of each group writes the group's parameters.
template <int D>
__device__ __forceinline__ bool group_leader() {
    return (threadIdx.x & (D == 128 ? 15 : 31)) == 0;
}

template <int D>
__device__ __forceinline__ void write_key(unsigned char *tile, int t, const float (&x)[CPL<D>], float *kval) {
    unsigned c[CPL<D>];
    float s, lo;
    quantise<D>(x, c, s, lo);
    const unsigned w = join_k<D>(c);
    const int lane = threadIdx.x & 31;
    constexpr int SH = D == 128 ? 2 : 4;  // lanes of a word
    if (lane % SH == 0) reinterpret_cast<unsigned *>(tile)[kv4_kword<D>(t, lane / SH)] = w;
    if (group_leader<D>())
        reinterpret_cast<unsigned *>(tile + Kv4<D>::CODES)[t * Kv4<D>::NG + lane_group<D>()] = pack_params(s, lo);
    if (kval)
#pragma unroll
        for (int i = 0; i < CPL<D>; ++i) kval[CPL<D> * lane + i] = __fmaf_rn(s, (float)c[i], lo);
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

template <int D, int P>
__global__ void __launch_bounds__(RW_THREADS) kv4_write_kernel(const __grid_constant__ Kv4RowArgs a) {
    pdl_wait();
    extern __shared__ float kval[];  // [P][D] dequantised keys (with metadata)
    PageJob j;
    if (!page_job<P>(a, blockIdx.x, j)) return;
    const int kvh = a.m.kv0 + blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *kt = a.k4 + kv4_tile<D>(j.blk, a.m.Hkv, kvh, P, 0);
    unsigned char *vt = a.v4 + kv4_tile<D>(j.blk, a.m.Hkv, kvh, P, 0);
    const bool meta = a.m.meta != nullptr;
    const uint16_t *kr = a.k_new + (j.row0 - j.t0) * a.stride + (size_t)kvh * D;  // row of slot 0
    const uint16_t *vr = a.v_new + (j.row0 - j.t0) * a.stride + (size_t)kvh * D;
    // the page's old keys, for the metadata
    if (meta)
        for (int t = warp; t < j.t0; t += RW_WARPS) {
            const unsigned char *tile = kt + (t >> 4) * Kv4<D>::TILE;
            unsigned c[CPL<D>];
            split_k<D>(reinterpret_cast<const unsigned *>(tile), t & 15, c);
            const unsigned pr =
                reinterpret_cast<const unsigned *>(tile + Kv4<D>::CODES)[(t & 15) * Kv4<D>::NG + lane_group<D>()];
#pragma unroll
            for (int i = 0; i < CPL<D>; ++i)
                kval[t * D + CPL<D> * lane + i] = __fmaf_rn(bf16lo(pr), (float)c[i], bf16hi(pr));
        }
    for (int pair = (j.t0 >> 1) + warp; 2 * pair < j.t1; pair += RW_WARPS) {
        const int t = 2 * pair;
        const bool has0 = t >= j.t0, has1 = t + 1 < j.t1;  // at least one of the pair is new
        float kx[2][CPL<D>] = {}, vx[2][CPL<D>] = {};
        if (has0) {
            load_row<D>(kr + t * a.stride, kx[0]);
            load_row<D>(vr + t * a.stride, vx[0]);
        }
        if (has1) {
            load_row<D>(kr + (t + 1) * a.stride, kx[1]);
            load_row<D>(vr + (t + 1) * a.stride, vx[1]);
        }
        unsigned char *ktile = kt + (t >> 4) * Kv4<D>::TILE, *vtile = vt + (t >> 4) * Kv4<D>::TILE;
        unsigned half[2] = {0u, 0u};
        unsigned *vp = reinterpret_cast<unsigned *>(vtile + Kv4<D>::CODES);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!(e ? has1 : has0)) continue;
            write_key<D>(ktile, (t + e) & 15, kx[e], meta ? kval + (t + e) * D : nullptr);
            unsigned c[CPL<D>];
            float s, lo;
            quantise<D>(vx[e], c, s, lo);
            half[e] = join_v<D>(c);
            if (group_leader<D>()) vp[((t + e) & 15) * Kv4<D>::NG + lane_group<D>()] = pack_params(s, lo);
        }
        constexpr int SH = D == 128 ? 1 : 2;
        if (lane % SH == 0) {
            unsigned *w = reinterpret_cast<unsigned *>(vtile) + kv4_vword<D>((t & 15) >> 1, lane / SH);
            unsigned v = half[0] | (half[1] << 16);
            if (!(has0 && has1)) {  // the other token of the pair keeps its half
                const unsigned old = *w;
                v = has0 ? (half[0] | (old & 0xffff0000u)) : ((half[1] << 16) | (old & 0xffffu));
            }
            *w = v;
        }
    }
    if (!meta) return;
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= D) return;
    float mn = INFINITY, mx = -INFINITY;
    bool nan = false;
    double s1 = 0.0, s2 = 0.0;
    for (int t = 0; t < j.n; ++t) {
        const float x = kval[t * D + c];
        nan |= x != x;
        mn = fminf(mn, x);
        mx = fmaxf(mx, x);
        const double xd = (double)x;
        s1 = __dadd_rn(s1, xd);
        s2 = __fma_rn(xd, xd, s2);
    }
    const double dn = (double)j.n;
    const double m = __ddiv_rn(s1, dn);
    double v = __dsub_rn(__ddiv_rn(s2, dn), __dmul_rn(m, m));
    if (v < 0.0) v = 0.0;
    if (nan) mn = mx = __int_as_float(0x7fc00000);
    const int sl = j.page % META_TILE;
    const long long T = ((long long)j.b * a.m.Hkv + kvh) * a.m.n_tiles + j.page / META_TILE;
    const int ch = c / 16, e = c % 16;
    uint8_t *bb = a.m.meta + T * 128 * D + ch * 2048;
    const int ob = sl * 32 + 16 * ((e >> 3) ^ ((sl >> 2) & 1)) + 2 * (e & 7);
    *reinterpret_cast<uint16_t *>(bb + ob) = bf16_down(mn);
    *reinterpret_cast<uint16_t *>(bb + 1024 + ob) = bf16_up(mx);
    uint8_t *mm = a.m.meta + a.m.n_tiles_total * 128 * D + T * 256 * D + ch * 4096;
    const int om = sl * 64 + 16 * ((e >> 2) ^ ((sl >> 1) & 3)) + 4 * (e & 3);
    *reinterpret_cast<float *>(mm + om) = (float)m;
    *reinterpret_cast<float *>(mm + 2048 + om) = (float)v;
}

// The lane's values of a row, to fp32 or bf16.
template <int D>
__device__ __forceinline__ void store_row(void *out, long long at, int f32, const unsigned (&c)[CPL<D>], unsigned pr) {
    const int lane = threadIdx.x & 31;
    float x[CPL<D>];
#pragma unroll
    for (int i = 0; i < CPL<D>; ++i) x[i] = __fmaf_rn(bf16lo(pr), (float)c[i], bf16hi(pr));
    if (f32) {
        float *o = static_cast<float *>(out) + at + CPL<D> * lane;
        if constexpr (D == 128) *reinterpret_cast<float4 *>(o) = make_float4(x[0], x[1], x[2], x[3]);
        else *reinterpret_cast<float2 *>(o) = make_float2(x[0], x[1]);
    } else {
        uint16_t *o = static_cast<uint16_t *>(out) + at + CPL<D> * lane;
        const unsigned w0 = (unsigned)f2bf(x[0]) | ((unsigned)f2bf(x[1]) << 16);
        if constexpr (D == 128) {
            const unsigned w1 = (unsigned)f2bf(x[2]) | ((unsigned)f2bf(x[3]) << 16);
            *reinterpret_cast<uint2 *>(o) = make_uint2(w0, w1);
        } else {
            *reinterpret_cast<unsigned *>(o) = w0;
        }
    }
}

template <int D, int P>
__global__ void __launch_bounds__(RW_THREADS) kv4_read_kernel(const __grid_constant__ Kv4RowArgs a) {
    pdl_wait();
    PageJob j;
    if (!page_job<P>(a, blockIdx.x, j)) return;
    const int kvh = a.m.kv0 + blockIdx.y;
    const int warp = threadIdx.x >> 5;
    const size_t page = kv4_tile<D>(j.blk, a.m.Hkv, kvh, P, 0);
    for (int t = j.t0 + warp; t < j.t1; t += RW_WARPS) {
        const size_t tile = page + (size_t)(t >> 4) * Kv4<D>::TILE;
        const long long at = (j.row0 + t - j.t0) * a.stride + (long long)kvh * D;
        const int p = (t & 15) * Kv4<D>::NG + lane_group<D>();
        unsigned c[CPL<D>];
        split_k<D>(reinterpret_cast<const unsigned *>(a.k4 + tile), t & 15, c);
        store_row<D>(a.k_out, at, a.f32, c, reinterpret_cast<const unsigned *>(a.k4 + tile + Kv4<D>::CODES)[p]);
        split_v<D>(reinterpret_cast<const unsigned *>(a.v4 + tile), t & 15, c);
        store_row<D>(a.v_out, at, a.f32, c, reinterpret_cast<const unsigned *>(a.v4 + tile + Kv4<D>::CODES)[p]);
    }
}

template <int D, int P>
cudaError_t write_t(const Kv4RowArgs &a, dim3 grid, cudaStream_t st) {
    return launch_pdl(kv4_write_kernel<D, P>, grid, dim3(RW_THREADS), a.m.meta ? (size_t)P * D * 4 : 0, st, a);
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
