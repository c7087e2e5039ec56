// kv4_decode.cu -- decode attention over the 4-bit cache, and its C entry
// points (include/entmaxkv_kv4.h).
//
// Mathematics.  With k_tj = s_tg c_tj + lo_tg for the coordinates j of group
// g, the score of token t is
//   q.k_t = sum_g [ s_tg sum_{j in g} q_j (c_tj - 8) + (lo_tg + 8 s_tg) sum_{j in g} q_j ],
// so the centred codes themselves are the tensor-core operand, in fp16: a code
// in the mantissa of 1024 is 1024 + c or 1024 + 16 c, and one packed
// multiply-add makes that c - 8, exactly (fp16 has room for two codes in a
// mantissa, so a word of eight codes needs one shift; bf16 would need three,
// and integer shifts and masks are what such a kernel is bound by).  The
// codes are centred because the tensor core truncates its fp32 sums: an offset
// common to all codes would be summed, truncated and cancelled again (with 16
// + c as the operand the softmax of 32k tokens was 5e-4 off, relatively).
//   keys    the query is scaled by a power of two per head, so that its
//           largest coordinate is near 2^13: coordinates down to 2^-27 of
//           that stay exact, smaller ones are off by 2^-38 of it at most
//   values  the weights p_t s_tg go in as two fp16 parts (22 bits together),
//           and sum_t p_t (lo_tg + 8 s_tg) is added at the end.  The
//           reference of a head's softmax is placed so that its largest p s
//           lies between 2^9 and 2^15: what is lost of a weight is below 2^-34
//           of the largest (values below 2^-86 get less).  Groups of four heads or fewer put the two parts
//           in the columns their heads leave free.  The sums move to a second
//           set of fp32 registers every few tiles, so that few truncations
//           meet a large sum.  With eight heads the lower parts would be
//           truncated against the sum of the upper ones, product by product
//           (124k tokens: 2.7e-6 off instead of 3.4e-7): there the products of
//           each tile and part begin at zero and move at once
//
// The chunks (16 or 32 tokens of one kv head) of all groups' page lists form one
// range that is cut evenly among the warps of a grid that fills the GPU once:
// ragged batches and any number of groups keep every SM busy to the end.  A
// warp takes its chunks through a ring of its own in shared memory, filled by
// bulk copies ahead of use, and reads each 16-token tile once for all query
// heads of the group (heads are the n dimension of m16n8k16, tokens or value
// coordinates the m dimension).
//   softmax  running max, sum and output per head, one partial for each warp
//            and group, merged by combine_kernel in token order
//   entmax   scan_kernel keeps the tokens whose z can still carry weight
//            (z > max so far - 1: no weight exceeds 1) as a list of (z, value
//            row) for each warp and group; tau_kernel, one CTA a head, drops
//            those below the head's max - 1, solves for tau and sums p v over
//            the support.  It counts z from the head's max: the differences
//            that matter are exact in fp32 and below 1, whatever the scores' size
//
// What bounds it: instructions, then memory.  A 16-token tile of 128
// coordinates (2304 bytes with its values) takes about 403 warp instructions
// with its values and 244 without, most of them to make operands of codes; the
// integer pipe is 44 to 48 % busy, the issue slots 60 to 65 %, the tensor
// pipe 16 to 20 %.  Softmax over 8 sequences of 16k to 32k tokens, 8 kv heads of 4,
// d = 128: 69 us, 236 MB at 3.4 TB/s (52 % of a copy's rate); entmax over 4
// of 64k to 128k: 117 us, of which the scan is 100 (271 MB at 2.7 TB/s).
// Tried and dropped: units of a quarter of a warp's share, taken from a queue
// in one CTA an SM (71 -> 84 us, 126 -> 145: each pays for its queries and its
// first copies again); key codes uncentred, straight from the mask (4 to 6 %
// faster, entmax 2.5 times as far off); the shift of a code word on the
// multiplier (71 -> 77 us); four stages to a ring (no gain);
// five CTAs an SM (96 registers a thread without spills; scan 121 -> 128 us,
// softmax of d = 64 82.5 -> 83.2).
#include <cfloat>
#include <cmath>
#include <cstring>

#include "../../include/entmaxkv_kv4.h"
#include "entmax.cuh"
#include "kv4.cuh"

namespace ekv {

namespace {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = AT_WARPS * 32;
constexpr int AT_MAX_WARPS = 148 * 5 * AT_WARPS;
constexpr int WHOLE_WARPS = 12;         // warps of a CTA that has a group to itself ...
constexpr int WHOLE_TILES = 16;         // ... and tiles for each of them at most, with many groups
constexpr int WHOLE_FEW = 5;            // and with few
constexpr int AT_MIN_CHUNKS = 2;        // chunks a warp gets at least ...
constexpr int AT_GROUP_PARTS = 512;     // ... and warps a group's list is cut among at most, on average
constexpr float AT_MAX_X = 32768.f;     // p s stays below this (fp16 ends at 65504) ...
constexpr int AT_TOP_X = 10;            // ... and is brought to 2^10 where a reference is set;
constexpr float AT_MAX_Y = 0x1p103f;    // so for p |lo + 8 s|, which matters where steps are far below the values,
constexpr int AT_TOP_Y = 96;            // and for p itself, which is all there is where values are zero.
constexpr int AT_UNIT = 8;              // Sums of the two are kept in units of 2^8: a list has fewer than 2^31 tokens,
constexpr float AT_PER_UNIT = 1.f / (1 << AT_UNIT);  // so they stay below 2^126

// CTAs an SM holds (registers bound the softmax, shared memory allows five).
template <int D, int G>
constexpr int softmax_ctas() { return D == 64 && G < 8 ? 4 : 3; }
constexpr int SCAN_CTAS = 4;

struct Kv4DecodeArgs {
    const uint16_t *q;
    const uint8_t *k4, *v4;
    const int *page_table, *seq_lens;
    const int *union_e, *union_blk, *union_cnt;  // the pages of each group (G > 1 with a selection),
    const int *sel, *cnt;                        // or of each head (G = 1); all null: every page
    float *out, *tau_out;
    float *part_o;        // [slots][G][d] softmax partials
    float2 *part_ml;      // [slots][G]
    float *cand_z;        // [B Hq][max_pages P]
    unsigned *cand_row;   // [B Hq][max_pages P]  blk P + slot
    int4 *seg;            // [slots][G] candidates of a warp's share of a group, their max, place of the first
    int2 *slots;          // [B Hkv] first and last slot of the group's shares
    int *zmax;            // [B Hq] running max of a head's z (order-mapped), null: none kept
    int W;                // warps that share the chunks at most
    int S;                // shares of a group, where every group's list is cut alike (else 0)
    int ct, lc;           // tiles of a chunk (1 or 2), log2 of the chunks of a page
    int npg;              // pages of a ring stage
    int B, Hq, Hkv, P, max_pages, num_blocks;
    int kv0, nk;
    float alpha;
    int r_int;
    unsigned one;         // 0x64006400: 1024 as two fp16, see code_f16
    int *status;
};

// --------------------------------------------------------------- the range of chunks

// Entries of the range: the sequences (nk groups each), or with selections the
// groups themselves.
__device__ __forceinline__ bool chosen(const Kv4DecodeArgs &a) { return a.union_e || a.sel; }
__device__ __forceinline__ int n_entries(const Kv4DecodeArgs &a) { return chosen(a) ? a.B * a.nk : a.B; }
__device__ __forceinline__ int groups_of_entry(const Kv4DecodeArgs &a) { return chosen(a) ? 1 : a.nk; }
__device__ __forceinline__ int tokens_of(const Kv4DecodeArgs &a, int b) {
    const int s = __ldg(a.seq_lens + b), cap = a.max_pages * a.P;
    return s < 0 ? 0 : min(s, cap);
}
// Chunks of each group of entry i.
__device__ __forceinline__ int entry_chunks(const Kv4DecodeArgs &a, int i) {
    if (!chosen(a)) return n_pages_of(tokens_of(a, i), a.P) << a.lc;
    int b, kvh;
    group_of(i, a.kv0, a.nk, b, kvh);
    if (a.union_e) return __ldg(a.union_cnt + b * a.Hkv + kvh) << a.lc;
    return max(0, min(__ldg(a.cnt + b * a.Hq + kvh), n_pages_of(tokens_of(a, b), a.P))) << a.lc;  // G = 1
}

// One warp's share of one group's list.
struct Share {
    int b, kvh, bk, g;  // g: group in the order of the range
    int U, seq;         // pages of the list, tokens of the sequence
    int first, last;    // chunks [first, last) of the list
    int T;              // chunks of the whole list
    int slot;           // where what the share gives is kept: consecutive for the shares of a group
    bool opens, closes; // its group's first, last share
};

// A warp's part of the range, from its first chunk on.  Every warp finds it by
// itself: lane i sums entries i C .. i C + C - 1.  The lists of selections are
// about alike in length and may be many: there each group's list is cut in
// a.S shares, and no warp has to know the other groups' (16 x 32 lists of 32
// pages: the scan 28 us with the range, 18 so).
struct Walk {
    int w;             // the warp, or its next share
    long long t, end;  // chunks [t, end) of the range are left
    int i;             // entry of chunk t or before,
    int T;             // the chunks of each of its groups,
    long long start;   // its first chunk
    Walk() = default;
    __device__ __forceinline__ Walk(const Kv4DecodeArgs &a, int w) {
        this->w = w;
        t = end = 0;
        if (w >= a.W) return;
        if (a.S) {
            end = (long long)a.B * a.nk * a.S;  // shares
            return;
        }
        const int n = n_entries(a), C = (n + 31) / 32, m = groups_of_entry(a), lane = threadIdx.x & 31;
        long long v = 0;
#pragma unroll 4
        for (int k = 0; k < C; ++k)
            if (lane * C + k < n) v += entry_chunks(a, lane * C + k);
        v *= m;
        long long x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL, x, o);
            if (lane >= o) x += y;
        }
        const long long total = __shfl_sync(FULL, x, 31);
        x -= v;
        // no more warps than chunks, so that every warp of them has one
        const int W = (int)min((long long)a.W, total);
        if (w >= W) return;
        t = total * w / W;
        end = total * (w + 1) / W;
        const int l = __popc(__ballot_sync(FULL, x <= t)) - 1;
        start = __shfl_sync(FULL, x, l);
        i = l * C;
        T = entry_chunks(a, i);
    }
    __device__ __forceinline__ bool more(const Kv4DecodeArgs &a) const { return a.S ? w < end : t < end; }
    __device__ __forceinline__ Share next(const Kv4DecodeArgs &a) {
        if (a.S) {
            Share s;
            s.g = w / a.S;
            const int k = w - s.g * a.S;
            group_of(s.g, a.kv0, a.nk, s.b, s.kvh);
            s.bk = s.b * a.Hkv + s.kvh;
            s.T = entry_chunks(a, chosen(a) ? s.g : s.b);
            s.U = s.T >> a.lc;
            s.seq = tokens_of(a, s.b);
            s.first = (int)((long long)s.T * k / a.S);
            s.last = (int)((long long)s.T * (k + 1) / a.S);
            s.slot = w;
            s.opens = k == 0;
            s.closes = k == a.S - 1;
            w += a.W;
            return s;
        }
        const int m = groups_of_entry(a);
        while (start + (long long)T * m <= t) {
            start += (long long)T * m;
            T = entry_chunks(a, ++i);
        }
        const int sub = m == 1 ? 0 : (int)(t - start) / T;
        Share s;
        s.g = i * m + sub;
        group_of(s.g, a.kv0, a.nk, s.b, s.kvh);
        s.bk = s.b * a.Hkv + s.kvh;
        s.U = T >> a.lc;
        s.T = T;
        s.seq = tokens_of(a, s.b);
        const long long at = start + (long long)sub * T;
        s.first = (int)(t - at);
        s.last = (int)min((long long)T, s.first + (end - t));
        t += s.last - s.first;
        s.slot = w + s.g;
        s.opens = s.first == 0;
        s.closes = s.last == T;
        return s;
    }
};

// Where a warp is.  It lies in shared memory while the warp reads a share's tiles,
// whose loop wants the registers: 8 x 32k softmax 75.4 -> 72.2 us, 4 x 128k entmax
// 124.2 -> 122.1 us.
struct Place {
    Walk walk;
    Share share;
    __device__ __forceinline__ void put(const Walk &w, const Share &s, int lane) {
        __syncwarp();
        if (lane == 0) {
            walk = w;
            share = s;
        }
        __syncwarp();
    }
};

// The shares of one group lie in consecutive slots, in the range w + g (both
// ascend along it, so no two shares meet); the first and the last leave word.
__device__ __forceinline__ void report_slot(const Kv4DecodeArgs &a, const Share &s) {
    if (s.opens) a.slots[s.bk].x = s.slot;
    if (s.closes) a.slots[s.bk].y = s.slot;
}
struct GroupShares {
    size_t slot;  // of the first share
    int n;
};
// The first slot of a call: every kv head has its own, for as many warps as a
// call on it alone may use, so calls on disjoint ranges share a workspace.
__host__ __device__ inline size_t slots_per_head(int B) { return (size_t)AT_MAX_WARPS + B; }

// What the host cannot see: a length or a count beyond the table.
__device__ __forceinline__ void report_limits(const Kv4DecodeArgs &a, int b, int kvh) {
    if (__ldg(a.seq_lens + b) > a.max_pages * a.P) atomicOr(a.status, ENTMAXKV_STATUS_BAD_LENGTH);
    if (a.sel && (unsigned)__ldg(a.cnt + b * a.Hq + kvh) > (unsigned)n_pages_of(tokens_of(a, b), a.P))
        atomicOr(a.status, ENTMAXKV_STATUS_BAD_SELECTION);
}
// Called by every thread of a head's CTA.
__device__ __forceinline__ GroupShares group_shares(const Kv4DecodeArgs &a, int b, int kvh) {
    const int2 s = __ldcg(a.slots + b * a.Hkv + kvh);
    const int T = entry_chunks(a, chosen(a) ? b * a.nk + kvh - a.kv0 : b);
    if (threadIdx.x == 0) report_limits(a, b, kvh);
    GroupShares r;
    r.n = T > 0 ? s.y - s.x + 1 : 0;
    r.slot = a.kv0 * slots_per_head(a.B) + (T > 0 ? s.x : 0);
    return r;
}

// --------------------------------------------------------------- the ring of tiles

// A stage holds four tiles (64 tokens): one, two or four pages of the list, of
// the keys and behind them of the values.  Each page is copied by the lane that
// has its entry, so a stage costs one pass of the warp whatever the page size
// (with a stage for every 32 tokens of a page instead: softmax of 8 x 32k
// tokens 87 us against 80 with pages of 16, 75 against 75 with 32; entmax of 4
// x 128k tokens 154 against 135 with 16, 125 against 117 with 64).
constexpr int RING_STAGES = 2;
template <int D, bool BOTH>
struct TileRing {
    static constexpr int HALF = 4 * Kv4<D>::TILE;
    static constexpr int STAGE = HALF * (BOTH ? 2 : 1);
    static constexpr int BYTES = RING_STAGES * STAGE;
    unsigned char *base;
    uint64_t *bar;
    int2 (*info)[4];         // of each page: its first cache row (block P + slot); valid tokens, and the head mask << 8
    int in = 0, out = 0;     // stages to fill and to take next
    unsigned parity = 0;     // of the stage to take
    int flying = 0;          // filled, not taken
    int e0 = 0;              // the lane's entry of 32 list entries from e0 on:
    int row = 0, tokens = 0, mask = 0;
    size_t at = 0;           // its byte offset in the cache

    __device__ __forceinline__ void init(const Kv4DecodeArgs &a, unsigned char *b, uint64_t *bars, int2 (*i)[4]) {
        base = b;
        bar = bars;
        info = i;
        if ((threadIdx.x & 31) == 0) {
            for (int s = 0; s < RING_STAGES; ++s) mbar_init(&bar[s], a.npg);
            mbar_fence_init();
        }
        __syncwarp();
    }
    __device__ __forceinline__ void start() { e0 = -(1 << 30); }  // a new list
    __device__ __forceinline__ void window(const Kv4DecodeArgs &a, const Share &s, int e) {
        const int i = e + (threadIdx.x & 31);
        e0 = e;
        tokens = 0;
        if (i >= s.U) return;
        int page = i, blk;
        mask = 0xff;
        if (a.sel) {  // strictly ascending, or the entry is left out
            const int *list = a.sel + (size_t)(s.b * a.Hq + s.kvh) * a.max_pages;
            page = __ldg(list + i);
            mask = 1;
            if (page < 0 || page >= n_pages_of(s.seq, a.P) || (i > 0 && page <= __ldg(list + i - 1))) {
                atomicOr(a.status, ENTMAXKV_STATUS_BAD_SELECTION);
                return;
            }
            blk = __ldg(a.page_table + (size_t)s.b * a.max_pages + page);
            if (blk < 0 || blk >= a.num_blocks) atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
        } else if (a.union_e) {
            const int ent = __ldg(a.union_e + (size_t)s.bk * a.max_pages + i);
            blk = __ldg(a.union_blk + (size_t)s.bk * a.max_pages + i);
            page = ent >> 8;
            mask = ent & 0xff;
        } else {
            blk = __ldg(a.page_table + (size_t)s.b * a.max_pages + i);
            if (blk < 0 || blk >= a.num_blocks) atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
        }
        if (blk < 0 || blk >= a.num_blocks) return;
        tokens = min(a.P, s.seq - page * a.P);
        row = (unsigned)blk * a.P;
        at = kv4_tile<D>(blk, a.Hkv, s.kvh, a.P, 0);
    }
    // Stages that a share takes.
    __device__ __forceinline__ int stages(const Kv4DecodeArgs &a, const Share &s) const {
        return s.last > s.first ? (((s.last - 1) >> a.lc) - (s.first >> a.lc)) / a.npg + 1 : 0;
    }
    // Starts the copies of stage k of a share into the next free stage.
    __device__ __forceinline__ void issue(const Kv4DecodeArgs &a, const Share &s, int k) {
        const int e = (s.first >> a.lc) + k * a.npg;
        if ((unsigned)(e - e0) >= 32u) window(a, s, e);
        const int piece = (int)(threadIdx.x & 31) - (e - e0);
        if ((unsigned)piece < (unsigned)a.npg) {  // the lanes that have the entries
            const int tp = a.ct << a.lc, t0 = (e + piece) * tp;  // the page's tiles; those of the share are
            const int lo = max(0, s.first * a.ct - t0), hi = min(tp, s.last * a.ct - t0);
            const int nval = max(0, min(16 * hi, tokens) - 16 * lo);
            info[in][piece] = make_int2(row + 16 * lo, nval | (mask << 8));
            if (nval > 0) {
                const unsigned bytes = ((nval + 15) >> 4) * Kv4<D>::TILE;
                const size_t o = at + lo * Kv4<D>::TILE;
                unsigned char *dst = base + in * STAGE + piece * tp * Kv4<D>::TILE;
                mbar_arrive_expect_tx(&bar[in], bytes * (BOTH ? 2 : 1));
                bulk_g2s(dst, a.k4 + o, bytes, &bar[in]);
                if (BOTH) bulk_g2s(dst + HALF, a.v4 + o, bytes, &bar[in]);
            } else {
                mbar_arrive(&bar[in]);
            }
        }
        in = in == RING_STAGES - 1 ? 0 : in + 1;
        ++flying;
    }
    __device__ __forceinline__ bool wait(const Kv4DecodeArgs &a) {
        const bool ok = mbar_wait(&bar[out], parity, a.status);
        --flying;
        return ok;
    }
    __device__ __forceinline__ void pass() {
        if (++out == RING_STAGES) {
            out = 0;
            parity ^= 1u;
        }
    }
    // Waits for the next stage.  False: it did not come (the status word says so).
    __device__ __forceinline__ bool take(const Kv4DecodeArgs &a, const int2 *&what, const unsigned char *&tiles) {
        const bool ok = wait(a);
        what = info[out];
        tiles = base + out * STAGE;
        pass();
        return __all_sync(FULL, ok);
    }
    // After a wait that ran out: the copies in flight have to land before the CTA ends.
    __device__ __forceinline__ void drain(const Kv4DecodeArgs &a) {
        while (flying > 0) {
            wait(a);
            pass();
        }
    }
};

// --------------------------------------------------------------- operands

// c - 8 of pair p of a word of eight codes (bits 4 p .. of each half), as two
// fp16.  one: 1024 twice, from a kernel argument: mask and or are one
// instruction only while the compiler does not know both constants (with a
// literal they were two; softmax over 8 x 32k tokens 84 us instead of 75).
template <int p>
__device__ __forceinline__ unsigned code_f16(unsigned w, unsigned one) {
    const unsigned x = p < 2 ? w : w >> 8;
    unsigned y;
    if constexpr (p % 2 == 0)  // 1024 + c, less 1032
        asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, 0x000f000f, %2, 0xea;\n\tadd.rn.f16x2 %0, t, %3;\n\t}"
            : "=r"(y)
            : "r"(x), "r"(one), "r"(0xe408e408u));
    else  // 1024 + 16 c, over 16 and less 72
        asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, 0x00f000f0, %2, 0xea;\n\tfma.rn.f16x2 %0, t, %3, %4;\n\t}"
            : "=r"(y)
            : "r"(x), "r"(one), "r"(0x2c002c00u), "r"(0xd480d480u));
    return y;
}
// Two floats as fp16, x0 in the low half.
__device__ __forceinline__ unsigned pack_f16(float x0, float x1) {
    unsigned y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(x1), "f"(x0));
    return y;
}
// What two floats exceed their fp16 parts by, as fp16 again.
__device__ __forceinline__ unsigned rest_f16(float x0, float x1, unsigned hi) {
    float h0, h1;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(h0), "=f"(h1)
        : "r"(hi));
    return pack_f16(x0 - h0, x1 - h1);
}
// The 8 x 8 matrix of 16-bit elements that the warp holds a row of in every
// four lanes, transposed.
__device__ __forceinline__ unsigned transpose8(unsigned x) {
    unsigned y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// D = A(16x16 fp16, row) * B(16x8 fp16, col), fp32 sums.
__device__ __forceinline__ void mul_f16_16816(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3,
                                              unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A(16x16 fp16, row) * B(16x8 fp16, col) + D, fp32 sums.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3,
                                              unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Off by 2^-22 of the result at most, as much as the weight's two fp16 parts leave.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int N>
__device__ __forceinline__ void load_words(const unsigned char *src, unsigned (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(src);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(src);
        w[0] = v.x;
        w[1] = v.y;
    }
}

// The G queries of a group as B fragments: column n holds head n % G, scaled
// by a power of two 2^e of its own; for the lane's two accumulator columns the
// sums of each coordinate group, in the units of the products, and the factor
// from those units to z.
template <int D, int G>
struct Queries {
    static constexpr int NE = G == 1 ? 1 : 2;  // distinct columns of a lane
    unsigned b[D / 16][2];
    float sum[Kv4<D>::NG][NE];
    float factor[NE];
    __device__ __forceinline__ void fetch(const uint16_t *q) {
        const int lane = threadIdx.x & 31, c = lane & 3;
        const unsigned *qw = reinterpret_cast<const unsigned *>(q + (size_t)((lane >> 2) % G) * D);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                b[i][x] = __ldg(qw + 32 * (i >> 2) + 8 * c + 4 * ((i >> 1) & 1) + 2 * (i & 1) + x);
    }
    __device__ __forceinline__ void finish(float scale) {
        const int lane = threadIdx.x & 31, c = lane & 3;
        float t[Kv4<D>::NG];
        unsigned top = 0;
#pragma unroll
        for (int g = 0; g < Kv4<D>::NG; ++g) {
            t[g] = 0.f;
#pragma unroll
            for (int i = 4 * g; i < 4 * g + 4; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    t[g] += bf16lo(b[i][x]) + bf16hi(b[i][x]);
                    top = max(top, max((b[i][x] >> 7) & 0xffu, (b[i][x] >> 23) & 0xffu));  // exponent fields
                }
            t[g] += __shfl_xor_sync(FULL, t[g], 1);
            t[g] += __shfl_xor_sync(FULL, t[g], 2);
        }
        top = max(top, __shfl_xor_sync(FULL, top, 1));
        top = max(top, __shfl_xor_sync(FULL, top, 2));
        const int e = min(13 - ((int)top - 127), 120);
        const float up = __uint_as_float((unsigned)(e + 127) << 23);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) b[i][x] = pack_f16(bf16lo(b[i][x]) * up, bf16hi(b[i][x]) * up);
#pragma unroll
        for (int v = 0; v < NE; ++v) {
            const int src = 4 * (2 * c + v);
            const float upc = __shfl_sync(FULL, up, src);
            factor[v] = scale / upc;
#pragma unroll
            for (int g = 0; g < Kv4<D>::NG; ++g) sum[g][v] = __shfl_sync(FULL, t[g], src) * upc;
        }
    }
};

// s and lo + 8 s of tokens lane / 4 and lane / 4 + 8.
template <int D>
struct Params {
    float s[2][Kv4<D>::NG], o[2][Kv4<D>::NG];
    __device__ __forceinline__ void load(const unsigned char *tile) {
        constexpr int NG = Kv4<D>::NG;
        const unsigned *pp = reinterpret_cast<const unsigned *>(tile + Kv4<D>::CODES) + ((threadIdx.x & 31) >> 2) * NG;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            unsigned w[NG];
            if constexpr (NG == 2) load_words<2>(reinterpret_cast<const unsigned char *>(pp + 8 * u * NG), w);
            else w[0] = pp[8 * u];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                s[u][g] = bf16lo(w[g]);
                o[u][g] = fmaf(8.f, s[u][g], bf16hi(w[g]));
            }
        }
    }
};

// z of the 16 tokens of a tile: z[e] token lane / 4, z[2 + e] token lane / 4 +
// 8, columns 2 (lane % 4) + e.
template <int D, int G>
__device__ __forceinline__ void tile_scores(const unsigned char *tile, const Queries<D, G> &Q, unsigned one,
                                            float (&z)[4]) {
    constexpr int NG = Kv4<D>::NG, WPL = Kv4<D>::WPL, NE = Queries<D, G>::NE;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    unsigned w0[WPL], w1[WPL];
    load_words<WPL>(tile + r * (D / 2) + c * (4 * WPL), w0);
    load_words<WPL>(tile + (r + 8) * (D / 2) + c * (4 * WPL), w1);
    Params<D> P;
    P.load(tile);
#pragma unroll
    for (int v = 0; v < 4; ++v) z[v] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 2 * g; i < 2 * g + 2; ++i) {
            mma_f16_16816(acc, code_f16<0>(w0[i], one), code_f16<0>(w1[i], one), code_f16<1>(w0[i], one),
                          code_f16<1>(w1[i], one), Q.b[2 * i][0], Q.b[2 * i][1]);
            mma_f16_16816(acc, code_f16<2>(w0[i], one), code_f16<2>(w1[i], one), code_f16<3>(w0[i], one),
                          code_f16<3>(w1[i], one), Q.b[2 * i + 1][0], Q.b[2 * i + 1][1]);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if ((v & 1) < NE)
                z[v] = fmaf(P.s[v >> 1][g], acc[v], fmaf(P.o[v >> 1][g], Q.sum[g][v & 1 & (NE - 1)], z[v]));
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if ((v & 1) < NE) z[v] *= Q.factor[v & 1 & (NE - 1)];
}
// Whether head n % G of the group selected the page, and whether all its heads
// see all tokens of a tile that has n valid ones.
template <int G>
__device__ __forceinline__ bool keeps(int mask, int n) { return (mask >> (n % G)) & 1; }
template <int G>
__device__ __forceinline__ bool whole(int mask, int n) { return n >= 16 && (~mask & ((1 << G) - 1)) == 0; }
// Tokens behind the sequence and heads that did not select the page: -inf.
template <int G>
__device__ __forceinline__ void mask_scores(int mask, int n, float (&z)[4]) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (r + 8 * (v >> 1) >= n || !keeps<G>(mask, 2 * c + (v & 1))) z[v] = -INFINITY;
}
struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// -------------------------------------------------------------- softmax

// 2^(x / 2).  References lie 96 above the largest score of their tokens (zero
// values) to 120 below it (values near 2^128): between two of them a weight's
// exponent may pass fp32's, though its product with the sum that it brings to
// the other reference does not.  Sums are therefore multiplied by the root twice.
__device__ __forceinline__ float half_weight(float x) { return exp2f(0.5f * x); }

// WHOLE: the CTA's warps share one group's list, and the CTA writes the result
// itself; else shares leave partials for combine_kernel.
template <int D, int G, int WARPS, bool WHOLE>
__global__ void __launch_bounds__(32 * WARPS, (WHOLE ? 1 : softmax_ctas<D, G>()))
    kv4_softmax_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    constexpr int NG = Kv4<D>::NG, WPL = Kv4<D>::WPL, MT = D / 16, NE = Queries<D, G>::NE;
    constexpr bool APART = G == 8;  // two products per value operand, one for each part (else one for both)
    constexpr int FLUSH = 8;        // tiles between flushes of the output sums (APART: one)
    using Ring = TileRing<D, true>;
    extern __shared__ __align__(128) unsigned char rings[];
    __shared__ uint64_t bars[WARPS][RING_STAGES];
    __shared__ int2 infos[WARPS][RING_STAGES][4];
    __shared__ Place places[WHOLE ? 1 : WARPS];
    __shared__ float2 parts[WHOLE ? WARPS : 1][G];  // reference and sum of the warps' shares
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    const int w = blockIdx.x * WARPS + warp;
    const unsigned one = a.one;
    const bool rest = G == 4 ? c >= 2 : G == 2 ? c & 1 : false;  // the lane's columns carry the lower parts
    Ring ring;
    ring.init(a, rings + warp * Ring::BYTES, bars[warp], infos[warp]);
    Walk walk(a, w);
    const int page_bytes = (a.ct << a.lc) * Kv4<D>::TILE;
    bool alive = true;  // no wait ran out so far
    while (walk.more(a)) {
        const Share to_do = walk.next(a);
        if (!WHOLE) places[warp].put(walk, to_do, lane);
        const Share &sh = WHOLE ? to_do : places[warp].share;
        Queries<D, G> Q;
        Q.fetch(a.q + ((size_t)sh.b * a.Hq + sh.kvh * G) * D);
        ring.start();
        const int stages = alive ? ring.stages(a, sh) : 0;
        for (int i = 0; i < RING_STAGES && i < stages; ++i) ring.issue(a, sh, i);
        Q.finish(1.4426950408889634f * rsqrtf((float)D));  // z in powers of two

        float acc[MT][4], tot[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][v] = tot[i][v] = 0.f;
        // per column of the lane: the reference (weights are 2^(z - ref)), the
        // sums of p and of p (lo + 8 s) over the lane's tokens
        float ref[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f}, off[NG][2] = {};
        int until = FLUSH;
        for (int i = 0; i < stages; ++i) {
            const int2 *whats;
            const unsigned char *stage;
            if (!ring.take(a, whats, stage)) {
                ring.drain(a);
                alive = false;  // the shares end empty, so that what reads them finds them whole
                break;
            }
#pragma unroll 1
            for (int page = 0; page < a.npg; ++page, stage += page_bytes) {
                const int what = whats[page].y, mask = what >> 8;
                int n = what & 0xff;
#pragma unroll 1
                for (const unsigned char *tile = stage; n > 0; n -= 16, tile += Kv4<D>::TILE) {
                    float z[4], p[4], x[NG][4], y[NG][2];
                    tile_scores<D, G>(tile, Q, a.one, z);
                    const unsigned char *vt = tile + Ring::HALF;
                    Params<D> P;
                    P.load(vt);
                    // weights p, the x = p s, and y, the sums of p (lo + 8 s)
                    auto weights = [&](auto masked) {
                        float sum = 0.f;
#pragma unroll
                        for (int e = 0; e < NE; ++e) {
                            p[e] = ex2(z[e] - ref[e]);
                            p[2 + e] = ex2(z[2 + e] - ref[e]);
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                x[g][e] = p[e] * P.s[0][g];
                                x[g][2 + e] = p[2 + e] * P.s[1][g];
                                y[g][e] = fmaf(p[e], P.o[0][g], p[2 + e] * P.o[1][g]);
                                // pages that the head did not select may hold anything
                                if (masked.value && !keeps<G>(mask, 2 * c + e)) x[g][e] = x[g][2 + e] = y[g][e] = 0.f;
                                sum = fmaf(fabsf(y[g][e]), AT_MAX_X / AT_MAX_Y, sum + (x[g][e] + x[g][2 + e]));
                            }
                            sum = fmaf(p[e] + p[2 + e], AT_MAX_X / AT_MAX_Y, sum);
                        }
                        return sum;
                    };
                    float sum;
                    const bool all = whole<G>(mask, n);
                    if (all) {
                        sum = weights(No{});
                    } else {
                        mask_scores<G>(mask, n, z);
                        // so may rows behind the sequence
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            if (r + 8 * u >= n)
#pragma unroll
                                for (int g = 0; g < NG; ++g) P.s[u][g] = P.o[u][g] = 0.f;
                        sum = weights(Yes{});
                    }
                    if (__any_sync(FULL, !(sum <= AT_MAX_X))) {
                        // the reference follows the largest p s, or p, or p |lo + 8 s|
                        float corr[2] = {1.f, 1.f};  // of the sums of p s, which are too small to count where it underflows
#pragma unroll
                        for (int e = 0; e < NE; ++e) {
                            float zm = fmaxf(z[e], z[2 + e]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) zm = fmaxf(zm, __shfl_xor_sync(FULL, zm, o));
                            float xm = 0.f, ym = 0.f;
                            const float p0 = exp2f(z[e] - zm), p1 = exp2f(z[2 + e] - zm);
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                xm = fmaxf(xm, fmaxf(p0 * P.s[0][g], p1 * P.s[1][g]));
                                ym = fmaxf(ym, fmaxf(p0 * fabsf(P.o[0][g]), p1 * fabsf(P.o[1][g])));
                            }
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) {
                                xm = fmaxf(xm, __shfl_xor_sync(FULL, xm, o));
                                ym = fmaxf(ym, __shfl_xor_sync(FULL, ym, o));
                            }
                            // below 2^(exponent + 1)
                            const int x_up = AT_TOP_X - ((int)(__float_as_uint(xm) >> 23) - 126);
                            const int y_up = AT_TOP_Y - ((int)(__float_as_uint(ym) >> 23) - 126);
                            const float nr = fmaxf(ref[e], zm - (float)max(-120, min(min(x_up, y_up), AT_TOP_Y)));
                            const float half = half_weight(ref[e] - nr);
                            corr[e] = half * half;
                            ref[e] = nr;
                            l[e] = l[e] * half * half;
#pragma unroll
                            for (int g = 0; g < NG; ++g) off[g][e] = off[g][e] * half * half;
                        }
                        if (NE == 1) corr[1] = corr[0];
#pragma unroll
                        for (int k = 0; k < MT; ++k)
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                if (!APART) acc[k][v] *= corr[v & 1];
                                tot[k][v] *= corr[v & 1];
                            }
                        weights(Yes{});
                    }
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
                        l[e] = fmaf(p[e] + p[2 + e], AT_PER_UNIT, l[e]);
#pragma unroll
                        for (int g = 0; g < NG; ++g) off[g][e] = fmaf(y[g][e], AT_PER_UNIT, off[g][e]);
                    }
                    unsigned w0[WPL], w1[WPL];
                    const int piece = (r ^ kv4_vswz<D>(c)) * (4 * WPL);  // pairs c and c + 4 have the same swizzle
                    load_words<WPL>(vt + c * D + piece, w0);
                    load_words<WPL>(vt + (c + 4) * D + piece, w1);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        // token by column, to column by token
                        unsigned bf[APART ? 2 : 1][2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float x0 = x[g][2 * u], x1 = x[g][2 * u + NE - 1];
                            const unsigned hi = pack_f16(x0, x1);
                            const unsigned lo = rest_f16(x0, x1, hi);
                            if constexpr (G == 8) {
                                bf[0][u] = transpose8(hi);
                                bf[1][u] = transpose8(lo);
                            } else if constexpr (G == 1) {
                                bf[0][u] = transpose8(__byte_perm(hi, lo, 0x5410));
                            } else {
                                bf[0][u] = transpose8(rest ? lo : hi);
                            }
                        }
                        auto sums = [&](int i, unsigned c0, unsigned c1, unsigned c2, unsigned c3) {
                            if constexpr (APART) {
#pragma unroll
                                for (int part = 0; part < 2; ++part) {
                                    float t[4];
                                    mul_f16_16816(t, c0, c1, c2, c3, bf[part][0], bf[part][1]);
#pragma unroll
                                    for (int v = 0; v < 4; ++v) tot[i][v] += t[v];
                                }
                            } else {
                                mma_f16_16816(acc[i], c0, c1, c2, c3, bf[0][0], bf[0][1]);
                            }
                        };
#pragma unroll
                        for (int k = 2 * g; k < 2 * g + 2; ++k) {
                            const unsigned a0 = code_f16<0>(w0[k], one), a1 = code_f16<1>(w0[k], one),
                                           a2 = code_f16<0>(w1[k], one), a3 = code_f16<1>(w1[k], one);
                            sums(2 * k, a0, a1, a2, a3);
                            const unsigned d0 = code_f16<2>(w0[k], one), d1 = code_f16<3>(w0[k], one),
                                           d2 = code_f16<2>(w1[k], one), d3 = code_f16<3>(w1[k], one);
                            sums(2 * k + 1, d0, d1, d2, d3);
                        }
                    }
                    if (!APART && --until == 0) {
                        until = FLUSH;
#pragma unroll
                        for (int k = 0; k < MT; ++k)
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                tot[k][v] += acc[k][v];
                                acc[k][v] = 0.f;
                            }
                    }
                }
            }
            __syncwarp();
            if (i + RING_STAGES < stages) ring.issue(a, sh, i + RING_STAGES);
        }
        // the share's partial: sums over the lanes of a column and over the
        // columns of a head, through the ring's memory (no copy is in flight)
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[e] += __shfl_xor_sync(FULL, l[e], o);
#pragma unroll
                for (int g = 0; g < NG; ++g) off[g][e] += __shfl_xor_sync(FULL, off[g][e], o);
            }
        const size_t slot = a.kv0 * slots_per_head(a.B) + sh.slot;
        if (!WHOLE && lane == 0) report_slot(a, sh);
        if (r == 0)
#pragma unroll
            for (int e = 0; e < NE; ++e)
                if (2 * c + e < G)
                    (WHOLE ? parts[warp][2 * c + e] : a.part_ml[slot * G + 2 * c + e]) = make_float2(ref[e], l[e]);
        float *merge = reinterpret_cast<float *>(ring.base);
#pragma unroll
        for (int k = 0; k < MT; ++k) {
            // tile k holds coordinates j (row r) and j + 1 (row r + 8)
            const int j = 64 * (k >> 2) + 8 * r + 4 * ((k >> 1) & 1) + 2 * (k & 1);
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (!APART) tot[k][v] += acc[k][v];
#pragma unroll
            for (int v = 0; v < 4; v += G == 1 ? 2 : 1) {
                float o = tot[k][v];
                if (G == 1) o += tot[k][v + 1];
                if (G == 2) o += __shfl_xor_sync(FULL, o, 1);
                if (G == 4) o += __shfl_xor_sync(FULL, o, 2);
                const int n = 2 * c + (v & 1);
                if (n < G) merge[n * D + j + (v >> 1)] = fmaf(o, AT_PER_UNIT, off[k >> 2][v & 1]);
            }
        }
        if (WHOLE) break;  // the one share
        walk = places[warp].walk;
        __syncwarp();
        for (int i = lane; i < G * D / 4; i += 32)
            reinterpret_cast<float4 *>(a.part_o + slot * G * D)[i] = reinterpret_cast<const float4 *>(merge)[i];
        // the next share's copies write over it
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }
    if constexpr (WHOLE) {
        __shared__ int strange[G];  // heads whose query is not finite
        int b, kvh;
        group_of(blockIdx.x, a.kv0, a.nk, b, kvh);
        const int h0 = b * a.Hq + kvh * G;
        if (threadIdx.x < G) strange[threadIdx.x] = 0;
        if (threadIdx.x == 0) report_limits(a, b, kvh);
        __syncthreads();
        for (int i = threadIdx.x; i < G * D; i += 32 * WARPS)
            if ((__ldg(a.q + (size_t)h0 * D + i) & 0x7f80u) == 0x7f80u) strange[i / D] = 1;
        __syncthreads();
        for (int i = threadIdx.x; i < G * D; i += 32 * WARPS) {
            const int h = i / D;
            float M = -INFINITY, den = 0.f, num = 0.f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) M = fmaxf(M, parts[k][h].x);
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                const float2 ml = parts[k][h];
                if (ml.y == 0.f) continue;  // no token of the head (NaN scores make it NaN)
                const float f = half_weight(ml.x - M);
                den = fmaf(f, f * ml.y, den);
                if (f != 0.f) num = fmaf(f, f * reinterpret_cast<const float *>(rings + k * Ring::BYTES)[i], num);
            }
            const float nan = __int_as_float(0x7fc00000);
            const bool fine = !strange[h], none = den == 0.f;
            a.out[(size_t)h0 * D + i] = !fine ? nan : none ? 0.f : num / den;
            if (i % D == 0) {
                if (!fine) atomicOr(a.status, ENTMAXKV_STATUS_NONFINITE);
                if (a.tau_out) a.tau_out[h0 + h] = !fine || none ? nan : 0.6931471805599453f * (M + (AT_UNIT + log2f(den)));
            }
        }
    }
}

// The shares of a head, merged in token order.
template <int D, int CB_NT>
__global__ void __launch_bounds__(CB_NT) kv4_combine_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    constexpr int SUB = CB_NT / D;
    extern __shared__ float weight[];  // of each share, its root
    __shared__ float red[2][CB_NT / 32];
    __shared__ float o_sh[SUB][D];
    const int G = a.Hq / a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int b, h;
    head_of(blockIdx.x, a.kv0 * G, a.nk * G, b, h);
    const int bh = b * a.Hq + h;
    const uint16_t qb = threadIdx.x < D ? a.q[(size_t)bh * D + threadIdx.x] : (uint16_t)0;
    const GroupShares gs = group_shares(a, b, h / G);
    const int n = gs.n;
    const size_t slot0 = gs.slot;
    const bool fine = __syncthreads_and((qb & 0x7f80u) != 0x7f80u);
    float M = -INFINITY;
    for (int s = threadIdx.x; s < n; s += CB_NT) M = fmaxf(M, __ldcg(&a.part_ml[(slot0 + s) * G + h % G]).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CB_NT / 32; ++i) M = fmaxf(M, red[0][i]);
    float den = 0.f;
    for (int s = threadIdx.x; s < n; s += CB_NT) {
        const float2 ml = __ldcg(&a.part_ml[(slot0 + s) * G + h % G]);
        const float f = ml.y == 0.f ? 0.f : half_weight(ml.x - M);  // no token of the head (NaN scores make it NaN)
        weight[s] = f;
        den = fmaf(f, f * ml.y, den);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(FULL, den, o);
    if (lane == 0) red[1][warp] = den;
    __syncthreads();
    den = 0.f;
#pragma unroll
    for (int i = 0; i < CB_NT / 32; ++i) den += red[1][i];
    const int j = threadIdx.x % D, sub = threadIdx.x / D;
    const float *p = a.part_o + (slot0 * G + h % G) * D + j;
    float num = 0.f;
#pragma unroll 8
    for (int s = sub; s < n; s += SUB) {
        const float f = weight[s], x = __ldcg(p + (size_t)s * G * D);
        if (f != 0.f) num = fmaf(f, f * x, num);
    }
    o_sh[sub][j] = num;
    __syncthreads();
    const float nan = __int_as_float(0x7fc00000);
    if (!fine && threadIdx.x == 0) atomicOr(a.status, ENTMAXKV_STATUS_NONFINITE);
    // den is 0 only without tokens (a share with tokens has a weight of 2^-128
    // at least, in units of 2^AT_UNIT); NaN scores make it NaN
    const bool none = den == 0.f;
    if (sub == 0) {
#pragma unroll
        for (int i = 1; i < SUB; ++i) num += o_sh[i][j];
        a.out[(size_t)bh * D + j] = !fine ? nan : none ? 0.f : num / den;
    }
    if (threadIdx.x == 0 && a.tau_out)
        a.tau_out[bh] = !fine || none ? nan : 0.6931471805599453f * (M + (AT_UNIT + log2f(den)));
}

// --------------------------------------------------------------- entmax

// What carries no weight beside a largest score m: scores up to m - 1, but
// never m itself (from 2^24 on, m - 1 may round to m).
__device__ __forceinline__ float no_weight(float m) { return fminf(m - 1.f, ord2f(f2ord(m) - 1)); }

__global__ void kv4_reset_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    const int G = a.Hq / a.Hkv, i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.B * a.nk * G) return;
    int b, h;
    head_of(i, a.kv0 * G, a.nk * G, b, h);
    a.zmax[b * a.Hq + h] = ORD_NEG_INF;
}

template <int D, int G>
__global__ void __launch_bounds__(AT_THREADS, SCAN_CTAS) kv4_scan_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    using Ring = TileRing<D, false>;
    constexpr int NE = Queries<D, G>::NE;
    extern __shared__ __align__(128) unsigned char rings[];
    __shared__ uint64_t bars[AT_WARPS][RING_STAGES];
    __shared__ int2 infos[AT_WARPS][RING_STAGES][4];
    __shared__ Place places[AT_WARPS];
    constexpr int EARLY = G == 8 ? 8 : 16;  // tiles a share begins with (8: 2 % slower)
    __shared__ float early[AT_WARPS][EARLY * 16 * G];
    __shared__ unsigned early_row[AT_WARPS][EARLY];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    const int w = blockIdx.x * AT_WARPS + warp;
    Ring ring;
    ring.init(a, rings + warp * Ring::BYTES, bars[warp], infos[warp]);
    const unsigned column = 0x11111111u << c, below = (1u << lane) - 1u;  // lanes of the same columns
    const size_t row_len = (size_t)a.max_pages * a.P;
    Walk walk(a, w);
    const int page_bytes = (a.ct << a.lc) * Kv4<D>::TILE;
    bool alive = true;  // no wait ran out so far
    while (walk.more(a)) {
        const Share to_do = walk.next(a);
        places[warp].put(walk, to_do, lane);
        const Share &sh = places[warp].share;
        const int h0 = sh.b * a.Hq + sh.kvh * G;
        Queries<D, G> Q;
        Q.fetch(a.q + (size_t)h0 * D);
        ring.start();
        const int stages = alive ? ring.stages(a, sh) : 0;
        for (int i = 0; i < RING_STAGES && i < stages; ++i) ring.issue(a, sh, i);
        Q.finish((a.alpha - 1.f) * rsqrtf((float)D));
        const size_t list = (size_t)(h0 + 2 * c) * row_len + (size_t)sh.first * (16 * a.ct);

        float m[2] = {-INFINITY, -INFINITY};      // the lane's max so far, of its columns
        float known[2] = {-INFINITY, -INFINITY};  // what other shares of the head have reported
        int next[2] = {ORD_NEG_INF, ORD_NEG_INF};
        float thr[2] = {-INFINITY, -INFINITY};    // below it a score carries no weight
        int n[2] = {0, 0};                        // candidates of the lane's columns
        bool bad[2] = {false, false};             // the lane saw a NaN score
        int held = 0;                             // early tiles held back, -1 once they are settled

        // Lists the tokens of a tile that can still carry weight.  A lane goes
        // by the largest score it knows of; a new one reaches the other lanes
        // through the head's shared max.
        auto test = [&](const float (&z)[4], unsigned row) {
            bool any = false;
#pragma unroll
            for (int e = 0; e < NE; ++e) any |= !(z[e] <= thr[e]) || !(z[2 + e] <= thr[e]);  // NaN stays a candidate
            if (!__any_sync(FULL, any)) return;
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                bad[e] |= z[e] != z[e] || z[2 + e] != z[2 + e];
                const float tm = fmaxf(z[e], z[2 + e]);
                if (tm > m[e]) {
                    m[e] = tm;
                    if (a.zmax && tm > known[e] && 2 * c + e < G) atomicMax(a.zmax + h0 + 2 * c + e, f2ord(tm));
                    thr[e] = fmaxf(thr[e], no_weight(tm));
                }
                const unsigned lo = __ballot_sync(FULL, !(z[e] <= thr[e])) & column;
                const unsigned hi = __ballot_sync(FULL, !(z[2 + e] <= thr[e])) & column;
                if (2 * c + e < G) {
                    const size_t at = list + e * row_len + n[e];
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
                }
                n[e] += __popc(lo) + __popc(hi);
            }
        };
        // The first tiles of a share are tested together, against the largest
        // score that the warps of the head have met in theirs (alone, a warp
        // lists nearly all of them, and the tau kernel has to drop them again:
        // entmax over 4 x 128k tokens took 206 us so, and 163 with it).
        auto settle = [&] {
#pragma unroll
            for (int e = 0; e < NE; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(FULL, m[e], o));
                if (a.zmax) {
                    if (r == 0 && 2 * c + e < G && m[e] > -INFINITY) atomicMax(a.zmax + h0 + 2 * c + e, f2ord(m[e]));
                    known[e] = ord2f(__ldcg(a.zmax + h0 + (2 * c + e) % G));
                }
                thr[e] = no_weight(fmaxf(m[e], known[e]));
            }
            __syncwarp();
#pragma unroll 1
            for (int k = 0; k < held; ++k) {
                const float *from = early[warp] + k * 16 * G;
                float z[4];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if ((v & 1) < NE) z[v] = from[(r + 8 * (v >> 1)) * G + (2 * c + (v & 1)) % G];
                test(z, early_row[warp][k] + r);
            }
            held = -1;
        };
        for (int i = 0; i < stages; ++i) {
            const int2 *whats;
            const unsigned char *stage;
            if (!ring.take(a, whats, stage)) {
                ring.drain(a);
                alive = false;  // the shares end empty, so that what reads them finds them whole
                break;
            }
            if (a.zmax && (i & 1)) {  // used two stages on: nothing waits for the load
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    known[e] = fmaxf(known[e], ord2f(next[e]));
                    thr[e] = no_weight(fmaxf(m[e], known[e]));
                    next[e] = __ldcg(a.zmax + h0 + (2 * c + e) % G);
                }
            }
#pragma unroll 1
            for (int page = 0; page < a.npg; ++page, stage += page_bytes) {
                const int2 what = whats[page];
                const int mask = what.y >> 8;
                int left = what.y & 0xff;
                unsigned row = (unsigned)what.x + r;
#pragma unroll 1
                for (const unsigned char *tile = stage; left > 0; left -= 16, tile += Kv4<D>::TILE, row += 16) {
                    float z[4];
                    tile_scores<D, G>(tile, Q, a.one, z);
                    if (!whole<G>(mask, left)) mask_scores<G>(mask, left, z);
                    if (held < 0) {
                        test(z, row);
                        continue;
                    }
                    float *to = early[warp] + held * 16 * G;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if ((v & 1) < NE && 2 * c + (v & 1) < G) to[(r + 8 * (v >> 1)) * G + 2 * c + (v & 1)] = z[v];
                    if (r == 0) early_row[warp][held] = row;
#pragma unroll
                    for (int e = 0; e < NE; ++e) m[e] = fmaxf(m[e], fmaxf(z[e], z[2 + e]));
                    if (++held == EARLY) settle();
                }
            }
            __syncwarp();
            if (i + RING_STAGES < stages) ring.issue(a, sh, i + RING_STAGES);
        }
        if (held >= 0) settle();
        walk = places[warp].walk;
        const size_t slot = a.kv0 * slots_per_head(a.B) + sh.slot;
        if (lane == 0) report_slot(a, sh);
#pragma unroll
        for (int e = 0; e < NE; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(FULL, m[e], o));
            // a NaN stays a candidate: its share may not be passed over for a low max
            if (__ballot_sync(FULL, bad[e]) & column) m[e] = __int_as_float(0x7fc00000);
            if (r == 0 && 2 * c + e < G)
                a.seg[slot * G + 2 * c + e] = make_int4(n[e], __float_as_int(m[e]), sh.first * (16 * a.ct), 0);
        }
    }
}

constexpr int TK_CAP = 4096;   // candidates held on chip
constexpr int TK_PASS = 1024;  // listed ones that the CTA takes at a time
constexpr int TK_BINS = 1024;

// One CTA a head: the candidates above the head's max - 1 in token order, their
// threshold, and the sum of p v over the support.  Where more of them are than
// fit on chip, a histogram first raises the cut: with every z of a bin
// taken for its lower edge e, the largest edge t with sum (e - t)_+^r >= 1 is
// below tau (alpha = 1.25 over 120k tokens: 1.7 ms without).  tau and what is
// held on chip are relative to the head's max: x = z - max in [-1, 0].
// What else the shares have listed depends on when they heard of each other's
// max, so nothing goes by the lists' lengths: the path is chosen by the number
// above the final cut, and a candidate's thread by its rank among those.
template <int D, int TK_NT>
__global__ void __launch_bounds__(TK_NT) kv4_tau_kernel(const __grid_constant__ Kv4DecodeArgs a) {
    pdl_wait();
    constexpr int TK_NW = TK_NT / 32, TK_EACH = TK_PASS / TK_NT;
    constexpr int NG = Kv4<D>::NG;
    extern __shared__ int dyn[];
    float *cz = reinterpret_cast<float *>(dyn);                     // [TK_CAP] the candidates' x ...
    unsigned *crow = reinterpret_cast<unsigned *>(dyn + TK_CAP);    // [TK_CAP] ... and their value rows
    __shared__ float o_sh[TK_NW][D];
    __shared__ float red[2][TK_NW][2];
    __shared__ float s_max[TK_NW];
    __shared__ int s_n[TK_NW * TK_EACH + 1];
    __shared__ int scan[72];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.Hq / a.Hkv;
    int b, h;
    head_of(blockIdx.x, a.kv0 * G, a.nk * G, b, h);
    const int bh = b * a.Hq + h, kvh = h / G;
    const float nan = __int_as_float(0x7fc00000);
    const uint16_t qb = threadIdx.x < D ? a.q[(size_t)bh * D + threadIdx.x] : (uint16_t)0;
    const GroupShares gs = group_shares(a, b, kvh);
    const int W = gs.n;
    const int4 *seg = a.seg + gs.slot * G + h % G;
    // place of each share's candidates among the head's, and in the head's list
    int *seg_at = dyn + 2 * TK_CAP, *seg_base = seg_at + W + 1;
    const bool fine = __syncthreads_and((qb & 0x7f80u) != 0x7f80u);
    if (!fine && threadIdx.x == 0) atomicOr(a.status, ENTMAXKV_STATUS_NONFINITE);

    float zmax = -INFINITY;
    int listed = 0;
    for (int i = threadIdx.x; i < W; i += TK_NT) {
        const int4 s = __ldcg(seg + (size_t)i * G);
        zmax = fmaxf(zmax, __int_as_float(s.y));
        listed |= s.x;
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

    const float r = 1.f / (a.alpha - 1.f);
    const int ri = a.r_int;
    const float thr = no_weight(zmax);
    float cut = -1.f;  // x below it carry no weight
    auto kept = [&](float z) { return !(z <= thr) && !(z - zmax < cut); };  // NaN stays
    float *zl = a.cand_z + (size_t)bh * a.max_pages * a.P;
    unsigned *rl = a.cand_row + (size_t)bh * a.max_pages * a.P;
    // listed candidates of a share that reaches the cut
    auto seg_size = [&](int w) {
        const int4 s = __ldcg(seg + (size_t)w * G);
        seg_base[w] = s.z;
        return __int_as_float(s.y) <= thr ? 0 : s.x;
    };
    // exclusive sums of f(w) over the shares, in seg_at; returns the total
    auto place = [&](auto f) {
        long long all = 0;
        for (int w0 = 0; w0 < W; w0 += TK_NT) {
            const int w = w0 + threadIdx.x;
            const int k = w < W ? f(w) : 0;
            int tot;
            const int at = block_excl_scan(k, scan, &tot);
            if (w < W) seg_at[w] = (int)all + at;
            all += tot;
        }
        if (threadIdx.x == 0) seg_at[W] = (int)all;
        __syncthreads();
        return (int)all;
    };
    const int R = place(seg_size);
    int nc;
    bool onchip = true, bad = false;
    // the kept candidates, a warp a share, once the lists hold no others:
    // f(place, index in the head's list)
    auto each = [&](auto f) {
        for (int w = warp; w < W; w += TK_NW) {
            const int at = seg_at[w], n = seg_at[w + 1] - at, src = seg_base[w];
#pragma unroll 4
            for (int i = lane; i < n; i += 32) f(at + i, src + i);
        }
    };
    if (R <= TK_CAP) {
        // the lists as one range, TK_EACH places a thread at a time
        nc = 0;
        for (int base = 0; base < R; base += TK_NT * TK_EACH) {
            float z[TK_EACH];
            unsigned row[TK_EACH];
#pragma unroll
            for (int u = 0; u < TK_EACH; ++u) {
                const int i = base + u * TK_NT + threadIdx.x;
                z[u] = -INFINITY;
                row[u] = 0u;
                if (i < R) {
                    int lo = 0, hi = W - 1;
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (seg_at[mid] <= i) lo = mid;
                        else hi = mid - 1;
                    }
                    const int at = seg_base[lo] + i - seg_at[lo];
                    z[u] = __ldcg(zl + at);
                    row[u] = __ldcg(rl + at);
                }
            }
            unsigned keep[TK_EACH];
#pragma unroll
            for (int u = 0; u < TK_EACH; ++u) {
                bad |= z[u] != z[u];
                keep[u] = __ballot_sync(FULL, kept(z[u]));
                if (lane == 0) s_n[u * TK_NW + warp] = __popc(keep[u]);
            }
            __syncthreads();
            if (threadIdx.x < 32) {
                static_assert(TK_EACH * TK_NW == 32, "a warp scans the counts");
                const int k = s_n[lane];
                int x = k;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(FULL, x, o);
                    if (lane >= o) x += y;
                }
                s_n[lane] = x - k;
                if (lane == 31) s_n[32] = x;
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < TK_EACH; ++u) {
                const int k = nc + s_n[u * TK_NW + warp] + __popc(keep[u] & ((1u << lane) - 1u));
                if (kept(z[u])) {
                    cz[k] = z[u] - zmax;
                    crow[k] = row[u];
                }
            }
            nc += s_n[32];
            __syncthreads();
        }
    } else {
        int *bins = dyn;
        for (int i = threadIdx.x; i < TK_BINS; i += TK_NT) bins[i] = 0;
        __syncthreads();
        for (int w = warp; w < W; w += TK_NW) {
            const int n = seg_size(w), src = seg_base[w];
#pragma unroll 4
            for (int i = lane; i < n; i += 32) {
                const float z = __ldcg(zl + src + i);
                if (z > thr) atomicAdd(&bins[min((int)(fmaxf(z - zmax + 1.f, 0.f) * TK_BINS), TK_BINS - 1)], 1);
            }
        }
        __syncthreads();
        int mine = 0, above;
        for (int i = threadIdx.x; i < TK_BINS; i += TK_NT) mine += bins[i];
        block_excl_scan(mine, scan, &above);
        int lo = 0;
        for (int top = above > TK_CAP ? TK_BINS - 1 : 0; lo < top;) {
            const int mid = (lo + top + 1) >> 1;
            __syncthreads();
            float sum = 0.f;
            for (int i = mid + threadIdx.x; i < TK_BINS; i += TK_NT)
                sum += bins[i] * pos_pow((i - mid) * (1.f / TK_BINS), r, ri);
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
            if (lane == 0) s_max[warp] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int w = 0; w < TK_NW; ++w) sum += s_max[w];
            if (sum >= 1.001f) lo = mid;
            else top = mid - 1;
        }
        __syncthreads();
        cut = fmaxf(-1.f, lo * (1.f / TK_BINS) - 1.f - 1e-6f);
        // each share's list without what is below the cut; how many stay, and where they go
        for (int w = warp; w < W; w += TK_NW) {
            const int n = seg_size(w);
            float *zs = zl + seg_base[w];
            unsigned *rs = rl + seg_base[w];
            int k = 0;
            for (int i0 = 0; i0 < n; i0 += 128) {
                float z[4];
                unsigned row[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = i0 + 32 * u + lane;
                    z[u] = i < n ? __ldcg(zs + i) : -INFINITY;
                    row[u] = i < n ? __ldcg(rs + i) : 0u;
                }
                __syncwarp();  // the pieces' places are read before any is written over
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool keep = kept(z[u]);
                    const unsigned bal = __ballot_sync(FULL, keep);
                    bad |= z[u] != z[u];
                    if (keep) {
                        const int to = k + __popc(bal & ((1u << lane) - 1u));
                        zs[to] = z[u];
                        rs[to] = row[u];
                    }
                    k += __popc(bal);
                }
            }
            __syncwarp();
            if (lane == 0) seg_at[w] = k;
        }
        __syncthreads();
        nc = place([&](int w) { return seg_at[w]; });
        onchip = nc <= TK_CAP;
        if (onchip)
            each([&](int at, int i) {
                cz[at] = __ldcg(zl + i) - zmax;
                crow[at] = __ldcg(rl + i);
            });
    }
    if (__syncthreads_or(bad)) {
        for (int j = threadIdx.x; j < D; j += TK_NT) a.out[(size_t)bh * D + j] = nan;
        if (threadIdx.x == 0 && a.tau_out) a.tau_out[bh] = nan;
        return;
    }
    const float hi = -powf((float)nc, 1.f - a.alpha);
    float tau = cut;
    EntmaxEdge edge;  // alpha > 2
    edge.lo = edge.hi = cut;
    if (nc > 1 && hi > cut) {
        // off chip every thread adds the candidates of its place, pass by pass
        auto solve = [&](auto for_each) {
            if (r >= 1.f) {
                tau = entmax_tau<TK_NT>(for_each, nc, cut, hi, 0.f, r, ri, red);
            } else {
                edge = entmax_tau_halving<TK_NT>(for_each, cut, hi, r, red);
                tau = (float)edge.lo;
            }
        };
        if (onchip) solve([&](auto add, int f, int st) { for (int i = f; i < nc; i += st) add(cz[i]); });
        else solve([&](auto add, int, int) { each([&](int, int i) { add(__ldcg(zl + i) - zmax); }); });
    }
    if (threadIdx.x == 0 && a.tau_out) a.tau_out[bh] = zmax + tau;
    auto weight = [&](float x) { return r >= 1.f ? pos_pow(x - tau, r, ri) : edge.weight(x, r); };

    // p v over the support.  A value word holds 4 coordinates of both tokens
    // of a pair: one word a lane is a row (d = 128), half a warp a row (64).
    constexpr int LPR = D / 4;        // lanes of a row
    constexpr int RPW = 32 / LPR;     // rows of a warp at a time
    const int ll = lane % LPR, sub = lane / LPR;
    const int piece = ll / Kv4<D>::WPL, wi = ll % Kv4<D>::WPL;
    // In fp32: a warp adds its share of a support that is mostly a few dozen tokens,
    // and outputs are 3 to 6e-7 off with it, as far as the scores' own rounding puts them.
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const size_t block = (size_t)(a.P / 16) * Kv4<D>::TILE;
    auto add_row = [&](float p, unsigned row) {
        const unsigned blk = row / (unsigned)a.P;
        const int slot = (int)(row - blk * a.P), t = slot & 15, pair = t >> 1;
        const unsigned char *tile = a.v4 + ((size_t)blk * a.Hkv + kvh) * block + (size_t)(slot >> 4) * Kv4<D>::TILE;
        // the lane's coordinate block keeps its place: read the word that holds it
        const unsigned w =
            __ldg(reinterpret_cast<const unsigned *>(tile) + pair * (D / 4) +
                  (piece ^ kv4_vswz<D>(pair)) * Kv4<D>::WPL + wi) >>
            (16 * (t & 1));
        const unsigned pr = __ldg(reinterpret_cast<const unsigned *>(tile + Kv4<D>::CODES) + t * NG + (wi >> 1));
        const float s = p * bf16lo(pr), lo = p * bf16hi(pr);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += fmaf(s, (float)((w >> (4 * i)) & 15u), lo);
    };
    if (onchip) {
        // the support alone, its weights and rows in place
        int ns = 0;
        for (int i0 = 0; i0 < nc; i0 += TK_NT) {
            const int i = i0 + threadIdx.x;
            const float p = i < nc ? weight(cz[i]) : 0.f;
            const unsigned row = i < nc ? crow[i] : 0u;
            const unsigned keep = __ballot_sync(FULL, p > 0.f);
            if (lane == 0) s_n[warp] = __popc(keep);
            __syncthreads();
            int at = ns;
#pragma unroll
            for (int w = 0; w < TK_NW; ++w) {
                if (w < warp) at += s_n[w];
                ns += s_n[w];
            }
            if (p > 0.f) {
                at += __popc(keep & ((1u << lane) - 1u));
                cz[at] = p;
                crow[at] = row;
            }
            __syncthreads();
        }
#pragma unroll 4
        for (int i = warp * RPW + sub; i < ns; i += TK_NW * RPW) add_row(cz[i], crow[i]);
    } else {
        for (int w = warp; w < W; w += TK_NW) {
            const int n = seg_at[w + 1] - seg_at[w], src = seg_base[w];
#pragma unroll 4
            for (int i = sub; i < n; i += RPW) {
                const float p = weight(__ldcg(zl + src + i) - zmax);
                if (p > 0.f) add_row(p, __ldcg(rl + src + i));
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

// Warps that share the chunks of a call over nk kv heads, on `ctas` CTAs an SM:
// the grid fills the GPU once, unless that leaves fewer than AT_MIN_CHUNKS
// chunks to a warp or cuts each group's list in more than AT_GROUP_PARTS.
void share_out(Kv4DecodeArgs &a, int sms, int ctas) {
    const long long groups = (long long)a.B * a.nk;
    const long long chunks = (groups * a.max_pages) << a.lc;
    long long W = (long long)sms * ctas * AT_WARPS;
    if (W > AT_MAX_WARPS) W = AT_MAX_WARPS;
    if (W > groups * AT_GROUP_PARTS) W = groups * AT_GROUP_PARTS;
    if (W > (chunks + AT_MIN_CHUNKS - 1) / AT_MIN_CHUNKS) W = (chunks + AT_MIN_CHUNKS - 1) / AT_MIN_CHUNKS;
    a.W = (int)W;
    a.S = 0;
    if (a.union_e || a.sel) {
        a.S = (int)(W / groups > 1 ? W / groups : 1);
        if (a.S * groups < W) a.W = (int)(a.S * groups);
    }
}

struct Carve {
    size_t part_o, part_ml, cand_z, cand_row, seg, slots, union_e, union_blk, union_cnt, zmax, counters, total;
};

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
    const size_t rows = s->Hq * slots_per_head(s->B);
    c.part_o = take(rows * s->d * 4);
    c.part_ml = take(rows * 8);
    c.cand_z = take(tokens * 4);
    c.cand_row = take(tokens * 4);
    c.seg = take(rows * 16);
    c.slots = take(groups * 8);
    c.union_e = take(groups * s->max_pages * 4);
    c.union_blk = take(groups * s->max_pages * 4);
    c.union_cnt = take(groups * 4);
    c.zmax = take(heads * 4);
    c.counters = take(groups * 4);
    c.total = off;
    return c;
}

template <class K>
cudaError_t run_shares(K k, const Kv4DecodeArgs &a, int warps, size_t ring, cudaStream_t st) {
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(k), warps * ring);
    return e != cudaSuccess ? e : launch_pdl(k, dim3(ceil_div(a.W, warps)), dim3(32 * warps), warps * ring, st, a);
}

template <int D, int G>
cudaError_t decode_t(Kv4DecodeArgs a, int sms, cudaStream_t st) {
    const int groups = a.B * a.nk, heads = groups * G;
    cudaError_t e;
    if (a.alpha == 1.f) {
        constexpr size_t ring = TileRing<D, true>::BYTES;
        // Short lists, or enough groups that a CTA for each fills the GPU: one
        // launch, each CTA a group.  us, so and cut over the GPU: 2 groups of
        // 701 tokens 11.3 and 15.6 (one call after another, the host's time
        // counts), 64 of 1500 16.5 and 20.6, 128 of 3000 23.2 and 27.3; but 16
        // of 1500 18.5 and 16.6, 8 of 3000 20.6 and 14.4
        const int tiles = a.max_pages * (a.ct << a.lc);
        if (groups <= sms && tiles <= WHOLE_WARPS * (3 * groups >= sms ? WHOLE_TILES : WHOLE_FEW)) {
            a.S = WHOLE_WARPS;
            a.W = groups * WHOLE_WARPS;
            return run_shares(kv4_softmax_kernel<D, G, WHOLE_WARPS, true>, a, WHOLE_WARPS, ring, st);
        }
        share_out(a, sms, softmax_ctas<D, G>());
        e = run_shares(kv4_softmax_kernel<D, G, AT_WARPS, false>, a, AT_WARPS, ring, st);
        if (e != cudaSuccess) return e;
        // heads of many shares get more threads while every SM has a place for
        // one (24 heads of 512 shares: 31 us in all with 1024 threads, 49 with
        // 256; 8 heads of 22 shares: 12.6 and 10.6)
        const bool few = heads <= sms && (long long)a.W > 64ll * a.B * a.nk;
        return launch_pdl(few ? kv4_combine_kernel<D, 1024> : kv4_combine_kernel<D, 256>, dim3(heads),
                          dim3(few ? 1024 : 256), (size_t)a.W * 4, st, a);
    }
    share_out(a, sms, SCAN_CTAS);
    // short shares list little that a common max would have cut: no launch to reset it
    const bool given = a.union_e;  // the union's kernel has reset it
    if (!given && ((long long)a.B * a.nk * a.max_pages) << a.lc < 4ll * a.W) a.zmax = nullptr;
    if (a.zmax && !given) {
        e = launch_pdl(kv4_reset_kernel, dim3(ceil_div(heads, 256)), dim3(256), 0, st, a);
        if (e != cudaSuccess) return e;
    }
    if ((e = run_shares(kv4_scan_kernel<D, G>, a, AT_WARPS, TileRing<D, false>::BYTES, st)) != cudaSuccess) return e;
    const size_t smem = (size_t)(2 * TK_CAP + 2 * a.W + 1) * 4;
    // More threads a head while every head's CTA finds a place at once (128
    // heads: 22 us with 512 threads, 25 with 256; 512 heads: 19 and 11)
    const bool many = heads > 2 * sms;
    auto k = many ? kv4_tau_kernel<D, 256> : kv4_tau_kernel<D, 512>;
    if ((e = ensure_smem(reinterpret_cast<const void *>(k), smem)) != cudaSuccess) return e;
    return launch_pdl(k, dim3(heads), dim3(many ? 256 : 512), smem, st, a);
}

template <int D>
cudaError_t decode_d(const Kv4DecodeArgs &a, int sms, cudaStream_t st) {
    switch (a.Hq / a.Hkv) {
        case 1: return decode_t<D, 1>(a, sms, st);
        case 2: return decode_t<D, 2>(a, sms, st);
        case 4: return decode_t<D, 4>(a, sms, st);
        default: return decode_t<D, 8>(a, sms, st);
    }
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
    a.part_o = reinterpret_cast<float *>(w + c.part_o);
    a.part_ml = reinterpret_cast<float2 *>(w + c.part_ml);
    a.cand_z = reinterpret_cast<float *>(w + c.cand_z);
    a.cand_row = reinterpret_cast<unsigned *>(w + c.cand_row);
    a.seg = reinterpret_cast<int4 *>(w + c.seg);
    a.slots = reinterpret_cast<int2 *>(w + c.slots);
    a.zmax = reinterpret_cast<int *>(w + c.zmax);
    a.B = s->B;
    a.Hq = s->Hq;
    a.Hkv = s->Hkv;
    a.P = s->page_size;
    a.max_pages = s->max_pages;
    a.num_blocks = s->num_blocks;
    kv_range(s, &a.kv0, &a.nk);
    a.ct = s->page_size == 16 ? 1 : 2;
    a.lc = s->page_size == 64 ? 1 : 0;
    a.npg = 64 / s->page_size;
    a.alpha = alpha;
    a.r_int = alpha > 1.f ? integer_r(alpha) : 0;
    a.one = 0x64006400u;
    a.status = di.status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (sel && s->Hq == s->Hkv) {  // a head's own list is its group's
        a.sel = sel;
        a.cnt = cnt;
    } else if (sel) {
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
    const cudaError_t e = s->d == 64 ? decode_d<64>(a, di.sms, st) : decode_d<128>(a, di.sms, st);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_ERR_CUDA;
}

}  // extern "C"
