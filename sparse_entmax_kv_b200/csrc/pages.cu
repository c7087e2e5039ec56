// pages.cu -- copying, forking, growing, compacting and freeing the pages of a
// cache (include/entmaxkv_pages.h), and their C entry points.
//
// Which blocks are free follows from the page table alone: the rows' blocks
// are marked in a bitmap (one bit a block), and one CTA turns the bitmap and
// the rows' needs into a plan (prefix sums in row and block order, so nothing
// depends on timing).  A second launch carries the plan out: new rows,
// metadata records, and the (src, dst) block pairs in every buffer, bound by
// memory bandwidth: 16-byte loads, several in flight a thread, row x tile and
// pair x buffer x chunk spread over a grid that fills the GPU.  With tables of
// up to SMALL_TABLE entries the planning CTA marks the blocks itself, in
// shared memory, and the two (grow: one) launches are all; larger ones are
// marked by the whole GPU in two launches before the plan.
#include <cstring>

#include "../../include/entmaxkv_pages.h"
#include "common.cuh"
#include "internal.h"

namespace ekv {

namespace {

constexpr int PL_NT = 1024;  // threads of the planning CTA
constexpr int SMALL_TABLE = 65536;   // entries, and ...
constexpr int SMALL_WORDS = 7168;    // ... words of the bitmap that it marks itself (28 KB, beside 17 KB of plan)
constexpr int SMALL_ROWS = 1024;     // rows whose plan stays in shared memory
constexpr int MV_NT = 256;
constexpr int MV_UNROLL = 8;
constexpr long long MV_CHUNK = (long long)MV_NT * MV_UNROLL * 16;  // bytes a CTA moves at a time

struct PageArgs {
    int B, P, max_pages, num_blocks;
    const int *table_in, *lens_in, *hold, *parent, *n_add;
    int *table_out, *lens_out;
    int in_place;
    unsigned *bits;      // [words] blocks in use
    int small;           // the planning CTA marks them itself
    int words;
    int *act;            // [B] parent each row really follows (-1: empty)
    int *fresh;          // [B] block of the row's copied page, -1 none left, -2 none needed
    int *first;          // [B] row that keeps the parent's partial page
    int *list;           // [num_blocks] free blocks, ascending
    int *pair_src, *pair_dst, *n_pairs;
    int *refs, *n_free, *remap, *n_live;
    int *status;
};

__device__ __forceinline__ int row_pages(const PageArgs &a, int b) {
    return n_pages_of(seq_len_of(a.lens_in, b, a.P, a.max_pages, a.status), a.P);
}
__device__ __forceinline__ bool block_ok(const PageArgs &a, int blk) { return blk >= 0 && blk < a.num_blocks; }

__global__ void clear_kernel(int *p, int n) {
    pdl_wait();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) p[i] = 0;
}

// Marks the blocks of the table's entries i0, i0 + step, ... and the held ones.
// I: 32 bits where the table is small (an entry's row is a division).
template <class I>
__device__ __forceinline__ void mark_blocks(const PageArgs &a, unsigned *bits, int i0, int step) {
    const I n = (I)a.B * (I)a.max_pages;
    const int cap = a.max_pages * a.P;
#pragma unroll 4
    for (I i = i0; i < n; i += step) {
        const int b = (int)(i / (unsigned)a.max_pages), p = (int)(i - (I)b * (unsigned)a.max_pages);
        const int len = __ldg(a.lens_in + b), blk = __ldg(a.table_in + i);
        if (p == 0 && len > cap) atomicOr(a.status, ENTMAXKV_STATUS_BAD_LENGTH);
        if ((long long)p * a.P >= len) continue;
        if (block_ok(a, blk)) atomicOr(&bits[blk >> 5], 1u << (blk & 31));
        else atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
    }
    if (a.hold)
        for (int i = i0; i < a.num_blocks; i += step)
            if (a.hold[i] > 0) atomicOr(&bits[i >> 5], 1u << (i & 31));
}
__global__ void mark_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    mark_blocks<long long>(a, a.bits, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
}

// The bitmap of blocks in use, as the planning CTA has it: marked before, or
// (small tables) marked here, in shared memory.
__device__ unsigned *marked_bits(const PageArgs &a, unsigned *sh) {
    if (!a.small) return a.bits;
    for (int i = threadIdx.x; i < a.words; i += PL_NT) sh[i] = 0u;
    __syncthreads();
    mark_blocks<unsigned>(a, sh, threadIdx.x, PL_NT);
    __syncthreads();
    return sh;
}

__global__ void refs_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int n = row_pages(a, b);
        for (int p = threadIdx.x; p < n; p += blockDim.x) {
            const int blk = a.table_in[(size_t)b * a.max_pages + p];
            if (block_ok(a, blk)) atomicAdd(&a.refs[blk], 1);
            else atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
        }
    }
    if (a.hold)
        for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.num_blocks; i += gridDim.x * blockDim.x)
            if (a.hold[i] > 0) atomicAdd(&a.refs[i], a.hold[i]);
}

__global__ void __launch_bounds__(PL_NT) count_free_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    __shared__ int sh[72];
    int n = 0, tot;
    for (int i = threadIdx.x; i < a.num_blocks; i += PL_NT) n += a.refs[i] == 0;
    block_excl_scan(n, sh, &tot);
    if (threadIdx.x == 0) *a.n_free = tot;
}

// Bits of word w that stand for blocks.
__device__ __forceinline__ unsigned word_mask(const PageArgs &a, int w) {
    const int left = a.num_blocks - 32 * w;
    return left >= 32 ? 0xffffffffu : (1u << left) - 1u;
}

// The first `want` free blocks, ascending, into list; returns how many.
__device__ int list_free(const PageArgs &a, const unsigned *bits, long long want, int *list, int *sh) {
    long long found = 0;
    for (int w0 = 0; w0 < a.words && found < want; w0 += PL_NT) {
        const int w = w0 + threadIdx.x;
        unsigned f = w < a.words ? ~bits[w] & word_mask(a, w) : 0u;
        int tot;
        long long at = found + block_excl_scan(__popc(f), sh, &tot);
        for (; f && at < want; f &= f - 1u, ++at) list[at] = 32 * w + __ffs(f) - 1;
        found += tot;
    }
    __syncthreads();  // the list is read by other threads of the CTA
    return (int)(found < want ? found : want);
}

__global__ void __launch_bounds__(PL_NT) plan_fork_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    extern __shared__ unsigned map[];
    __shared__ int sh[72];
    __shared__ int s_act[SMALL_ROWS], s_first[SMALL_ROWS], s_list[SMALL_ROWS], s_len[SMALL_ROWS];
    const bool few = a.B <= SMALL_ROWS;
    int *act = few ? s_act : a.act, *first = few ? s_first : a.first, *list = few ? s_list : a.list;
    for (int b = threadIdx.x; b < a.B; b += PL_NT) {
        int p = a.parent[b];
        bool bad = p < -1 || p >= a.B;
        if (a.in_place && !bad && p >= 0 && p != b) bad = a.parent[p] != p;
        if (bad) {
            atomicOr(a.status, ENTMAXKV_STATUS_BAD_ROW);
            p = a.in_place ? b : -1;
        }
        act[b] = p;
        if (few) {
            a.act[b] = p;
            s_len[b] = seq_len_of(a.lens_in, b, a.P, a.max_pages, nullptr);
        }
        first[b] = 0x7fffffff;
    }
    const unsigned *bits = marked_bits(a, map);
    __syncthreads();
    // the parent's own row keeps the partial page, else the first child
    for (int b = threadIdx.x; b < a.B; b += PL_NT) {
        const int p = act[b];
        if (p >= 0) atomicMin(&first[p], p == b ? -1 : b);
    }
    __syncthreads();
    auto length = [&](int p) { return few ? s_len[p] : seq_len_of(a.lens_in, p, a.P, a.max_pages, nullptr); };
    auto needs = [&](int b) {
        if (b >= a.B) return 0;
        const int p = act[b];
        return p >= 0 && length(p) % a.P != 0 && first[p] != (p == b ? -1 : b) ? 1 : 0;
    };
    long long want = 0;
    for (int b0 = 0; b0 < a.B; b0 += PL_NT) {
        int tot;
        block_excl_scan(needs(b0 + threadIdx.x), sh, &tot);
        want += tot;
    }
    const int have = list_free(a, bits, want < a.num_blocks ? want : a.num_blocks, list, sh);
    int rank = 0, pairs = 0;
    for (int b0 = 0; b0 < a.B; b0 += PL_NT) {
        const int b = b0 + threadIdx.x;
        int src = -1, tot, n_pairs;
        const int need = needs(b);
        if (need) src = __ldg(a.table_in + (size_t)act[b] * a.max_pages + length(act[b]) / a.P);
        const int at = rank + block_excl_scan(need, sh, &tot);
        rank += tot;
        int blk = -2;
        if (need) {
            blk = at < have ? list[at] : -1;
            if (blk < 0) atomicOr(a.status, ENTMAXKV_STATUS_NO_BLOCK);
        }
        const bool copy = blk >= 0 && block_ok(a, src);
        const int k = pairs + block_excl_scan(copy, sh, &n_pairs);
        pairs += n_pairs;
        if (copy) {
            a.pair_src[k] = src;
            a.pair_dst[k] = blk;
        }
        if (b < a.B) a.fresh[b] = blk;
    }
    if (threadIdx.x == 0) *a.n_pairs = pairs;
}

__global__ void __launch_bounds__(PL_NT) plan_grow_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    extern __shared__ unsigned map[];
    __shared__ int sh[72];
    __shared__ long long s_sum[PL_NT / 32];
    __shared__ int s_list[SMALL_ROWS];
    const long long cap = (long long)a.max_pages * a.P;
    // pages sequence b needs, its pages and new length; -1: it does not grow
    auto need = [&](int b, int &n0, long long &L) {
        if (b >= a.B) return -1;
        const int add = a.n_add[b];
        if (add <= 0) return -1;
        const int L0 = seq_len_of(a.lens_in, b, a.P, a.max_pages, nullptr);
        L = (long long)L0 + add;
        if (L > cap) {
            atomicOr(a.status, ENTMAXKV_STATUS_BAD_LENGTH);
            return -1;
        }
        n0 = n_pages_of(L0, a.P);
        return (int)((L + a.P - 1) / a.P) - n0;
    };
    // inclusive sums in 64 bits, and their total
    auto scan64 = [&](long long x, long long &total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) s_sum[warp] = x;
        __syncthreads();
        total = 0;
#pragma unroll 4
        for (int w = 0; w < PL_NT / 32; ++w) {
            if (w < warp) x += s_sum[w];
            total += s_sum[w];
        }
        return x;
    };
    long long want = 0, tot, L = 0, end = 0;
    int n0 = 0, k = need(threadIdx.x, n0, L);  // of the first rows, which mostly are all
    const unsigned *bits = marked_bits(a, map);
    end = scan64(max(0, k), tot);
    want = tot;
    const long long first = tot;
    for (int b0 = PL_NT; b0 < a.B; b0 += PL_NT) {
        int n;
        long long l;
        scan64(max(0, need(b0 + threadIdx.x, n, l)), tot);
        want += tot;
    }
    int *list = want <= SMALL_ROWS ? s_list : a.list;
    const int have = list_free(a, bits, want < a.num_blocks ? want : a.num_blocks, list, sh);
    long long used = first;
    for (int b0 = 0; b0 < a.B; b0 += PL_NT) {
        const int b = b0 + threadIdx.x;
        if (b0) {
            k = need(b, n0, L);
            end = used + scan64(max(0, k), tot);
            used += tot;
        }
        if (end > have && k > 0) {
            atomicOr(a.status, ENTMAXKV_STATUS_NO_BLOCK);
            k = -1;
        }
        // the warp's rows one after another, a lane a page
        for (unsigned some = __ballot_sync(FULL, k > 0); some; some &= some - 1u) {
            const int l = __ffs(some) - 1, kk = __shfl_sync(FULL, k, l);
            const long long from = __shfl_sync(FULL, end, l) - kk;
            int *row = a.table_out + (size_t)__shfl_sync(FULL, b, l) * a.max_pages + __shfl_sync(FULL, n0, l);
            for (int i = threadIdx.x & 31; i < kk; i += 32) row[i] = list[from + i];
        }
        if (k >= 0) a.lens_out[b] = (int)L;
    }
}

__global__ void __launch_bounds__(PL_NT) plan_compact_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    extern __shared__ unsigned map[];
    __shared__ int sh[72];
    const unsigned *bits = marked_bits(a, map);
    int n = 0, n_live;
    for (int w = threadIdx.x; w < a.words; w += PL_NT) n += __popc(bits[w]);
    block_excl_scan(n, sh, &n_live);
    int holes = 0, moves = 0;
    for (int w0 = 0; w0 < a.words; w0 += PL_NT) {
        const int w = w0 + threadIdx.x;
        const unsigned live = w < a.words ? bits[w] : 0u;
        const unsigned valid = w < a.words ? word_mask(a, w) : 0u;
        const int left = n_live - 32 * w;  // blocks of the word below n_live
        const unsigned low = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
        int th, tm;
        int h = holes + block_excl_scan(__popc(~live & valid & low), sh, &th);
        int m = moves + block_excl_scan(__popc(live & ~low), sh, &tm);
        for (unsigned f = ~live & valid & low; f; f &= f - 1u) a.pair_dst[h++] = 32 * w + __ffs(f) - 1;
        for (unsigned f = live & ~low; f; f &= f - 1u) a.pair_src[m++] = 32 * w + __ffs(f) - 1;
        holes += th;
        moves += tm;
    }
    for (int i = threadIdx.x; i < a.num_blocks; i += PL_NT)
        if (i < n_live || !((bits[i >> 5] >> (i & 31)) & 1u)) a.remap[i] = (bits[i >> 5] >> (i & 31)) & 1u ? i : -1;
    __syncthreads();  // holes == moves: the pairs are complete
    for (int i = threadIdx.x; i < moves; i += PL_NT) a.remap[a.pair_src[i]] = a.pair_dst[i];
    if (threadIdx.x == 0) {
        *a.n_live = n_live;
        *a.n_pairs = moves;
    }
}

// ------------------------------------------------------------ carrying it out

// One row of the new table.
__device__ __forceinline__ void fork_row(const PageArgs &a, int b) {
    const int p = a.act[b];
    if (a.in_place && p == b) return;
    int L = p >= 0 ? seq_len_of(a.lens_in, p, a.P, a.max_pages, nullptr) : 0;
    const int fresh = a.fresh[b];
    if (fresh == -1) L -= L % a.P;
    const int n = n_pages_of(L, a.P);
    for (int i = threadIdx.x; i < a.max_pages; i += blockDim.x) {
        int blk = -1;
        if (i < n) blk = fresh >= 0 && i == n - 1 ? fresh : a.table_in[(size_t)p * a.max_pages + i];
        a.table_out[(size_t)b * a.max_pages + i] = blk;
    }
    if (threadIdx.x == 0) a.lens_out[b] = L;
}
__device__ __forceinline__ void remap_row(const PageArgs &a, int b) {
    const int n = n_pages_of(seq_len_of(a.lens_in, b, a.P, a.max_pages, nullptr), a.P);
    for (int i = threadIdx.x; i < a.max_pages; i += blockDim.x) {
        const size_t at = (size_t)b * a.max_pages + i;
        const int blk = i < n ? a.table_in[at] : -1;
        a.table_out[at] = block_ok(a, blk) ? a.remap[blk] : -1;
    }
}

// Up to MV_CHUNK bytes (a multiple of 16), all loads before the stores.
__device__ __forceinline__ void move_chunk(const char *from, char *to, long long bytes) {
    const uint4 *src = reinterpret_cast<const uint4 *>(from);
    uint4 *dst = reinterpret_cast<uint4 *>(to);
    const int m = (int)(bytes < MV_CHUNK ? bytes : MV_CHUNK) / 16;
    uint4 v[MV_UNROLL];
#pragma unroll
    for (int u = 0; u < MV_UNROLL; ++u)
        if (u * MV_NT + threadIdx.x < m) v[u] = src[u * MV_NT + threadIdx.x];
#pragma unroll
    for (int u = 0; u < MV_UNROLL; ++u)
        if (u * MV_NT + threadIdx.x < m) dst[u * MV_NT + threadIdx.x] = v[u];
}

// Buffers that a launch has room for: its arguments are copied with it, and
// few buffers are the common case.
constexpr int FEW = 16;

template <int N>
struct ApplyArgs {
    PageArgs p;
    int bufs, metas;
    long long bytes;  // of a block
    int Hkv, n_tiles;
    long long region, tile[2];  // bytes of the bound region, and of a tile in it and in the other
    char *buf[N];
    const char *meta_in[N];
    char *meta_out[N];
};

// Rows, then metadata tiles (of both regions; they follow their rows), then
// chunks of the block pairs, item after item.
template <bool FORK, int N>
__global__ void __launch_bounds__(MV_NT, 4) apply_kernel(const __grid_constant__ ApplyArgs<N> a) {
    pdl_wait();
    const PageArgs &p = a.p;
    const long long per = (a.bytes + MV_CHUNK - 1) / MV_CHUNK;  // chunks of a block
    const long long meta0 = p.B, n_meta = FORK ? (long long)a.metas * p.B * a.Hkv * a.n_tiles : 0;
    const long long move0 = meta0 + n_meta;
    const long long total = move0 + per * a.bufs * (a.bufs ? *p.n_pairs : 0);
    for (long long k = blockIdx.x; k < total; k += gridDim.x) {
        if (k >= move0) {
            const long long pb = (k - move0) / per, off = ((k - move0) - pb * per) * MV_CHUNK;
            const int pair = (int)(pb / a.bufs);
            char *base = a.buf[pb - (long long)pair * a.bufs] + off;
            move_chunk(base + p.pair_src[pair] * a.bytes, base + p.pair_dst[pair] * a.bytes, a.bytes - off);
        } else if (k >= meta0) {
            long long i = k - meta0;
            const int t = (int)(i % a.n_tiles);
            i /= a.n_tiles;
            const int h = (int)(i % a.Hkv);
            i /= a.Hkv;
            const int b = (int)(i % p.B), m = (int)(i / p.B), from = p.act[b];
            if (from < 0 || (p.in_place && from == b)) continue;
            if ((long long)t * META_TILE * p.P >= seq_len_of(p.lens_in, from, p.P, p.max_pages, nullptr)) continue;
            const long long s = ((long long)from * a.Hkv + h) * a.n_tiles + t;
            const long long d = ((long long)b * a.Hkv + h) * a.n_tiles + t;
#pragma unroll 1
            for (int r = 0; r < 2; ++r) {
                const long long base = r ? a.region : 0;
                move_chunk(a.meta_in[m] + base + s * a.tile[r], a.meta_out[m] + base + d * a.tile[r], a.tile[r]);
            }
        } else if (FORK) {
            fork_row(p, (int)k);
        } else {
            remap_row(p, (int)k);
        }
    }
}

template <int N>
struct MoveArgs {
    const char *src[N];
    char *dst[N];
    const int *src_ids, *dst_ids;
    int n, bufs, src_blocks, dst_blocks;
    long long bytes;   // of a block
    int *status;
};

// Block pairs, every buffer: chunk after chunk of MV_CHUNK bytes.
template <int N>
__global__ void __launch_bounds__(MV_NT) move_kernel(const __grid_constant__ MoveArgs<N> a) {
    pdl_wait();
    const long long per = (a.bytes + MV_CHUNK - 1) / MV_CHUNK;  // chunks of a block
    const long long total = per * a.bufs * a.n;
    for (long long k = blockIdx.x; k < total; k += gridDim.x) {
        const long long pb = k / per, off = (k - pb * per) * MV_CHUNK;
        const int pair = (int)(pb / a.bufs), buf = (int)(pb - (long long)pair * a.bufs);
        const int s = a.src_ids[pair], d = a.dst_ids[pair];
        if (s < 0 || s >= a.src_blocks || d < 0 || d >= a.dst_blocks) {
            if (threadIdx.x == 0) atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
            continue;
        }
        move_chunk(a.src[buf] + s * a.bytes + off, a.dst[buf] + d * a.bytes + off, a.bytes - off);
    }
}

// ---------------------------------------------------------------- host side

int check_pages_shape(const entmaxkv_shape *s) {
    const int rc = check_shape(s);
    if (rc) return rc;
    return s->kv_begin || s->kv_count ? ENTMAXKV_ERR_SHAPE : ENTMAXKV_OK;
}

int check_buffers(const entmaxkv_buffers *b, bool blocks) {
    if (!b || (b->count > 0 && !b->base)) return ENTMAXKV_ERR_NULL;
    if (b->count < 0 || b->count > ENTMAXKV_MAX_BUFFERS) return ENTMAXKV_ERR_SHAPE;
    if (blocks && b->count && (b->block_bytes <= 0 || b->block_bytes % 16)) return ENTMAXKV_ERR_SHAPE;
    for (int i = 0; i < b->count; ++i) {
        if (!b->base[i]) return ENTMAXKV_ERR_NULL;
        if (!aligned16(b->base[i])) return ENTMAXKV_ERR_ALIGN;
    }
    return ENTMAXKV_OK;
}

struct Carve {
    size_t bits, act, fresh, first, list, pair_src, pair_dst, counts, refs, total;
};
Carve carve(const entmaxkv_shape *s) {
    Carve c;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off += (bytes + 255) & ~(size_t)255;
        return o;
    };
    const size_t nb = s->num_blocks, B = s->B;
    c.bits = take((nb + 31) / 32 * 4);
    c.act = take(B * 4);
    c.fresh = take(B * 4);
    c.first = take(B * 4);
    c.list = take(nb * 4);
    c.pair_src = take((nb > B ? nb : B) * 4);
    c.pair_dst = take((nb > B ? nb : B) * 4);
    c.counts = take(16);
    c.refs = take(nb * 4);
    c.total = off;
    return c;
}

// Checks of the calls that plan on a table, and what they share.
int fill_pages(const entmaxkv_shape *s, const int32_t *table, const int32_t *lens, const int32_t *hold, void *ws,
               size_t ws_bytes, PageArgs *a) {
    int rc = check_pages_shape(s);
    if (rc) return rc;
    if (!table || !lens) return ENTMAXKV_ERR_NULL;
    const Carve c = carve(s);
    if (!ws || ws_bytes < c.total) return ENTMAXKV_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return ENTMAXKV_ERR_ALIGN;
    char *w = static_cast<char *>(ws);
    *a = PageArgs{};
    a->B = s->B;
    a->P = s->page_size;
    a->max_pages = s->max_pages;
    a->num_blocks = s->num_blocks;
    a->table_in = table;
    a->lens_in = lens;
    a->hold = hold;
    a->bits = reinterpret_cast<unsigned *>(w + c.bits);
    a->words = (s->num_blocks + 31) / 32;
    a->act = reinterpret_cast<int *>(w + c.act);
    a->fresh = reinterpret_cast<int *>(w + c.fresh);
    a->first = reinterpret_cast<int *>(w + c.first);
    a->list = reinterpret_cast<int *>(w + c.list);
    a->pair_src = reinterpret_cast<int *>(w + c.pair_src);
    a->pair_dst = reinterpret_cast<int *>(w + c.pair_dst);
    a->n_pairs = reinterpret_cast<int *>(w + c.counts);
    a->refs = reinterpret_cast<int *>(w + c.refs);
    return ENTMAXKV_OK;
}

// The device's status word, once every argument has been checked.
int on_device(PageArgs *a) {
    DevInfo di;
    const int rc = device_info(&di);
    if (!rc) a->status = di.status;
    return rc;
}

constexpr int GRID = 148 * 16;  // two or more rounds of CTAs even the rows and chunks out (148 * 8: 4% slower)

// The planning launch, after the marking ones where the table is large.
template <class K>
cudaError_t plan(K k, PageArgs &a, cudaStream_t st) {
    const long long entries = (long long)a.B * a.max_pages;
    a.small = entries <= SMALL_TABLE && a.words <= SMALL_WORDS;
    if (!a.small) {
        cudaError_t e = launch_pdl(clear_kernel, dim3(min(ceil_div(a.words, 256), GRID)), dim3(256), 0, st,
                                   reinterpret_cast<int *>(a.bits), (int)a.words);
        if (e != cudaSuccess) return e;
        const long long items = a.hold && a.num_blocks > entries ? a.num_blocks : entries;
        const long long ctas = (items + 255) / 256;
        e = launch_pdl(mark_kernel, dim3((unsigned)(ctas < GRID ? ctas : GRID)), dim3(256), 0, st, a);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(k, dim3(1), dim3(PL_NT), a.small ? (size_t)a.words * 4 : 0, st, a);
}

// The second launch; pairs: how many blocks move at most.
template <bool FORK, int N>
cudaError_t apply_n(const PageArgs &p, const entmaxkv_buffers *bufs, const entmaxkv_shape *s, long long pairs,
                  const entmaxkv_buffers *meta_in, const entmaxkv_buffers *meta_out, cudaStream_t st) {
    ApplyArgs<N> a;
    a.p = p;
    a.bufs = bufs->count;
    a.bytes = bufs->count ? bufs->block_bytes : 0;
    for (int i = 0; i < bufs->count; ++i) a.buf[i] = static_cast<char *>(bufs->base[i]);
    a.metas = meta_in ? meta_in->count : 0;
    for (int i = 0; i < a.metas; ++i) {
        a.meta_in[i] = static_cast<const char *>(meta_in->base[i]);
        a.meta_out[i] = static_cast<char *>(meta_out->base[i]);
    }
    a.Hkv = s->Hkv;
    a.n_tiles = meta_tiles(s->max_pages);
    a.tile[0] = 128ll * s->d;
    a.tile[1] = 256ll * s->d;
    a.region = (long long)s->B * s->Hkv * a.n_tiles * a.tile[0];
    static_assert(256 * 128 <= MV_CHUNK, "a metadata tile is one chunk");
    const long long items = s->B + (long long)a.metas * s->B * s->Hkv * a.n_tiles +
                            (a.bytes + MV_CHUNK - 1) / MV_CHUNK * a.bufs * pairs;
    return launch_pdl(apply_kernel<FORK, N>, dim3((unsigned)(items < GRID ? items : GRID)), dim3(MV_NT), 0, st, a);
}
template <bool FORK>
cudaError_t apply(const PageArgs &p, const entmaxkv_buffers *bufs, const entmaxkv_shape *s, long long pairs,
                  const entmaxkv_buffers *meta_in, const entmaxkv_buffers *meta_out, cudaStream_t st) {
    const bool few = bufs->count <= FEW && (!meta_in || meta_in->count <= FEW);
    return few ? apply_n<FORK, FEW>(p, bufs, s, pairs, meta_in, meta_out, st)
               : apply_n<FORK, ENTMAXKV_MAX_BUFFERS>(p, bufs, s, pairs, meta_in, meta_out, st);
}

template <int N>
cudaError_t move(const entmaxkv_buffers *src, int src_blocks, const entmaxkv_buffers *dst, int dst_blocks,
                 const int *src_ids, const int *dst_ids, int n, int *status, cudaStream_t st) {
    MoveArgs<N> m;
    m.bufs = src->count;
    m.bytes = src->block_bytes;
    for (int i = 0; i < src->count; ++i) {
        m.src[i] = static_cast<const char *>(src->base[i]);
        m.dst[i] = static_cast<char *>(dst->base[i]);
    }
    m.src_ids = src_ids;
    m.dst_ids = dst_ids;
    m.n = n;
    m.src_blocks = src_blocks;
    m.dst_blocks = dst_blocks;
    m.status = status;
    const long long chunks = (m.bytes + MV_CHUNK - 1) / MV_CHUNK * m.bufs * n;
    return launch_pdl(move_kernel<N>, dim3((unsigned)(chunks < GRID ? chunks : GRID)), dim3(MV_NT), 0, st, m);
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_ERR_CUDA; }

}  // namespace

}  // namespace ekv

using namespace ekv;

extern "C" {

size_t entmaxkv_pages_workspace_size(const entmaxkv_shape *s) {
    if (check_pages_shape(s)) return (size_t)-1;
    return carve(s).total;
}

int entmaxkv_pages_refs(const entmaxkv_shape *s, const int32_t *page_table, const int32_t *seq_lens,
                        const int32_t *hold, int32_t *refs, int32_t *n_free, void *workspace, size_t ws_bytes,
                        void *stream) {
    PageArgs a;
    if (!refs && !n_free) return ENTMAXKV_ERR_NULL;
    int rc = fill_pages(s, page_table, seq_lens, hold, workspace, ws_bytes, &a);
    if (rc || (rc = on_device(&a))) return rc;
    if (refs) a.refs = refs;
    a.n_free = n_free;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pdl(clear_kernel, dim3(min(ceil_div(a.num_blocks, 256), GRID)), dim3(256), 0, st, a.refs,
                               (int)a.num_blocks);
    if (e == cudaSuccess) e = launch_pdl(refs_kernel, dim3(hold ? GRID : min(a.B, GRID)), dim3(256), 0, st, a);
    if (e == cudaSuccess && n_free) e = launch_pdl(count_free_kernel, dim3(1), dim3(PL_NT), 0, st, a);
    return rc_of(e);
}

int entmaxkv_pages_fork(const entmaxkv_shape *s, const int32_t *parent, const int32_t *table_in,
                        const int32_t *lens_in, const int32_t *hold, int32_t *table_out, int32_t *lens_out,
                        const entmaxkv_buffers *bufs, const entmaxkv_buffers *meta_in,
                        const entmaxkv_buffers *meta_out, void *workspace, size_t ws_bytes, void *stream) {
    PageArgs a;
    int rc = fill_pages(s, table_in, lens_in, hold, workspace, ws_bytes, &a);
    if (rc) return rc;
    if (!parent || !table_out || !lens_out || (meta_in == nullptr) != (meta_out == nullptr)) return ENTMAXKV_ERR_NULL;
    if ((rc = check_buffers(bufs, true))) return rc;
    a.in_place = table_out == table_in;
    if ((lens_out == lens_in) != (a.in_place != 0)) return ENTMAXKV_ERR_SHAPE;
    if (meta_in) {
        if ((rc = check_buffers(meta_in, false)) || (rc = check_buffers(meta_out, false))) return rc;
        if (meta_in->count != meta_out->count) return ENTMAXKV_ERR_SHAPE;
        for (int i = 0; i < meta_in->count; ++i)
            if ((meta_in->base[i] == meta_out->base[i]) != (a.in_place != 0)) return ENTMAXKV_ERR_SHAPE;
    }
    if ((rc = on_device(&a))) return rc;
    a.parent = parent;
    a.table_out = table_out;
    a.lens_out = lens_out;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = plan(plan_fork_kernel, a, st);
    if (e == cudaSuccess) e = apply<true>(a, bufs, s, s->B, meta_in, meta_out, st);
    return rc_of(e);
}

int entmaxkv_pages_grow(const entmaxkv_shape *s, const int32_t *n_add, const int32_t *hold, int32_t *page_table,
                        int32_t *seq_lens, void *workspace, size_t ws_bytes, void *stream) {
    PageArgs a;
    int rc = fill_pages(s, page_table, seq_lens, hold, workspace, ws_bytes, &a);
    if (rc) return rc;
    if (!n_add) return ENTMAXKV_ERR_NULL;
    if ((rc = on_device(&a))) return rc;
    a.n_add = n_add;
    a.table_out = page_table;
    a.lens_out = seq_lens;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return rc_of(plan(plan_grow_kernel, a, st));
}

int entmaxkv_pages_compact(const entmaxkv_shape *s, const int32_t *table_in, const int32_t *seq_lens,
                           const int32_t *hold, int32_t *table_out, const entmaxkv_buffers *bufs, int32_t *remap,
                           int32_t *n_live, void *workspace, size_t ws_bytes, void *stream) {
    PageArgs a;
    int rc = fill_pages(s, table_in, seq_lens, hold, workspace, ws_bytes, &a);
    if (rc) return rc;
    if (!table_out || !remap || !n_live) return ENTMAXKV_ERR_NULL;
    if ((rc = check_buffers(bufs, true)) || (rc = on_device(&a))) return rc;
    a.table_out = table_out;
    a.remap = remap;
    a.n_live = n_live;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = plan(plan_compact_kernel, a, st);
    if (e == cudaSuccess) e = apply<false>(a, bufs, s, s->num_blocks, nullptr, nullptr, st);
    return rc_of(e);
}

int entmaxkv_pages_copy(const entmaxkv_buffers *src, int32_t src_blocks, const entmaxkv_buffers *dst,
                        int32_t dst_blocks, const int32_t *src_ids, const int32_t *dst_ids, int32_t n, void *stream) {
    int rc = check_buffers(src, true);
    if (rc || (rc = check_buffers(dst, true))) return rc;
    if (src->count != dst->count || (src->count && src->block_bytes != dst->block_bytes)) return ENTMAXKV_ERR_SHAPE;
    if (n < 0 || src_blocks < 1 || dst_blocks < 1) return ENTMAXKV_ERR_SHAPE;
    if (n == 0 || src->count == 0) return ENTMAXKV_OK;
    if (!src_ids || !dst_ids) return ENTMAXKV_ERR_NULL;
    DevInfo di;
    if ((rc = device_info(&di))) return rc;
    auto run = src->count <= FEW ? move<FEW> : move<ENTMAXKV_MAX_BUFFERS>;
    return rc_of(run(src, src_blocks, dst, dst_blocks, src_ids, dst_ids, n, di.status, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
