// pages.cu -- copying, forking, growing, compacting and freeing the pages of a
// cache (include/entmaxkv_pages.h), and their C entry points.
//
// Which blocks are free follows from the page table alone: the rows' blocks
// are marked in a bitmap (one bit a block), and one CTA turns the bitmap and
// the rows' needs into a plan (prefix sums in row and block order, so nothing
// depends on timing).  Moving the pages is then a copy of (src, dst) block
// pairs in every buffer, bound by memory bandwidth: 16-byte loads, several in
// flight a thread, pair x buffer x chunk spread over a persistent grid.
#include <cstring>

#include "../../include/entmaxkv_pages.h"
#include "common.cuh"
#include "internal.h"

namespace ekv {

namespace {

constexpr int PL_NT = 1024;  // threads of the planning CTA
constexpr int MV_NT = 256;
constexpr int MV_UNROLL = 8;
constexpr long long MV_CHUNK = (long long)MV_NT * MV_UNROLL * 16;  // bytes a CTA moves at a time

struct PageArgs {
    int B, P, max_pages, num_blocks;
    const int *table_in, *lens_in, *hold, *parent, *n_add;
    int *table_out, *lens_out;
    int in_place;
    unsigned *bits;      // [words] blocks in use
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

// Marks the blocks of the rows (one CTA a row, then the held ones).
__global__ void mark_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int n = row_pages(a, b);
        for (int p = threadIdx.x; p < n; p += blockDim.x) {
            const int blk = a.table_in[(size_t)b * a.max_pages + p];
            if (block_ok(a, blk)) atomicOr(&a.bits[blk >> 5], 1u << (blk & 31));
            else atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
        }
    }
    if (a.hold)
        for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.num_blocks; i += gridDim.x * blockDim.x)
            if (a.hold[i] > 0) atomicOr(&a.bits[i >> 5], 1u << (i & 31));
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

// The first `want` free blocks, ascending, into a.list; returns how many.
__device__ int list_free(const PageArgs &a, long long want, int *sh) {
    long long found = 0;
    for (int w0 = 0; w0 < a.words && found < want; w0 += PL_NT) {
        const int w = w0 + threadIdx.x;
        unsigned f = w < a.words ? ~a.bits[w] & word_mask(a, w) : 0u;
        int tot;
        long long at = found + block_excl_scan(__popc(f), sh, &tot);
        for (; f && at < want; f &= f - 1u, ++at) a.list[at] = 32 * w + __ffs(f) - 1;
        found += tot;
    }
    __syncthreads();  // the list is read by other threads of the CTA
    return (int)(found < want ? found : want);
}

__global__ void __launch_bounds__(PL_NT) plan_fork_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    __shared__ int sh[72];
    for (int b = threadIdx.x; b < a.B; b += PL_NT) {
        int p = a.parent[b];
        bool bad = p < -1 || p >= a.B;
        if (a.in_place && !bad && p >= 0 && p != b) bad = a.parent[p] != p;
        if (bad) {
            atomicOr(a.status, ENTMAXKV_STATUS_BAD_ROW);
            p = a.in_place ? b : -1;
        }
        a.act[b] = p;
        a.first[b] = 0x7fffffff;
    }
    __syncthreads();
    // the parent's own row keeps the partial page, else the first child
    for (int b = threadIdx.x; b < a.B; b += PL_NT) {
        const int p = a.act[b];
        if (p >= 0) atomicMin(&a.first[p], p == b ? -1 : b);
    }
    __syncthreads();
    auto needs = [&](int b, int &src) {
        if (b >= a.B) return 0;
        const int p = a.act[b];
        if (p < 0) return 0;
        const int L = seq_len_of(a.lens_in, p, a.P, a.max_pages, a.status);
        if (L % a.P == 0 || a.first[p] == (p == b ? -1 : b)) return 0;
        src = a.table_in[(size_t)p * a.max_pages + L / a.P];
        return 1;
    };
    long long want = 0;
    for (int b0 = 0; b0 < a.B; b0 += PL_NT) {
        int src, tot;
        block_excl_scan(needs(b0 + threadIdx.x, src), sh, &tot);
        want += tot;
    }
    const int have = list_free(a, want, sh);
    int rank = 0, pairs = 0;
    for (int b0 = 0; b0 < a.B; b0 += PL_NT) {
        const int b = b0 + threadIdx.x;
        int src = -1, tot, n_pairs;
        const int need = needs(b, src);
        const int at = rank + block_excl_scan(need, sh, &tot);
        rank += tot;
        int blk = -2;
        if (need) {
            blk = at < have ? a.list[at] : -1;
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

// The new rows of the table, one CTA a row.
__global__ void fork_rows_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int p = a.act[b];
        if (a.in_place && p == b) continue;
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
}

struct MetaMove {
    const char *in[ENTMAXKV_MAX_BUFFERS];
    char *out[ENTMAXKV_MAX_BUFFERS];
    const int *act, *lens;
    int in_place, B, Hkv, d, P, max_pages, n_tiles;
    long long n_tiles_total;
};

// Metadata tiles follow their rows: one CTA per (row, kv head) and buffer.
__global__ void fork_meta_kernel(const __grid_constant__ MetaMove a) {
    pdl_wait();
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    const int p = a.act[b];
    if (p < 0 || (a.in_place && p == b)) return;
    const int n = n_pages_of(seq_len_of(a.lens, p, a.P, a.max_pages, nullptr), a.P);
    const int tiles = (n + META_TILE - 1) / META_TILE;
    const char *in = a.in[blockIdx.y];
    char *out = a.out[blockIdx.y];
    const long long src = ((long long)p * a.Hkv + h) * a.n_tiles, dst = ((long long)b * a.Hkv + h) * a.n_tiles;
#pragma unroll
    for (int region = 0; region < 2; ++region) {
        const long long tile = (region ? 256 : 128) * a.d, base = region ? a.n_tiles_total * 128 * a.d : 0;
        const uint4 *s = reinterpret_cast<const uint4 *>(in + base + src * tile);
        uint4 *o = reinterpret_cast<uint4 *>(out + base + dst * tile);
        for (long long i = threadIdx.x; i < tiles * tile / 16; i += blockDim.x) o[i] = s[i];
    }
}

__global__ void __launch_bounds__(PL_NT) plan_grow_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    __shared__ int sh[72];
    __shared__ long long s_at[PL_NT];
    const long long cap = (long long)a.max_pages * a.P;
    // pages sequence b needs, its pages and new length; -1: it does not grow
    auto need = [&](int b, int &n0, long long &L) {
        if (b >= a.B) return -1;
        const int add = a.n_add[b];
        if (add <= 0) return -1;
        const int L0 = seq_len_of(a.lens_in, b, a.P, a.max_pages, a.status);
        L = (long long)L0 + add;
        if (L > cap) {
            atomicOr(a.status, ENTMAXKV_STATUS_BAD_LENGTH);
            return -1;
        }
        n0 = n_pages_of(L0, a.P);
        return (int)((L + a.P - 1) / a.P) - n0;
    };
    // inclusive sums of the needs in 64 bits (a round of PL_NT at a time)
    auto scan64 = [&](long long v) {
        s_at[threadIdx.x] = v;
        __syncthreads();
        for (int o = 1; o < PL_NT; o <<= 1) {
            const long long x = threadIdx.x >= o ? s_at[threadIdx.x - o] : 0;
            __syncthreads();
            s_at[threadIdx.x] += x;
            __syncthreads();
        }
        const long long r = s_at[threadIdx.x];
        return r;
    };
    long long want = 0;
    for (int b0 = 0; b0 < a.B; b0 += PL_NT) {
        int n0;
        long long L;
        scan64(max(0, need(b0 + threadIdx.x, n0, L)));
        want += s_at[PL_NT - 1];
        __syncthreads();
    }
    const int have = list_free(a, want < a.num_blocks ? want : a.num_blocks, sh);
    long long used = 0;
    for (int b0 = 0; b0 < a.B; b0 += PL_NT) {
        const int b = b0 + threadIdx.x;
        int n0 = 0;
        long long L = 0;
        const int k = need(b, n0, L);
        const long long end = used + scan64(max(0, k));
        used += s_at[PL_NT - 1];
        __syncthreads();
        if (k < 0) continue;
        if (end > have && k > 0) {
            atomicOr(a.status, ENTMAXKV_STATUS_NO_BLOCK);
            continue;
        }
        for (int i = 0; i < k; ++i) a.table_out[(size_t)b * a.max_pages + n0 + i] = a.list[end - k + i];
        a.lens_out[b] = (int)L;
    }
}

__global__ void __launch_bounds__(PL_NT) plan_compact_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    __shared__ int sh[72];
    int n = 0, n_live;
    for (int w = threadIdx.x; w < a.words; w += PL_NT) n += __popc(a.bits[w]);
    block_excl_scan(n, sh, &n_live);
    int holes = 0, moves = 0;
    for (int w0 = 0; w0 < a.words; w0 += PL_NT) {
        const int w = w0 + threadIdx.x;
        const unsigned live = w < a.words ? a.bits[w] : 0u;
        const unsigned valid = w < a.words ? word_mask(a, w) : 0u;
        const int left = n_live - 32 * w;  // blocks of the word below n_live
        const unsigned low = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
        int th, tm;
        int h = holes + block_excl_scan(__popc(~live & valid & low), sh, &th);
        int m = moves + block_excl_scan(__popc(live & ~low), sh, &tm);
        for (unsigned f = ~live & valid & low; f; f &= f - 1u) a.pair_dst[h++] = 32 * w + __ffs(f) - 1;
        for (unsigned f = live & ~low; f; f &= f - 1u) a.pair_src[m++] = 32 * w + __ffs(f) - 1;
        for (unsigned f = valid; f; f &= f - 1u) {
            const int i = __ffs(f) - 1;
            a.remap[32 * w + i] = ((live & low) >> i) & 1u ? 32 * w + i : -1;
        }
        holes += th;
        moves += tm;
    }
    __syncthreads();  // holes == moves: the pairs are complete
    for (int i = threadIdx.x; i < moves; i += PL_NT) a.remap[a.pair_src[i]] = a.pair_dst[i];
    if (threadIdx.x == 0) {
        *a.n_live = n_live;
        *a.n_pairs = moves;
    }
}

__global__ void remap_rows_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int n = n_pages_of(seq_len_of(a.lens_in, b, a.P, a.max_pages, nullptr), a.P);
        for (int i = threadIdx.x; i < a.max_pages; i += blockDim.x) {
            const size_t at = (size_t)b * a.max_pages + i;
            const int blk = i < n ? a.table_in[at] : -1;
            a.table_out[at] = block_ok(a, blk) ? a.remap[blk] : -1;
        }
    }
}

struct MoveArgs {
    const char *src[ENTMAXKV_MAX_BUFFERS];
    char *dst[ENTMAXKV_MAX_BUFFERS];
    const int *src_ids, *dst_ids;
    const int *n_dev;  // pairs, on the device (else n)
    int n, bufs, src_blocks, dst_blocks;
    long long bytes;   // of a block
    int *status;
};

// Block pairs, every buffer: chunk after chunk of MV_CHUNK bytes.
__global__ void __launch_bounds__(MV_NT) move_kernel(const __grid_constant__ MoveArgs a) {
    pdl_wait();
    const int n = a.n_dev ? *a.n_dev : a.n;
    const long long per = (a.bytes + MV_CHUNK - 1) / MV_CHUNK;  // chunks of a block
    const long long total = per * a.bufs * n;
    for (long long k = blockIdx.x; k < total; k += gridDim.x) {
        const long long pb = k / per;
        const int pair = (int)(pb / a.bufs), buf = (int)(pb % a.bufs);
        const int s = a.src_ids[pair], d = a.dst_ids[pair];
        if (s < 0 || s >= a.src_blocks || d < 0 || d >= a.dst_blocks) {
            if (threadIdx.x == 0) atomicOr(a.status, ENTMAXKV_STATUS_BAD_PAGE);
            continue;
        }
        const long long off = (k % per) * MV_CHUNK;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.src[buf] + s * a.bytes + off);
        uint4 *dst = reinterpret_cast<uint4 *>(a.dst[buf] + d * a.bytes + off);
        const long long left = (a.bytes - off) / 16;
        const int m = (int)(left < MV_CHUNK / 16 ? left : MV_CHUNK / 16);
        uint4 v[MV_UNROLL];
#pragma unroll
        for (int u = 0; u < MV_UNROLL; ++u)
            if (u * MV_NT + threadIdx.x < m) v[u] = src[u * MV_NT + threadIdx.x];
#pragma unroll
        for (int u = 0; u < MV_UNROLL; ++u)
            if (u * MV_NT + threadIdx.x < m) dst[u * MV_NT + threadIdx.x] = v[u];
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

constexpr int GRID = 148 * 8;

cudaError_t mark(const PageArgs &a, cudaStream_t st) {
    cudaError_t e = launch_pdl(clear_kernel, dim3(min(ceil_div(a.words, 256), GRID)), dim3(256), 0, st,
                               reinterpret_cast<int *>(a.bits), (int)a.words);
    if (e != cudaSuccess) return e;
    return launch_pdl(mark_kernel, dim3(a.hold ? GRID : min(a.B, GRID)), dim3(256), 0, st, a);
}

void fill_move(MoveArgs *m, const entmaxkv_buffers *src, const entmaxkv_buffers *dst) {
    *m = MoveArgs{};
    m->bufs = src->count;
    m->bytes = src->block_bytes;
    for (int i = 0; i < src->count; ++i) {
        m->src[i] = static_cast<const char *>(src->base[i]);
        m->dst[i] = static_cast<char *>(dst->base[i]);
    }
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
    cudaError_t e = mark(a, st);
    if (e == cudaSuccess) e = launch_pdl(plan_fork_kernel, dim3(1), dim3(PL_NT), 0, st, a);
    if (e == cudaSuccess) e = launch_pdl(fork_rows_kernel, dim3(min(a.B, GRID)), dim3(256), 0, st, a);
    if (e == cudaSuccess && bufs->count) {
        MoveArgs m;
        fill_move(&m, bufs, bufs);
        m.src_ids = a.pair_src;
        m.dst_ids = a.pair_dst;
        m.n_dev = a.n_pairs;
        m.src_blocks = m.dst_blocks = s->num_blocks;
        m.status = a.status;
        e = launch_pdl(move_kernel, dim3(GRID), dim3(MV_NT), 0, st, m);
    }
    if (e == cudaSuccess && meta_in && meta_in->count) {
        MetaMove m{};
        for (int i = 0; i < meta_in->count; ++i) {
            m.in[i] = static_cast<const char *>(meta_in->base[i]);
            m.out[i] = static_cast<char *>(meta_out->base[i]);
        }
        m.act = a.act;
        m.lens = lens_in;
        m.in_place = a.in_place;
        m.B = s->B;
        m.Hkv = s->Hkv;
        m.d = s->d;
        m.P = s->page_size;
        m.max_pages = s->max_pages;
        m.n_tiles = meta_tiles(s->max_pages);
        m.n_tiles_total = (long long)s->B * s->Hkv * m.n_tiles;
        e = launch_pdl(fork_meta_kernel, dim3(s->B * s->Hkv, meta_in->count), dim3(256), 0, st, m);
    }
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
    cudaError_t e = mark(a, st);
    if (e == cudaSuccess) e = launch_pdl(plan_grow_kernel, dim3(1), dim3(PL_NT), 0, st, a);
    return rc_of(e);
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
    cudaError_t e = mark(a, st);
    if (e == cudaSuccess) e = launch_pdl(plan_compact_kernel, dim3(1), dim3(PL_NT), 0, st, a);
    if (e == cudaSuccess) e = launch_pdl(remap_rows_kernel, dim3(min(a.B, GRID)), dim3(256), 0, st, a);
    if (e == cudaSuccess && bufs->count) {
        MoveArgs m;
        fill_move(&m, bufs, bufs);
        m.src_ids = a.pair_src;
        m.dst_ids = a.pair_dst;
        m.n_dev = a.n_pairs;
        m.src_blocks = m.dst_blocks = s->num_blocks;
        m.status = a.status;
        e = launch_pdl(move_kernel, dim3(GRID), dim3(MV_NT), 0, st, m);
    }
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
    MoveArgs m;
    fill_move(&m, src, dst);
    m.src_ids = src_ids;
    m.dst_ids = dst_ids;
    m.n = n;
    m.src_blocks = src_blocks;
    m.dst_blocks = dst_blocks;
    m.status = di.status;
    const long long chunks = (m.bytes + MV_CHUNK - 1) / MV_CHUNK * m.bufs * n;
    return rc_of(launch_pdl(move_kernel, dim3((unsigned)(chunks < GRID ? chunks : GRID)), dim3(MV_NT), 0,
                            static_cast<cudaStream_t>(stream), m));
}

}  // extern "C"
