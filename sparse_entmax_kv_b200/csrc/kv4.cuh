// kv4.cuh -- the 4-bit cache's layout (include/entmaxkv_kv4.h): where a
// token's codes and parameters lie inside a 16-token tile, and the arguments
// of the kernels that write, read and attend over it.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace ekv {

constexpr int KV4_GROUP = 64;  // coordinates that share s and lo

template <int D>
struct Kv4 {
    static constexpr int NG = D / KV4_GROUP;  // groups of a row
    static constexpr int WPL = D / 32;        // 32-bit code words a lane of the attention kernel owns in a row
    static constexpr int CODES = 8 * D;       // bytes of a tile's codes
    static constexpr int TILE = 9 * D;        // bytes of a 16-token tile
};

// Byte address of tile `t16` of (block, kv head).
template <int D>
__device__ __forceinline__ size_t kv4_tile(int blk, int Hkv, int kvh, int P, int t16) {
    return (((size_t)blk * Hkv + kvh) * (P / 16) + t16) * Kv4<D>::TILE;
}

// Word index (within the tile) of the 8 coordinates 8 q8 .. 8 q8 + 7 of the
// key of token t; coordinate n of them at bits 16 (n & 1) + 4 (n >> 1).
template <int D>
__device__ __forceinline__ int kv4_kword(int t, int q8) {
    return t * (D / 8) + ((q8 >> 1) & 3) * Kv4<D>::WPL + 2 * (q8 >> 3) + (q8 & 1);
}
// XOR on the position of a value word's row piece, by token pair.
template <int D>
__device__ __forceinline__ int kv4_vswz(int pair) {
    return D == 128 ? 2 * (pair & 3) : 4 * ((pair >> 1) & 1);
}
// Word index of the 4 coordinates 4 q4 .. 4 q4 + 3 of the values of token
// pair `pair`; coordinate n of the pair's token e at bits 16 e + 4 n.
template <int D>
__device__ __forceinline__ int kv4_vword(int pair, int q4) {
    return pair * (D / 4) + (((q4 >> 1) & 7) ^ kv4_vswz<D>(pair)) * Kv4<D>::WPL + 2 * (q4 >> 4) + (q4 & 1);
}

struct Kv4RowArgs {
    const uint16_t *k_new, *v_new;  // write
    void *k_out, *v_out;            // read
    long long stride;               // elements between rows
    const int *row_start;           // null: row b for sequence b
    int n_rows;
    const int *page_table, *seq_lens;
    uint8_t *k4, *v4;
    MetaArgs m;  // metadata (m.meta null: none), shape fields, kv-head range, status
    int f32;     // read: fp32 rows
    unsigned big;  // the bits of 2^23
};
cudaError_t launch_kv4_write(const Kv4RowArgs &a, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4RowArgs &a, cudaStream_t st);

}  // namespace ekv
