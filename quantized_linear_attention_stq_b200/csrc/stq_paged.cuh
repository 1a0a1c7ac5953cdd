// stq_paged.cuh -- how one attention call over the paged cache is split over thread blocks, and the
// partial results that its parts leave for the join.
//
// The work of a call is a line of tiles of TK cached tokens: request after request, inside a request
// unit after unit (a unit: up to 16 query heads of one key-value head), inside a unit tile after
// tile. Block c of C takes tiles [W c / C, W (c + 1) / C) of the W tiles, whatever requests they
// belong to: the blocks' shares differ by one tile at most, however ragged the lengths. A unit that
// lies in one block's share is finished there. Another unit is cut in pieces; a block keeps at most
// two, one that began before its share (piece 0) and one that goes on behind it (piece 1).
#pragma once

#include "stq_internal.cuh"

namespace stq {
namespace paged {

constexpr int TK = 64;          // cached tokens of a tile
constexpr int ROWS = 16;        // query heads of a unit, at most
constexpr int kMaxBlocks = 592; // blocks of a split call, at most (the workspace is sized for them)

struct Params {
    const void *q;                        // [B][Hq][d]
    const void *k_pages, *v_pages;        // [num_pages][Hkv][page][d]
    const int32_t *table, *lens;          // [B][W], [B]
    float *o;                             // [B][Hq][d]
    float *pieces;                        // [blocks][2][ROWS][d + 2]: sums, running maximum, running sum
    long long *first_tile;                // [B + 1]: tiles of the requests before, per unit
    int32_t *status;
    float scale2;                         // scale * log2(e)
    int32_t B, Hq, Hkv, group, row_tiles; // group = Hq / Hkv, row_tiles = ceil(group / ROWS)
    int32_t W, page, num_pages;
    int32_t split;                        // 1: shares of the line of tiles; 0: one block per unit
};

#ifdef __CUDACC__
// Cached tokens of request b; one outside [0, W * page] counts as none.
__device__ __forceinline__ int cached_length(const Params &p, int b, bool *bad)
{
    const int n = p.lens[b];
    *bad = n < 0 || (long long)n > (long long)p.W * p.page;
    return *bad ? 0 : n;
}
__device__ __forceinline__ int tiles_of(int len) { return (int)(((long long)len + TK - 1) / TK); }

// Blocks that get work: each a tile at least.
__device__ __forceinline__ int busy_blocks(long long W, int most) { return W < most ? (W > 0 ? (int)W : 1) : most; }
// First tile of block c's share of W tiles over C blocks, and the block that holds tile t.
__device__ __forceinline__ long long share_begin(long long W, int c, int C) { return W * c / C; }
__device__ __forceinline__ int block_of(long long W, long long t, int C) { return (int)(((t + 1) * C - 1) / W); }
#endif

}  // namespace paged
}  // namespace stq
