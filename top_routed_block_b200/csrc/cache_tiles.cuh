// cache_tiles.cuh -- attention of many query rows over an 8-bit cache: what the expansion of the
// pages (cache_attend.cu) and the tile kernel (attn_fwd.cu) share.
#pragma once

#include "cache.cuh"
#include "cache_index.h"

namespace fvattn {

constexpr int kTileRows = 128, kTileKeys = 128;

// Attention of many new query rows per sequence over an 8-bit cache, whose pages lie expanded as bf16
// [B * heads, cap, d] (the tensor maps of AttnLaunch, boxes of 128 tokens).  Rows of one key head are
// its `group` query heads times M new tokens; an item is 128 of them.  The first n_whole items (a
// multiple of the grid) come whole from the queue, in order, so that the SMs share one head's keys
// in L2; the n_rest behind them, fewer than the grid, are cut into equal stretches of key tiles, one
// a CTA, and joined (a last wave of whole items would leave most SMs idle).
struct CacheTiles {
    int32_t *rest;       // [n_rest + 1] key tiles before each of the rest
    float2 *part_stats;  // [2 * grid, 128] m, l of the partial rows
    float *part_acc;     // [2 * grid, 128, d]
    int n_rest;
    AttendLaunch a;
    int64_t cap;         // tokens of a head's expanded K or V: the table's, rounded up to 128
    void *K, *V;
    int32_t *nan_first;  // [B * heads, d]: 2^31 - 1 - first token whose V was NaN there, 0 none
    int rows, row_tiles, n_whole, ctas;
};

// Expands the pages, checks the call and plans the rest.
cudaError_t launch_cache_expand(const CacheTiles &ct, cudaStream_t stream);

#ifdef __CUDACC__

// ------------------------------------------------- cached keys (CacheTiles)
// Row r of item `item`: one query token of one query head, and what it sees.
struct CacheRow {
    bool valid;          // a row of the head's, and its token one of the sequence's new ones
    int limit;           // it sees cached tokens [0, limit)
    int64_t q_at, o_at;  // its first element in Q and O
    int64_t lse_at;
};

__device__ __forceinline__ CacheRow cache_row(const CacheTiles &ct, int item, int r) {
    const AttendLaunch &a = ct.a;
    const int bh = item / ct.row_tiles, row = (item % ct.row_tiles) * kTileRows + r;
    const int b = bh / a.pool.heads, h = bh % a.pool.heads;
    const Seq seq = sequence(a, b);
    const int m = row % a.M;
    CacheRow c;
    c.valid = row < ct.rows && m < seq.n_new;
    const int64_t hq = c.valid ? h * a.group + row / a.M : 0, tok = c.valid ? m : 0;
    c.limit = c.valid ? row_limit(a, seq, m) : 0;
    c.q_at = b * a.q_b + hq * a.q_h + tok * a.q_n;
    c.o_at = b * a.o_b + hq * a.o_h + tok * a.o_n;
    c.lse_at = (static_cast<int64_t>(b) * a.pool.heads * a.group + hq) * a.M + tok;
    return c;
}

// Key tiles an item walks: up to the last token that one of its rows sees.
__device__ __forceinline__ int cache_tiles_of(const CacheTiles &ct, int item) {
    const AttendLaunch &a = ct.a;
    const int bh = item / ct.row_tiles, row0 = (item % ct.row_tiles) * kTileRows;
    const Seq seq = sequence(a, bh / a.pool.heads);
    if (seq.n_new == 0) return 0;
    const int row1 = min(row0 + kTileRows, ct.rows) - 1;
    const int last = row0 / a.M == row1 / a.M ? min(row1 % a.M, seq.n_new - 1) : seq.n_new - 1;
    return (row_limit(a, seq, last) + kTileKeys - 1) / kTileKeys;
}

// The items behind the whole ones (CacheTiles), cut into equal stretches of their key tiles.
struct CacheRest {
    int64_t at, end;  // this CTA's stretch
    bool opened;

    __device__ __forceinline__ void open(const CacheTiles &ct, int cta) {
        opened = true;
        const int64_t total = ct.n_rest > 0 ? ct.rest[ct.n_rest] : 0;
        const int n = stretches(total, ct.ctas);
        at = cta < n ? stretch_start(cta, total, n) : 0;
        end = cta < n ? stretch_start(cta + 1, total, n) : 0;
    }
    // The next piece: {item, first key tile << 1 | whether others have the rest of it, key tiles, -}.
    __device__ __forceinline__ bool next(const CacheTiles &ct, int4 &piece) {
        if (at >= end) return false;
        int lo = 0, hi = ct.n_rest - 1;
        while (lo < hi) {  // the last item that begins at or before `at`
            const int mid = (lo + hi + 1) >> 1;
            if (__ldcg(ct.rest + mid) <= at) lo = mid;
            else hi = mid - 1;
        }
        const int begin = __ldcg(ct.rest + lo), units = __ldcg(ct.rest + lo + 1) - begin;
        const int off = static_cast<int>(at) - begin;
        const int n = static_cast<int>(min(static_cast<int64_t>(units - off), end - at));
        at += n;
        // (an item without key tiles has one unit, so that its rows are written)
        const int tiles = max(min(cache_tiles_of(ct, ct.n_whole + lo) - off, n), 0);
        piece = make_int4(ct.n_whole + lo, off << 1 | (n < units ? 1 : 0), tiles, ct.n_whole + lo + 1);
        return true;
    }
};

// A row of a piece whose item others share: its sums to the partials' place.  Slot 2 cta + 1: of the
// item that the CTA's stretch ends in; 2 cta: of the one it begins in.
__device__ __forceinline__ int64_t cache_part_row(bool begins, int cta, int r) {
    return (static_cast<int64_t>(2 * cta) + (begins ? 1 : 0)) * kTileRows + r;
}

#endif

}  // namespace fvattn
