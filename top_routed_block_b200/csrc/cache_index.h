// cache_index.h -- the index arithmetic of the paged 8-bit cache, for the kernels and
// for checks on the host: which tokens are cached, which slots of which pages a call
// touches, and how attention splits the cached tokens into work items.  Plain C++ when
// compiled without nvcc.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FVATTN_HD __host__ __device__ __forceinline__
#else
#define FVATTN_HD inline
#endif

namespace fvattn {

// A length or start from device memory, held inside [0, most].
FVATTN_HD int64_t clamp_len(int64_t n, int64_t most) { return n < 0 ? 0 : n > most ? most : n; }

// A page table entry: the page, or -1 where the entry names none of the pool's.
FVATTN_HD int checked_page(int page, int num_pages) { return page >= 0 && page < num_pages ? page : -1; }

// The part of page number pg (of a sequence) that n new tokens behind `start` cached ones
// fill: slots [lo, hi) of the page, the first from new token `token`.  Empty: lo >= hi.
struct PageSpan {
    int lo, hi;
    int64_t token;
};

FVATTN_HD PageSpan page_span(int64_t start, int64_t n, int64_t pg, int block) {
    const int64_t first = pg * block;
    int64_t lo = start > first ? start : first;
    int64_t hi = start + n < first + block ? start + n : first + block;
    if (hi < lo) hi = lo;
    return PageSpan{static_cast<int>(lo - first < block ? lo - first : block),
                    static_cast<int>(hi - first < block ? (hi - first > 0 ? hi - first : 0) : block), lo - start};
}

// Pages that T new tokens can touch at most, wherever they start.
FVATTN_HD int64_t max_touched_pages(int64_t T, int block) { return T <= 0 ? 0 : (T + block - 2) / block + 1; }

// New tokens a call appends to a sequence: none where the start is not a length, and no
// more than the page table has room for.
FVATTN_HD int64_t append_count(int64_t start, int64_t n, int64_t T, int64_t capacity) {
    if (start < 0 || start > capacity) return 0;
    n = clamp_len(n, T);
    return n < capacity - start ? n : capacity - start;
}

// Attention of a few rows cuts the line of all segments' units of `unit` tokens into equal
// stretches.  Units of a segment of `len` cached tokens (an empty one still writes its rows):
FVATTN_HD int64_t segment_units(int64_t len, int unit) { return len <= 0 ? 1 : (len + unit - 1) / unit; }

// How many stretches for up to `ctas` CTAs: none is empty.
FVATTN_HD int stretches(int64_t total, int ctas) { return total < ctas ? static_cast<int>(total) : ctas; }

// Stretch c of n is [stretch_start(c), stretch_start(c + 1)) of `total` units ...
FVATTN_HD int64_t stretch_start(int64_t c, int64_t total, int64_t n) { return c * total / n; }
// ... and unit u lies in stretch
FVATTN_HD int stretch_of(int64_t u, int64_t total, int64_t n) { return static_cast<int>(((u + 1) * n - 1) / total); }

}  // namespace fvattn
