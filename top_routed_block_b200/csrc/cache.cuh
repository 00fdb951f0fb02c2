// cache.cuh -- internal interface of the paged 8-bit key/value cache: appending
// (cache_append.cu) and attention (cache_attend.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "cache_index.h"
#include "common.cuh"
#include "rope.cuh"

namespace fvattn {

// The pool: page p, head h, slot s, channel c at ((p * heads + h) * block + s) * d + c.
struct CachePool {
    uint8_t *k, *v;        // e4m3 codes
    int32_t *ke, *ve;      // power-of-two scale exponents [num_pages, heads]
    int num_pages, heads, block, d;
    const int32_t *table;  // [B, max_pages]
    int max_pages;
};

// Exponent of a page that holds only zeros: below what any fp32 value asks for, so that
// the next tokens set the scale.
constexpr int kZeroPageExp = -160;

struct AppendLaunch {
    CachePool pool;
    const void *K, *V;  // bf16 [B, heads, T, d] with strides
    int64_t k_b, k_h, k_n, v_b, v_h, v_n;
    int B, T;
    const int32_t *start, *new_lens;  // new_lens may be null: all T
    const int32_t *pos;               // null: no rotation
    int64_t pos_b;
    bool half;
    RopeParams rope;
    int32_t *dev_status;
};

cudaError_t launch_cache_append(const AppendLaunch &a, int sms, cudaStream_t stream);

struct AttendLaunch {
    CachePool pool;
    const void *Q;  // bf16 [B, heads * group, M, d] with strides
    void *O;
    float *LSE;     // [B, heads * group, M]
    int64_t q_b, q_h, q_n, o_b, o_h, o_n;
    int B, group, M;
    const int32_t *lens, *new_lens;  // new_lens may be null: all M
    int causal;
    int32_t *dev_status;
    void *workspace;
    int sms;
};

// Rows of one key head: its query heads times M new tokens.
inline int64_t attend_rows(int group, int M) { return static_cast<int64_t>(group) * M; }
// Whether the call takes the few-rows kernel (else the pages are expanded and the tensor
// cores' 128-row tiles run over them).
bool attend_few_rows(int group, int M, int64_t capacity);
size_t attend_few_workspace(int d, int sms);
cudaError_t launch_attend_few(const AttendLaunch &a, cudaStream_t stream);
#ifdef __CUDACC__

// x * 2^e for |e| up to 252: two exact factors (a single 2^e may lie outside fp32).  Exact
// unless the result is subnormal.
__device__ __forceinline__ float scale_pow2(float x, int e) {
    const int h = e / 2;
    return x * __int_as_float((h + 127) << 23) * __int_as_float((e - h + 127) << 23);
}
__device__ __forceinline__ int clamp_exp(int e) { return max(-250, min(e, 250)); }

// Whether any of the four e4m3 codes of w is a NaN (0x7F or 0xFF).
__device__ __forceinline__ bool any_nan_e4m3(uint32_t w) {
    return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;
}

struct Seq {
    int len;    // cached tokens (a page table holds fewer than 2^31)
    int n_new;  // of them new: the queries
};

__device__ __forceinline__ Seq sequence(const AttendLaunch &a, int b) {
    const int64_t cap = static_cast<int64_t>(a.pool.max_pages) * a.pool.block;
    Seq s;
    s.len = static_cast<int>(clamp_len(a.lens[b], cap));
    s.n_new = static_cast<int>(clamp_len(a.new_lens ? a.new_lens[b] : a.M, a.M));
    return s;
}

// Tokens that query token m sees: [0, limit).
__device__ __forceinline__ int row_limit(const AttendLaunch &a, const Seq &s, int m) {
    if (m >= s.n_new) return 0;
    return a.causal ? static_cast<int>(clamp_len(static_cast<int64_t>(s.len) - s.n_new + m + 1, s.len)) : s.len;
}

// Lengths, counts and (TABLE) the page table entries in use: those of sequences with queries.  One CTA,
// writes the status word.
template <bool TABLE>
__device__ __forceinline__ void check_attend(const AttendLaunch &a) {
    const int64_t cap = static_cast<int64_t>(a.pool.max_pages) * a.pool.block;
    bool bad = false;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int64_t len = a.lens[b], n = a.new_lens ? a.new_lens[b] : a.M;
        if (len < 0 || len > cap || n < 0 || n > a.M) bad = true;
    }
    const int all = TABLE ? a.B * a.pool.max_pages : 0, stride = static_cast<int>(blockDim.x);
    for (int i0 = threadIdx.x; i0 < all; i0 += 4 * stride) {
        int page[4];
        int used[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // four entries' loads at a time
            const int i = i0 + k * stride;
            page[k] = i < all ? __ldcg(a.pool.table + i) : 0;
            const Seq seq = i < all ? sequence(a, i / a.pool.max_pages) : Seq{0, 0};
            used[k] = seq.n_new > 0 ? seq.len : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * stride;
            if (i < all && static_cast<int64_t>(i % a.pool.max_pages) * a.pool.block < used[k] &&
                checked_page(page[k], a.pool.num_pages) < 0)
                bad = true;
        }
        if (all - i0 <= 4 * stride) break;  // i0 + 4 stride may pass 2^31
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.dev_status = any ? FVATTN_ERR_BAD_PAGE : FVATTN_OK;
}

#endif

}  // namespace fvattn
