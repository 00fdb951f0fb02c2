// cache_append.cu -- new keys and values into a paged cache of e4m3 codes with one
// power-of-two scale per (page, head), the keys turned by their rotary positions on
// the way.
//
// Mathematics: a page of one head holds codes c and an exponent e, value = c 2^e, in
// the format of fvattn_quant_e4m3.  Appending tokens with largest magnitude a to a
// page asks for need = the smallest e with a 2^-e <= 448; the page's exponent becomes
// max(e, need) if older tokens are in it and need otherwise.  New values are turned in
// fp32 and rounded once, from fp32 to e4m3 (nearest, ties to even, saturating; never
// through bf16, which would round twice).  Where the exponent grows, the older codes go
// to the new scale; the powers of two make that exact except for codes that become
// subnormal, which are rounded again.  A page whose tokens are all zero keeps an
// exponent below every need, so that it does not fix the scale of what follows.
//
// What bounds it: HBM for long calls (2 bytes in, 1 byte out per element), launch
// latency for single tokens.  One CTA per (sequence, touched page, head, K or V): it
// owns the page's exponent and rows, so there are no atomics and nothing is written
// twice.  The values stay in registers between the maximum and the rounding: one read.
// CTA 0 does no work of its own: it checks starts, counts and page table entries and
// writes the status word, so that the call is one launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "cache.cuh"
#include "common.cuh"

namespace fvattn {

namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 values2(uint32_t two_codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two_codes)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The exponent a largest magnitude asks for (an infinity: 2^0, as the quantizer does).
__device__ __forceinline__ int need_exp(float amax) {
    if (amax == 0.0f) return kZeroPageExp;
    if (isinf(amax)) return 0;
    int e = ilogbf(amax) - 8;  // amax 2^-e in [256, 512)
    if (scale_pow2(amax, -e) > 448.0f) ++e;
    return e;
}

struct AppendArgs {
    AppendLaunch a;
    int touched;  // pages a sequence's new tokens can touch
};

__device__ void check_append(const AppendArgs &g) {
    const AppendLaunch &a = g.a;
    const int64_t capacity = static_cast<int64_t>(a.pool.max_pages) * a.pool.block;
    bool bad = false;
    const int64_t all = static_cast<int64_t>(a.B) * g.touched;
    for (int64_t i = threadIdx.x; i < all; i += kAppendThreads) {
        const int64_t b = i / g.touched;
        const int64_t start = a.start[b], n = a.new_lens ? a.new_lens[b] : a.T;
        if (start < 0 || n < 0 || n > a.T || start + n > capacity) bad = true;
        const int64_t count = append_count(start, n, a.T, capacity);
        if (count <= 0) continue;
        const int64_t pg = start / a.pool.block + i % g.touched;
        const PageSpan sp = page_span(start, count, pg, a.pool.block);
        if (sp.lo < sp.hi && checked_page(a.pool.table[b * a.pool.max_pages + pg], a.pool.num_pages) < 0) bad = true;
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.dev_status = any ? FVATTN_ERR_BAD_PAGE : FVATTN_OK;
}

template <int D, int BS, bool HALF>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs g) {
    constexpr int TPT = D / 16;                  // threads of a token: two vectors of 8 channels each
    constexpr int TOKS = kAppendThreads / TPT;   // tokens a pass covers
    constexpr int PASSES = BS > TOKS ? BS / TOKS : 1;
    __shared__ float warp_max[kAppendThreads / 32];
    const AppendLaunch &a = g.a;
    if (blockIdx.x == 0) {
        check_append(g);
        return;
    }
    int64_t x = static_cast<int64_t>(blockIdx.x) - 1;
    const bool is_v = x & 1;
    x >>= 1;
    const int h = static_cast<int>(x % a.pool.heads);
    x /= a.pool.heads;
    const int j = static_cast<int>(x % g.touched);
    const int64_t b = x / g.touched;

    const int64_t capacity = static_cast<int64_t>(a.pool.max_pages) * BS;
    const int64_t start = a.start[b];
    const int64_t n = append_count(start, a.new_lens ? a.new_lens[b] : a.T, a.T, capacity);
    if (n <= 0) return;
    const int64_t pg = start / BS + j;
    const PageSpan sp = page_span(start, n, pg, BS);
    if (sp.lo >= sp.hi) return;
    const int page = checked_page(a.pool.table[b * a.pool.max_pages + pg], a.pool.num_pages);
    if (page < 0) return;

    const int64_t ph = static_cast<int64_t>(page) * a.pool.heads + h;
    uint8_t *codes = (is_v ? a.pool.v : a.pool.k) + ph * (BS * D);
    int32_t *exps = (is_v ? a.pool.ve : a.pool.ke) + ph;
    const __nv_bfloat16 *src = is_v ? static_cast<const __nv_bfloat16 *>(a.V) + b * a.v_b + h * a.v_h
                                    : static_cast<const __nv_bfloat16 *>(a.K) + b * a.k_b + h * a.k_h;
    const int64_t src_n = is_v ? a.v_n : a.k_n;
    const bool turn = !is_v && a.pos != nullptr;
    const bool older = sp.lo > 0;  // slots before the first new token hold older ones
    const int e_old = older ? clamp_exp(*exps) : kZeroPageExp;

    // the thread's two vectors: D/2 channels apart, or the two halves of the pairs' channels
    const int i = threadIdx.x % TPT;
    int ca = 8 * i, cb = 8 * i + D / 2;
    uint32_t on = 0;  // pairs that turn
    int pa = ca / 2, pb = cb / 2;
    if (HALF && turn) {
        const int half = a.rope.n_pairs / 8;
        if (i < half) {
            cb = ca + a.rope.n_pairs;
            on = 0xffu;
        } else {
            ca = 2 * a.rope.n_pairs + 16 * (i - half);
            cb = ca + 8;
        }
        pa = 8 * i;
        pb = 8 * i + 4;
    } else if (turn) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            on |= (pa + w < a.rope.n_pairs ? 1u : 0u) << w;
            on |= (pb + w < a.rope.n_pairs ? 1u : 0u) << (4 + w);
        }
    }

    uint4 ra[PASSES], rb[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int slot = sp.lo + p * TOKS + static_cast<int>(threadIdx.x) / TPT;
        ra[p] = rb[p] = make_uint4(0, 0, 0, 0);
        if (slot < sp.hi) {
            const __nv_bfloat16 *row = src + (sp.token + (slot - sp.lo)) * src_n;
            ra[p] = __ldg(reinterpret_cast<const uint4 *>(row + ca));
            rb[p] = __ldg(reinterpret_cast<const uint4 *>(row + cb));
        }
    }
    float v[PASSES][16];
    float amax = 0.0f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int slot = sp.lo + p * TOKS + static_cast<int>(threadIdx.x) / TPT;
        const uint32_t w[8] = {ra[p].x, ra[p].y, ra[p].z, ra[p].w, rb[p].x, rb[p].y, rb[p].z, rb[p].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[p][2 * k] = rope_bf16_lo(w[k]);
            v[p][2 * k + 1] = rope_bf16_hi(w[k]);
        }
        if (turn && slot < sp.hi) {
            const int64_t t = sp.token + (slot - sp.lo);
            const RopePos x = rope_load_pos(a.pos + b * a.pos_b + t * a.rope.n_axes, a.rope.n_axes);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (!((on >> k) & 1u)) continue;
                const int pair = k < 4 ? pa + k : pb + k - 4;
                float c, s;
                rope_cos_sin(rope_coord(x, a.rope.axis[pair]), a.rope.turns[pair], c, s);
                // interleaved: channels 2k, 2k+1 of the 16; half: k and 8 + k
                const int m0 = HALF ? k : 2 * k, m1 = HALF ? 8 + k : 2 * k + 1;
                const float y0 = v[p][m0], y1 = v[p][m1];
                v[p][m0] = fmaf(y0, c, -y1 * s);
                v[p][m1] = fmaf(y1, c, y0 * s);
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(v[p][k]));  // fmaxf leaves NaN out
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
    const int need = need_exp(amax);
    const int e = max(e_old, need);
    if (threadIdx.x == 0) *exps = e;

    if (older && e > e_old) {
        const int shift = max(e_old - e, -250);
        uint4 *old = reinterpret_cast<uint4 *>(codes);
        for (int q = threadIdx.x; q < sp.lo * (D / 16); q += kAppendThreads) {
            const uint4 c4 = old[q];
            uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x0 = values2(c[k] & 0xffffu), x1 = values2(c[k] >> 16);
                c[k] = codes2(scale_pow2(x0.x, shift), scale_pow2(x0.y, shift)) |
                       (codes2(scale_pow2(x1.x, shift), scale_pow2(x1.y, shift)) << 16);
            }
            old[q] = make_uint4(c[0], c[1], c[2], c[3]);
        }
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int slot = sp.lo + p * TOKS + static_cast<int>(threadIdx.x) / TPT;
        if (slot >= sp.hi) continue;
        uint32_t c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            c[k] = codes2(scale_pow2(v[p][2 * k], -e), scale_pow2(v[p][2 * k + 1], -e));
        uint8_t *row = codes + slot * D;
        *reinterpret_cast<uint2 *>(row + ca) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        *reinterpret_cast<uint2 *>(row + cb) = make_uint2(c[4] | (c[5] << 16), c[6] | (c[7] << 16));
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendLaunch &a, cudaStream_t stream) {
    AppendArgs g{a, static_cast<int>(max_touched_pages(a.T, a.pool.block))};
    const int64_t ctas = static_cast<int64_t>(a.B) * g.touched * a.pool.heads * 2 + 1;
    const unsigned grid = static_cast<unsigned>(ctas);
#define FVATTN_APPEND(D_, B_) \
    (a.half ? append_kernel<D_, B_, true><<<grid, kAppendThreads, 0, stream>>>(g) \
            : append_kernel<D_, B_, false><<<grid, kAppendThreads, 0, stream>>>(g))
    if (a.pool.d == 128) a.pool.block == 128 ? FVATTN_APPEND(128, 128) : FVATTN_APPEND(128, 64);
    else a.pool.block == 128 ? FVATTN_APPEND(64, 128) : FVATTN_APPEND(64, 64);
#undef FVATTN_APPEND
    return cudaGetLastError();
}

}  // namespace fvattn
