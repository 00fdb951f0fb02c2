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
// What bounds it: HBM for long calls (2 bytes in, 1 byte out per element), launch latency
// for single tokens.  One group of threads owns the page of a head while it is appended to, its
// exponent and its rows: no atomics, nothing written twice.  The values stay in registers
// between the maximum and the rounding: one read.
//   Up to 8 tokens: a warp per (sequence, touched page, head, K or V), 4 to a CTA.
//   More: a CTA of 512 threads per (sequence, touched page, K or V) and group of heads.  The
//   angles belong to the tokens, so it computes their cosines and sines once, keeps them in
//   registers and walks its heads, the next head's rows in flight.  (With a CTA per head, each
//   computing its angles, 4680 tokens of 40 heads, d 128, took 85 us.)
// The CTA behind the last does no work of its own: it checks starts, counts and page table entries
// and writes the status word, so that the call is one launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "cache.cuh"
#include "common.cuh"

namespace fvattn {

namespace {

constexpr int kFewTokens = 8;   // up to here a warp per page
constexpr int kFewWarps = 4;    // of them in a CTA

// Threads of a CTA that owns a page: two vectors of 8 channels each per pass, at most 512.
constexpr int append_threads(int d, int block) { return block * d / 16 < 512 ? block * d / 16 : 512; }

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
    int touched;          // pages a sequence's new tokens can touch
    int heads_per_group;  // heads a group of threads walks
    int groups;
};

__device__ void check_append(const AppendArgs &g) {
    const AppendLaunch &a = g.a;
    const int64_t capacity = static_cast<int64_t>(a.pool.max_pages) * a.pool.block;
    bool bad = false;
    const int64_t all = static_cast<int64_t>(a.B) * g.touched;
    for (int64_t i = threadIdx.x; i < all; i += blockDim.x) {
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

// THREADS threads (a warp, or the whole CTA) own a page; tokens beyond PASSES times what they cover
// at once do not occur (a page's slots, or kFewTokens).
template <int D, bool HALF, int THREADS, int PASSES>
__global__ void __launch_bounds__(THREADS == 32 ? 32 * kFewWarps : THREADS)
    append_kernel(const __grid_constant__ AppendArgs g) {
    constexpr int TPT = D / 16;            // threads of a token: two vectors of 8 channels each
    constexpr int TOKS = THREADS / TPT;    // tokens a pass covers
    constexpr int WARPS = THREADS / 32;
    __shared__ float warp_max[2][WARPS];   // by turns, so that one barrier a head is enough
    const AppendLaunch &a = g.a;
    if (blockIdx.x == gridDim.x - 1) {
        check_append(g);
        return;
    }
    const int tid = static_cast<int>(threadIdx.x) % THREADS;
    int64_t x = THREADS == 32 ? static_cast<int64_t>(blockIdx.x) * kFewWarps + threadIdx.x / 32 : blockIdx.x;
    const bool is_v = x & 1;
    x >>= 1;
    const int h0 = static_cast<int>(x % g.groups) * g.heads_per_group;
    const int h1 = min(h0 + g.heads_per_group, a.pool.heads);
    x /= g.groups;
    const int j = static_cast<int>(x % g.touched);
    const int64_t b = x / g.touched;
    if (b >= a.B) return;  // (warps: the last CTA may have more than there are pages)

    const int BS = a.pool.block;
    const int64_t capacity = static_cast<int64_t>(a.pool.max_pages) * BS;
    const int64_t start = a.start[b];
    const int64_t n = append_count(start, a.new_lens ? a.new_lens[b] : a.T, a.T, capacity);
    if (n <= 0) return;
    const int64_t pg = start / BS + j;
    const PageSpan sp = page_span(start, n, pg, BS);
    if (sp.lo >= sp.hi) return;
    const int page = checked_page(a.pool.table[b * a.pool.max_pages + pg], a.pool.num_pages);
    if (page < 0) return;

    uint8_t *codes = (is_v ? a.pool.v : a.pool.k) + static_cast<int64_t>(page) * a.pool.heads * BS * D;
    int32_t *exps = (is_v ? a.pool.ve : a.pool.ke) + static_cast<int64_t>(page) * a.pool.heads;
    const __nv_bfloat16 *src = is_v ? static_cast<const __nv_bfloat16 *>(a.V) + b * a.v_b
                                    : static_cast<const __nv_bfloat16 *>(a.K) + b * a.k_b;
    const int64_t src_n = is_v ? a.v_n : a.k_n, src_h = is_v ? a.v_h : a.k_h;
    const bool turn = !is_v && a.pos != nullptr;
    const bool older = sp.lo > 0;  // slots before the first new token hold older ones

    // the thread's two vectors: D/2 channels apart, or the two halves of the pairs' channels
    const int i = tid % TPT;
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
    const int slot0 = sp.lo + tid / TPT;  // of pass 0
    uint4 ra[PASSES], rb[PASSES];
    auto load = [&](int h) {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int slot = slot0 + p * TOKS;
            ra[p] = rb[p] = make_uint4(0, 0, 0, 0);
            if (slot < sp.hi) {
                const __nv_bfloat16 *row = src + h * src_h + (sp.token + (slot - sp.lo)) * src_n;
                ra[p] = __ldg(reinterpret_cast<const uint4 *>(row + ca));
                rb[p] = __ldg(reinterpret_cast<const uint4 *>(row + cb));
            }
        }
    };
    load(h0);
    int e_next = older ? exps[h0] : kZeroPageExp;
    float c[PASSES][8], s[PASSES][8];
    if (turn) {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int slot = slot0 + p * TOKS;
            if (slot >= sp.hi) continue;
            const RopePos at = rope_load_pos(a.pos + b * a.pos_b + (sp.token + (slot - sp.lo)) * a.rope.n_axes, a.rope.n_axes);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                c[p][k] = 1.0f;
                s[p][k] = 0.0f;
                const int pair = k < 4 ? pa + k : pb + k - 4;
                if ((on >> k) & 1u) rope_cos_sin(rope_coord(at, a.rope.axis[pair]), a.rope.turns[pair], c[p][k], s[p][k]);
            }
        }
    }
    for (int h = h0; h < h1; ++h) {
        const int e_old = clamp_exp(e_next);
        float v[PASSES][16];
        float amax = 0.0f;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const uint32_t w[8] = {ra[p].x, ra[p].y, ra[p].z, ra[p].w, rb[p].x, rb[p].y, rb[p].z, rb[p].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[p][2 * k] = rope_bf16_lo(w[k]);
                v[p][2 * k + 1] = rope_bf16_hi(w[k]);
            }
        }
        if (h + 1 < h1) {
            load(h + 1);
            e_next = older ? exps[h + 1] : kZeroPageExp;
        }
        if (turn) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                if (slot0 + p * TOKS >= sp.hi) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    // interleaved: channels 2k, 2k+1 of the 16; half: k and 8 + k
                    const int m0 = HALF ? k : 2 * k, m1 = HALF ? 8 + k : 2 * k + 1;
                    const float y0 = v[p][m0], y1 = v[p][m1];
                    if ((on >> k) & 1u) {
                        v[p][m0] = fmaf(y0, c[p][k], -y1 * s[p][k]);
                        v[p][m1] = fmaf(y1, c[p][k], y0 * s[p][k]);
                    }
                }
            }
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
#pragma unroll
            for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(v[p][k]));  // fmaxf leaves NaN out
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if constexpr (WARPS > 1) {
            float *wm = warp_max[(h - h0) & 1];
            if ((tid & 31) == 0) wm[tid >> 5] = amax;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WARPS; ++w) amax = fmaxf(amax, wm[w]);
        }
        const int e = max(e_old, need_exp(amax));
        if (tid == 0) exps[h] = e;
        uint8_t *rows = codes + static_cast<int64_t>(h) * BS * D;
        if (older && e > e_old) {
            const int shift = max(e_old - e, -250);
            uint4 *old = reinterpret_cast<uint4 *>(rows);
            for (int q = tid; q < sp.lo * (D / 16); q += THREADS) {
                const uint4 c4 = old[q];
                uint32_t o4[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x0 = values2(o4[k] & 0xffffu), x1 = values2(o4[k] >> 16);
                    o4[k] = codes2(scale_pow2(x0.x, shift), scale_pow2(x0.y, shift)) |
                            (codes2(scale_pow2(x1.x, shift), scale_pow2(x1.y, shift)) << 16);
                }
                old[q] = make_uint4(o4[0], o4[1], o4[2], o4[3]);
            }
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int slot = slot0 + p * TOKS;
            if (slot >= sp.hi) continue;
            uint32_t q[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) q[k] = codes2(scale_pow2(v[p][2 * k], -e), scale_pow2(v[p][2 * k + 1], -e));
            uint8_t *row = rows + slot * D;
            *reinterpret_cast<uint2 *>(row + ca) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
            *reinterpret_cast<uint2 *>(row + cb) = make_uint2(q[4] | (q[5] << 16), q[6] | (q[7] << 16));
        }
    }
}

template <int D, bool HALF>
cudaError_t launch_append_t(AppendArgs &g, int sms, cudaStream_t stream) {
    const AppendLaunch &a = g.a;
    const int64_t pages = static_cast<int64_t>(a.B) * g.touched * 2;  // K and V apart
    if (a.T <= kFewTokens) {
        g.heads_per_group = 1;
        g.groups = a.pool.heads;
        const unsigned ctas = static_cast<unsigned>(ceil_div(pages * g.groups, kFewWarps)) + 1;
        append_kernel<D, HALF, 32, kFewTokens * (D / 16) / 32><<<ctas, 32 * kFewWarps, 0, stream>>>(g);
        return cudaGetLastError();
    }
    // heads to a CTA: as many as leave about four CTAs per SM
    const int64_t per = pages * a.pool.heads / (4LL * sms);
    g.heads_per_group = static_cast<int>(per < 1 ? 1 : per < a.pool.heads ? per : a.pool.heads);
    g.groups = static_cast<int>(ceil_div(a.pool.heads, g.heads_per_group));
    const unsigned ctas = static_cast<unsigned>(pages * g.groups) + 1;
    if (a.pool.block == 128) {
        constexpr int T = append_threads(D, 128);
        append_kernel<D, HALF, T, 128 * (D / 16) / T><<<ctas, T, 0, stream>>>(g);
    } else {
        constexpr int T = append_threads(D, 64);
        append_kernel<D, HALF, T, 64 * (D / 16) / T><<<ctas, T, 0, stream>>>(g);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const AppendLaunch &a, int sms, cudaStream_t stream) {
    AppendArgs g{a, static_cast<int>(max_touched_pages(a.T, a.pool.block)), 1, 1};
    if (a.pool.d == 128) return a.half ? launch_append_t<128, true>(g, sms, stream) : launch_append_t<128, false>(g, sms, stream);
    return a.half ? launch_append_t<64, true>(g, sms, stream) : launch_append_t<64, false>(g, sms, stream);
}

}  // namespace fvattn
