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
//   Up to 16 tokens (32 at d 64): a warp per (sequence, touched page, head, K or V), 4 to a CTA.
//   More: a resident grid of CTAs with 16 channels of a page to a thread.  All (sequence, touched
//   page, head) form a line of which each takes an equal stretch.  The angles belong to
//   the tokens, so it computes their cosines and sines once a page, keeps them in registers and
//   walks the heads, the next head's rows in flight.  (With a CTA per head, each computing its
//   angles, 4680 tokens of 40 heads, d 128, took 85 us; with as many CTAs as there are groups of
//   5 heads, which leaves the last wave of them mostly empty, 61.)
// Measured: those 4680 tokens 39 us, 3.7 TB/s (a head's maximum needs a barrier of the CTA before its
// rounding, and with one CTA of 1024 threads an SM nothing else runs meanwhile: 62 % of the issue slots);
// 333 ragged tokens of 5 sequences 5.9 us, one token 4.1 us: latency.
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

constexpr int kFewWarps = 4;   // warps that own a page each, in a CTA
constexpr int kFewPasses = 4;  // tokens such a warp takes at most, over those it covers at once

__device__ __forceinline__ float2 values2(uint32_t two_codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two_codes)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The exponent a largest magnitude (not negative) asks for (an infinity: 2^0, as the quantizer
// does): from amax = m 2^x with m in [1, 2), x - 8, and one more if m > 448 / 256.
__device__ __forceinline__ int need_exp(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    if (bits >= 0x7f800000u) return 0;
    if (bits < 0x00800000u) {  // zero or subnormal
        if (bits == 0) return kZeroPageExp;
        const int e = ilogbf(amax) - 8;
        return scale_pow2(amax, -e) > 448.0f ? e + 1 : e;
    }
    return static_cast<int>(bits >> 23) - 135 + ((bits & 0x007fffffu) > 0x00600000u ? 1 : 0);
}

// Largest magnitude of three; NaN is left out.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Four values -> four codes, the first in the low byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{.reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1; cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3; mov.b32 %0, {lo, hi};}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Sixteen values times 2^-e as codes.
__device__ __forceinline__ void codes16(const float (&v)[16], int e, uint32_t (&q)[4]) {
    if (e >= -127 && e <= 126) {  // 2^-e is a normal number
        const float f = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = codes4(v[4 * k] * f, v[4 * k + 1] * f, v[4 * k + 2] * f, v[4 * k + 3] * f);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            q[k] = codes4(scale_pow2(v[4 * k], -e), scale_pow2(v[4 * k + 1], -e), scale_pow2(v[4 * k + 2], -e),
                          scale_pow2(v[4 * k + 3], -e));
    }
}

struct AppendArgs {
    AppendLaunch a;
    int touched;    // pages a sequence's new tokens can touch
    int64_t pages;  // (sequence, touched page, head), in this order
    bool apart;     // K and V of one of them to a warp, or a CTA, each
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

// K (TURN) or V of items [item, item_end) by THREADS threads (a warp, or the whole CTA); tokens
// beyond PASSES times what they cover at once do not occur.
template <int D, bool HALF, bool FULL, int THREADS, int PASSES, bool TURN>
__device__ __forceinline__ void append_items(const AppendArgs &g, int64_t item, int64_t item_end, const RopeTable &table,
                                             float (*warp_max)[THREADS / 32], int &barriers) {
    constexpr int TPT = D / 16;          // threads of a token: two vectors of 8 channels each
    constexpr int TOKS = THREADS / TPT;  // tokens a pass covers
    constexpr int WARPS = THREADS / 32;
    const AppendLaunch &a = g.a;
    const int tid = static_cast<int>(threadIdx.x) % THREADS;
    const int H = a.pool.heads, BS = a.pool.block;
    const int64_t capacity = static_cast<int64_t>(a.pool.max_pages) * BS;
    const int64_t src_b = TURN ? a.k_b : a.v_b, src_h = TURN ? a.k_h : a.v_h, src_n = TURN ? a.k_n : a.v_n;

    // the thread's two vectors: D/2 channels apart, or the two halves of the pairs' channels
    const int i = tid % TPT;
    int ca = 8 * i, cb = 8 * i + D / 2;
    uint32_t on = 0;  // pairs that turn
    int pa = ca / 2, pb = cb / 2;
    const bool turn = TURN && a.pos != nullptr;
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
    while (item < item_end) {
        // heads [h0, h1) of one page
        const int h0 = static_cast<int>(item % H), h1 = static_cast<int>(min(static_cast<int64_t>(H), h0 + (item_end - item)));
        const int64_t x = item / H;
        item += h1 - h0;
        const int j = static_cast<int>(x % g.touched);
        const int64_t b = x / g.touched;
        const int64_t start = a.start[b];
        const int64_t n = append_count(start, a.new_lens ? a.new_lens[b] : a.T, a.T, capacity);
        if (n <= 0) continue;
        const int64_t pg = start / BS + j;
        const PageSpan sp = page_span(start, n, pg, BS);
        if (sp.lo >= sp.hi) continue;
        const int page = checked_page(a.pool.table[b * a.pool.max_pages + pg], a.pool.num_pages);
        if (page < 0) continue;

        const bool older = sp.lo > 0;         // slots before the first new token hold older ones
        const int slot0 = sp.lo + tid / TPT;  // of pass 0
        const int64_t ph = static_cast<int64_t>(page) * H + h0;
        uint8_t *codes = (TURN ? a.pool.k : a.pool.v) + ph * BS * D;
        int32_t *exps = (TURN ? a.pool.ke : a.pool.ve) + ph;
        // the next head's rows, and the exponent its older tokens have
        const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(TURN ? a.K : a.V) + b * src_b + h0 * src_h +
                                    (sp.token + tid / TPT) * src_n;
        uint4 ra[PASSES], rb[PASSES];
        int e_next = kZeroPageExp;
        auto load = [&](int ahead) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                if (slot0 + p * TOKS < sp.hi) {
                    ra[p] = __ldcg(reinterpret_cast<const uint4 *>(from + p * TOKS * src_n + ca));
                    rb[p] = __ldcg(reinterpret_cast<const uint4 *>(from + p * TOKS * src_n + cb));
                }
            }
            from += src_h;
            if (older) e_next = exps[ahead];
        };
        load(0);
        extern __shared__ float4 angles[];  // two pairs' cosines and sines to a float4, the thread's own
        float4 *mine = angles + threadIdx.x;
        const int stride = static_cast<int>(blockDim.x);
        if (turn) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int slot = slot0 + p * TOKS;
                if (slot >= sp.hi) continue;
                const RopePos at =
                    rope_load_pos(a.pos + b * a.pos_b + (sp.token + (slot - sp.lo)) * a.rope.n_axes, a.rope.n_axes);
#pragma unroll
                for (int w = 0; w < 8; w += 2) {
                    float4 cs = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
                    const int pair = w < 4 ? pa + w : pb + w - 4;
                    if ((on >> w) & 1u) rope_cos_sin(rope_coord(at, table.axis[pair]), table.step[pair], cs.x, cs.y);
                    if ((on >> w) & 2u) rope_cos_sin(rope_coord(at, table.axis[pair + 1]), table.step[pair + 1], cs.z, cs.w);
                    mine[(p * 4 + w / 2) * stride] = cs;
                }
            }
        }
        for (int h = h0; h < h1; ++h) {
            const int e_old = clamp_exp(e_next);
            float y[PASSES][16];
            float amax = 0.0f;
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                if (slot0 + p * TOKS >= sp.hi) continue;
                const uint32_t w[8] = {ra[p].x, ra[p].y, ra[p].z, ra[p].w, rb[p].x, rb[p].y, rb[p].z, rb[p].w};
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    y[p][2 * q] = rope_bf16_lo(w[q]);
                    y[p][2 * q + 1] = rope_bf16_hi(w[q]);
                }
            }
            if (h + 1 < h1) load(1);
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                if (slot0 + p * TOKS >= sp.hi) continue;
                if (turn) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 cs = mine[(p * 4 + q / 2) * stride];
                        const float c = q & 1 ? cs.z : cs.x, s = q & 1 ? cs.w : cs.y;
                        // interleaved: channels 2q, 2q+1 of the 16; half: q and 8 + q
                        const int m0 = HALF ? q : 2 * q, m1 = HALF ? 8 + q : 2 * q + 1;
                        const float y0 = y[p][m0], y1 = y[p][m1];
                        if (FULL || ((on >> q) & 1u)) {
                            y[p][m0] = fmaf(y0, c, -y1 * s);
                            y[p][m1] = fmaf(y1, c, y0 * s);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < 16; q += 2) amax = max_abs(amax, y[p][q], y[p][q + 1]);
            }
            // (numbers that are not negative order as their bits do)
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            if constexpr (WARPS > 1) {
                float *wm = warp_max[barriers++ & 1];
                if ((tid & 31) == 0) wm[tid >> 5] = amax;
                __syncthreads();
                const float mine = (tid & 31) < WARPS ? wm[tid & 31] : 0.0f;
                amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine)));
            }
            const int e = max(e_old, need_exp(amax));
            if (tid == 0) *exps = e;
            if (older && e > e_old) {
                const int shift = max(e_old - e, -250);
                uint4 *old = reinterpret_cast<uint4 *>(codes);
                for (int q = tid; q < sp.lo * (D / 16); q += THREADS) {
                    const uint4 c4 = old[q];
                    uint32_t o4[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float2 x0 = values2(o4[w] & 0xffffu), x1 = values2(o4[w] >> 16);
                        o4[w] = codes4(scale_pow2(x0.x, shift), scale_pow2(x0.y, shift), scale_pow2(x1.x, shift),
                                       scale_pow2(x1.y, shift));
                    }
                    old[q] = make_uint4(o4[0], o4[1], o4[2], o4[3]);
                }
            }
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int slot = slot0 + p * TOKS;
                if (slot >= sp.hi) continue;
                uint32_t q[4];
                codes16(y[p], e, q);
                uint8_t *row = codes + slot * D;
                *reinterpret_cast<uint2 *>(row + ca) = make_uint2(q[0], q[1]);
                *reinterpret_cast<uint2 *>(row + cb) = make_uint2(q[2], q[3]);
            }
            codes += BS * D;
            ++exps;
        }
    }
}

template <int D, bool HALF, bool FULL, int THREADS, int PASSES>
__global__ void __launch_bounds__(THREADS == 32 ? 32 * kFewWarps : THREADS, THREADS == 32 ? 1 : 1024 / THREADS)
    append_kernel(const __grid_constant__ AppendArgs g) {
    __shared__ float warp_max[2][THREADS / 32];  // by turns, so that one barrier a head is enough
    __shared__ RopeTable table;
    table.fill(g.a.rope);
    __syncthreads();
    wait_for_stream();
    if (blockIdx.x == gridDim.x - 1) {
        check_append(g);
        return;
    }
    int barriers = 0;
    if (THREADS == 32 || g.apart) {
        const int64_t x = THREADS == 32 ? static_cast<int64_t>(blockIdx.x) * kFewWarps + threadIdx.x / 32 : blockIdx.x;
        const int64_t item = x >> 1, end = min(item + 1, g.pages);
        if (x & 1) append_items<D, HALF, FULL, THREADS, PASSES, false>(g, item, end, table, warp_max, barriers);
        else append_items<D, HALF, FULL, THREADS, PASSES, true>(g, item, end, table, warp_max, barriers);
    } else {  // K, then V, of a stretch of them
        const int64_t item = stretch_start(blockIdx.x, g.pages, gridDim.x - 1);
        const int64_t end = stretch_start(blockIdx.x + 1, g.pages, gridDim.x - 1);
        append_items<D, HALF, FULL, THREADS, PASSES, true>(g, item, end, table, warp_max, barriers);
        append_items<D, HALF, FULL, THREADS, PASSES, false>(g, item, end, table, warp_max, barriers);
    }
}

// The angles' place in shared memory: 64 bytes a thread and pass.
template <int D, bool HALF, bool FULL, int THREADS, int PASSES>
cudaError_t launch_append_k(const AppendArgs &g, int64_t ctas, cudaStream_t stream) {
    constexpr int threads = THREADS == 32 ? 32 * kFewWarps : THREADS, smem = PASSES * 64 * threads;
    const cudaError_t e = allow_shared_memory<append_kernel<D, HALF, FULL, THREADS, PASSES>>(smem);
    if (e != cudaSuccess) return e;
    const cudaLaunchConfig_t cfg = early_launch(dim3(static_cast<unsigned>(ctas) + 1), threads, smem, stream);  // one checks
    return cudaLaunchKernelEx(&cfg, append_kernel<D, HALF, FULL, THREADS, PASSES>, g);
}

template <int D, bool HALF, bool FULL, int THREADS>
cudaError_t launch_append_ctas(AppendArgs g, int sms, cudaStream_t stream) {
    const int64_t resident = static_cast<int64_t>(sms) * (1024 / THREADS) - 1;
    g.apart = 2 * g.pages <= resident;
    const int64_t ctas = g.apart ? 2 * g.pages : g.pages < resident ? g.pages : resident;
    return launch_append_k<D, HALF, FULL, THREADS, 1>(g, ctas, stream);
}

template <int D, bool HALF, bool FULL>
cudaError_t launch_append_t(const AppendArgs &g, int sms, cudaStream_t stream) {
    const AppendLaunch &a = g.a;
    constexpr int covered = 512 / D;  // tokens of a warp at once
    const int64_t few_ctas = ceil_div(2 * g.pages, kFewWarps);
    if (a.T <= covered) return launch_append_k<D, HALF, FULL, 32, 1>(g, few_ctas, stream);
    if (a.T <= kFewPasses * covered) return launch_append_k<D, HALF, FULL, 32, kFewPasses>(g, few_ctas, stream);
    return a.pool.block == 128 ? launch_append_ctas<D, HALF, FULL, 128 * D / 16>(g, sms, stream)
                               : launch_append_ctas<D, HALF, FULL, 64 * D / 16>(g, sms, stream);
}

}  // namespace

cudaError_t launch_cache_append(const AppendLaunch &a, int sms, cudaStream_t stream) {
    const int64_t touched = max_touched_pages(a.T, a.pool.block);
    const AppendArgs g{a, static_cast<int>(touched), a.B * touched * a.pool.heads, true};
    const bool full = !a.pos || 2 * a.rope.n_pairs == a.pool.d;  // every channel turns
#define FVATTN_APPEND(D_) \
    (a.half ? full ? launch_append_t<D_, true, true>(g, sms, stream) : launch_append_t<D_, true, false>(g, sms, stream) \
            : full ? launch_append_t<D_, false, true>(g, sms, stream) : launch_append_t<D_, false, false>(g, sms, stream))
    return a.pool.d == 128 ? FVATTN_APPEND(128) : FVATTN_APPEND(64);
#undef FVATTN_APPEND
}

}  // namespace fvattn
