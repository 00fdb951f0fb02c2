// cache_attend.cu -- attention of a few new queries per sequence over a paged cache of
// e4m3 keys and values (one power-of-two scale per page and head), and the expansion
// of the pages that the many-queries path reads.
//
// Mathematics: for query row r of key head h (its G query heads times the M new tokens)
// and cached token u of a page with exponents ek, ev:
//   s_u = q_r . k_u 2^ek log2(e)/sqrt(d),   O_r = sum_u 2^(s_u - m) v_u 2^ev / l,
//   l = sum_u 2^(s_u - m),  LSE = (m + log2 l) ln 2.
// One pass with running maxima.  Two of them: m, of the scores, for l; and m + w, of
// s_u + ev, for the products with V, so that the weights 2^(s_u - m + ev - w) <= 1 of pages of
// very different scales stay in range (w is kept relative to m: beside a large score its
// low bits would be lost).  They are scaled by 2^15 and rounded to fp16 (relative
// 2^-11; a weight below 2^-29 of the largest loses bits, below 2^-40 it is zero).  Codes
// convert to fp16 without loss, and so do the query's values after a power-of-two scale per
// row that puts its largest in [2^14, 2^15) (bf16 has fewer bits; values 2^-31 below the
// largest lose bits).  So the products are exact in the tensor cores' fp32 sums.
//
// What bounds it: HBM.  Each cached byte is read once and used for 2 * 8 rows of a matrix
// instruction; one row or eight cost the same.
//
// Why mma.sync: with 1 to 16 rows a tcgen05 tile (M = 64 or 128) would be almost empty, and
// its operands would have to be converted from e4m3 to 16 bits through shared memory.  Here
// the tokens are the M side: S^T = K Q^T and O^T = V^T P^T with m16n8k16, the rows are
// its N = 8, and the A fragments are the cached bytes themselves, loaded from global
// memory straight into the lanes that use them (the order of the channels inside a product
// is free, so each lane takes 16 contiguous bytes) and converted in registers: no shared
// memory, no barrier, each warp its own tokens.  P^T goes from the accumulators' layout to
// the B operand's by one 8x8 transpose per 8 tokens.
//
// Split: the cached tokens of a (sequence, key head, row tile) are cut into chunks, planned
// on the device from the lengths so that the host never waits for them; a persistent grid
// takes the chunks in turn.  A chunk's four warps take 32 tokens at a time, join in shared
// memory, and write either the result (one chunk) or a partial, which a second kernel joins
// in chunk order: no atomics, the same bits every time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <math_constants.h>

#include "cache.cuh"
#include "common.cuh"

namespace fvattn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;               // tokens a warp takes at a time (inside one page: pages hold 64 or 128)
constexpr int kChunkStep = kStep * kWarps;
constexpr int kCtasPerSm = 3;
constexpr int kItemsPerCta = 4;         // chunks a CTA of the grid gets on average
constexpr int kJoinThreads = 128;
constexpr float kWeightLog2 = 15.0f;    // weights are scaled by 2^15 before fp16

// Work plan, written to the workspace by CTA 0 for the joining kernel (and recomputed by
// every CTA for itself): prefix[b] = first work item of sequence b.
struct FewWorkspace {
    size_t prefix, stats, acc, total;
    int64_t items;
};

FewWorkspace few_layout(int B, int64_t groups, int rows, int d, int64_t capacity, int ctas) {
    FewWorkspace w{};
    Carver c;
    w.items = max_items(B, groups, capacity, ctas, kItemsPerCta, kChunkStep);
    w.prefix = c.take<int32_t>(static_cast<size_t>(B) + 1);
    w.stats = c.take<float>(static_cast<size_t>(w.items) * rows * 4);
    w.acc = c.take<float>(static_cast<size_t>(w.items) * rows * d);
    w.total = align_up(c.off, 256);
    return w;
}

struct FewArgs {
    AttendLaunch a;
    int32_t *prefix;
    float4 *stats;  // [items, tile rows]: m, l, w
    float *acc;     // [items, tile rows, d]
    float scale_log2;
    int row_tiles;
    int work_ctas;
    bool join;      // whether a sequence may have more than one chunk
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t two_codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two_codes)));
    return h;
}

__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// D (16 x 8) += A (16 x 16) B (16 x 8), fp16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of the warp's 8x8 matrix of 16-bit values.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// The cached bytes: not kept in L1 (this SM reads them once), kept in L2 as usual (another
// row tile may read them).
__device__ __forceinline__ uint4 load16(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load8(const uint8_t *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
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

// Lengths, counts and the page table entries in use; one CTA, writes the status word.
__device__ void check_attend(const AttendLaunch &a) {
    const int64_t cap = static_cast<int64_t>(a.pool.max_pages) * a.pool.block;
    bool bad = false;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int64_t len = a.lens[b], n = a.new_lens ? a.new_lens[b] : a.M;
        if (len < 0 || len > cap || n < 0 || n > a.M) bad = true;
    }
    const int all = a.B * a.pool.max_pages, stride = static_cast<int>(blockDim.x);
    for (int i0 = threadIdx.x; i0 < all; i0 += 4 * stride) {
        int page[4];
        int64_t len[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // four entries' loads at a time
            const int i = i0 + k * stride;
            page[k] = i < all ? __ldg(a.pool.table + i) : 0;
            len[k] = i < all ? __ldg(a.lens + i / a.pool.max_pages) : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * stride;
            if (i < all && static_cast<int64_t>(i % a.pool.max_pages) * a.pool.block < clamp_len(len[k], cap) &&
                checked_page(page[k], a.pool.num_pages) < 0)
                bad = true;
        }
        if (all - i0 <= 4 * stride) break;  // i0 + 4 stride may pass 2^31
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.dev_status = any ? FVATTN_ERR_BAD_PAGE : FVATTN_OK;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Every CTA makes the same plan from the lengths: the chunk (returned) and the first work
// item of each sequence (prefix[0..B], shared memory).  One warp, the others wait.
__device__ int make_plan(const FewArgs &g, int *prefix, int *chunk_s) {
    const AttendLaunch &a = g.a;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int64_t cap = static_cast<int64_t>(a.pool.max_pages) * a.pool.block;
        const int64_t groups = static_cast<int64_t>(a.pool.heads) * g.row_tiles;
        int64_t tokens = 0;
        for (int b = lane; b < a.B; b += 32) {
            const int64_t len = clamp_len(a.lens[b], cap);
            tokens += len > 0 ? len : 1;
        }
        tokens = warp_sum(tokens);
        int64_t chunk = chunk_tokens(tokens, groups, g.work_ctas, kItemsPerCta, kChunkStep);
        chunk = chunk < (1 << 30) ? chunk : (1 << 30);
        int before = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int n = b < a.B ? static_cast<int>(chunks_of(clamp_len(a.lens[b], cap), chunk) * groups) : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
            }
            if (b < a.B) prefix[b] = before + inc - n;
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            prefix[a.B] = before;
            *chunk_s = static_cast<int>(chunk);
        }
    }
    __syncthreads();
    return *chunk_s;
}

// Largest b with prefix[b] <= item.
__device__ __forceinline__ int find_sequence(const int *prefix, int B, int item) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= item) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A row's sums: l = sum 2^(s - m), acc = 2^15 sum 2^(s - m + ev - w) v.  Without a token m = w =
// -inf and both are 0.
__device__ __forceinline__ float out_factor(float l, float w) {
    return l == 0.0f ? 0.0f : ex2(w - kWeightLog2) / l;
}
// m_old - m_new for a maximum that moved from m_old (or -inf) to m_new.
__device__ __forceinline__ float moved_by(float m_old, float m_new) { return m_old == m_new ? 0.0f : m_old - m_new; }
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
}

// Bytes per lane of one V row: 16 at d 128, 8 at d 64.
template <int D>
struct VRow;
template <>
struct VRow<128> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint8_t *p) {
        const uint4 x = load16(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
};
template <>
struct VRow<64> {
    uint32_t w[2];
    __device__ __forceinline__ void load(const uint8_t *p) {
        const uint2 x = load8(p);
        w[0] = x.x, w[1] = x.y;
    }
};

// One warp's 32 tokens of K and V as the lanes use them.
// K: lane (g = lane / 4, q = lane % 4) has bytes c * 64 + q * 16 .. + 15 (c < D / 64) of tokens
// mt * 16 + half * 8 + g.  V: bytes g * D/8 .. of tokens kg * 16 + {2q, 2q+1, 2q+8, 2q+9}.
template <int D>
struct StepK {
    uint4 x[2][2][D / 64];
};
template <int D>
struct StepV {
    VRow<D> x[2][4];
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? kCtasPerSm : 2) attend_few_kernel(const __grid_constant__ FewArgs g) {
    constexpr int ROWS = 8 * NT;
    constexpr int KS = D / 16;   // k16 steps of K Q^T
    constexpr int MT = D / 16;   // m16 tiles of V^T P^T
    constexpr int VW = D / 32;   // words of a lane's V row
    extern __shared__ int prefix[];
    __shared__ int chunk_s;
    __shared__ float4 stat_s[kWarps][ROWS];
    __shared__ float acc_s[kWarps][8][D];
    const AttendLaunch &a = g.a;
    if (blockIdx.x == 0) {
        make_plan(g, prefix, &chunk_s);
        if (g.join) {
            for (int b = threadIdx.x; b <= a.B; b += kThreads) g.prefix[b] = prefix[b];
        }
        check_attend(a);
        return;
    }
    const int chunk = make_plan(g, prefix, &chunk_s);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = lane >> 2, lq = lane & 3;
    const int BS = a.pool.block, H = a.pool.heads;
    const int R = a.group * a.M;
    const int n_items = prefix[a.B];

    for (int item = static_cast<int>(blockIdx.x) - 1; item < n_items; item += g.work_ctas) {
        const int b = find_sequence(prefix, a.B, item);
        const Seq seq = sequence(a, b);
        const int n_chunks = static_cast<int>(chunks_of(seq.len, chunk));
        int x = item - prefix[b];
        const int ci = x % n_chunks;
        x /= n_chunks;
        const int rt = x % g.row_tiles;
        const int h = x / g.row_tiles;
        const int row0 = rt * ROWS;
        const int rows = min(ROWS, R - row0);

        // query fragments: row nt * 8 + lg, scaled by 2^-sq into fp16
        uint32_t qf[NT][KS][2];
        int sq[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = row0 + nt * 8 + lg;
            const bool in = r < R && r % a.M < seq.n_new;
            const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(a.Q) + b * a.q_b;
            if (in) qr += static_cast<int64_t>(h * a.group + r / a.M) * a.q_h + static_cast<int64_t>(r % a.M) * a.q_n;
            float top = 0.0f;
            uint32_t raw[KS][2];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
#pragma unroll
                for (int w2 = 0; w2 < 2; ++w2) {
                    const uint4 v = in ? __ldg(reinterpret_cast<const uint4 *>(qr + c * 64 + lq * 16 + w2 * 8))
                                       : make_uint4(0, 0, 0, 0);
                    raw[c * 4 + w2 * 2][0] = v.x;
                    raw[c * 4 + w2 * 2][1] = v.y;
                    raw[c * 4 + w2 * 2 + 1][0] = v.z;
                    raw[c * 4 + w2 * 2 + 1][1] = v.w;
                }
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float lo = fabsf(rope_bf16_lo(raw[k][e])), hi = fabsf(rope_bf16_hi(raw[k][e]));
                    if (lo < CUDART_INF_F) top = fmaxf(top, lo);
                    if (hi < CUDART_INF_F) top = fmaxf(top, hi);
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            sq[nt] = top > 0.0f ? ilogbf(top) - 14 : 0;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    qf[nt][k][e] = f16x2_of(scale_pow2(rope_bf16_lo(raw[k][e]), -sq[nt]),
                                            scale_pow2(rope_bf16_hi(raw[k][e]), -sq[nt]));
            }
        }
        // per lane, rows nt * 8 + 2 lq + e: scale exponent, visible tokens, running statistics
        int sqr[NT][2];
        int lim[NT][2];
        float m[NT][2], w[NT][2], l[NT][2];
        int min_lim = seq.len;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = 2 * lq + e, r = row0 + nt * 8 + rr;
                sqr[nt][e] = __shfl_sync(0xffffffffu, sq[nt], rr * 4);
                const int tok = r < R ? r % a.M : a.M;
                lim[nt][e] = r < R ? row_limit(a, seq, tok) : 0;
                if (r < R && tok < seq.n_new) min_lim = min(min_lim, lim[nt][e]);
                m[nt][e] = w[nt][e] = -CUDART_INF_F;
                l[nt][e] = 0.0f;
            }
        }
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 1));
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 2));
        float o[NT][MT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.0f;

        // (2^31 tokens: ci * chunk < len + chunk stays below 2^32)
        const int c0 = static_cast<int>(min(static_cast<int64_t>(ci) * chunk, static_cast<int64_t>(seq.len)));
        const int c1 = seq.n_new == 0 ? c0 : c0 + min(chunk, seq.len - c0);
        const int32_t *table = a.pool.table + static_cast<int64_t>(b) * a.pool.max_pages;
        // the page and head of the step at `tok` (or -1), and its first byte
        auto page_at = [&](int tok) -> int64_t {
            if (tok >= c1) return -1;
            const int p = checked_page(__ldg(table + tok / BS), a.pool.num_pages);
            return p < 0 ? -1 : static_cast<int64_t>(p) * H + h;
        };
        StepK<D> kx;
        StepV<D> vx;
        int ek = 0, ev = 0;
        auto load_k = [&](int64_t ph, int tok) {
            if (ph < 0) return;
            const uint8_t *p = a.pool.k + (ph * BS + (tok & (BS - 1))) * D + lg * D + lq * 16;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) kx.x[mt][hf][c] = load16(p + (mt * 16 + hf * 8) * D + c * 64);
        };
        auto load_v = [&](int64_t ph, int tok) {
            if (ph < 0) return;
            const uint8_t *p = a.pool.v + (ph * BS + (tok & (BS - 1))) * D + lg * (D / 8) + 2 * lq * D;
#pragma unroll
            for (int kg = 0; kg < 2; ++kg)
#pragma unroll
                for (int t = 0; t < 4; ++t) vx.x[kg][t].load(p + (kg * 16 + (t >> 1) * 8 + (t & 1)) * D);
        };
        int tok = c0 + warp * kStep;
        int64_t ph = page_at(tok), ph_next = page_at(tok + kChunkStep);
        load_k(ph, tok);
        load_v(ph, tok);
        if (ph >= 0) {
            ek = __ldg(a.pool.ke + ph);
            ev = __ldg(a.pool.ve + ph);
        }
        for (; tok < c1; tok += kChunkStep) {
            const int tok_next = tok + kChunkStep;
            const int64_t ph_after = page_at(tok_next + kChunkStep);
            int ek_next = 0, ev_next = 0;
            if (ph_next >= 0) {
                ek_next = __ldg(a.pool.ke + ph_next);
                ev_next = __ldg(a.pool.ve + ph_next);
            }
            if (ph < 0) {  // a page table entry outside the pool: its tokens are left out
                load_k(ph_next, tok_next);
                load_v(ph_next, tok_next);
                ph = ph_next, ph_next = ph_after, ek = ek_next, ev = ev_next;
                continue;
            }
            // S^T = K Q^T
            float s[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[nt][mt][k] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint4 &x0 = kx.x[mt][0][k >> 2], &x1 = kx.x[mt][1][k >> 2];
                    const uint32_t w0 = (k & 3) == 0 ? x0.x : (k & 3) == 1 ? x0.y : (k & 3) == 2 ? x0.z : x0.w;
                    const uint32_t w1 = (k & 3) == 0 ? x1.x : (k & 3) == 1 ? x1.y : (k & 3) == 2 ? x1.z : x1.w;
                    const uint32_t a0 = f16x2_of_codes(w0 & 0xffffu), a1 = f16x2_of_codes(w1 & 0xffffu);
                    const uint32_t a2 = f16x2_of_codes(w0 >> 16), a3 = f16x2_of_codes(w1 >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[nt][mt], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
                }
            }
            load_k(ph_next, tok_next);
            const bool edge = tok + kStep > min_lim;
            const float evf = static_cast<float>(clamp_exp(ev));
            // weights for V, transposed into the B operand
            uint32_t pf[NT][2][2];
            float alpha[NT][2];
            bool moved = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = ldexpf(g.scale_log2, sqr[nt][e] + clamp_exp(ek));
                    float mx = -CUDART_INF_F;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            float &v = s[nt][mt][2 * hf + e];
                            v *= f;
                            if (edge && tok + mt * 16 + hf * 8 + lg >= lim[nt][e]) v = -CUDART_INF_F;
                            mx = fmaxf(mx, v);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float m_new = fmaxf(m[nt][e], mx);
                    const float m_ref = m_new == -CUDART_INF_F ? 0.0f : m_new;
                    const float shift = moved_by(m[nt][e], m_new);
                    const float w_old = w[nt][e] + shift;
                    const float w_new = fmaxf(w_old, mx - m_ref + evf);
                    const float w_off = w_new == -CUDART_INF_F ? 0.0f : evf + kWeightLog2 - w_new;
                    const float al = ex2(shift);
                    const bool grew = w_new != w_old && w_old != -CUDART_INF_F;
                    alpha[nt][e] = grew ? ex2(w_old - w_new) : 1.0f;
                    moved |= grew;
                    float sum = 0.0f;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            float &v = s[nt][mt][2 * hf + e];
                            const float t = v - m_ref;
                            sum += ex2(t);
                            v = ex2(t + w_off);
                        }
                    l[nt][e] = l[nt][e] * al + sum;
                    m[nt][e] = m_new;
                    w[nt][e] = w_new;
                }
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        pf[nt][mt][hf] = transpose8x8(f16x2_of(s[nt][mt][2 * hf], s[nt][mt][2 * hf + 1]));
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[nt][i][k] *= alpha[nt][k & 1];
            }
            // A step that some row sees only in part (the sequence's end, the causal edge): a
            // NaN among the values of a token that a row does not see must not reach it through
            // 0 * NaN.  NaN codes become zero, and the rows that do see one get it back below: what
            // a row sees is a prefix, so the first NaN of a channel decides.
            bool nan_here = false;
            if (edge) {
#pragma unroll
                for (int kg = 0; kg < 2; ++kg)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int k = 0; k < VW; ++k) nan_here |= any_nan_e4m3(vx.x[kg][t].w[k]);
                nan_here = __any_sync(0xffffffffu, nan_here);
            }
            if (nan_here) {
                for (int i = 0; i < MT; ++i) {
                    for (int half = 0; half < 2; ++half) {
                        const int byte = 2 * i + half, word = byte >> 2, sh = (byte & 3) * 8;
                        int first = kStep;
#pragma unroll
                        for (int kg = 0; kg < 2; ++kg)
#pragma unroll
                            for (int t = 0; t < 4; ++t)
#pragma unroll
                                for (int k = 0; k < VW; ++k)
                                    if (k == word && ((vx.x[kg][t].w[k] >> sh) & 0x7fu) == 0x7fu) {
                                        first = min(first, kg * 16 + (t >> 1) * 8 + (t & 1) + 2 * lq);
                                        vx.x[kg][t].w[k] &= ~(0xffu << sh);
                                    }
                        first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
                        first = min(first, __shfl_xor_sync(0xffffffffu, first, 2));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int ii = 0; ii < MT; ++ii)
                                    if (ii == i && first < kStep && tok + first < lim[nt][e]) {
                                        if (half) o[nt][ii][2 + e] = CUDART_NAN_F;
                                        else o[nt][ii][e] = CUDART_NAN_F;
                                    }
                    }
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int kg = 0; kg < 2; ++kg) {
#pragma unroll
                for (int k = 0; k < VW; ++k) {
#pragma unroll
                    for (int pair = 0; pair < 2; ++pair) {  // bytes 0, 1 and 2, 3 of the word: channels 4k + 2 pair, + 1
                        const uint32_t sel = pair ? 0x7362u : 0x5140u;
                        const uint32_t x01 = prmt(vx.x[kg][0].w[k], vx.x[kg][1].w[k], sel);
                        const uint32_t x23 = prmt(vx.x[kg][2].w[k], vx.x[kg][3].w[k], sel);
                        const uint32_t a0 = f16x2_of_codes(x01 & 0xffffu), a1 = f16x2_of_codes(x01 >> 16);
                        const uint32_t a2 = f16x2_of_codes(x23 & 0xffffu), a3 = f16x2_of_codes(x23 >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[nt][2 * k + pair], a0, a1, a2, a3, pf[nt][kg][0], pf[nt][kg][1]);
                    }
                }
            }
            load_v(ph_next, tok_next);
            ph = ph_next, ph_next = ph_after, ek = ek_next, ev = ev_next;
        }

        // join the warps: statistics, then eight rows at a time
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (lg == 0) stat_s[warp][nt * 8 + 2 * lq + e] = make_float4(m[nt][e], sum, w[nt][e], 0.0f);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt * 8 >= rows) break;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int ch = lg * (D / 8) + 2 * i;
                if (nt * 8 + 2 * lq < rows)
                    *reinterpret_cast<float2 *>(&acc_s[warp][2 * lq][ch]) = make_float2(o[nt][i][0], o[nt][i][2]);
                if (nt * 8 + 2 * lq + 1 < rows)
                    *reinterpret_cast<float2 *>(&acc_s[warp][2 * lq + 1][ch]) = make_float2(o[nt][i][1], o[nt][i][3]);
            }
            __syncthreads();
            for (int y = threadIdx.x; y < min(8, rows - nt * 8) * (D / 4); y += kThreads) {
                const int rr = y / (D / 4), ch = (y % (D / 4)) * 4;
                const int r = row0 + nt * 8 + rr;
                float mm = -CUDART_INF_F, ww = -CUDART_INF_F;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, stat_s[k][nt * 8 + rr].x);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float4 st = stat_s[k][nt * 8 + rr];
                    ww = fmaxf(ww, st.z + moved_by(st.x, mm));
                }
                float ll = 0.0f;
                float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float4 st = stat_s[k][nt * 8 + rr];
                    const float4 v = *reinterpret_cast<const float4 *>(&acc_s[k][rr][ch]);
                    const float shift = moved_by(st.x, mm);
                    // (without a token the sums are 0, or NaN)
                    ll += st.x == -CUDART_INF_F ? st.y : st.y * ex2(shift);
                    const float f = st.z == -CUDART_INF_F ? 1.0f : ex2(st.z + shift - ww);
                    sum.x += v.x * f, sum.y += v.y * f, sum.z += v.z * f, sum.w += v.w * f;
                }
                if (n_chunks > 1) {
                    const int64_t at = static_cast<int64_t>(item) * ROWS + nt * 8 + rr;
                    if (ch == 0) g.stats[at] = make_float4(mm, ll, ww, 0.0f);
                    *reinterpret_cast<float4 *>(g.acc + at * D + ch) = sum;
                } else if (r % a.M < seq.n_new) {
                    const int64_t hq = h * a.group + r / a.M, tokq = r % a.M;
                    const float f = out_factor(ll, ww);
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.O) + b * a.o_b + hq * a.o_h + tokq * a.o_n + ch;
                    const __nv_bfloat162 p0 = __floats2bfloat162_rn(sum.x * f, sum.y * f);
                    const __nv_bfloat162 p1 = __floats2bfloat162_rn(sum.z * f, sum.w * f);
                    *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&p0),
                                                                 *reinterpret_cast<const uint32_t *>(&p1));
                    if (ch == 0)
                        a.LSE[(static_cast<int64_t>(b) * H * a.group + hq) * a.M + tokq] = lse_of(mm, ll);
                }
            }
            __syncthreads();
        }
    }
}

// Joins the chunks of one row: grid (row of the tile's heads, sequence).  The chunks go to the
// CTA's groups of D / 4 threads in turn and the groups are added in order.
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const __grid_constant__ FewArgs g) {
    constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
    __shared__ float4 acc_s[GROUPS][LANES];
    __shared__ float3 stat_s[GROUPS];
    const AttendLaunch &a = g.a;
    const int b = blockIdx.y;
    const int R = a.group * a.M;
    const int h = blockIdx.x / R, r = blockIdx.x % R;
    const Seq seq = sequence(a, b);
    const int groups = a.pool.heads * g.row_tiles;
    const int first_item = g.prefix[b];
    const int n_chunks = (g.prefix[b + 1] - first_item) / groups;
    if (n_chunks <= 1 || r % a.M >= seq.n_new) return;
    const int rt = r / ROWS;
    const int64_t at0 = (static_cast<int64_t>(first_item) + static_cast<int64_t>(h * g.row_tiles + rt) * n_chunks) * ROWS +
                        r % ROWS;
    const int grp = threadIdx.x / LANES, ch = (threadIdx.x % LANES) * 4;
    float m = -CUDART_INF_F, w = -CUDART_INF_F, l = 0.0f;
    for (int c = grp; c < n_chunks; c += GROUPS) m = fmaxf(m, g.stats[at0 + static_cast<int64_t>(c) * ROWS].x);
    for (int c = grp; c < n_chunks; c += GROUPS) {
        const float4 st = g.stats[at0 + static_cast<int64_t>(c) * ROWS];
        w = fmaxf(w, st.z + moved_by(st.x, m));
    }
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = grp; c < n_chunks; c += GROUPS) {
        const int64_t at = at0 + static_cast<int64_t>(c) * ROWS;
        const float4 st = g.stats[at];
        const float4 v = *reinterpret_cast<const float4 *>(g.acc + at * D + ch);
        const float shift = moved_by(st.x, m);
        l += st.x == -CUDART_INF_F ? st.y : st.y * ex2(shift);
        const float f = st.z == -CUDART_INF_F ? 1.0f : ex2(st.z + shift - w);
        sum.x += v.x * f, sum.y += v.y * f, sum.z += v.z * f, sum.w += v.w * f;
    }
    acc_s[grp][threadIdx.x % LANES] = sum;
    if (ch == 0) stat_s[grp] = make_float3(m, l, w);
    __syncthreads();
    if (grp != 0) return;
    float mm = -CUDART_INF_F, ww = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) mm = fmaxf(mm, stat_s[k].x);
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) ww = fmaxf(ww, stat_s[k].z + moved_by(stat_s[k].x, mm));
    float ll = 0.0f;
    float4 all = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
        const float3 st = stat_s[k];
        const float4 v = acc_s[k][threadIdx.x];
        const float shift = moved_by(st.x, mm);
        ll += st.x == -CUDART_INF_F ? st.y : st.y * ex2(shift);
        const float f = st.z == -CUDART_INF_F ? 1.0f : ex2(st.z + shift - ww);
        all.x += v.x * f, all.y += v.y * f, all.z += v.z * f, all.w += v.w * f;
    }
    const int64_t hq = h * a.group + r / a.M, tokq = r % a.M;
    const float f = out_factor(ll, ww);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.O) + b * a.o_b + hq * a.o_h + tokq * a.o_n + ch;
    const __nv_bfloat162 p0 = __floats2bfloat162_rn(all.x * f, all.y * f);
    const __nv_bfloat162 p1 = __floats2bfloat162_rn(all.z * f, all.w * f);
    *reinterpret_cast<uint2 *>(out) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&p0), *reinterpret_cast<const uint32_t *>(&p1));
    if (ch == 0) a.LSE[(static_cast<int64_t>(b) * a.pool.heads * a.group + hq) * a.M + tokq] = lse_of(mm, ll);
}

// ---------------------------------------------------------------- pages as bf16

// Every cached token of every head as bf16 (exact: a code has 4 bits, its scale is a power of
// two), for the 128-row tiles of the tensor cores.  CTA = (page, head, sequence); CTA 0 only
// checks.  Tokens from the sequence's end to the next multiple of 128 are zeros: the tiles read
// them.  NaN codes of V become zero in the copy and the first of each channel is kept in
// nan_first, so that a NaN that a query does not see cannot reach it through 0 * NaN.
constexpr int kExpandThreads = 256;

struct ExpandArgs {
    AttendLaunch a;
    int64_t cap;
    __nv_bfloat16 *K, *V;
    int32_t *nan_first;
    int pages;
};

__device__ __forceinline__ uint4 expand8(uint32_t lo, uint32_t hi, int e) {
    uint32_t out[4];
    const uint32_t c[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = f16x2_of_codes(c[i]);
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        const __nv_bfloat162 y = __floats2bfloat162_rn(scale_pow2(v.x, e), scale_pow2(v.y, e));
        out[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

__global__ void __launch_bounds__(kExpandThreads) cache_expand_kernel(const __grid_constant__ ExpandArgs g) {
    const AttendLaunch &a = g.a;
    if (blockIdx.x == 0) {
        check_attend(a);
        return;
    }
    int64_t x = static_cast<int64_t>(blockIdx.x) - 1;
    const int pg = static_cast<int>(x % g.pages);
    x /= g.pages;
    const int h = static_cast<int>(x % a.pool.heads);
    const int b = static_cast<int>(x / a.pool.heads);
    const int BS = a.pool.block, D = a.pool.d;
    const int64_t len = sequence(a, b).len;
    const int64_t tok0 = static_cast<int64_t>(pg) * BS;
    if (tok0 >= static_cast<int64_t>(align_up(static_cast<size_t>(len), 128))) return;
    const int fill = static_cast<int>(clamp_len(len - tok0, BS));  // cached slots of the page
    const int page = fill > 0 ? checked_page(a.pool.table[static_cast<int64_t>(b) * a.pool.max_pages + pg], a.pool.num_pages) : -1;
    const int64_t ph = static_cast<int64_t>(page < 0 ? 0 : page) * a.pool.heads + h;
    const int64_t bh = static_cast<int64_t>(b) * a.pool.heads + h;
    const int ek = page < 0 ? 0 : clamp_exp(a.pool.ke[ph]), ev = page < 0 ? 0 : clamp_exp(a.pool.ve[ph]);
    const uint2 *kc = reinterpret_cast<const uint2 *>(a.pool.k + ph * BS * D);
    const uint2 *vc = reinterpret_cast<const uint2 *>(a.pool.v + ph * BS * D);
    uint4 *ko = reinterpret_cast<uint4 *>(g.K + (bh * g.cap + tok0) * D);
    uint4 *vo = reinterpret_cast<uint4 *>(g.V + (bh * g.cap + tok0) * D);
    const int per_row = D / 8;
    for (int i = threadIdx.x; i < BS * per_row; i += kExpandThreads) {
        const int slot = i / per_row;
        if (page < 0 || slot >= fill) {
            ko[i] = vo[i] = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint2 kk = __ldcs(kc + i);
        uint2 vv = __ldcs(vc + i);
        ko[i] = expand8(kk.x, kk.y, ek);
        if (any_nan_e4m3(vv.x) || any_nan_e4m3(vv.y)) {
            for (int y = 0; y < 8; ++y) {
                uint32_t &word = y < 4 ? vv.x : vv.y;
                const int sh = (y & 3) * 8;
                if (((word >> sh) & 0x7fu) == 0x7fu) {
                    word &= ~(0xffu << sh);
                    atomicMax(g.nan_first + bh * D + (i % per_row) * 8 + y,
                              0x7fffffff - static_cast<int>(tok0 + slot));
                }
            }
        }
        vo[i] = expand8(vv.x, vv.y, ev);
    }
}

int few_row_tile(int64_t rows) { return rows <= 8 ? 8 : 16; }

// CTAs that take chunks: the resident ones but for the one that checks.
int few_work_ctas(int row_tile, int sms) { return sms * (row_tile == 8 ? kCtasPerSm : 2) - 1; }

}  // namespace

bool attend_few_rows(int group, int M) { return attend_rows(group, M) <= 32; }

size_t attend_few_workspace(int B, int heads, int group, int M, int d, int block, int max_pages, int sms) {
    const int64_t rows = attend_rows(group, M);
    const int tile = few_row_tile(rows);
    return few_layout(B, heads * ceil_div(rows, tile), tile, d, static_cast<int64_t>(max_pages) * block,
                      few_work_ctas(tile, sms)).total;
}

template <int D, int NT>
static cudaError_t launch_few_t(FewArgs &g, int64_t items, cudaStream_t stream) {
    const AttendLaunch &a = g.a;
    const int64_t ctas = items < g.work_ctas ? items : g.work_ctas;
    const size_t smem = (static_cast<size_t>(a.B) + 1) * sizeof(int);
    attend_few_kernel<D, NT><<<static_cast<unsigned>(ctas) + 1, kThreads, smem, stream>>>(g);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !g.join) return e;
    const dim3 grid(static_cast<unsigned>(a.pool.heads * attend_rows(a.group, a.M)), static_cast<unsigned>(a.B));
    attend_join_kernel<D, 8 * NT><<<grid, kJoinThreads, 0, stream>>>(g);
    return cudaGetLastError();
}

cudaError_t launch_attend_few(const AttendLaunch &a, cudaStream_t stream) {
    const int64_t rows = attend_rows(a.group, a.M);
    const int tile = few_row_tile(rows);
    FewArgs g{};
    g.a = a;
    g.row_tiles = static_cast<int>(ceil_div(rows, tile));
    g.work_ctas = few_work_ctas(tile, a.sms);
    const int64_t capacity = static_cast<int64_t>(a.pool.max_pages) * a.pool.block;
    const FewWorkspace w = few_layout(a.B, static_cast<int64_t>(a.pool.heads) * g.row_tiles, tile, a.pool.d, capacity,
                                      g.work_ctas);
    char *ws = static_cast<char *>(a.workspace);
    g.prefix = reinterpret_cast<int32_t *>(ws + w.prefix);
    g.stats = reinterpret_cast<float4 *>(ws + w.stats);
    g.acc = reinterpret_cast<float *>(ws + w.acc);
    g.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(a.pool.d)));
    g.join = capacity > kChunkStep;
    if (a.pool.d == 128) return tile == 8 ? launch_few_t<128, 1>(g, w.items, stream) : launch_few_t<128, 2>(g, w.items, stream);
    return tile == 8 ? launch_few_t<64, 1>(g, w.items, stream) : launch_few_t<64, 2>(g, w.items, stream);
}

cudaError_t launch_cache_expand(const AttendLaunch &a, int64_t cap, void *K, void *V, int32_t *nan_first,
                                cudaStream_t stream) {
    ExpandArgs g{a, cap, static_cast<__nv_bfloat16 *>(K), static_cast<__nv_bfloat16 *>(V), nan_first,
                 static_cast<int>(cap / a.pool.block)};
    const int64_t ctas = static_cast<int64_t>(a.B) * a.pool.heads * g.pages + 1;
    cache_expand_kernel<<<static_cast<unsigned>(ctas), kExpandThreads, 0, stream>>>(g);
    return cudaGetLastError();
}

}  // namespace fvattn
