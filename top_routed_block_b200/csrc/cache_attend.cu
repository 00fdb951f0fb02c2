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
// 2^-11; a weight below 2^-29 of the largest loses bits, below 2^-40 it is zero), and the
// codes of V convert to fp16 without loss.  K takes part as it is, in e4m3: a query's value,
// scaled per row by a power of two, is the sum of two e4m3 numbers, its first 4 bits and 16 times
// the next 4 (bf16 has 8; what is left of values below 2^-15 of the row's largest is at most
// 2^-22 of that).  So the products are exact in the tensor cores' fp32 sums.
//
// What bounds it: HBM.  Each cached byte is read once and used for the 8 rows of a matrix
// instruction; one row or eight cost the same.  More rows take more row tiles of 8, which read
// the same bytes from L2.  (Tiles of 16 and 24 rows, which convert V once for all of them, have no
// registers left to hide latency: 20 rows over 4 x 8 heads x 20 k tokens, d 128, took 116 us as one
// tile of 24 and 83 us as three of 8; 16 rows 62 and 61 us.)
//
// Why mma.sync: with 1 to 8 rows a tcgen05 tile (M = 64 or 128) would be almost empty, and
// its V would have to be converted from e4m3 to 16 bits through shared memory.  Here the
// tokens are the M side: S^T = K Q^T with m16n8k32 (e4m3, once for each half of the queries)
// and O^T = V^T P^T with m16n8k16 (fp16), the rows are N = 8, and the A fragments are the
// cached bytes in the lanes that use them (the order of the channels inside a product is free,
// so each lane takes 16 contiguous bytes): each warp its own tokens, no barrier.  P^T
// goes from the accumulators' layout to the B operand's by one 8x8 transpose per 8 tokens.
//
// Loads: a warp copies its tokens (contiguous in a page) into its own part of shared memory,
// 512 contiguous bytes an instruction (cp.async), the next step's K once this one's scores are
// done and its V once this one's products are; loads in flight cost no registers and warps do not
// wait for each other.  The 16-byte chunks of a 128-byte line are permuted so that both the copies
// and the lanes' reads in fragment order are free of bank conflicts.  (Copied in fragment
// order straight from the pages, 64 bytes of 8 rows at a time, reads stop at 5.0 TB/s; in
// whole lines they reach 6.8: a copy loop alone, 900 MB of pages in random order.)
//
// Split: the work is planned on the device from the lengths, so that the host never waits for
// them.  A segment is one (sequence, key head), its units the tokens that a CTA's warps take at
// once.  Much work (8 units for each resident CTA, or more): the line of all segments' units is cut
// into equal stretches; a CTA does whole segments in passing and leaves partials of the two it
// shares with its neighbours.  Little work: each segment is cut into its own chunks, as small as
// the resident CTAs allow, one a CTA, because beginning a segment costs as much as two units.  With
// several row tiles each stretch or chunk goes to as many neighbouring CTAs, which read the
// same tokens at about the same time: from HBM once.  A second kernel joins partials in order: no
// atomics, the same bits every time.  Caches of at most 512 tokens take one CTA a segment and row
// tile, and one launch.
//
// Measured: one token of 8 sequences x 40 heads, 88 k tokens, d 128 (902 MB) 144.5 us with the join (4.4 alone),
// 6.2 TB/s.  Row tiles beyond the first are bound by the conversion of V (the ALU pipe is busy 48 % of
// the time, 12 warps an SM hide no more): 20 rows of 4 x 8 heads, 20 k tokens (41 MB) 27 + 4 us.  Short
// segments cost their beginning and end: 256 sequences of 200 to 2000 tokens x 8 heads (590 MB) 143 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <math_constants.h>

#include "cache_tiles.cuh"
#include "common.cuh"

namespace fvattn {

namespace {

constexpr int kWarps = 4;  // of a CTA.  Short caches in so few CTAs that each has an SM to itself: 8, which halves
                           // the steps one after another (64 CTAs, 500 tokens, d 128: 7.7 us, with 4 8.6; 90 tokens
                           // 6.1 and 5.8; in a second wave, 160 CTAs, it loses: 14.2 and 10.4).
constexpr int kMoreWarps = 8;
constexpr int kRows = 8;                // rows of a tile
// Tokens a warp takes at a time (inside one page: pages hold 64 or 128); a unit is what the CTA's
// warps take.  One row tile, bound by HBM: 32, whose finer cut of the work balances better (8 x 40
// heads, 88 k tokens, d 128: 141 us, with 64 149).  More tiles, bound by the warps: 64, which
// spends less on each token (20 rows, 4 x 8 heads, 20 k tokens: 27 us, with 32 34).
constexpr int kOneTileStep = 32, kMoreTilesStep = 64;
// Tables of at most so many tokens: a CTA takes a whole segment, in one launch without a plan.  us, whole / split, in
// tables of just the cached tokens, one row (20 rows):
//   cached tokens           250                    500                     1000                    2000
//   8 heads, d 64            5.2 /  9.5 (5.4, 9.9)   6.1 /  9.8 (6.4, 10.7)   8.2 /  9.7 (8.4, 10.7)  12.0 /  9.9 (12.4, 11.0)
//   8 heads, d 128           6.3 / 10.4 (7.4, 12.2)  7.6 / 10.7 (8.7, 12.7)  10.2 / 11.1 (11.4, 13.0) 15.5 / 11.4 (16.9, 14.0)
//   8 sequences x 40, d 128  8.9 / 13.8             12.6 / 17.4             19.7 / 24.5             35.6 / 38.5
// They meet between 1000 and 1500 tokens, later with more segments; 512 lies on the safe side.  The rule
// sees the table's width, not the lengths, which are on the device: the same 500 tokens of 8 heads, d 128, take 7.6 us
// in a table of 512 and 10.9 in one of 65536.
constexpr int kWholeTokens = 512;
constexpr int kCtasPerSm = 3;           // by shared memory (64 KB each at d 128) and registers
constexpr int kChunkShare = 8;          // units per CTA below which segments are cut into chunks
constexpr int kChunkSequences = 64;     // more sequences are not worth the search for the chunk
constexpr int kMostCtas = 512;          // stretches (444 CTAs are resident on 148 SMs)
constexpr int kJoinThreads = 128;
constexpr int kMostScale = 125;         // largest power of two in the scores' factor
constexpr float kWeightLog2 = 15.0f;    // weights are scaled by 2^15 before fp16
constexpr float kNegInf = -__builtin_huge_valf();

struct FewWorkspace {
    size_t split, stats, acc, total;
};

FewWorkspace few_layout(int d, int ctas) {
    FewWorkspace w{};
    Carver c;
    w.split = c.take<int4>(static_cast<size_t>(ctas));
    w.stats = c.take<float4>(static_cast<size_t>(ctas) * 2 * kRows);
    w.acc = c.take<float>(static_cast<size_t>(ctas) * 2 * kRows * d);
    w.total = align_up(c.off, 256);
    return w;
}

struct FewArgs {
    AttendLaunch a;
    int4 *split;      // [ctas] the segment that begins in a stretch and ends behind it: sequence, key head,
                      // parts (0: none); and whether the stretch met a bad page table entry
    int unit;         // tokens
    float4 *stats;    // [2 * ctas, kRows]: m, l, w
    float *acc;       // [2 * ctas, kRows, d]
    float scale_log2;
    int row_tiles;
    int ctas;         // stretches of the work; each is done by row_tiles neighbouring CTAs
    bool whole;       // a CTA per segment and row tile
    int log2_block;
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

// Two fp32 values -> two e4m3 codes in the low half, nearest, saturating.
__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// D (16 x 8) += A (16 x 16) B (16 x 8), fp16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D (16 x 8) += A (16 x 32) B (32 x 8), e4m3 operands, fp32 sums.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of the warp's 8x8 matrix of 16-bit values.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// ------------------------------------------------------------------ the plan

__device__ __forceinline__ int units_of(const FewArgs &g, int len) {
    return static_cast<int>(segment_units(len, g.unit));
}

// The plan, in shared memory: first[b] = what comes before sequence b, for b = 0 .. B, in units
// (stretches) or in chunks of at most first[B + 1] units; first[B + 1] = 0 says stretches.
// Every CTA makes the same plan in its shared memory: all load the lengths, one warp adds.
__device__ __forceinline__ void make_plan(const FewArgs &g, int *first, int *lens) {
    const AttendLaunch &a = g.a;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const Seq seq = sequence(a, b);
        lens[b] = seq.n_new > 0 ? seq.len : 0;  // (nothing to write)
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int groups = a.pool.heads;
        int total = 0;
        for (int b = lane; b < a.B; b += 32) total += units_of(g, lens[b]) * groups;
        total = __reduce_add_sync(0xffffffffu, total);
        // the smallest chunk, of 1 .. 32 units, with which every chunk gets its own CTA
        int chunk = 0;
        if (total < kChunkShare * g.ctas && a.B <= kChunkSequences) {
            int n = 0;
            for (int b = 0; b < a.B; ++b) n += (units_of(g, lens[b]) + lane) / (lane + 1);
            const uint32_t fits = __ballot_sync(0xffffffffu, n * groups <= g.ctas);
            chunk = __ffs(static_cast<int>(fits));  // 0: none
        }
        int before = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            const int u = b < a.B ? units_of(g, lens[b]) : 0;
            const int n = (chunk ? (u + chunk - 1) / chunk : u) * groups;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
            }
            if (b < a.B) first[b] = before + inc - n;
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            first[a.B] = before;
            first[a.B + 1] = chunk;
        }
    }
    __syncthreads();
}

// Largest b with first[b] <= x.
__device__ __forceinline__ int find_sequence(const int *first, int B, int x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ------------------------------------------------------------------ a row's sums

// l = sum 2^(s - m), acc = 2^15 sum 2^(s - m + ev - w) v.  Without a token m = w = -inf, both are 0.
// acc 2^(w - 15) / l, the power of two in two factors: w goes with V's exponents, and 2^(w - 15) alone may
// lie outside fp32 where the result does not (a page of values near 2^-120, or a channel of zeros in a
// page of exponent 200).
struct OutFactor {
    float inv_l, half;
    __device__ __forceinline__ OutFactor(float l, float w)
        : inv_l(l == 0.0f ? 0.0f : 1.0f / l), half(l == 0.0f ? 0.0f : ex2((w - kWeightLog2) * 0.5f)) {}
    __device__ __forceinline__ float operator()(float acc) const { return acc * inv_l * half * half; }
};
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}
// m_old - m_new for a maximum that moved from m_old (or -inf) to m_new.
__device__ __forceinline__ float moved_by(float m_old, float m_new) { return m_old == m_new ? 0.0f : m_old - m_new; }

// N partial sums of one row as one: their statistics (m, l, w), and the factor of each one's acc.
struct Joined {
    float m, w, l;
    __device__ __forceinline__ Joined() : m(kNegInf), w(kNegInf), l(0.0f) {}
    __device__ __forceinline__ void top(float m_k) { m = fmaxf(m, m_k); }                        // first all of these,
    __device__ __forceinline__ void weight(float m_k, float w_k) { w = fmaxf(w, w_k + moved_by(m_k, m)); }  // then these,
    __device__ __forceinline__ float add(float m_k, float l_k, float w_k) {                      // then these
        const float shift = moved_by(m_k, m);
        l += m_k == kNegInf ? l_k : l_k * ex2(shift);  // (without a token 0, or NaN)
        return w_k == kNegInf ? 1.0f : ex2(w_k + shift - w);
    }
};

__device__ __forceinline__ void add_scaled(float4 &sum, const float4 &v, float f) {
    sum.x += v.x * f, sum.y += v.y * f, sum.z += v.z * f, sum.w += v.w * f;
}

// Four channels of row r (of key head h) from its sums, and the LSE with the first of them.
__device__ __forceinline__ void write_row(const AttendLaunch &a, int b, int h, int r, int ch, const float4 &sum,
                                          const Joined &j) {
    const int64_t hq = h * a.group + r / a.M, tok = r % a.M;
    const OutFactor f(j.l, j.w);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.O) + b * a.o_b + hq * a.o_h + tok * a.o_n + ch;
    const __nv_bfloat162 p0 = __floats2bfloat162_rn(f(sum.x), f(sum.y));
    const __nv_bfloat162 p1 = __floats2bfloat162_rn(f(sum.z), f(sum.w));
    *reinterpret_cast<uint2 *>(out) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&p0), *reinterpret_cast<const uint32_t *>(&p1));
    if (ch == 0) a.LSE[(static_cast<int64_t>(b) * a.pool.heads * a.group + hq) * a.M + tok] = lse_of(j.m, j.l);
}

// ------------------------------------------------------------------ loads

// A warp's part of shared memory: a step of K, then one of V, rows in order.  The 16-byte chunks of
// each 128-byte line (one row at d 128, two at d 64) are permuted by exclusive or with a number
// that depends on the line.
template <int D, int STEP>
struct Step {
    static constexpr int BYTES = STEP * D;

    // K's reads take 4 chunks of two neighbouring rows at a time, V's two chunks of every other row
    // of 8 (d 64: half rows): both hit 8 different chunk places.
    static __device__ __forceinline__ int mix(int line) {
        return D == 128 ? (((line >> 1) & 3) << 1) ^ ((line & 1) << 2) : (line & 3) << 1;
    }
    // Place of byte `at` (a multiple of 8) of row `row`.
    static __device__ __forceinline__ int place(int row, int at) {
        const int byte = row * D + at, line = byte >> 7;
        return (line << 7) + ((((byte >> 4) & 7) ^ mix(line)) << 4) + (byte & 8);
    }
    // place() as a lane's constant and an immediate.  Copy i of a step covers lines 4 i .. 4 i + 3, 8
    // lanes each; whether i (d 128) is odd flips the chunks' upper bit.
    static __device__ __forceinline__ int copy_lane(int lane) {
        const int line = lane >> 3;
        return (line << 7) + (((lane & 7) ^ mix(line)) << 4);
    }
    static __device__ __forceinline__ int copy_at(int c, int i) { return (D == 128 && (i & 1) ? c ^ 64 : c) + i * 512; }
    // Rows g + 8 k, channels c * 64 + q * 16 ..: the row's last 3 bits are g's.
    static __device__ __forceinline__ int key_lane(int g, int q) { return place(g, q * 16); }
    static __device__ __forceinline__ int key_at(int c, int rows8, int half) { return (half ? c ^ 64 : c) + rows8 * 8 * D; }
    // Rows 2 q + odd + 8 k, channels g * D/8 ..
    static __device__ __forceinline__ int value_lane(int g, int q) { return place(2 * q, g * (D / 8)); }
    static __device__ __forceinline__ int value_at(int c, int rows8, int odd) {
        return (odd ? (c ^ 64) + (D == 128 ? 128 : 0) : c) + rows8 * 8 * D;
    }
    // One step of K or V from its first byte in the page (`src`: this lane's 16 bytes of the first copy).
    static __device__ __forceinline__ void copy(uint32_t dst, const uint8_t *src, int lane_place) {
#pragma unroll
        for (int i = 0; i < BYTES / 512; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + copy_at(lane_place, i)), "l"(src + i * 512)
                         : "memory");
    }
};

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();  // the other lanes' copies too
}

// ------------------------------------------------------------------ the kernel

template <int D, int STEP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == kWarps ? kCtasPerSm : 1) attend_few_kernel(const __grid_constant__ FewArgs g) {
    constexpr int KW = D / 16;      // words of a lane's part of a query or key row
    constexpr int MT = D / 16;      // m16 tiles of V^T P^T
    constexpr int VW = D / 32;      // words of a lane's V row
    constexpr int ST = STEP / 16;   // 16-token tiles of a step
    constexpr int UNIT = STEP * WARPS, THREADS = WARPS * 32;
    using S_ = Step<D, STEP>;
    extern __shared__ __align__(128) unsigned char smem[];  // whole lines (16 bytes off: 142 -> 159 us)
    unsigned char *kr = smem + (threadIdx.x >> 5) * 2 * S_::BYTES, *vr = kr + S_::BYTES;  // this warp's K and V
    float *acc_s = reinterpret_cast<float *>(smem);  // [WARPS][kRows][D], between segments
    int *first = reinterpret_cast<int *>(smem + WARPS * 2 * S_::BYTES);
    int *lens = first + g.a.B + 2;
    __shared__ float4 stat_s[WARPS][kRows];
    __shared__ int4 split_s;
    static_assert(kRows * D * 4 <= 2 * S_::BYTES, "the sums reuse the steps' place");
    const AttendLaunch &a = g.a;
    wait_for_stream();
    if (threadIdx.x == 0) split_s = make_int4(0, 0, 0, 0);
    if (!g.whole && blockIdx.x > 0) make_plan(g, first, lens);
    if (blockIdx.x == 0) {  // (with a plan, the others check the table's entries as they meet them)
        if (g.whole) check_attend<true>(a);
        else check_attend<false>(a);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = lane >> 2, lq = lane & 3;
    const int BS = a.pool.block, H = a.pool.heads;
    const int R = a.group * a.M;
    const int cta = static_cast<int>(blockIdx.x) - 1;
    const int copy_place = S_::copy_lane(lane), key_place = S_::key_lane(lg, lq), value_place = S_::value_lane(lg, lq);
    const uint32_t k_at = static_cast<uint32_t>(__cvta_generic_to_shared(kr)), v_at = k_at + S_::BYTES;

    const int rt = cta % g.row_tiles, stretch = cta / g.row_tiles;
    const int row0 = rt * kRows, rows = min(kRows, R - row0);
    int unit = stretch, unit_end = stretch + 1, chunk = 0;
    if (!g.whole) {
        const int total = first[a.B];
        chunk = first[a.B + 1];
        const int n = stretches(total, g.ctas);
        if (stretch >= n) {
            unit_end = unit;  // nothing left for it
        } else if (!chunk) {
            unit = static_cast<int>(stretch_start(stretch, total, n));
            unit_end = static_cast<int>(stretch_start(stretch + 1, total, n));
        }
    }
    while (unit < unit_end) {
        // the segment, and units [off, off + n_units) of its
        int b, h, off = 0, n_units, all;
        Seq seq;
        if (g.whole) {
            b = stretch / H;
            h = stretch % H;
            seq = sequence(a, b);
            n_units = all = units_of(g, seq.len);
            unit = unit_end;
        } else {
            b = find_sequence(first, a.B, unit);
            seq = Seq{lens[b], a.new_lens ? static_cast<int>(clamp_len(a.new_lens[b], a.M)) : a.M};
            all = units_of(g, seq.len);
            const int at = unit - first[b];
            if (chunk) {  // its chunks are as even as can be
                const int n = (all + chunk - 1) / chunk;
                h = at / n;
                off = static_cast<int>(stretch_start(at % n, all, n));
                n_units = static_cast<int>(stretch_start(at % n + 1, all, n)) - off;
                unit = unit_end;
                if (off == 0 && threadIdx.x == 0) split_s.x = b, split_s.y = h, split_s.z = n;
            } else {
                h = at / all;
                off = at % all;
                n_units = min(all - off, unit_end - unit);
                unit += n_units;
                if (off == 0 && n_units < all && threadIdx.x == 0) {
                    const int total = first[a.B], last = first[b] + (h + 1) * all - 1;
                    split_s.x = b, split_s.y = h;
                    split_s.z = stretch_of(last, total, stretches(total, g.ctas)) - stretch + 1;
                }
            }
        }

        const int c1 = seq.n_new == 0 ? 0 : min(seq.len, (off + n_units) * UNIT);
        const int32_t *table = a.pool.table + static_cast<int64_t>(b) * a.pool.max_pages;
        // the page and head of the step at `tok`, or -1: behind the end, or an entry outside the pool
        auto page_at = [&](int tok) -> int64_t {
            if (tok >= c1) return -1;
            const int p = checked_page(table[tok >> g.log2_block], a.pool.num_pages);
            return p < 0 ? -1 : static_cast<int64_t>(p) * H + h;
        };
        // this warp's step at tok is on its way (copy groups K, V); the page of the next is looked up.  (The
        // table is read before the length says whether its entry counts, so that the two loads overlap.)
        int tok = off * UNIT + warp * STEP;
        const int entry = table[min(tok >> g.log2_block, a.pool.max_pages - 1)];
        const int entry_next = table[min((tok + UNIT) >> g.log2_block, a.pool.max_pages - 1)];
        const int p0 = tok < c1 ? checked_page(entry, a.pool.num_pages) : -1;
        const int p1 = tok + UNIT < c1 ? checked_page(entry_next, a.pool.num_pages) : -1;
        int64_t ph = p0 < 0 ? -1 : static_cast<int64_t>(p0) * H + h;
        int64_t ph_next = p1 < 0 ? -1 : static_cast<int64_t>(p1) * H + h;
        int ek = 0, ev = 0;
        {
            const int64_t at = (ph * BS + (tok & (BS - 1))) * D + lane * 16;
            if (ph >= 0) {
                S_::copy(k_at, a.pool.k + at, copy_place);
                ek = a.pool.ke[ph];
                ev = a.pool.ve[ph];
            }
            copies_commit();
            if (ph >= 0) S_::copy(v_at, a.pool.v + at, copy_place);
            copies_commit();
        }

        // query fragments: row lg, scaled by 2^-sq to at most 448 and split: qh + ql / 16.
        // Word w of chunk c holds channels c * 64 + lq * 16 + 4 w .. + 3, as K's words do.
        uint32_t qh[KW], ql[KW];
        int sq;
        {
            const int r = row0 + lg;
            const bool in = r < R && r % a.M < seq.n_new;
            const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(a.Q) + b * a.q_b;
            if (in) qr += static_cast<int64_t>(h * a.group + r / a.M) * a.q_h + static_cast<int64_t>(r % a.M) * a.q_n;
            uint32_t raw[KW][2];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
#pragma unroll
                for (int w2 = 0; w2 < 2; ++w2) {
                    const uint4 v = in ? *reinterpret_cast<const uint4 *>(qr + c * 64 + lq * 16 + w2 * 8)
                                       : make_uint4(0, 0, 0, 0);
                    raw[c * 4 + w2 * 2][0] = v.x;
                    raw[c * 4 + w2 * 2][1] = v.y;
                    raw[c * 4 + w2 * 2 + 1][0] = v.z;
                    raw[c * 4 + w2 * 2 + 1][1] = v.w;
                }
            }
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float lo = fabsf(rope_bf16_lo(raw[k][e])), hi = fabsf(rope_bf16_hi(raw[k][e]));
                    if (lo < CUDART_INF_F) top = fmaxf(top, lo);
                    if (hi < CUDART_INF_F) top = fmaxf(top, hi);
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            sq = top > 0.0f ? ilogbf(top) - 8 : 0;
            if (scale_pow2(top, -sq) > 448.0f) ++sq;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                uint32_t code[2], rest[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x0 = scale_pow2(rope_bf16_lo(raw[k][e]), -sq);
                    float x1 = scale_pow2(rope_bf16_hi(raw[k][e]), -sq);
                    if (isinf(x0)) x0 = CUDART_NAN_F;  // an infinite query has no softmax either
                    if (isinf(x1)) x1 = CUDART_NAN_F;
                    code[e] = codes_of(x0, x1);
                    const uint32_t y = f16x2_of_codes(code[e]);
                    const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&y));
                    rest[e] = codes_of((x0 - z.x) * 16.0f, (x1 - z.y) * 16.0f);
                }
                qh[k] = code[0] | (code[1] << 16);
                ql[k] = rest[0] | (rest[1] << 16);
            }
        }
        // per lane, rows 2 lq + e: scale exponent, visible tokens, running statistics
        int sqr[2], lim[2];
        float m[2], w[2], l[2];
        int min_lim = seq.len;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rr = 2 * lq + e, r = row0 + rr;
            sqr[e] = __shfl_sync(0xffffffffu, sq, rr * 4);
            const int m_tok = r < R ? r % a.M : a.M;
            lim[e] = r < R ? row_limit(a, seq, m_tok) : 0;
            if (r < R && m_tok < seq.n_new) min_lim = min(min_lim, lim[e]);
            m[e] = w[e] = kNegInf;
            l[e] = 0.0f;
        }
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 1));
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 2));
        float o[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;

        for (; tok < c1; tok += UNIT) {
            const bool here = ph >= 0, more = ph_next >= 0;
            const int64_t at_next = (ph_next * BS + ((tok + UNIT) & (BS - 1))) * D + lane * 16;
            const int ek_here = clamp_exp(ek);
            const float evf = static_cast<float>(clamp_exp(ev));
            if (more) {
                ek = a.pool.ke[ph_next];
                ev = a.pool.ve[ph_next];
            }
            ph = ph_next;
            ph_next = page_at(tok + 2 * UNIT);
            copies_wait<1>();  // K of this step
            if (!here) {       // an entry outside the pool: its tokens are left out
                split_s.w = 1;
                copies_wait<0>();
                if (more) S_::copy(k_at, a.pool.k + at_next, copy_place);
                copies_commit();
                if (more) S_::copy(v_at, a.pool.v + at_next, copy_place);
                copies_commit();
                continue;
            }
            // S^T = K Q^T, the second half of the queries' bits apart
            float s[ST][4];
#pragma unroll
            for (int mt = 0; mt < ST; ++mt) {
                float lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) s[mt][k] = lo[k] = 0.0f;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    // rows g and g + 8 of the tile, channels c * 64 + q * 16 .. + 15
                    const uint4 x0 = *reinterpret_cast<const uint4 *>(kr + S_::key_at(key_place, 2 * mt, c));
                    const uint4 x1 = *reinterpret_cast<const uint4 *>(kr + S_::key_at(key_place, 2 * mt + 1, c));
                    mma_e4m3(s[mt], x0.x, x1.x, x0.y, x1.y, qh[c * 4], qh[c * 4 + 1]);
                    mma_e4m3(lo, x0.x, x1.x, x0.y, x1.y, ql[c * 4], ql[c * 4 + 1]);
                    mma_e4m3(s[mt], x0.z, x1.z, x0.w, x1.w, qh[c * 4 + 2], qh[c * 4 + 3]);
                    mma_e4m3(lo, x0.z, x1.z, x0.w, x1.w, ql[c * 4 + 2], ql[c * 4 + 3]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) s[mt][k] = fmaf(lo[k], 0.0625f, s[mt][k]);
            }
            __syncwarp();  // read by all lanes
            if (more) S_::copy(k_at, a.pool.k + at_next, copy_place);
            copies_commit();
            const bool edge = tok + STEP > min_lim;
            // the weights, transposed into the B operand
            float alpha[2];
            bool moved = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int fe = clamp_exp(sqr[e] + ek_here);
                const float f = scale_pow2(g.scale_log2, min(fe, kMostScale));
                if (fe > kMostScale) {  // what is above that on its own, so that a product of zero stays zero
                    const float above = __int_as_float((fe - kMostScale + 127) << 23);
#pragma unroll
                    for (int mt = 0; mt < ST; ++mt) s[mt][e] *= above, s[mt][2 + e] *= above;
                }
                float mx = kNegInf;
#pragma unroll
                for (int mt = 0; mt < ST; ++mt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float &v = s[mt][2 * hf + e];
                        v *= f;
                        if (edge && tok + mt * 16 + hf * 8 + lg >= lim[e]) v = kNegInf;
                        mx = fmaxf(mx, v);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float m_new = fmaxf(m[e], mx);
                const float m_ref = m_new == kNegInf ? 0.0f : m_new;
                const float shift = moved_by(m[e], m_new);
                const float w_old = w[e] + shift;
                const float w_new = fmaxf(w_old, mx - m_ref + evf);
                const float w_off = w_new == kNegInf ? 0.0f : evf + kWeightLog2 - w_new;
                const float al = ex2(shift);
                const bool grew = w_new != w_old && w_old != kNegInf;
                alpha[e] = grew ? ex2(w_old - w_new) : 1.0f;
                moved |= grew;
                float sum = 0.0f;
#pragma unroll
                for (int mt = 0; mt < ST; ++mt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float &v = s[mt][2 * hf + e];
                        const float t = v - m_ref;
                        sum += ex2(t);
                        v = ex2(t + w_off);
                    }
                l[e] = l[e] * al + sum;
                m[e] = m_new;
                w[e] = w_new;
            }
            uint32_t pf[ST][2];
#pragma unroll
            for (int mt = 0; mt < ST; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) pf[mt][hf] = transpose8x8(f16x2_of(s[mt][2 * hf], s[mt][2 * hf + 1]));
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[i][k] *= alpha[k & 1];
            }
            copies_wait<1>();  // V of this step
            // A step that some row sees only in part (the sequence's end, the causal edge): a
            // NaN among the values of a token that a row does not see must not reach it through
            // 0 * NaN.  The lane makes its NaN codes zero, and the rows that do see one get it back
            // here: what a row sees is a prefix, so the first NaN of a channel decides.
            bool nan_here = false;
            if (edge) {
#pragma unroll 4
                for (int i = lane; i < S_::BYTES / 16; i += 32) {
                    const uint4 x = reinterpret_cast<const uint4 *>(vr)[i];
                    nan_here |= any_nan_e4m3(x.x) || any_nan_e4m3(x.y) || any_nan_e4m3(x.z) || any_nan_e4m3(x.w);
                }
                nan_here = __any_sync(0xffffffffu, nan_here);
            }
            if (nan_here) {
#pragma unroll
                for (int byte = 0; byte < D / 8; ++byte) {
                    const int at = lg * (D / 8) + byte;
                    int seen = STEP;
#pragma unroll 1
                    for (int row = 2 * lq; row < STEP; row += (row & 1) ? 7 : 1) {  // this lane's: 2q, 2q + 1 of each 8
                        unsigned char &code = vr[S_::place(row, at & ~7) + (at & 7)];
                        if ((code & 0x7fu) != 0x7fu) continue;
                        code = 0;
                        seen = min(seen, row);
                    }
                    seen = min(seen, __shfl_xor_sync(0xffffffffu, seen, 1));
                    seen = min(seen, __shfl_xor_sync(0xffffffffu, seen, 2));
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (seen < STEP && tok + seen < lim[e]) o[byte / 2][(byte & 1) * 2 + e] = CUDART_NAN_F;
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int kg = 0; kg < ST; ++kg) {
                uint32_t vx[4][VW];
#pragma unroll
                for (int t = 0; t < 4; ++t) {  // tokens 2q, 2q + 1, 2q + 8, 2q + 9 of the 16, channels g * D/8 ..
                    const unsigned char *x = vr + S_::value_at(value_place, 2 * kg + (t >> 1), t & 1);
                    if constexpr (D == 128) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(x);
                        vx[t][0] = y.x, vx[t][1] = y.y, vx[t][2] = y.z, vx[t][3] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2 *>(x);
                        vx[t][0] = y.x, vx[t][1] = y.y;
                    }
                }
#pragma unroll
                for (int k = 0; k < VW; ++k) {
#pragma unroll
                    for (int pair = 0; pair < 2; ++pair) {  // bytes 0, 1 and 2, 3 of the word: channels 4k + 2 pair, + 1
                        const uint32_t sel = pair ? 0x7362u : 0x5140u;
                        const uint32_t x01 = __byte_perm(vx[0][k], vx[1][k], sel);
                        const uint32_t x23 = __byte_perm(vx[2][k], vx[3][k], sel);
                        mma_f16(o[2 * k + pair], f16x2_of_codes(x01 & 0xffffu), f16x2_of_codes(x01 >> 16),
                                f16x2_of_codes(x23 & 0xffffu), f16x2_of_codes(x23 >> 16), pf[kg][0], pf[kg][1]);
                    }
                }
            }
            __syncwarp();
            if (more) S_::copy(v_at, a.pool.v + at_next, copy_place);
            copies_commit();
        }
        copies_wait<0>();
        __syncthreads();  // the steps' place becomes the sums'

        // join the warps
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[e];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            if (lg == 0) stat_s[warp][2 * lq + e] = make_float4(m[e], sum, w[e], 0.0f);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int ch = lg * (D / 8) + 2 * i;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (2 * lq + e < rows)
                    *reinterpret_cast<float2 *>(acc_s + (warp * kRows + 2 * lq + e) * D + ch) = make_float2(o[i][e], o[i][2 + e]);
        }
        __syncthreads();
        const bool complete = n_units == all;
        const int slot = 2 * cta + (off == 0 ? 1 : 0);
        for (int y = threadIdx.x; y < rows * (D / 4); y += THREADS) {
            const int rr = y / (D / 4), ch = (y % (D / 4)) * 4;
            Joined j;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) j.top(stat_s[k][rr].x);
#pragma unroll
            for (int k = 0; k < WARPS; ++k) j.weight(stat_s[k][rr].x, stat_s[k][rr].z);
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                const float4 st = stat_s[k][rr];
                add_scaled(sum, *reinterpret_cast<const float4 *>(acc_s + (k * kRows + rr) * D + ch), j.add(st.x, st.y, st.z));
            }
            if (!complete) {
                const int64_t at = static_cast<int64_t>(slot) * kRows + rr;
                if (ch == 0) g.stats[at] = make_float4(j.m, j.l, j.w, 0.0f);
                *reinterpret_cast<float4 *>(g.acc + at * D + ch) = sum;
            } else if ((row0 + rr) % a.M < seq.n_new) {
                write_row(a, b, h, row0 + rr, ch, sum, j);
            }
        }
        __syncthreads();
    }
    if (!g.whole && rt == 0 && threadIdx.x == 0) g.split[stretch] = split_s;
}

// Joins the partials of one row: grid (row, stretch), of the segment that begins in the stretch and goes on
// behind it.  They go to the CTA's groups of D / 4 threads in turn, and the groups are added in order.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const __grid_constant__ FewArgs g) {
    constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
    __shared__ float4 part_s[kMostCtas];
    __shared__ float4 acc_s[GROUPS][LANES];
    __shared__ float3 stat_s[GROUPS];
    wait_for_stream();  // launched while the partials are still made
    const AttendLaunch &a = g.a;
    const int r = blockIdx.x, from = blockIdx.y;
    if (r == 0 && from == 0) {
        bool bad = false;
        for (int i = threadIdx.x; i < g.ctas; i += kJoinThreads) bad |= g.split[i].w != 0;
        if (bad) *a.dev_status = FVATTN_ERR_BAD_PAGE;
    }
    const int4 split = g.split[from];
    const int b = split.x, h = split.y, n_parts = split.z;
    if (n_parts <= 1 || r % a.M >= sequence(a, b).n_new) return;
    const int rt = r / kRows;
    // a segment's first part is the second partial of its CTA (of the segment that CTA ends in), the
    // others are the first of theirs
    auto part = [&](int c) {
        return (2 * (static_cast<int64_t>(from + c) * g.row_tiles + rt) + (c == 0 ? 1 : 0)) * kRows + r % kRows;
    };
    for (int c = threadIdx.x; c < n_parts; c += kJoinThreads) part_s[c] = g.stats[part(c)];
    __syncthreads();
    const int grp = threadIdx.x / LANES, ch = (threadIdx.x % LANES) * 4;
    Joined j;
    for (int c = grp; c < n_parts; c += GROUPS) j.top(part_s[c].x);
    for (int c = grp; c < n_parts; c += GROUPS) j.weight(part_s[c].x, part_s[c].z);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int c = grp; c < n_parts; c += GROUPS) {
        const float4 st = part_s[c];
        add_scaled(sum, *reinterpret_cast<const float4 *>(g.acc + part(c) * D + ch), j.add(st.x, st.y, st.z));
    }
    acc_s[grp][threadIdx.x % LANES] = sum;
    if (ch == 0) stat_s[grp] = make_float3(j.m, j.l, j.w);
    __syncthreads();
    if (grp != 0) return;
    Joined k;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) k.top(stat_s[i].x);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) k.weight(stat_s[i].x, stat_s[i].z);
    sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i)
        add_scaled(sum, acc_s[i][threadIdx.x], k.add(stat_s[i].x, stat_s[i].y, stat_s[i].z));
    write_row(a, b, h, r, ch, sum, k);
}

// ---------------------------------------------------------------- pages as bf16

// Every cached token of every head as bf16, for the 128-row tiles of the tensor cores.  Exact (a code
// has 4 bits and its scale is a power of two) from 2^-133, bf16's smallest step, up to its largest
// number, which stands for all above it: an infinity would reach the rows that do not see it, as
// 0 * inf.  A CTA takes pages of one (sequence, head); CTA 0 only checks.  Tokens from the
// sequence's end to the next multiple of 128 are zeros: the tiles read them.  NaN codes of V become
// zero in the copy and the first of each channel is kept in nan_first, so that a NaN that a query
// does not see cannot reach it through 0 * NaN.
constexpr int kExpandThreads = 256;
// CTAs for each SM at most; those of a head take its pages in turn.  (A CTA a page: 8 x 8 heads with 16 of
// 1024 pages in use 82 us, now 26; 40 heads with 256 of 256, 162 and 165.)
constexpr int kExpandPerSm = 64;

// By the checking CTA: key tiles (at least one each) before each of the rest items.
__device__ void plan_rest(const CacheTiles &ct) {
    __shared__ int sums[kExpandThreads];
    const int i = static_cast<int>(threadIdx.x);  // (there are fewer of them than SMs)
    const int n = i < ct.n_rest ? max(cache_tiles_of(ct, ct.n_whole + i), 1) : 0;
    sums[i] = n;
    __syncthreads();
    for (int o = 1; o < kExpandThreads; o <<= 1) {
        const int t = i >= o ? sums[i - o] : 0;
        __syncthreads();
        sums[i] += t;
        __syncthreads();
    }
    if (i < ct.n_rest) ct.rest[i] = sums[i] - n;
    if (i == 0) ct.rest[ct.n_rest] = sums[kExpandThreads - 1];
}

constexpr float kMostBf16 = 3.38953139e38f;  // 255 2^120
constexpr int kMostPlainExp = 119;           // 448 2^119 is below it

// Inside bf16's range; a NaN stays.
__device__ __forceinline__ float held(float x) { return x > kMostBf16 ? kMostBf16 : x < -kMostBf16 ? -kMostBf16 : x; }

// Eight codes times 2^e (f, where that is a normal number and no product passes bf16's range).
__device__ __forceinline__ uint4 expand8(uint2 codes, int e, bool plain, float f) {
    uint32_t out[4];
    const uint32_t c[4] = {codes.x & 0xffffu, codes.x >> 16, codes.y & 0xffffu, codes.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = f16x2_of_codes(c[i]);
        float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        if (plain) v = make_float2(v.x * f, v.y * f);
        else v = make_float2(held(scale_pow2(v.x, e)), held(scale_pow2(v.y, e)));
        const __nv_bfloat162 y = __floats2bfloat162_rn(v.x, v.y);
        out[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D>
__device__ __forceinline__ void expand_page(const CacheTiles &ct, const Seq &seq, int b, int h, int pg) {
    constexpr int PER_ROW = D / 8, AHEAD = 64 * PER_ROW / kExpandThreads;  // a vector: 8 codes; 64 rows at a time
    const AttendLaunch &a = ct.a;
    const int BS = a.pool.block;
    const int tok0 = pg * BS;
    const int fill = max(min(seq.len - tok0, BS), 0);  // cached slots of the page
    const int page =
        fill > 0 ? checked_page(a.pool.table[static_cast<int64_t>(b) * a.pool.max_pages + pg], a.pool.num_pages) : -1;
    const int64_t ph = static_cast<int64_t>(page < 0 ? 0 : page) * a.pool.heads + h;
    const int64_t bh = static_cast<int64_t>(b) * a.pool.heads + h;
    const int rows = page < 0 ? 0 : fill;
#pragma unroll 1
    for (int part = 0; part < BS / 32; ++part) {  // K, then V, 64 rows at a time
        const bool is_v = part >= BS / 64;
        const int row0 = (is_v ? part - BS / 64 : part) * 64;
        const int e = page < 0 ? 0 : clamp_exp((is_v ? a.pool.ve : a.pool.ke)[ph]);
        const bool plain = e >= -126 && e <= kMostPlainExp;
        const float f = plain ? __int_as_float((e + 127) << 23) : 0.0f;
        const uint2 *src = reinterpret_cast<const uint2 *>((is_v ? a.pool.v : a.pool.k) + (ph * BS + row0) * D);
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(is_v ? ct.V : ct.K) + (bh * ct.cap + tok0 + row0) * D);
        uint2 c[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = i * kExpandThreads + threadIdx.x;
            c[i] = row0 + at / PER_ROW < rows ? __ldcs(src + at) : make_uint2(0, 0);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = i * kExpandThreads + threadIdx.x;
            if (is_v && (any_nan_e4m3(c[i].x) || any_nan_e4m3(c[i].y))) {
                for (int y = 0; y < 8; ++y) {
                    uint32_t &word = y < 4 ? c[i].x : c[i].y;
                    const int sh = (y & 3) * 8;
                    if (((word >> sh) & 0x7fu) != 0x7fu) continue;
                    word &= ~(0xffu << sh);
                    atomicMax(ct.nan_first + bh * D + at % PER_ROW * 8 + y, 0x7fffffff - (tok0 + row0 + at / PER_ROW));
                }
            }
            dst[at] = expand8(c[i], e, plain, f);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kExpandThreads) cache_expand_kernel(const __grid_constant__ CacheTiles ct, int per_head) {
    const AttendLaunch &a = ct.a;
    if (blockIdx.x == 0) {
        plan_rest(ct);
        check_attend<true>(a);
        return;
    }
    const int x = static_cast<int>(blockIdx.x) - 1, bh = x / per_head;
    const int b = bh / a.pool.heads, h = bh % a.pool.heads;
    const Seq seq = sequence(a, b);
    if (seq.n_new == 0) return;
    const int pages = static_cast<int>(align_up(static_cast<size_t>(seq.len), 128)) / a.pool.block;
#pragma unroll 1
    for (int pg = x % per_head; pg < pages; pg += per_head) expand_page<D>(ct, seq, b, h, pg);
}

// CTAs that take work: the resident ones but for the one that checks.
int few_ctas(int sms) { return sms * kCtasPerSm - 1; }

}  // namespace

// The few-rows kernel's time grows with its row tiles; the other one pays for expanding the pages
// and is the same from 1 to 128 rows.  They meet at about 64 (us, few / tiles: d 128, 4 x 8 heads, 93 k
// tokens in all: 48 rows 148 / 183, 64 rows 189 / 184, 96 rows 283 / 185; 23 k tokens: 54 / 64, 67 / 63,
// 94 / 64; d 64, 23 k: 36 / 49, 44 / 48, 61 / 49), and at 128 where a CTA takes a whole cache and nothing
// is joined (500 tokens: 96 rows 15 / 23, 128 rows 20 / 23; that is for few segments: 100 rows of 8 heads, d 128, with 8
// sequences 27 / 35, with 32 97 / 64).
bool attend_few_rows(int group, int M, int64_t capacity) {
    return attend_rows(group, M) <= (capacity <= kWholeTokens ? 128 : 64);
}

size_t attend_few_workspace(int d, int sms) { return few_layout(d, few_ctas(sms)).total; }

template <int D, int STEP, int WARPS>
static cudaError_t launch_few_t(FewArgs g, cudaStream_t stream) {
    const AttendLaunch &a = g.a;
    g.unit = STEP * WARPS;
    constexpr size_t steps = static_cast<size_t>(WARPS) * 2 * Step<D, STEP>::BYTES;
    const size_t smem = steps + (2 * static_cast<size_t>(a.B) + 2) * sizeof(int);
    cudaError_t e = allow_shared_memory<attend_few_kernel<D, STEP, WARPS>>(static_cast<int>(steps + (2 * kMaxHeads + 2) * sizeof(int)));
    if (e != cudaSuccess) return e;
    const cudaLaunchConfig_t work = early_launch(dim3(static_cast<unsigned>(g.ctas * g.row_tiles) + 1), WARPS * 32, smem, stream);
    e = cudaLaunchKernelEx(&work, attend_few_kernel<D, STEP, WARPS>, g);
    if (e != cudaSuccess || g.whole) return e;
    cudaLaunchConfig_t cfg = early_launch(
        dim3(static_cast<unsigned>(attend_rows(a.group, a.M)), static_cast<unsigned>(g.ctas)), kJoinThreads, 0, stream);
    return cudaLaunchKernelEx(&cfg, attend_join_kernel<D>, g);
}

cudaError_t launch_attend_few(const AttendLaunch &a, cudaStream_t stream) {
    FewArgs g{};
    g.a = a;
    g.row_tiles = static_cast<int>(ceil_div(attend_rows(a.group, a.M), kRows));
    g.whole = static_cast<int64_t>(a.pool.max_pages) * a.pool.block <= kWholeTokens;
    const int most = few_ctas(a.sms);
    if (most > kMostCtas) return cudaErrorInvalidValue;
    const FewWorkspace w = few_layout(a.pool.d, most);
    g.ctas = g.whole ? a.B * a.pool.heads : most / g.row_tiles;
    g.log2_block = a.pool.block == 128 ? 7 : 6;
    char *ws = static_cast<char *>(a.workspace);
    g.split = reinterpret_cast<int4 *>(ws + w.split);
    g.stats = reinterpret_cast<float4 *>(ws + w.stats);
    g.acc = reinterpret_cast<float *>(ws + w.acc);
    g.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(a.pool.d)));
    const bool alone = g.whole && static_cast<int64_t>(g.ctas) * g.row_tiles < a.sms;
#define FVATTN_FEW(D_) \
    (alone               ? launch_few_t<D_, kOneTileStep, kMoreWarps>(g, stream) \
     : g.row_tiles == 1 ? launch_few_t<D_, kOneTileStep, kWarps>(g, stream) \
                         : launch_few_t<D_, kMoreTilesStep, kWarps>(g, stream))
    return a.pool.d == 128 ? FVATTN_FEW(128) : FVATTN_FEW(64);
#undef FVATTN_FEW
}

cudaError_t launch_cache_expand(const CacheTiles &ct, cudaStream_t stream) {
    const AttendLaunch &a = ct.a;
    const int64_t heads = static_cast<int64_t>(a.B) * a.pool.heads, pages = ct.cap / a.pool.block;
    const int64_t even = ceil_div(static_cast<int64_t>(a.sms) * kExpandPerSm, heads);
    const int per_head = static_cast<int>(ceil_div(pages, ceil_div(pages, even)));  // equal shares
    const unsigned ctas = static_cast<unsigned>(heads * per_head + 1);
    if (a.pool.d == 128) cache_expand_kernel<128><<<ctas, kExpandThreads, 0, stream>>>(ct, per_head);
    else cache_expand_kernel<64><<<ctas, kExpandThreads, 0, stream>>>(ct, per_head);
    return cudaGetLastError();
}

}  // namespace fvattn
