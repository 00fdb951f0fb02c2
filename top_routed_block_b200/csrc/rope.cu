// rope.cu -- rotary positions with several axes (time, height, width of a video's
// tokens) applied to Q and K before routing and attention, and the inverse rotation
// for their gradients.
//
// Mathematics: channel pair j of a head is turned by the angle
//   theta = position[axis_j] * inv_freq_j,
//   (x, y) -> (x cos theta - y sin theta, y cos theta + x sin theta);
// the two channels of pair j are 2j and 2j+1 ("interleaved") or j and j + n_pairs
// ("half").  A rotation's transpose is its inverse, so the gradient is the same
// kernel with the sine's sign changed.
//
// What bounds it: HBM.  Every element is read once and written once (4 bytes of
// traffic for 3 flop).  The angles belong to a token, not to a head, so a thread
// keeps the cosines and sines of its 8 channel pairs in registers and walks the
// heads of both tensors; a pair's angle is paid for once per head group.
//
// Layout of the work: a thread owns two 16-byte vectors (8 channels each) of one
// token, d/16 threads share a token, and a CTA of 256 threads covers 32 (d 128) or 64
// (d 64) tokens.  The vectors are d/2 channels apart (half the rotated channels apart
// for the "half" pairing, which puts both channels of a pair in the same thread), so
// that the threads of a token read and write contiguous 128-byte (64-byte) runs.
// The input may have any strides between tokens and heads (the projections'
// [B, N, H, d] or a fused [B, N, 3, H, d]); no copy to [B, H, N, d] is needed before.
//
// Measured: Q and K of 40 heads x 32760 tokens, d 128 (1.34 GB) 209 us, 6.4 TB/s; of 8 x 32768, d 64 (134 MB)
// 24.9 us, 5.4 TB/s; 2 x 512 tokens 3.0 us, of which nearly all is the launch.
#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "rope.cuh"

namespace fvattn {

namespace {

constexpr int kRopeThreads = 256;
// Heads whose loads a thread has outstanding (two 16-byte loads each): 8 in long calls, where a
// thread walks all heads; 2 in short ones, whose few heads to a thread leave more CTAs resident.
constexpr int kLongAhead = 8, kShortAhead = 2;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// One token's two vectors of a head, turned.  Interleaved: word w of a vector is pair w of
// it.  Half: words w of the two vectors are the x and the y of pairs 2w and 2w+1.
// `on`: one bit per pair that turns (the others keep their values, whatever they are).
template <bool HALF, bool FULL>
__device__ __forceinline__ void turn(uint4 &va, uint4 &vb, const float (&c)[8], const float (&s)[8], uint32_t on) {
    uint32_t a[4] = {va.x, va.y, va.z, va.w}, b[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float a0 = rope_bf16_lo(a[w]), a1 = rope_bf16_hi(a[w]);
        const float b0 = rope_bf16_lo(b[w]), b1 = rope_bf16_hi(b[w]);
        if constexpr (HALF) {
            const int p = 2 * w;
            const uint32_t na = pack2(fmaf(a0, c[p], -b0 * s[p]), fmaf(a1, c[p + 1], -b1 * s[p + 1]));
            const uint32_t nb = pack2(fmaf(b0, c[p], a0 * s[p]), fmaf(b1, c[p + 1], a1 * s[p + 1]));
            if (FULL || on) {
                a[w] = na;
                b[w] = nb;
            }
        } else {
            const uint32_t na = pack2(fmaf(a0, c[w], -a1 * s[w]), fmaf(a1, c[w], a0 * s[w]));
            const uint32_t nb = pack2(fmaf(b0, c[4 + w], -b1 * s[4 + w]), fmaf(b1, c[4 + w], b0 * s[4 + w]));
            if (FULL || ((on >> w) & 1u)) a[w] = na;
            if (FULL || ((on >> (4 + w)) & 1u)) b[w] = nb;
        }
    }
    va = make_uint4(a[0], a[1], a[2], a[3]);
    vb = make_uint4(b[0], b[1], b[2], b[3]);
}

template <bool HALF, bool FULL, int AHEAD>
__device__ __forceinline__ void walk_heads(const RopeTensor &x, int h0, int h1, int64_t b, int64_t t, int ca, int cb,
                                           const float (&c)[8], const float (&s)[8], uint32_t on) {
    const __nv_bfloat16 *in = static_cast<const __nv_bfloat16 *>(x.in) + b * x.in_b + t * x.in_n;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(x.out) + b * x.out_b + t * x.out_n;
    for (int h = h0; h < h1; h += AHEAD) {
        uint4 va[AHEAD], vb[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (h + i < h1) {
                const __nv_bfloat16 *p = in + (h + i) * x.in_h;
                va[i] = *reinterpret_cast<const uint4 *>(p + ca);
                vb[i] = *reinterpret_cast<const uint4 *>(p + cb);
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (h + i < h1) {
                turn<HALF, FULL>(va[i], vb[i], c, s, on);
                __nv_bfloat16 *p = out + (h + i) * x.out_h;
                *reinterpret_cast<uint4 *>(p + ca) = va[i];
                *reinterpret_cast<uint4 *>(p + cb) = vb[i];
            }
        }
    }
}

// grid: (token tiles, head groups, B); the heads of q come before those of k.
template <int D, bool HALF, bool FULL, int AHEAD>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeTensor q, const __grid_constant__ RopeTensor k,
                const int32_t *pos, int64_t pos_b, int N, int heads_per_group, float sign,
                const __grid_constant__ RopeParams p) {
    constexpr int TPT = D / 16;  // threads of a token
    __shared__ RopeTable table;
    table.fill(p);
    __syncthreads();
    wait_for_stream();
    const int i = threadIdx.x % TPT;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / TPT) + threadIdx.x / TPT;
    if (t >= N) return;
    const int64_t b = blockIdx.z;
    const int total = q.heads + k.heads;
    const int h0 = blockIdx.y * heads_per_group, h1 = min(total, h0 + heads_per_group);

    // the two vectors' first channels, and the first pair of each
    int ca, cb, pa, pb;
    uint32_t on = 0;
    if (HALF) {
        const int half = p.n_pairs / 8;  // vectors of each half (n_pairs is a multiple of 8)
        const bool turns = FULL || i < half;
        ca = turns ? 8 * i : 2 * p.n_pairs + 16 * (i - half);
        cb = turns ? ca + p.n_pairs : ca + 8;
        pa = 8 * i;
        pb = 8 * i + 4;
        on = turns ? 0xffu : 0u;
    } else {
        ca = 8 * i;
        cb = 8 * i + D / 2;
        pa = ca / 2;
        pb = cb / 2;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            on |= (pa + w < p.n_pairs ? 1u : 0u) << w;
            on |= (pb + w < p.n_pairs ? 1u : 0u) << (4 + w);
        }
    }
    float c[8], s[8];
    const RopePos x = rope_load_pos(pos + b * pos_b + t * p.n_axes, p.n_axes);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const int j = w < 4 ? pa + w : pb + w - 4;
        c[w] = 1.0f;
        s[w] = 0.0f;
        if (FULL || ((on >> w) & 1u)) rope_cos_sin(rope_coord(x, table.axis[j]), table.step[j], c[w], s[w]);
        s[w] *= sign;
    }
    if (h0 < q.heads) walk_heads<HALF, FULL, AHEAD>(q, h0, min(h1, q.heads), b, t, ca, cb, c, s, on);
    if (h1 > q.heads) walk_heads<HALF, FULL, AHEAD>(k, max(h0 - q.heads, 0), h1 - q.heads, b, t, ca, cb, c, s, on);
}

}  // namespace

cudaError_t launch_rope(const RopeTensor &q, const RopeTensor &k, const int32_t *pos, int64_t pos_b, int B, int N,
                        int d, bool half, bool inverse, const RopeParams &p, int sms, cudaStream_t stream) {
    const int tokens = kRopeThreads / (d / 16);
    const int64_t tiles = ceil_div(N, tokens);
    const int heads = q.heads + k.heads;
    // Two token tiles per SM or more: one group of all heads, so that a token's angles are computed
    // once.  Fewer: the heads are split until there are about three CTAs per SM.  Measured on both sides
    // of the switch, Q and K of so many heads each, d 128, us, short form / long form:
    //   token tiles per SM    0.25         0.5          1            2            3            8
    //   40 heads              10.9 / 21.3  18.8 / 23.4  34.8 / 32.8  69.2 / 68.4  103 / 95.5   254 / 240
    //    8 heads               3.5 / 5.4    6.1 / 6.7    9.2 / 9.1   15.7 / 15.1  21.8 / 21.3  53.2 / 50.1
    //    2 heads               2.4 / 3.4    3.0 / 3.5    3.4 / 4.0    6.0 / 6.2    7.3 / 10.6  15.8 / 22.0
    // (d 64 alike.)  They meet between one and two tiles per SM.  With fewer heads than the long form
    // has in flight (2 + 2 of 8) it stays behind throughout; the rule does not look at that.
    const bool is_long = tiles * B >= 2LL * sms;
    const int64_t groups_wanted = is_long ? 1 : ceil_div(3LL * sms, tiles * B);
    const int per_group = static_cast<int>(ceil_div(heads, groups_wanted < heads ? groups_wanted : heads));
    const int groups = static_cast<int>(ceil_div(heads, per_group));
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(groups), static_cast<unsigned>(B));
    const cudaLaunchConfig_t cfg = early_launch(grid, kRopeThreads, 0, stream);
    const bool full = 2 * p.n_pairs == d;
    const float sign = inverse ? -1.0f : 1.0f;
#define FVATTN_ROPE(D_, H_, F_, A_) \
    cudaLaunchKernelEx(&cfg, rope_kernel<D_, H_, F_, A_>, q, k, pos, pos_b, N, per_group, sign, p)
#define FVATTN_ROPE_F(D_, H_, A_) (full ? FVATTN_ROPE(D_, H_, true, A_) : FVATTN_ROPE(D_, H_, false, A_))
#define FVATTN_ROPE_H(D_, A_) (half ? FVATTN_ROPE_F(D_, true, A_) : FVATTN_ROPE_F(D_, false, A_))
    if (d == 128) return is_long ? FVATTN_ROPE_H(128, kLongAhead) : FVATTN_ROPE_H(128, kShortAhead);
    return is_long ? FVATTN_ROPE_H(64, kLongAhead) : FVATTN_ROPE_H(64, kShortAhead);
#undef FVATTN_ROPE_H
#undef FVATTN_ROPE_F
#undef FVATTN_ROPE
}

}  // namespace fvattn
