// rope.cuh -- rotary positions with several axes: the parameters the host passes and
// the device helpers shared by the rotation (rope.cu) and the cache append
// (cache_append.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fvattn {

constexpr int kMaxRopePairs = 64;  // d / 2 at d = 128
constexpr int kMaxRopeAxes = 4;

// By value in the kernels' parameters: what one channel pair is turned by.
struct RopeParams {
    uint64_t step[kMaxRopePairs];  // revolutions per unit of position, modulo 1 in 2^-64 (rope_step.h)
    uint8_t axis[kMaxRopePairs];   // which coordinate of the position turns the pair
    int n_pairs;                   // pairs that turn; 2 n_pairs <= d, the other channels pass through
    int n_axes;
};

// One tensor of a rotation: element (b, h, t, c) at b * sb + h * sh + t * sn + c (in elements).
struct RopeTensor {
    const void *in;
    void *out;
    int64_t in_b, in_h, in_n, out_b, out_h, out_n;
    int heads;
};

cudaError_t launch_rope(const RopeTensor &q, const RopeTensor &k, const int32_t *pos, int64_t pos_b, int B, int N,
                        int d, bool half, bool inverse, const RopeParams &p, int sms, cudaStream_t stream);

#ifdef __CUDACC__

__device__ __forceinline__ float rope_bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float rope_bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// What a CTA's threads look up by pair, in shared memory: neighbouring threads want different
// pairs, which the kernel parameters' constant bank would serve one after the other.
struct RopeTable {
    uint64_t step[kMaxRopePairs];
    int axis[kMaxRopePairs];

    // By the first threads of the CTA; a barrier follows.
    __device__ __forceinline__ void fill(const RopeParams &p) {
        if (threadIdx.x < kMaxRopePairs) {
            step[threadIdx.x] = p.step[threadIdx.x];
            axis[threadIdx.x] = p.axis[threadIdx.x];
        }
    }
};

// Cosine and sine of pos steps.  A position is a whole number, so whole revolutions drop out of the
// 64-bit product by themselves, and the angle is exact but for the step's last bit (2^-64 of a
// revolution, 1e-9 radians at 2^31).  Of its upper 32 bits the first two, rounded, are the
// quarter turn; the rest is an angle x in [-pi/4, pi/4), good to 2^-24 of itself, whose sine
// and cosine come from their Taylor series up to x^9 and x^8 (what is left out is below 2e-9 and
// 3e-8).  (The same through fp64 products and sincospif took most of an append's time.)
__device__ __forceinline__ void rope_cos_sin(int pos, uint64_t step, float &c, float &s) {
    const uint32_t turn = static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(pos)) * step) >> 32) + 0x20000000u;
    const float x = static_cast<float>(static_cast<int32_t>(turn & 0x3fffffffu) - 0x20000000) * 1.4629180792671596e-9f;  // 2 pi 2^-32
    const float x2 = x * x;
    float sn = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, -1/7!
    sn = fmaf(x2, sn, 8.3333333e-3f);                     // 1/5!
    sn = fmaf(x2, sn, -1.6666667e-1f);                    // -1/3!
    sn = fmaf(x * x2, sn, x);
    float cs = fmaf(x2, 2.4801587e-5f, -1.3888889e-3f);  // 1/8!, -1/6!
    cs = fmaf(x2, cs, 4.1666667e-2f);                     // 1/4!
    cs = fmaf(x2, cs, -0.5f);
    cs = fmaf(x2, cs, 1.0f);
    // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
    const bool odd = turn & 0x40000000u;
    c = __uint_as_float(__float_as_uint(odd ? sn : cs) ^ ((turn ^ (turn << 1)) & 0x80000000u));
    s = __uint_as_float(__float_as_uint(odd ? cs : sn) ^ (turn & 0x80000000u));
}

// The coordinates of one token.
struct RopePos {
    int x[kMaxRopeAxes];
};

__device__ __forceinline__ RopePos rope_load_pos(const int32_t *p, int n_axes) {
    RopePos r;
#pragma unroll
    for (int a = 0; a < kMaxRopeAxes; ++a) r.x[a] = a < n_axes ? p[a] : 0;
    return r;
}

__device__ __forceinline__ int rope_coord(const RopePos &p, int axis) {
    return axis == 0 ? p.x[0] : axis == 1 ? p.x[1] : axis == 2 ? p.x[2] : p.x[3];
}

#endif

}  // namespace fvattn
