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
    double turns[kMaxRopePairs];   // revolutions per unit of position: inv_freq / (2 pi)
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

// Cosine and sine of pos * turns revolutions.  The product and its reduction to half a
// revolution run in fp64, so that a position of 2^31 still has an angle good to about
// 1e-6; what is left is below pi and goes through the fp32 sincospif.
__device__ __forceinline__ void rope_cos_sin(int pos, double turns, float &c, float &s) {
    double t = static_cast<double>(pos) * turns;
    t -= rint(t);
    sincospif(static_cast<float>(2.0 * t), &s, &c);
}

// The coordinates of one token.
struct RopePos {
    int x[kMaxRopeAxes];
};

__device__ __forceinline__ RopePos rope_load_pos(const int32_t *p, int n_axes) {
    RopePos r;
#pragma unroll
    for (int a = 0; a < kMaxRopeAxes; ++a) r.x[a] = a < n_axes ? __ldg(p + a) : 0;
    return r;
}

__device__ __forceinline__ int rope_coord(const RopePos &p, int axis) {
    return axis == 0 ? p.x[0] : axis == 1 ? p.x[1] : axis == 2 ? p.x[2] : p.x[3];
}

#endif

}  // namespace fvattn
