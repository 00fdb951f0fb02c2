// common.cuh -- status codes, device-status helpers and small utilities shared
// by the routing, ordering and attention kernels of libfvattn.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "fvattn.h"

namespace fvattn {

// First device error wins: the status word holds 0 until some thread records
// an error, after which it is never overwritten.
__device__ __forceinline__ void record_error(int32_t *dev_status, int32_t code) {
    if (dev_status) atomicCAS(reinterpret_cast<int *>(dev_status), 0, code);
}

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Host side: records the reason of the calling thread's latest FVATTN_ERR_CUDA (a
// static string), read back through fvattn_last_error().
void set_last_error(const char *what);
__host__ __device__ constexpr size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Workspace carving: every region starts on a 256-byte boundary.
struct Carver {
    size_t off = 0;
    template <class T>
    size_t take(size_t count) {
        size_t at = align_up(off, 256);
        off = at + count * sizeof(T);
        return at;
    }
};

// A launch that may begin before the kernel in front of it in the stream has ended: the kernel waits for
// that one itself (wait_for_stream) before it reads or writes anything, so that only the launch is
// overlapped.  It saves about 1 us a call where calls for single tokens follow each other.  What the
// kernel in front may have written is not read through the read-only path (__ldg): that is for data
// that nobody writes while the kernel lives, and this one lives already.
inline cudaLaunchConfig_t early_launch(dim3 grid, unsigned threads, size_t smem, cudaStream_t stream) {
    static cudaLaunchAttribute early = [] {
        cudaLaunchAttribute a{};
        a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        a.val.programmaticStreamSerializationAllowed = 1;
        return a;
    }();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cfg;
}

// Lets a kernel use `bytes` of dynamic shared memory, on its first launch on each device (the attribute
// belongs to the device's own copy of the function).
template <auto Kernel>
cudaError_t allow_shared_memory(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load() & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

constexpr int kMaxRouteBlocks = 1024;   // routing keeps one row's scores in shared memory
constexpr int kMaxCount = 4096;         // largest key-block count a row may hold
constexpr int kMaxHeads = 4096;         // largest B*H of the attention call (head ordering in one CTA)

}  // namespace fvattn
