// Shared by the training operators' kernels (layer norm, recurrence, AdamW): element
// types, loads and stores of short vectors, warp sums, and host-side checks.
#pragma once

#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "adacomp.h"
#include "adacomp_internal.cuh"

namespace adacomp {

adacomp_status launch_result(cudaError_t e, cudaStream_t stream);  // abi.cu

namespace {

// ---------------------------------------------------------------- host
struct TrainRange {  // a named range on the host timeline, as for the compressor's calls
    explicit TrainRange(const char* name) { nvtxRangePushA(name); }
    ~TrainRange() { nvtxRangePop(); }
    TrainRange(const TrainRange&) = delete;
    TrainRange& operator=(const TrainRange&) = delete;
};

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool known_dtype(int32_t t) { return t == ADACOMP_F32 || t == ADACOMP_BF16; }
inline int dtype_bytes(int32_t t) { return t == ADACOMP_BF16 ? 2 : 4; }

// Multiprocessors of the current device, looked up once per device (by any of several host threads).
inline cudaError_t sm_count(int* out)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return cudaSuccess;
}

// Lets a kernel have `shared` bytes of dynamic shared memory, and (kClusters) clusters of more than
// eight CTAs, once per device; of several host threads that come first, each does.
template <auto kern, bool kClusters = false> cudaError_t allow(int shared)
{
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
    if (kClusters && e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

// ---------------------------------------------------------------- device
using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- pairs
// Two fp32 values that one instruction computes with. Every operation rounds as its scalar
// form does (.rn: no contraction).
struct Pair {
    unsigned long long b;
};

__device__ __forceinline__ Pair pair(float x, float y)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.b) : "f"(x), "f"(y));
    return p;
}

__device__ __forceinline__ Pair pair(float x) { return pair(x, x); }

__device__ __forceinline__ void split(Pair p, float& x, float& y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p.b));
}

__device__ __forceinline__ float both(Pair p)  // the sum of the two
{
    float x, y;
    split(p, x, y);
    return x + y;
}

__device__ __forceinline__ Pair operator*(Pair x, Pair y)
{
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.b) : "l"(x.b), "l"(y.b));
    return p;
}

__device__ __forceinline__ Pair fma2(Pair x, Pair y, Pair z)
{
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.b) : "l"(x.b), "l"(y.b), "l"(z.b));
    return p;
}

__device__ __forceinline__ Pair operator+(Pair x, Pair y) { return fma2(x, pair(1.0f), y); }  // x + y, in any company

}  // namespace
}  // namespace adacomp
