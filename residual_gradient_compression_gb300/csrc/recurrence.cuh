// Shared by the recurrence's kernels: their arguments, the gate, and addresses of rows.
#pragma once

#include <type_traits>

#include "train_common.cuh"

namespace adacomp {

constexpr int kRecChunk = ADACOMP_RECURRENCE_CHUNK;  // steps between kept states

struct RecSeq {  // one strided [batch, steps, channels] tensor
    void* p;
    int64_t batch, step;
};

struct RecArgs {
    RecSeq z, x, y, dy, dz, dx;
    const float *h0, *dh_last;
    const int32_t* lengths;
    float *h_last, *dh0, *carry;
    int64_t batch, steps, channels, chunks;
};

// The kernels that split the steps over clusters (recurrence_split.cu), for few columns. `by`:
// the bytes at a time that rows can be copied by.
template <typename T> cudaError_t rec_split_forward(const RecArgs& p, int by, cudaStream_t stream);
template <typename T> cudaError_t rec_split_backward(const RecArgs& p, int by, cudaStream_t stream);

namespace {

// a = sigmoid(z) and 1 - a = sigmoid(-z), neither formed by a subtraction: with
// e = exp(-|z|), 1 / (1 + e) is the larger of the two and e / (1 + e) the smaller. exp is to
// 2 + 1.2 |z| units in the last place and 0 from |z| = 87.4 on; NaN stays NaN.
__device__ __forceinline__ void gate(float z, float* a, float* b)
{
    float e = -1.44269504f * fabsf(z), r = 1.0f;
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e));
    r += e;
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r));
    const float s = e * r;
    const bool open = z >= 0.0f;
    *a = open ? r : s;
    *b = open ? s : r;
}

__device__ __forceinline__ int64_t length_of(const RecArgs& p, int64_t b)
{
    if (!p.lengths) return p.steps;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : n > p.steps ? p.steps : n;
}

template <typename T> __device__ __forceinline__ T* at(const RecSeq& s, int64_t b, int64_t t, int64_t c)
{
    return static_cast<T*>(s.p) + b * s.batch + t * s.step + c;
}

template <typename T> __device__ __forceinline__ T* moved(T* p, int64_t bytes)
{
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + bytes);
}

// Distances between rows, in bytes: in 32 bits where the rows are read 16 bytes at a time
// (the host sees to it), so that an address is one instruction.
template <int kBytes>
using Distance = typename std::conditional<kBytes == 16 || kBytes < 0, int32_t, int64_t>::type;

}  // namespace
}  // namespace adacomp
