// Shared by the recurrence's kernels: their arguments, the gate, and addresses of rows.
#pragma once

#include <initializer_list>
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
    uint32_t timeout;  // of a wait for the other CTAs of a cluster, in 1024 ns
    uint32_t silent;   // test only: the CTA of every cluster that writes nothing to the others
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

__device__ __forceinline__ float least3(float x, float y, float z)
{
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

__device__ __forceinline__ float not_below(float x, float least)  // NaN stays NaN
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(least));
    return r;
}

// The product of gates, which is 0 only if one of them is: what vanishes in fp32 is rounded up to
// kLeast and not down to 0, so that an infinite state stays infinite behind it, as it does step
// by step (0 * infinity is not a number). The states wait for nothing that this adds.
constexpr float kLeast = 0x1p-149f;

__device__ __forceinline__ float product(float A, float a) { return not_below(A * a, least3(A, a, kLeast)); }

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

// kBytes, by which the kernels take a tensor's rows: 16, 4 or 2 bytes at a time as they are
// aligned, or less than zero: rows of elements of -kBytes bytes without alignment, by the
// aligned 16 bytes that hold them (a copy of four bytes costs as much as one of 16).
// Tiles are then of one sequence's channels (kApart), and otherwise of all sequences'
// numbered through, so that few channels fill a tile too.
template <int kBytes> constexpr bool kApart = kBytes == 16 || kBytes < 0;

// Distances between rows, in bytes: in 32 bits where the rows are read 16 bytes at a time
// (the host sees to it), so that an address is one instruction.
template <int kBytes> using Distance = typename std::conditional<kApart<kBytes>, int32_t, int64_t>::type;

// Whether rows without alignment are taken by the aligned 16 bytes that hold them, in tiles of
// `cols` of one sequence's channels: unless that makes more tiles than channels that are numbered
// through do by `through`, and more than `most`.
inline bool by_granules(const RecArgs& p, int64_t cols, int64_t through, int64_t most,
                        std::initializer_list<const RecSeq*> seqs)
{
    const int64_t apart = p.batch * ((p.channels + cols - 1) / cols), tiles = (p.batch * p.channels + through - 1) / through;
    bool fits = p.channels >= 32 && (4 * apart <= 5 * tiles || apart <= most);
    for (const RecSeq* s : seqs) fits = fits && s->step < (int64_t)1 << 22;  // a tile's steps span less than 2^31 bytes
    return fits;
}

}  // namespace
}  // namespace adacomp
