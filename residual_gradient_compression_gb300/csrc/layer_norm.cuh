// Shared by layer norm's kernels: their arguments, and rows in pieces of up to 16 bytes.
#pragma once

#include <initializer_list>

#include "train_common.cuh"

namespace adacomp {

struct LnArgs {
    const void *x, *dy, *w, *b;
    void *y, *dx, *dw, *db;
    float *mean, *rstd;          // outputs of the forward pass
    const float *mean_in, *rstd_in;
    float* part;                 // [slices][2][dim], and a pair of sums per row where rows are wide
    int64_t rows, dim, x_stride, y_stride, dy_stride, dx_stride;
    int32_t slices;              // of the rows, each with partial sums of dw and db
    int32_t group;               // threads of a row
    float eps;
};

// The backward pass (layer_norm_backward.cu), and the bytes of its workspace.
template <typename X, typename W> cudaError_t ln_backward(const LnArgs& a, cudaStream_t stream);
size_t ln_backward_bytes(int64_t rows, int64_t dim);

namespace {

// N consecutive elements as they lie in memory: 16, 8, 4 or 2 bytes, as the rows' alignment allows.
template <int kBytes> struct RawOf;
template <> struct RawOf<16> {
    using type = uint4;
};
template <> struct RawOf<8> {
    using type = uint2;
};
template <> struct RawOf<4> {
    using type = uint32_t;
};
template <> struct RawOf<2> {
    using type = uint16_t;
};

template <typename X, int N> struct Piece {
    static constexpr int kBytes = N * (int)sizeof(X);
    using Raw = typename RawOf<kBytes>::type;
    Raw q;
    __device__ __forceinline__ void load(const X* p) { q = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ void zero() { q = Raw{}; }
    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (kBytes == 16) {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            if constexpr (sizeof(X) == 4) return __uint_as_float(w[j]);
            else return j & 1 ? bf16_high(w[j / 2]) : bf16_low(w[j / 2]);
        } else if constexpr (kBytes == 8) {
            return j & 1 ? bf16_high(j < 2 ? q.x : q.y) : bf16_low(j < 2 ? q.x : q.y);
        } else if constexpr (sizeof(X) == 4) {
            return __uint_as_float(q);
        } else {
            return j & 1 ? bf16_high(q) : bf16_low(q);
        }
    }
};

// The elements of a thread's pieces, two at a time, across the pieces where they are single.
template <typename X, int N, int kPieces> __device__ __forceinline__ Pair pair_of(const Piece<X, N> (&p)[kPieces], int i)
{
    return pair(p[2 * i / N].get(2 * i % N), p[(2 * i + 1) / N].get((2 * i + 1) % N));
}

template <int N> __device__ __forceinline__ void put_piece(float* p, const float (&v)[N])
{
    if constexpr (N == 1) *p = v[0];
    else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

template <int N> __device__ __forceinline__ void put_piece(bf16* p, const float (&v)[N])
{
    if constexpr (N == 1) {
        *p = from_f32<bf16>(v[0]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
    } else if constexpr (N == 4) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&t);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// N weights from p on (4 or 8 of them: from a 16-byte boundary).
template <int N> __device__ __forceinline__ void weights(const float* p, float (&v)[N])
{
    if constexpr (N < 4) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = p[j];
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 q = *reinterpret_cast<const float4*>(p + j);
            v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
        }
    }
}

template <int N> __device__ __forceinline__ void weights(const bf16* p, float (&v)[N])
{
    if constexpr (N < 4) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = to_f32(p[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const uint2 q = *reinterpret_cast<const uint2*>(p + j);
            v[j] = bf16_low(q.x), v[j + 1] = bf16_high(q.x), v[j + 2] = bf16_low(q.y), v[j + 3] = bf16_high(q.y);
        }
    }
}

// Where rows are long a thread adds runs of kLnRun terms, and the runs' sums with what their
// additions round off: a sum of millions of terms in sequence would lose their last bits, all in
// one direction if they are alike. (fp64 sums instead: 4096 x 12288 bf16 backward 145 us, not 98.)
constexpr int kLnRun = 256;

struct RunSum {
    float sum = 0.0f, rest = 0.0f;
    __device__ __forceinline__ void add(float v)  // D. Knuth's exact sum of two
    {
        const float t = sum + v, from_v = t - sum;
        rest += (sum - (t - from_v)) + (v - from_v);
        sum = t;
    }
    __device__ __forceinline__ float value() const { return sum + rest; }
};

// The sum over the lanes of a group of up to 32 (a power of two).
__device__ __forceinline__ float group_sum(float v, int group)
{
    for (int o = group >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- host
// How many elements of the rows can be read and written at a time: 16 bytes of them, 4 or one.
int piece_of(const LnArgs& a, int ex, std::initializer_list<const void*> p, std::initializer_list<int64_t> strides,
             std::initializer_list<const void*> weights)
{
    int64_t bits = a.dim * ex;
    for (const void* q : p) bits |= (int64_t)reinterpret_cast<uintptr_t>(q);
    if (a.rows > 1)
        for (int64_t s : strides) bits |= s * ex;
    bool whole = bits % 16 == 0;
    for (const void* q : weights) whole = whole && is_aligned(q, 16);
    return whole ? 16 / ex : bits % 4 == 0 ? 4 / ex : 1;
}

int group_of(int64_t places, int most)  // the smallest power of two with room for them
{
    int g = 1;
    while (g < most && g < places) g *= 2;
    return g;
}

}  // namespace
}  // namespace adacomp
