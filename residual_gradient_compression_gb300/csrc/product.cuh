// Shared by the linear layers and the losses over a vocabulary: what is done with a product's sums (the
// epilogues).
//
// A product is C(m, n) = sum over k of A(m, k) B(n, k). A warp of the kernel that forms it has 32 rows' sums in
// registers, 128 columns of a row per thread, and hands them to an epilogue in two steps: rows(), a thread its
// row (from column c up to `last`, the strip-th of the row), with what begin() loaded before the sums were
// there; and chunk(), the warp 32 columns at a time through shared memory, so that what it reads and writes in
// global memory are whole pieces of rows (a thread that writes its own row takes 32 cache lines at a time: a
// linear layer's forward product of 8192 x 2048 x 16384 bf16 took 369 us so, and 313 without its stores).
// kExact: the results are held in fp32, so the sums are formed in short runs. kPieces: a thread may also hand
// over columns on their own, piece(). kFetches: there may be a matrix that the chunks are added to: begin()
// brings it into L2, and fetch() loads a chunk while the one before is worked on (a chunk's loads in its turn: a
// layer of 16384 x 2048 x 8192 bf16 with a residual 608 us, and 414 so). kPatches: patch() changes single
// columns of a chunk in shared memory. kParts: part() takes the sums of a part of the terms.
#pragma once

#include "train_common.cuh"

namespace adacomp {

// Parts of a caller's workspace, one after the other; without a base, only their sizes.
struct Carve {
    char* base = nullptr;
    size_t at = 0;
    template <typename T> T* take(int64_t n)
    {
        const size_t from = at;
        at += ((size_t)(n < 0 ? 0 : n) * sizeof(T) + 255) & ~(size_t)255;
        return base ? reinterpret_cast<T*>(base + from) : nullptr;
    }
};

namespace {

constexpr int kStrip = 128;  // columns of a row that a thread has; a softmax's partial sums are kept for each
constexpr int kRows = 128;   // rows of a tile

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// ---------------------------------------------------------------- a row's columns, eight or a multiple of them
template <typename T, int N> __device__ __forceinline__ void put_chunk(T* p, const float (&v)[N], int64_t left, bool whole)
{
    if (whole && left >= N) {
        uint4* q = reinterpret_cast<uint4*>(p);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                q[i / 4] = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                                      __float_as_uint(v[i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 t = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&t);
                }
                q[i / 8] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) p[i] = from_f32<T>(v[i]);
}

template <typename T, int N> __device__ __forceinline__ void get_chunk(const T* p, float (&v)[N], int64_t left, bool whole)
{
    if (whole && left >= N) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
        for (int i = 0; i < N * (int)sizeof(T) / 16; ++i) {
            const uint4 u = q[i];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    v[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    v[8 * i + 2 * j] = bf16_low(w[j]);
                    v[8 * i + 2 * j + 1] = bf16_high(w[j]);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
}

// N columns of a row: four that are aligned to as many, or one.
template <int N> struct Cols {
    float v[N];
    __device__ __forceinline__ Cols operator+(const Cols& o) const
    {
        Cols s;
#pragma unroll
        for (int i = 0; i < N; ++i) s.v[i] = v[i] + o.v[i];
        return s;
    }
};

template <typename T, int N> __device__ __forceinline__ void put(T* p, const Cols<N>& c, int32_t left)
{
    if constexpr (N == 4) {
        if (left >= 4) {
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(p) = make_float4(c.v[0], c.v[1], c.v[2], c.v[3]);
            } else {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(c.v[0], c.v[1]), hi = __floats2bfloat162_rn(c.v[2], c.v[3]);
                *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) p[i] = from_f32<T>(c.v[i]);
}

template <int N, typename T> __device__ __forceinline__ Cols<N> get(const T* p, int32_t left)
{
    Cols<N> c;
    if constexpr (N == 4) {
        if (left >= 4) {
            if constexpr (sizeof(T) == 4) {
                const float4 w = *reinterpret_cast<const float4*>(p);
                c.v[0] = w.x, c.v[1] = w.y, c.v[2] = w.z, c.v[3] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(p);
                c.v[0] = bf16_low(w.x), c.v[1] = bf16_high(w.x), c.v[2] = bf16_low(w.y), c.v[3] = bf16_high(w.y);
            }
            return c;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) c.v[i] = i < left ? to_f32(p[i]) : 0.0f;
    return c;
}

// A warp's 32 rows of 32 columns in shared memory; a row's 16-byte pieces lie where no two rows of eight share banks.
struct Stage {
    float4* p;
    __device__ __forceinline__ float4& at(int row, int piece) const { return p[row * 8 + (piece ^ (row & 7))]; }
};

// A thread's own row: 32 of its columns to shared memory, and one of them there.
__device__ __forceinline__ void put_row(const Stage& s, const float (&v)[kStrip], int from)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) s.at(lane, i) = make_float4(v[from + 4 * i], v[from + 4 * i + 1], v[from + 4 * i + 2], v[from + 4 * i + 3]);
}

__device__ __forceinline__ void put_chunk_of(const Stage& s, const float (&v)[kStrip], int chunk)  // in loops that are not unrolled
{
    switch (chunk) {
    case 0: put_row(s, v, 0); break;
    case 1: put_row(s, v, 32); break;
    case 2: put_row(s, v, 64); break;
    default: put_row(s, v, 96);
    }
}

__device__ __forceinline__ float& row_value(const Stage& s, int col)
{
    return reinterpret_cast<float*>(&s.at(threadIdx.x & 31, col / 4))[col & 3];
}

// How a warp takes a chunk: in turns of four rows, of which a lane has four columns, or, where rows do not begin
// at such places, of one row, of which it has one.
template <int N> struct Turns {
    static constexpr int kCount = N == 4 ? 8 : 32;
    int row, col;
    __device__ __forceinline__ Turns()
    {
        const int lane = threadIdx.x & 31;
        row = N == 4 ? lane / 8 : 0;
        col = N == 4 ? (lane & 7) * 4 : lane;
    }
    __device__ __forceinline__ int row_of(int turn) const { return turn * (32 / kCount) + row; }
    __device__ __forceinline__ Cols<N> read(const Stage& s, int turn) const
    {
        const float4& v = s.at(row_of(turn), col / 4);
        Cols<N> c;
        if constexpr (N == 4) c.v[0] = v.x, c.v[1] = v.y, c.v[2] = v.z, c.v[3] = v.w;
        else c.v[0] = reinterpret_cast<const float*>(&v)[col & 3];
        return c;
    }
    __device__ __forceinline__ void write(const Stage& s, int turn, const Cols<N>& c) const
    {
        float4& v = s.at(row_of(turn), col / 4);
        if constexpr (N == 4) v = make_float4(c.v[0], c.v[1], c.v[2], c.v[3]);
        else reinterpret_cast<float*>(&v)[col & 3] = c.v[0];
    }
};

inline bool whole_rows(const void* p, int64_t stride, int64_t rows, int bytes)
{
    return is_aligned(p, 16) && (rows < 2 || stride * bytes % 16 == 0);
}

// A chunk of a matrix that an epilogue reads, as a warp takes it, on its way while the chunk before is worked on.
struct Fetched {
    uint32_t w[32];
    template <typename T, int N> __device__ __forceinline__ void load(int turn, const T* p, int32_t left)
    {
        constexpr int kWords = N == 1 ? 1 : (int)sizeof(T);
        uint32_t* to = w + turn * kWords;
        if constexpr (N == 4) {
            if (left >= 4) {
                if constexpr (sizeof(T) == 4) {
                    const uint4 q = *reinterpret_cast<const uint4*>(p);
                    to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
                } else {
                    const uint2 q = *reinterpret_cast<const uint2*>(p);
                    to[0] = q.x, to[1] = q.y;
                }
                return;
            }
        }
        const Cols<N> c = get<N>(p, left);
        if constexpr (N == 4 && sizeof(T) == 2) {
            to[0] = __float_as_uint(c.v[0]) >> 16 | (__float_as_uint(c.v[1]) & 0xffff0000u);
            to[1] = __float_as_uint(c.v[2]) >> 16 | (__float_as_uint(c.v[3]) & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) to[i] = __float_as_uint(c.v[i]);
        }
    }
    template <typename T, int N> __device__ __forceinline__ Cols<N> use(int turn) const
    {
        constexpr int kWords = N == 1 ? 1 : (int)sizeof(T);
        const uint32_t* from = w + turn * kWords;
        Cols<N> c;
        if constexpr (N == 4 && sizeof(T) == 2) {
            c.v[0] = bf16_low(from[0]), c.v[1] = bf16_high(from[0]), c.v[2] = bf16_low(from[1]), c.v[3] = bf16_high(from[1]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) c.v[i] = __uint_as_float(from[i]);
        }
        return c;
    }
    template <typename T, int N>
    __device__ __forceinline__ void load_all(const T* p, int64_t stride, int32_t n, int32_t r0, int32_t end, int32_t c0)
    {
        const Turns<N> turn;
        const int32_t c = c0 + turn.col, left = n - c;
#pragma unroll
        for (int i = 0; i < Turns<N>::kCount; ++i) {
            const int32_t r = r0 + turn.row_of(i);
            load<T, N>(i, p + r * stride + c, r < end ? left : 0);
        }
    }
};

// Brings a row's columns from p on into L2.
template <typename T> __device__ __forceinline__ void prefetch_row(const T* p, int32_t left)
{
    const char* q = reinterpret_cast<const char*>(p);
    const int32_t bytes = (left < kStrip ? left : kStrip) * (int32_t)sizeof(T);
    for (int32_t i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i));
}

// Of a matrix in a workspace: rows begin with a cache line, unless they are shorter than one.
inline int64_t pitch_of(int64_t cols) { return round_up(cols, cols < 64 ? 8 : 64); }

// ---------------------------------------------------------------- fp32 numbers in parts
constexpr int kPlanes = 4;  // of bf16 numbers for an fp32 matrix

// x = top + mid + low exactly (but for what is below 2^-133), each a bf16 number. A value that is not finite has
// only a top; the fourth plane is the top without such values, for the products with the other operand's lower
// parts (infinity times a part that is 0 would be NaN).
__device__ __forceinline__ void split_parts(float x, bf16 (&part)[kPlanes])
{
    part[0] = __float2bfloat16_rn(x);
    part[1] = part[2] = part[3] = __float2bfloat16_rn(0.0f);
    if (!(fabsf(x) <= 3.402823466e38f)) return;
    if (__hisinf(part[0])) part[0] = __float2bfloat16_rz(x);  // rounded past the largest bf16 number
    const float rest = x - __bfloat162float(part[0]);
    part[1] = __float2bfloat16_rn(rest);
    part[2] = __float2bfloat16_rn(rest - __bfloat162float(part[1]));
    part[3] = part[0];
}

// The same by cutting bits off instead of rounding, in fewer instructions, for an epilogue (a training step of
// cross entropy 2003 x 501 x 10007 396 and 378 us); each part the upper half of a word. The other operand's
// parts are rounded, so what their products leave out has no sign in common.
__device__ __forceinline__ void cut_parts(float x, uint32_t (&part)[kPlanes])
{
    const bool finite = fabsf(x) <= 3.402823466e38f;
    part[0] = x != x ? 0x7fff0000u : __float_as_uint(x) & 0xffff0000u;
    const float rest = finite ? x - __uint_as_float(part[0]) : 0.0f;
    part[1] = __float_as_uint(rest) & 0xffff0000u;
    part[2] = __float_as_uint(rest - __uint_as_float(part[1])) & 0xffff0000u;
    part[3] = finite ? part[0] : 0u;
}

// A value in two parts of one sign, so that an infinite factor meets no 0 or other sign in the second: what bf16
// has of its bits, and the rest, or where there is none 2^-24 of it.
__device__ __forceinline__ float first_of(float v) { return __bfloat162float(__float2bfloat16_rz(v)); }
__device__ __forceinline__ float rest_of(float v)
{
    if (isinf(v)) return copysignf(1.0f, v);
    const float rest = v - first_of(v);
    return rest == 0.0f ? v * 5.9604645e-8f : rest;
}

// The gradient of bf16 products is an operand of two more. It is rounded to bf16 for them, by 2^-9 of each value
// at random, which is less than their results' own rounding where sums of many rows or columns are formed; of up
// to kFewRows rows, whose few values may share one rounding, it is taken in two parts (the products' time is
// that of reading and writing the weights).
constexpr int64_t kFewRows = 32;

// A row's columns as operands of another product: bf16 numbers, two planes of them, or, of an fp32 matrix, four.
template <typename T, int N> __device__ __forceinline__ void put_parts(bf16* p, int64_t plane, const float (&v)[N], int64_t left, bool two)
{
    if constexpr (sizeof(T) == 2) {
        if (!two) {
            put_chunk(p, v, left, true);
            return;
        }
        float part[N];
#pragma unroll
        for (int i = 0; i < N; ++i) part[i] = first_of(v[i]);
        put_chunk(p, part, left, true);
#pragma unroll
        for (int i = 0; i < N; ++i) part[i] = rest_of(v[i]);
        put_chunk(p + plane, part, left, true);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            float part[kPlanes][8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                bf16 each[kPlanes];
                split_parts(v[i + c], each);
#pragma unroll
                for (int j = 0; j < kPlanes; ++j) part[j][c] = __bfloat162float(each[j]);
            }
#pragma unroll
            for (int j = 0; j < kPlanes; ++j) put_chunk(p + j * plane + i, part[j], left - i, true);
        }
    }
}

// ---------------------------------------------------------------- activations
// None of them is formed as a difference that cancels: far below 0 each is right relative to itself. Of bf16 layers by
// quick functions, as the epilogue of a product of 2048 terms has no time for more. 1 + erf(x) of x = z / sqrt 2, and exp(-x^2), of
// two values at a time: erfc(|x|) = exp(-x^2) t p(t) with t = 1 / (1 + 0.411 |x|), whose coefficients are fitted here
// (linear program over 0 <= x <= 9.4: 1.1e-7 at most, and 7.3e-5 of erfc where that is less). With the exponential's
// argument it is off by 3.5e-7 or 1.2e-4 of erfc, whichever is less: far below what bf16 results are rounded to.
__device__ __forceinline__ Pair quick_one_plus_erf(Pair z, Pair& bell)
{
    float z0, z1, e0, e1, d0, d1, r0, r1;
    split(z, z0, z1);
    split(z * z * pair(-0.72134752f), e0, e1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(e0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(e1));
    bell = pair(r0, r1);
    split(fma2(pair(fabsf(z0), fabsf(z1)), pair(0.29062089f), pair(1.0f)), d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
    const Pair t = pair(r0, r1);
    const Pair p = fma2(t, fma2(t, fma2(t, fma2(t, fma2(t, pair(-0.17731535f), pair(0.56442744f)), pair(-0.18067640f)), pair(0.35698659f)),
                                pair(0.20235198f)), pair(0.23422568f));
    const Pair tail = t * p * bell;  // erfc(|x|)
    split(tail, e0, e1);
    split(fma2(tail, pair(-1.0f), pair(2.0f)), r0, r1);
    return pair(z0 < 0.0f ? e0 : r0, z1 < 0.0f ? e1 : r1);
}

__device__ __forceinline__ float quick_sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

template <typename T, int kKind> __device__ __forceinline__ float activate(float z)
{
    constexpr bool kQuick = sizeof(T) == 2;
    if constexpr (kKind == ADACOMP_ACT_RELU) {
        return z < 0.0f ? 0.0f : z;
    } else if constexpr (kKind == ADACOMP_ACT_GELU) {
        return 0.5f * z * erfcf(-0.70710678f * z);
    } else if constexpr (kKind == ADACOMP_ACT_GELU_TANH) {  // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        const float u = 0.79788456f * (z + 0.044715f * z * z * z);
        if (kQuick) return z * quick_sigmoid(2.0f * u);
        return z / (1.0f + expf(-2.0f * u));
    } else if constexpr (kKind == ADACOMP_ACT_SILU) {
        if (kQuick) return z * quick_sigmoid(z);
        return z / (1.0f + expf(-z));
    } else {
        return z;
    }
}

template <typename T, int kKind> __device__ __forceinline__ float slope(float z)
{
    constexpr bool kQuick = sizeof(T) == 2;
    if constexpr (kKind == ADACOMP_ACT_RELU) {
        return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;  // NaN stays NaN
    } else if constexpr (kKind == ADACOMP_ACT_GELU) {
        return 0.5f * erfcf(-0.70710678f * z) + z * expf(-0.5f * z * z) * 0.39894228f;
    } else if constexpr (kKind == ADACOMP_ACT_GELU_TANH) {  // s = (1 + tanh u) / 2: s + 2 z s (1 - s) du/dz
        const float u = 0.79788456f * (z + 0.044715f * z * z * z);
        const float s = kQuick ? quick_sigmoid(2.0f * u) : 1.0f / (1.0f + expf(-2.0f * u));
        const float c = fmaxf(fminf(z, 100.0f), -100.0f);  // where s is 0 or 1, and z z might overflow
        return s * (1.0f + c * (1.0f - s) * 1.5957691f * (1.0f + 0.134145f * c * c));
    } else if constexpr (kKind == ADACOMP_ACT_SILU) {
        const float g = kQuick ? quick_sigmoid(z) : 1.0f / (1.0f + expf(-z));
        return g * (1.0f + z * (1.0f - g));
    } else {
        return 1.0f;
    }
}

// N values at a time, an even number of them or one.
template <typename T, int kKind, int N> __device__ __forceinline__ void activate_all(float (&v)[N])
{
    if constexpr (sizeof(T) == 2 && kKind == ADACOMP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const Pair z = pair(v[i], v[N == 1 ? i : i + 1]);
            Pair bell;
            float a, b;
            split(z * pair(0.5f) * quick_one_plus_erf(z, bell), a, b);
            v[i] = a;
            if (N > 1) v[N == 1 ? i : i + 1] = b;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = activate<T, kKind>(v[i]);
    }
}

template <typename T, int kKind, int N> __device__ __forceinline__ void slope_all(float (&v)[N])
{
    if constexpr (sizeof(T) == 2 && kKind == ADACOMP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const Pair z = pair(v[i], v[i + 1]);
            Pair bell;
            const Pair c = quick_one_plus_erf(z, bell) * pair(0.5f);
            split(fma2(z * pair(0.39894228f), bell, c), v[i], v[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = slope<T, kKind>(v[i]);
    }
}

// ---------------------------------------------------------------- epilogues
// y = act(sum + bias) + residual, and the value before the activation.
template <typename T> struct EpiLinear {
    // fp32: one copy of the instructions, which a CTA with one or two tiles waits to be loaded (a training step
    // of 3001 x 1001 x 777 187 and 165 us); bf16: four, whose stores overlap (gelu of 16384 x 2048 x 8192 with
    // both outputs 432 and 378)
    static constexpr int kUnroll = sizeof(T) == 4 ? 1 : 4;
    static constexpr bool kExact = sizeof(T) == 4, kChunks = true, kPieces = true, kFetches = true, kPatches = false, kParts = false;
    T *y, *pre;
    const T *bias, *residual;
    int64_t y_stride, pre_stride, residual_stride;
    int32_t n, act;
    bool whole;  // all of them
    struct State {};
    __device__ __forceinline__ bool fetches() const { return residual != nullptr; }
    __device__ __forceinline__ State begin(int32_t r, int32_t c) const
    {
        if (residual) prefetch_row(residual + r * residual_stride + c, n - c);
        return {};
    }
    __device__ __forceinline__ void rows(const Stage&, const State&, int32_t, int32_t, int32_t, int32_t, bool, float (&)[kStrip]) const {}

    __device__ __forceinline__ void fetch(Fetched& f, int32_t r0, int32_t end, int32_t c0) const
    {
        if (whole) f.load_all<T, 4>(residual, residual_stride, n, r0, end, c0);
        else f.load_all<T, 1>(residual, residual_stride, n, r0, end, c0);
    }

    // (Little unrolled: what a CTA runs once or a few times costs as much as its instructions take to be loaded.)
    template <int N, typename F>
    __device__ __forceinline__ void turns(const Stage& stage, const Fetched& fetched, int32_t r0, int32_t end, int32_t c0, F f) const
    {
        constexpr int kCount = Turns<N>::kCount;
        const Turns<N> turn;
        const int32_t c = c0 + turn.col, left = n - c;
        Cols<N> b = {};
        if (bias) b = get<N>(bias + c, left);
#pragma unroll(N == 4 ? 2 : 4)
        for (int i = 0; i < kCount; ++i) {
            const int32_t r = r0 + turn.row_of(i);
            const Cols<N> z = turn.read(stage, i) + b;
            if (pre && r < end) put(pre + r * pre_stride + c, z, left);
            const Cols<N> v = f(z);
            if (residual) turn.write(stage, i, v);
            else if (r < end) put(y + r * y_stride + c, v, left);
        }
        if (!residual) return;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int32_t r = r0 + turn.row_of(i);
            const Cols<N> v = turn.read(stage, i) + fetched.use<T, N>(i);
            if (r < end) put(y + r * y_stride + c, v, left);
        }
    }

    template <int kKind, int N> static __device__ __forceinline__ Cols<N> each(Cols<N> c)
    {
        activate_all<T, kKind>(c.v);
        return c;
    }

    template <typename G> __device__ __forceinline__ void with_act(G g) const
    {
        switch (act) {
        case ADACOMP_ACT_RELU: g([](auto v) { return each<ADACOMP_ACT_RELU>(v); }); break;
        case ADACOMP_ACT_GELU: g([](auto v) { return each<ADACOMP_ACT_GELU>(v); }); break;
        case ADACOMP_ACT_GELU_TANH: g([](auto v) { return each<ADACOMP_ACT_GELU_TANH>(v); }); break;
        case ADACOMP_ACT_SILU: g([](auto v) { return each<ADACOMP_ACT_SILU>(v); }); break;
        default: g([](auto v) { return v; });
        }
    }

    __device__ __forceinline__ void chunk(const Stage& stage, const State&, const Fetched& fetched, int32_t r0, int32_t end, int32_t c) const
    {
        if (whole) with_act([&](auto f) { turns<4>(stage, fetched, r0, end, c, f); });
        else with_act([&](auto f) { turns<1>(stage, fetched, r0, end, c, f); });
    }

    // columns, by a thread on its own
    template <int N> __device__ __forceinline__ void piece(int32_t r, int32_t c, Cols<N> v) const
    {
        const int32_t left = n - c;
        if (bias) v = v + get<N>(bias + c, left);
        if (pre) put(pre + r * pre_stride + c, v, left);
        with_act([&](auto f) { v = f(v); });
        if (residual) v = v + get<N>(residual + r * residual_stride + c, left);
        put(y + r * y_stride + c, v, left);
    }
};

// The sums themselves, in rows that `map` may move; with acc, added up over several products in fp32 (first:
// nothing to add to yet) and rounded by the last one only. Of a product whose terms are split, the parts' sums
// go to acc, split_stride apart (and neither first nor last is asked).
template <typename T> struct EpiStore {
    static constexpr int kUnroll = sizeof(T) == 4 ? 1 : 4;
    static constexpr bool kExact = sizeof(T) == 4, kChunks = true, kPieces = true, kFetches = true, kPatches = false, kParts = true;
    T* out;
    float* acc;
    const int32_t* map;
    int64_t stride, acc_stride, split_stride;
    int32_t n;
    bool first, last, whole;
    struct State {
        int32_t to;
    };
    __device__ __forceinline__ bool fetches() const { return !first; }
    __device__ __forceinline__ State begin(int32_t r, int32_t c) const
    {
        if (!first) prefetch_row(acc + r * acc_stride + c, n - c);
        return {map ? map[r] : r};
    }
    __device__ __forceinline__ void rows(const Stage&, const State&, int32_t, int32_t, int32_t, int32_t, bool, float (&)[kStrip]) const {}

    __device__ __forceinline__ void fetch(Fetched& f, int32_t r0, int32_t end, int32_t c0) const
    {
        f.load_all<float, 4>(acc, acc_stride, n, r0, end, c0);
    }

    template <int N, typename O>
    __device__ __forceinline__ void turns(const Stage& stage, int32_t to, O* p, int64_t pitch, int32_t r0, int32_t end, int32_t c0) const
    {
        const Turns<N> turn;
        const int32_t c = c0 + turn.col, left = n - c;
#pragma unroll
        for (int i = 0; i < Turns<N>::kCount; ++i) {
            const int32_t r = __shfl_sync(0xffffffffu, to, turn.row_of(i));
            if (r0 + turn.row_of(i) < end) put(p + r * pitch + c, turn.read(stage, i), left);
        }
    }

    __device__ __forceinline__ void part(const Stage& stage, int split, int32_t r0, int32_t end, int32_t c0) const
    {
        turns<4>(stage, r0 + (int32_t)(threadIdx.x & 31), acc + split * split_stride, acc_stride, r0, end, c0);
    }

    __device__ __forceinline__ void chunk(const Stage& stage, const State& s, const Fetched& fetched, int32_t r0, int32_t end, int32_t c0) const
    {
        if (!first) {
            const Turns<4> turn;
#pragma unroll
            for (int i = 0; i < 8; ++i) turn.write(stage, i, turn.read(stage, i) + fetched.use<float, 4>(i));
            __syncwarp();
        }
        if (!last) turns<4>(stage, r0 + (int32_t)(threadIdx.x & 31), acc, acc_stride, r0, end, c0);
        else if (whole) turns<4>(stage, s.to, out, stride, r0, end, c0);
        else turns<1>(stage, s.to, out, stride, r0, end, c0);
    }

    template <int N> __device__ __forceinline__ void piece(int32_t r, int32_t c, Cols<N> v) const
    {
        const int32_t left = n - c;
        if (!first) v = v + get<N>(acc + r * acc_stride + c, left);
        if (last) put(out + (map ? map[r] : r) * stride + c, v, left);
        else put(acc + r * acc_stride + c, v, left);
    }
};

// exp of differences from a row's maximum or logarithm: the quick form's error (2 + 1.2 |x| units
// of 2^-24) is far below what bf16 inputs are rounded to; fp32 inputs take expf (2 units).
template <typename T> __device__ __forceinline__ float exp_of(float x)
{
    if constexpr (sizeof(T) == 4) return expf(x);
    else return __expf(x);
}

// What each row is compared with: k tokens in ascending order (those past the list's end are
// INT32_MAX), with their weights, of the rows in their own order; map: the rows that have a loss.
struct Lists {
    const int32_t* index;
    const float* q;
    const int32_t* map;
    int32_t k;
};

// Where a row's list begins, its first place that is not before column c, and the token there.
struct Place {
    int64_t list = 0;
    int32_t at = 0, token = INT32_MAX;
};

__device__ __forceinline__ Place place_of(const Lists& l, int64_t row, int32_t c)
{
    Place p;
    p.list = row * l.k;
    const int32_t* index = l.index + p.list;
    for (int hi = l.k; p.at < hi;) {
        const int mid = (p.at + hi) / 2;
        if (index[mid] < c) p.at = mid + 1;
        else hi = mid;
    }
    if (p.at < l.k) p.token = index[p.at];
    return p;
}

__device__ __forceinline__ int32_t next_token(const Lists& l, const Place& p, int32_t at)
{
    return at < l.k ? l.index[p.list + at] : INT32_MAX;
}

// Of each strip of up to 128 logits of a row: their maximum and the sum of exp(z - maximum); and the logits
// of the listed tokens.
template <typename T> struct EpiSoftmax {
    static constexpr bool kExact = true, kChunks = false, kPieces = false, kFetches = false, kPatches = false, kParts = false;
    float2* part;  // [strips][row_stride]
    float* picked;
    Lists lists;
    int64_t row_stride;
    float scale;  // of the logits: 1 / temperature
    using State = Place;
    __device__ __forceinline__ State begin(int32_t r, int32_t c) const { return place_of(lists, lists.map[r], c); }
    __device__ __forceinline__ void rows(const Stage& stage, const State& s, int32_t r, int32_t c, int32_t last, int32_t strip, bool live,
                                         float (&v)[kStrip]) const
    {
        const int32_t end = !live ? c : last - c < kStrip ? last : c + kStrip;
#pragma unroll
        for (int i = 0; i < kStrip; ++i) v[i] *= scale;
        if (__any_sync(0xffffffffu, live && s.token < end)) {  // by shared memory, where a column can be an index
            int32_t at = s.at, token = live ? s.token : INT32_MAX;
#pragma unroll 1
            for (int q = 0; q < kStrip; q += 32) {
                put_chunk_of(stage, v, q / 32);
                for (; token < end && token < c + q + 32; token = next_token(lists, s, ++at)) picked[s.list + at] = row_value(stage, token - c - q);
            }
        }
        if (!live) return;
        if (end < c + kStrip) {
#pragma unroll
            for (int i = 0; i < kStrip; ++i) v[i] = i < end - c ? v[i] : -INFINITY;
        }
        float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int i = 4; i < kStrip; ++i) top[i & 3] = fmaxf(top[i & 3], v[i]);
        top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const float less = top[0] == -INFINITY ? 0.0f : top[0];  // nothing but -inf: all terms are 0
        float sum[4] = {};
#pragma unroll
        for (int i = 0; i < kStrip; ++i) sum[i & 3] += exp_of<T>(v[i] - less);
        part[strip * row_stride + r] = make_float2(top[0], (sum[0] + sum[1]) + (sum[2] + sum[3]));
    }
    __device__ __forceinline__ void chunk(const Stage&, const State&, const Fetched&, int32_t, int32_t, int32_t) const {}
};

// The logits' gradient (p - q) * dloss * temperature of columns first .. first + n - 1: rounded to
// bf16, or in parts. Rows past the last one, up to a tile's end, are zeros: they are terms of a product.
template <typename T> struct EpiGradient {
    static constexpr int kUnroll = sizeof(T) == 4 ? 1 : 4;
    static constexpr bool kExact = sizeof(T) == 4, kChunks = true, kPieces = false, kFetches = false, kPatches = true, kParts = false;
    bf16* dz;  // [planes][room][stride]
    Lists lists;
    const float *lse, *dloss, *given;
    int64_t stride, plane, dloss_stride;
    int32_t room, n, first;
    float scale, temperature;
    bool two;  // parts of bf16 results
    struct State {
        Place place;
        float lse, factor;
    };
    __device__ __forceinline__ State begin(int32_t r, int32_t c) const
    {
        const int64_t row = lists.map[r];
        State s = {place_of(lists, row, first + c), lse[row], dloss[row * dloss_stride] * temperature};
        if (given[row] != given[row]) s.factor = given[row];  // a row that has no value
        return s;
    }
    __device__ __forceinline__ void rows(const Stage&, const State& s, int32_t, int32_t, int32_t, int32_t, bool live, float (&v)[kStrip]) const
    {
        if (live) {
#pragma unroll
            for (int i = 0; i < kStrip; ++i) v[i] = exp_of<T>(fmaf(v[i], scale, -s.lse)) * s.factor;
        } else {
#pragma unroll
            for (int i = 0; i < kStrip; ++i) v[i] = 0.0f;
        }
    }
    // The listed tokens among the 32 columns from c on, which lie in shared memory, a thread its row's.
    __device__ __forceinline__ void patch(const Stage& stage, State& s, int32_t c) const
    {
        while (s.place.token < first + c + 32) {
            float& v = row_value(stage, s.place.token - first - c);
            v = fmaf(-lists.q[s.place.list + s.place.at], s.factor, v);
            s.place.token = next_token(lists, s.place, ++s.place.at);
        }
    }
    __device__ __forceinline__ void chunk(const Stage& stage, const State&, const Fetched&, int32_t r0, int32_t, int32_t c0) const
    {
        const Turns<4> turn;
        const int32_t c = c0 + turn.col, left = n - c;
#pragma unroll(sizeof(T) == 2 ? 8 : 1)
        for (int i = 0; i < 8; ++i) {
            const int32_t r = r0 + turn.row_of(i);
            if (r >= room) continue;
            const Cols<4> v = turn.read(stage, i);
            bf16* to = dz + r * stride + c;
            if constexpr (sizeof(T) == 2) {
                if (!two) {
                    put(to, v, left);
                    continue;
                }
                Cols<4> part;
#pragma unroll
                for (int j = 0; j < 4; ++j) part.v[j] = first_of(v.v[j]);
                put(to, part, left);
#pragma unroll
                for (int j = 0; j < 4; ++j) part.v[j] = rest_of(v.v[j]);
                put(to + plane, part, left);
            } else {
                uint32_t part[kPlanes][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t each[kPlanes];
                    cut_parts(v.v[j], each);
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p) part[p][j] = each[p];
                }
#pragma unroll
                for (int p = 0; p < kPlanes; ++p) {
                    uint16_t* at = reinterpret_cast<uint16_t*>(to + p * plane);
                    if (left >= 4) {
                        *reinterpret_cast<uint2*>(at) = make_uint2(__byte_perm(part[p][0], part[p][1], 0x7632), __byte_perm(part[p][2], part[p][3], 0x7632));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < left) at[j] = (uint16_t)(part[p][j] >> 16);
                    }
                }
            }
        }
    }
};

}  // namespace
}  // namespace adacomp
