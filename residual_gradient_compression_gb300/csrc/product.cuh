// Shared by the linear layers and the losses over a vocabulary: what is done with a product's
// sums (the epilogues), a product for operands of any layout, and rows that are copied together.
//
// A product is C(m, n) = sum over k of A(m, k) B(n, k). Whichever kernel forms it hands an epilogue
// the sums of one row, 32 columns at a time and in ascending order within a strip, in one thread's
// registers: begin(row), chunk(columns) for the strip's columns, end(strip). kZeros: rows past the last one, up to
// a tile's end, are set to zeros.
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

constexpr int kCols = 32;    // columns of a chunk
constexpr int kStrip = 128;  // of a strip: what a softmax's partial sums are kept for
constexpr int kRows = 128;   // rows of a tile

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// ---------------------------------------------------------------- rows of 32 columns
template <typename T> __device__ __forceinline__ void put_chunk(T* p, const float (&v)[kCols], int64_t left, bool whole)
{
    if (whole && left >= kCols) {
        uint4* q = reinterpret_cast<uint4*>(p);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kCols; i += 4)
                q[i / 4] = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                                      __float_as_uint(v[i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < kCols; i += 8) {
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
    for (int i = 0; i < kCols; ++i)
        if (i < left) p[i] = from_f32<T>(v[i]);
}

template <typename T> __device__ __forceinline__ void get_chunk(const T* p, float (&v)[kCols], int64_t left, bool whole)
{
    if (whole && left >= kCols) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
        for (int i = 0; i < kCols * (int)sizeof(T) / 16; ++i) {
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
    for (int i = 0; i < kCols; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
}

inline bool whole_rows(const void* p, int64_t stride, int64_t rows, int bytes)
{
    return is_aligned(p, 16) && (rows < 2 || stride * bytes % 16 == 0);
}

// ---------------------------------------------------------------- fp32 numbers in parts
constexpr int kPlanes = 4;  // of bf16 numbers for an fp32 matrix

// x = top + mid + low exactly (but for what is below 2^-133), each a bf16 number. A value that is not finite has only a
// top; the fourth plane is the top without such values, for the products with the other operand's lower parts
// (infinity times a part that is 0 would be NaN).
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

// A row's columns as operands of another product: bf16 numbers, or, of an fp32 matrix, planes of them.
template <typename T> __device__ __forceinline__ void put_parts(bf16* p, int64_t plane, const float (&v)[kCols], int64_t left)
{
    if constexpr (sizeof(T) == 2) {
        put_chunk(p, v, left, true);
    } else {
        float part[kPlanes][kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            bf16 each[kPlanes];
            split_parts(v[i], each);
#pragma unroll
            for (int j = 0; j < kPlanes; ++j) part[j][i] = __bfloat162float(each[j]);
        }
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) put_chunk(p + j * plane, part[j], left, true);
    }
}

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float activate(float z, int kind)
{
    switch (kind) {
    case ADACOMP_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case ADACOMP_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    case ADACOMP_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
    case ADACOMP_ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
    }
}

__device__ __forceinline__ float slope(float z, int kind)
{
    switch (kind) {
    case ADACOMP_ACT_RELU: return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;  // NaN stays NaN
    case ADACOMP_ACT_GELU:
        return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * expf(-0.5f * z * z) * 0.39894228f;
    case ADACOMP_ACT_GELU_TANH: {
        const float t = tanhf(0.79788456f * (z + 0.044715f * z * z * z));
        return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * 0.79788456f * (1.0f + 0.134145f * z * z);
    }
    case ADACOMP_ACT_SILU: {
        const float g = 1.0f / (1.0f + expf(-z));
        return g * (1.0f + z * (1.0f - g));
    }
    default: return 1.0f;
    }
}

// ---------------------------------------------------------------- epilogues
// y = act(sum + bias) + residual, and the value before the activation.
template <typename T> struct EpiLinear {
    T *y, *pre;
    const T *bias, *residual;
    int64_t y_stride, pre_stride, residual_stride, n;
    int32_t act;
    bool y_whole, pre_whole, bias_whole, residual_whole;
    static constexpr bool kZeros = false;
    struct State {};
    __device__ __forceinline__ void begin(State&, int64_t, int64_t, int) const {}
    __device__ __forceinline__ void chunk(State&, int64_t r, int64_t c, float (&v)[kCols]) const
    {
        if (c >= n) return;
        const int64_t left = n - c;
        if (bias) {
            float b[kCols];
            get_chunk(bias + c, b, left, bias_whole);
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] += b[i];
        }
        if (pre) put_chunk(pre + r * pre_stride + c, v, left, pre_whole);
        if (act != ADACOMP_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = activate(v[i], act);
        }
        if (residual) {
            float b[kCols];
            get_chunk(residual + r * residual_stride + c, b, left, residual_whole);
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] += b[i];
        }
        put_chunk(y + r * y_stride + c, v, left, y_whole);
    }
    __device__ __forceinline__ void end(State&, int64_t, int64_t) const {}
    __device__ __forceinline__ void zeros(int64_t, int64_t) const {}
};

// The sums themselves, in rows that `map` may move; with acc, added up over several products in
// fp32 (first: nothing to add to yet) and rounded by the last one only.
template <typename T> struct EpiStore {
    T* out;
    float* acc;
    const int32_t* map;
    int64_t stride, acc_stride, n, split_stride;  // split_stride: between the parts of a product whose terms are split
    bool first, last, whole;
    static constexpr bool kZeros = false;
    struct State {
        T* to;
    };
    __device__ __forceinline__ void begin(State& s, int64_t r, int64_t, int split) const
    {
        s.to = out + split * split_stride + (map ? map[r] : r) * stride;
    }
    __device__ __forceinline__ void chunk(State& s, int64_t r, int64_t c, float (&v)[kCols]) const
    {
        if (c >= n) return;
        const int64_t left = n - c;
        if (!first) {
            float b[kCols];
            get_chunk(acc + r * acc_stride + c, b, left, true);
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] += b[i];
        }
        if (last) put_chunk(s.to + c, v, left, whole);
        else put_chunk(acc + r * acc_stride + c, v, left, true);
    }
    __device__ __forceinline__ void end(State&, int64_t, int64_t) const {}
    __device__ __forceinline__ void zeros(int64_t, int64_t) const {}
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

// A row's first place in its list that is not before column c.
__device__ __forceinline__ int first_place(const int32_t* index, int k, int64_t c)
{
    int lo = 0, hi = k;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (index[mid] < c) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Of each strip of 128 logits of a row: their maximum and the sum of exp(z - maximum), in one pass
// over the sums as they come; and the logits of the listed tokens.
template <typename T> struct EpiSoftmax {
    float2* part;  // [strips][rows]
    float* picked;
    Lists lists;
    int64_t n, rows;
    float scale;  // of the logits: 1 / temperature
    static constexpr bool kZeros = false;
    struct State {
        float top, sum;
        const int32_t* index;
        float* picked;
        int at, next;
    };
    __device__ __forceinline__ void begin(State& s, int64_t r, int64_t c, int) const
    {
        const int64_t row = lists.map[r];
        s.top = -INFINITY;
        s.sum = 0.0f;
        s.index = lists.index + row * lists.k;
        s.picked = picked + row * lists.k;
        s.at = first_place(s.index, lists.k, c);
        s.next = s.at < lists.k ? s.index[s.at] : INT32_MAX;
    }
    __device__ __forceinline__ void chunk(State& s, int64_t, int64_t c, float (&v)[kCols]) const
    {
        if (c >= n) return;
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] *= scale;
        while (s.next < c + kCols && s.next < n) {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < kCols; ++i) z = s.next == c + i ? v[i] : z;
            s.picked[s.at] = z;
            s.next = ++s.at < lists.k ? s.index[s.at] : INT32_MAX;
        }
        if (n - c < kCols) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = i < n - c ? v[i] : -INFINITY;
        }
        float top = s.top;
#pragma unroll
        for (int i = 0; i < kCols; ++i) top = fmaxf(top, v[i]);
        const float from = top == -INFINITY ? 0.0f : top;  // nothing but -inf so far: all terms are 0
        float sum[4] = {s.sum * exp_of<T>(s.top - from), 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i & 3] += exp_of<T>(v[i] - from);
        s.sum = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        s.top = top;
    }
    __device__ __forceinline__ void end(State& s, int64_t r, int64_t strip) const
    {
        part[strip * rows + r] = make_float2(s.top, s.sum);
    }
    __device__ __forceinline__ void zeros(int64_t, int64_t) const {}
};

// The logits' gradient (p - q) * dloss * temperature of columns first .. first + n - 1: rounded to
// bf16, or, of fp32 operands, in parts.
template <typename T> struct EpiGradient {
    bf16* dz;  // [planes][rows][stride]
    Lists lists;
    const float *lse, *dloss, *given;
    int64_t stride, plane, rows, n, first, dloss_stride;  // rows: that there is room for
    float scale, temperature;
    static constexpr bool kZeros = true;
    struct State {
        float lse, factor;
        const int32_t* index;
        const float* q;
        int at;
        int64_t next;
    };
    __device__ __forceinline__ void begin(State& s, int64_t r, int64_t c, int) const
    {
        const int64_t row = lists.map[r];
        s.lse = lse[row];
        s.factor = dloss[row * dloss_stride] * temperature;
        if (given[row] != given[row]) s.factor = given[row];  // a row that has no value
        s.index = lists.index + row * lists.k;
        s.q = lists.q + row * lists.k;
        s.at = first_place(s.index, lists.k, first + c);
        s.next = s.at < lists.k ? s.index[s.at] - first : INT64_MAX;
    }
    __device__ __forceinline__ void chunk(State& s, int64_t r, int64_t c, float (&v)[kCols]) const
    {
        if (c >= n) return;
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] = exp_of<T>(fmaf(v[i], scale, -s.lse));
        while (s.next < c + kCols) {
            const float q = s.q[s.at];
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] -= s.next == c + i ? q : 0.0f;
            s.next = ++s.at < lists.k ? s.index[s.at] - first : INT64_MAX;
        }
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] *= s.factor;
        put_parts<T>(dz + r * stride + c, plane, v, n - c);
    }
    __device__ __forceinline__ void end(State&, int64_t, int64_t) const {}
    __device__ __forceinline__ void zeros(int64_t r, int64_t c) const
    {
        if (r >= rows || c >= n) return;
        float v[kCols] = {};
        put_parts<T>(dz + r * stride + c, plane, v, n - c);
    }
};

// ---------------------------------------------------------------- operands of any layout
struct Operand {
    const void* p;
    int64_t outer, inner;  // strides between rows, and along a row
};

struct SimpleArgs {
    Operand a, b;
    int64_t m, n, k;
    const int32_t *m_count, *k_count;  // how many of the rows m, or terms k, there are; NULL: all
    int64_t strip;                     // columns of a CTA's tile: a multiple of kCols
};

template <typename T, bool kInner>
__device__ __forceinline__ void simple_load(float* to, int row_pitch, const Operand& o, int rows, int64_t r0, int64_t r_end,
                                            int64_t k0, int64_t k_end)
{
    constexpr int kDepth = 16;
    const T* p = static_cast<const T*>(o.p);
    for (int i = threadIdx.x; i < rows * kDepth; i += kRows) {
        const int k = kInner ? i % kDepth : i / rows, r = kInner ? i / kDepth : i % rows;
        const bool there = r0 + r < r_end && k0 + k < k_end;
        to[k * row_pitch + r] = there ? to_f32(p[(r0 + r) * o.outer + (k0 + k) * o.inner]) : 0.0f;
    }
}

// A thread has a row and 32 columns; 16 terms at a time in shared memory, summed in fp32 one after the
// other.
template <typename T, typename Epi>
__global__ void __launch_bounds__(kRows) product_simple_kernel(const SimpleArgs g, const Epi epi)
{
    constexpr int kDepth = 16;
    __shared__ __align__(16) float sa[kDepth][kRows + 1], sb[kDepth][kCols + 4];
    ptx::griddep_wait();
    const int64_t m = g.m_count ? *g.m_count : g.m, terms = g.k_count ? *g.k_count : g.k;
    const int64_t strips = (g.n + g.strip - 1) / g.strip, tiles = (m + kRows - 1) / kRows * strips;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t strip = tile % strips, r0 = tile / strips * kRows, r = r0 + threadIdx.x, c0 = strip * g.strip;
        typename Epi::State state;
        if (r < m) epi.begin(state, r, c0, 0);
        for (int64_t c = c0; c < c0 + g.strip && c < g.n; c += kCols) {
            float v[kCols] = {};
            for (int64_t k = 0; k < terms; k += kDepth) {
                if (g.a.inner == 1) simple_load<T, true>(&sa[0][0], kRows + 1, g.a, kRows, r0, m, k, terms);
                else simple_load<T, false>(&sa[0][0], kRows + 1, g.a, kRows, r0, m, k, terms);
                if (g.b.inner == 1) simple_load<T, true>(&sb[0][0], kCols + 4, g.b, kCols, c, g.n, k, terms);
                else simple_load<T, false>(&sb[0][0], kCols + 4, g.b, kCols, c, g.n, k, terms);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kDepth; ++i) {
                    const float x = sa[i][threadIdx.x];
#pragma unroll
                    for (int j = 0; j < kCols; j += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(&sb[i][j]);
                        v[j] = fmaf(x, w.x, v[j]);
                        v[j + 1] = fmaf(x, w.y, v[j + 1]);
                        v[j + 2] = fmaf(x, w.z, v[j + 2]);
                        v[j + 3] = fmaf(x, w.w, v[j + 3]);
                    }
                }
                __syncthreads();
            }
            if (r < m) epi.chunk(state, r, c, v);
        }
        if (r < m) epi.end(state, r, strip);
    }
}

template <typename T, typename Epi> cudaError_t product_simple(const SimpleArgs& g, const Epi& epi, cudaStream_t stream)
{
    if (g.m <= 0 || g.n <= 0) return cudaSuccess;
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (g.m + kRows - 1) / kRows * ((g.n + g.strip - 1) / g.strip), most = (int64_t)sms * 8;
    return launch_after(product_simple_kernel<T, Epi>, dim3((unsigned)(tiles < most ? tiles : most)), dim3(kRows), 0, stream, g, epi);
}

}  // namespace
}  // namespace adacomp
