// Layer norm, forward and backward with the gradients of the weight and the bias:
// kernels and C entry points (adacomp.h).
#include <initializer_list>
#include <new>

#include "train_common.cuh"

struct adacomp_layer_norm {
    int64_t dim = 0;
    int32_t x_dtype = ADACOMP_F32, w_dtype = ADACOMP_F32;
    float eps = 0.0f;
};

namespace adacomp {
namespace {

constexpr int kLnThreads = 256;   // rows that are too wide for the registers of a CTA's turn
constexpr int kLnBack = 512;      // the others
constexpr int kLnParts = 304;     // CTAs of a backward pass at most, each with partial sums of dw and db
constexpr int kLnCols = 16;       // columns of a thread there, at most
constexpr int64_t kLnDim = (int64_t)kLnBack * kLnCols;
constexpr int kLnWideSlices = 128;

struct LnArgs {
    const void *x, *dy, *w, *b;
    void *y, *dx, *dw, *db;
    float *mean, *rstd;          // outputs of the forward pass
    const float *mean_in, *rstd_in;
    float* part;                 // [slices][2][dim] partial sums of dw and db
    int64_t rows, dim, x_stride, y_stride, dy_stride, dx_stride;
    int32_t slices;
    int32_t group;               // threads of a row
    float eps;
};

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

// The sum over the lanes of a group of up to 32 (a power of two).
__device__ __forceinline__ float group_sum(float v, int group)
{
    for (int o = group >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void group_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// How many rows of x and dy a thread of the backward pass has on their way, and the shared memory
// for them.
template <typename X, int N> struct LnRing {
    // pieces of two bytes cannot be copied so: half the columns, and one row ahead in registers
    static constexpr bool kRing = Piece<X, N>::kBytes >= 4;
    static constexpr int kCols = kRing ? kLnCols : kLnCols / 2;
    static constexpr int kRow = (kCols / N) * 2 * kLnBack * Piece<X, N>::kBytes;
    static constexpr int kStages = sizeof(X) == 2 ? 6 : 3;
    static constexpr int kBytes = kRing ? kStages * kRow : 0;
};

template <int kBytes> __device__ __forceinline__ void copy_piece(void* to, const void* from)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(from) : "memory");
}

// ---------------------------------------------------------------- forward
// Bound by memory: x is read once and y written. A row is held in registers as it lies in
// memory, kCols elements per thread, by a group of a.group lanes (kWarps 0), by a warp or by a
// CTA of kWarps warps; the mean and the sum of the squared deviations from it are two sums over
// the row's threads. The weights come from L1 for every row, so a thread's pieces are no longer
// than four 32-bit weights, which keeps its 16-byte loads of them side by side (pieces of eight
// bf16 elements: 33 us instead of 28 at 16384 rows of 2048, bound by L1). Nothing is loaded
// ahead: the other rows on the SM hide a row's loads (a persistent CTA with its weights in
// registers and the rows to come in shared memory took 33 us there, and 79 us instead of 50 at
// 8192 rows of 8192 bf16, with two barriers for each row in turn).
//
// With 32-bit weights, all in us: 16384 x 2048 bf16 25 (5.3 TB/s; 65536 rows 84, 6.4 TB/s), fp32
// 41 (6.5 TB/s); 8192 x 8192 bf16 50, fp32 79 (6.8 TB/s); 32768 x 1001 fp32 46 (5.7 TB/s).
// Odd rows of bf16 are bound by their two-byte loads and stores: 32768 x 1001 47 (2.8 TB/s).
template <int kWarps> constexpr int kLnRowThreads = kWarps > 1 ? 32 * kWarps : 128;  // a CTA's

template <typename X, typename W, int N, int kCols, int kWarps>
__global__ void __launch_bounds__(kLnRowThreads<kWarps>,
                                  (kCols == 64 ? 768 : kCols == 32 ? 1024 : 1536) / kLnRowThreads<kWarps>)
    ln_forward_row_kernel(const LnArgs a)
{
    constexpr int kPieces = kCols / N, kThreads = kLnRowThreads<kWarps>;
    __shared__ float sums[2][kThreads / 32];
    ptx::griddep_wait();
    if (kWarps < 2) ptx::griddep_launch();  // the next kernel's launch is under way while the last rows are
    const int group = kWarps == 0 ? a.group : 32 * kWarps, place = threadIdx.x & (group - 1);
    const int64_t row = (int64_t)blockIdx.x * (kThreads / group) + threadIdx.x / group;
    if (kWarps && row >= a.rows) return;
    const float n = (float)a.dim;
    const int dim = row < a.rows ? (int)a.dim : 0;  // lanes without a row take part in the sums
    const auto sum = [&](float v, int turn) {
        if (kWarps == 0) return group_sum(v, group);
        v = warp_sum(v);
        if (kWarps == 1) return v;
        if ((threadIdx.x & 31) == 0) sums[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) v += sums[turn][i];
        return v;
    };
    const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
    Piece<X, N> r[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int c = (k * group + place) * N;
        r[k].zero();
        if (c < dim) r[k].load(x + c);
    }
    Pair s[2] = {pair(0.0f), pair(0.0f)};
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) s[i & 1] = s[i & 1] + pair_of(r, i);
    const float mean = sum(both(s[0] + s[1]), 0) / n;
    const Pair minus = pair(-mean);
    s[0] = s[1] = pair(0.0f);
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
        if ((k * group + place) * N < dim) {
            if constexpr (N > 1) {
#pragma unroll
                for (int i = k * N / 2; i < (k + 1) * N / 2; ++i) {
                    const Pair d = pair_of(r, i) + minus;
                    s[i & 1] = fma2(d, d, s[i & 1]);
                }
            } else {
                const Pair d = pair(r[k].get(0) - mean, 0.0f);
                s[k & 1] = fma2(d, d, s[k & 1]);
            }
        }
    const float rstd = 1.0f / sqrtf(sum(both(s[0] + s[1]), 1) / n + a.eps);
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    X* y = static_cast<X*>(a.y) + row * a.y_stride;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int c = (k * group + place) * N;
        if (c < dim) {
            float wv[N], bv[N] = {}, v[N];
            weights<N>(w + c, wv);
            if (b) weights<N>(b + c, bv);
            if constexpr (N > 1) {
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    const Pair d = (pair_of(r, (k * N + j) / 2) + minus) * pair(rstd);
                    split(fma2(d, pair(wv[j], wv[j + 1]), pair(bv[j], bv[j + 1])), v[j], v[j + 1]);
                }
            } else {
                v[0] = fmaf((r[k].get(0) - mean) * rstd, wv[0], bv[0]);
            }
            put_piece<N>(y + c, v);
        }
    }
    if (place == 0 && (kWarps || row < a.rows)) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// Rows too wide for registers: a CTA per row, three passes over it (the second and third
// from L2).
template <typename X, typename W> __global__ void __launch_bounds__(kLnThreads) ln_forward_long_kernel(const LnArgs a)
{
    __shared__ float shared[2][kLnThreads / 32];
    ptx::griddep_wait();
    const int64_t row = blockIdx.x;
    const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
    X* y = static_cast<X*>(a.y) + row * a.y_stride;
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    const auto sum = [&](float v, int turn) {
        v = warp_sum(v);
        if ((threadIdx.x & 31) == 0) shared[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
        for (int i = 0; i < kLnThreads / 32; ++i) v += shared[turn][i];
        return v;
    };
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.dim; i += kLnThreads) s += to_f32(x[i]);
    const float mean = sum(s, 0) / (float)a.dim;
    s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.dim; i += kLnThreads) {
        const float d = to_f32(x[i]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(sum(s, 1) / (float)a.dim + a.eps);
    for (int64_t i = threadIdx.x; i < a.dim; i += kLnThreads)
        y[i] = from_f32<X>(fmaf((to_f32(x[i]) - mean) * rstd, to_f32(w[i]), b ? to_f32(b[i]) : 0.0f));
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// ---------------------------------------------------------------- backward
// Bound by memory: dy and x are read once and dx written. A group of threads (1 to 512, a
// power of two) has a row, 16 columns per thread at most, and goes from row to row, so that
// the weights, and the sums for dw and db over its rows, stay in its registers. The rows to
// come are copied to shared memory four ahead (every thread its own pieces: no barrier);
// pieces of single elements are loaded one row ahead. The two sums of a row need one
// barrier of the group where it is more than a warp. At the end the CTA's groups add their
// column sums in order, and a second kernel adds the CTAs'.
template <typename X, typename W, int N>
__global__ void __launch_bounds__(kLnBack, 1) ln_backward_kernel(const LnArgs a)
{
    using Ring = LnRing<X, N>;
    constexpr int kCols = Ring::kCols, kPieces = kCols / N, kPairs = kCols / 2;
    constexpr int kBytes = Piece<X, N>::kBytes, kStages = Ring::kStages;
    constexpr bool kRing = Ring::kRing;
    using Raw = typename Piece<X, N>::Raw;
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    __shared__ float2 sums[2][kLnBack / 32];
    ptx::griddep_wait();
    const int group = a.group, place = threadIdx.x & (group - 1), dim = (int)a.dim;
    const int groups = kLnBack / group, which = threadIdx.x / group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_n = 1.0f / (float)dim;
    const X* x = static_cast<const X*>(a.x);
    const X* dy = static_cast<const X*>(a.dy);
    X* dx = static_cast<X*>(a.dx);
    Pair w[kPairs], dw[kPairs], db[kPairs];
    {
        float v[kCols] = {};
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int c = (k * group + place) * N;
            if (c < dim) weights<N>(static_cast<const W*>(a.w) + c, *reinterpret_cast<float(*)[N]>(v + k * N));
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            w[i] = pair(v[2 * i], v[2 * i + 1]);
            dw[i] = db[i] = pair(0.0f);
        }
    }
    // the ring: [stage][piece][x, dy][thread]
    const auto slot = [&](int stage, int k, int tensor) {
        return reinterpret_cast<Raw*>(shared_bytes) + ((stage * kPieces + k) * 2 + tensor) * kLnBack + threadIdx.x;
    };
    const int64_t stride = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + which;
    const auto stage_row = [&](int64_t r, int stage) {
        if constexpr (kRing) {
            if (r < a.rows) {
#pragma unroll
                for (int k = 0; k < kPieces; ++k) {
                    const int c = (k * group + place) * N;
                    if (c < dim) {
                        copy_piece<kBytes>(slot(stage, k, 0), x + r * a.x_stride + c);
                        copy_piece<kBytes>(slot(stage, k, 1), dy + r * a.dy_stride + c);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    Piece<X, N> px[kPieces], pd[kPieces], next_x[kPieces], next_d[kPieces];
    const auto load_next = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int c = (k * group + place) * N;
            next_x[k].zero();
            next_d[k].zero();
            if (r < a.rows && c < dim) {
                next_x[k].load(x + r * a.x_stride + c);
                next_d[k].load(dy + r * a.dy_stride + c);
            }
        }
    };
    float mean = 0.0f, rstd = 0.0f;
    if (row < a.rows) mean = a.mean_in[row], rstd = a.rstd_in[row];
    if (kRing) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) stage_row(row + i * stride, i);
    } else {
        load_next(row);
    }
    // every lane of a warp takes part as long as the warp's first group has a row
    const int64_t lead = (int64_t)blockIdx.x * groups + (group < 32 ? warp * (32 / group) : which);
    int stage = 0, turn = 0;
    for (int64_t at = lead; at < a.rows; at += stride, row += stride) {
        const bool on = row < a.rows;
        float mean_next = 0.0f, rstd_next = 0.0f;
        if (row + stride < a.rows) mean_next = a.mean_in[row + stride], rstd_next = a.rstd_in[row + stride];
        if (kRing) asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            if (kRing) {
                px[k].zero();
                pd[k].zero();
                if (on && (k * group + place) * N < dim) {
                    px[k].q = *slot(stage, k, 0);
                    pd[k].q = *slot(stage, k, 1);
                }
            } else {
                px[k] = next_x[k];
                pd[k] = next_d[k];
            }
        }
        if (kRing) {
            stage_row(row + kStages * stride, stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
        } else {
            load_next(row + stride);
        }
        // with d = x - mean: xh = rstd * d, and the sum of g * xh is rstd times that of g * d
        Pair d[kPairs], g[kPairs], t0 = pair(0.0f), t1 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const Pair v = pair_of(pd, i);
            d[i] = pair_of(px, i) + pair(-mean);
            g[i] = v * w[i];
            db[i] = db[i] + v;
            dw[i] = fma2(v * pair(rstd), d[i], dw[i]);
            t0 = t0 + g[i];
            t1 = fma2(g[i], d[i], t1);
        }
        float s0 = both(t0), s1 = both(t1) * rstd;
        const int within = group < 32 ? group : 32;
        s0 = group_sum(s0, within);
        s1 = group_sum(s1, within);
        if (group > 32) {
            if (lane == 0) sums[turn][warp] = make_float2(s0, s1);
            group_barrier(1 + which, group);
            const int first = which * (group >> 5);
            s0 = s1 = 0.0f;
            for (int i = 0; i < group >> 5; ++i) {
                s0 += sums[turn][first + i].x;
                s1 += sums[turn][first + i].y;
            }
            turn ^= 1;
        }
        if (on) {
            // dx = rstd * (g - s0 / n - xh * s1 / n)
            const Pair scale = pair(rstd), k0 = pair(-(s0 * inv_n) * rstd), k1 = pair(-(s1 * inv_n) * rstd * rstd);
            float v[kCols];
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                split(fma2(g[i], scale, fma2(d[i], k1, k0)), v[2 * i], v[2 * i + 1]);
            X* const to = dx + row * a.dx_stride;
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const int c = (k * group + place) * N;
                if (c < dim) put_piece<N>(to + c, *reinterpret_cast<const float(*)[N]>(v + k * N));
            }
        }
        mean = mean_next;
        rstd = rstd_next;
    }
    if (kRing) asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the ring is free: it takes the groups' column sums, [group or warp][2][dim]
    float* const total = reinterpret_cast<float*>(shared_bytes);
    float sw[kCols], sb[kCols];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        split(dw[i], sw[2 * i], sw[2 * i + 1]);
        split(db[i], sb[2 * i], sb[2 * i + 1]);
    }
    if (group < 32) {  // the warp's groups first
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            for (int o = group; o < 32; o <<= 1) {
                sw[i] += __shfl_xor_sync(0xffffffffu, sw[i], o);
                sb[i] += __shfl_xor_sync(0xffffffffu, sb[i], o);
            }
    }
    const int owners = group < 32 ? kLnBack / 32 : groups, mine = group < 32 ? warp : which;
    if (group >= 32 || lane < group) {
        float* const to = total + mine * 2 * dim;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int c = (k * group + place) * N;
            if (c < dim)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    to[c + j] = sw[k * N + j];
                    to[dim + c + j] = sb[k * N + j];
                }
        }
    }
    __syncthreads();
    float* const part = a.part + (int64_t)blockIdx.x * 2 * dim;
    for (int i = threadIdx.x; i < 2 * dim; i += kLnBack) {
        float v = total[i];
        for (int o = 1; o < owners; ++o) v += total[o * 2 * dim + i];
        part[i] = v;
    }
}

// Adds the partial sums: 32 columns per CTA, 32 rows of threads that each add every 32nd.
constexpr int kLnJoin = 1024;

template <typename W> __global__ void __launch_bounds__(kLnJoin) ln_join_kernel(const LnArgs a)
{
    __shared__ float shared[kLnJoin / 32][33];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, n = 2 * a.dim;
    float s = 0.0f;
    if (i < n)
#pragma unroll 5
        for (int p = row; p < a.slices; p += kLnJoin / 32) s += a.part[p * n + i];
    shared[row][lane] = s;
    __syncthreads();
    s = warp_sum(shared[lane][row]);  // column `row` of the CTA's
    const int64_t c = (int64_t)blockIdx.x * 32 + row;
    if (lane != 0 || c >= n) return;
    if (c < a.dim) static_cast<W*>(a.dw)[c] = from_f32<W>(s);
    else if (a.db) static_cast<W*>(a.db)[c - a.dim] = from_f32<W>(s);
}

// Rows too wide for the registers of a CTA: the column sums by one thread per column and
// slice of the rows (before dx is written, which may be in place of dy or x), then dx by a
// CTA per row, in two passes.
template <typename X> __global__ void __launch_bounds__(kLnThreads) ln_columns_kernel(const LnArgs a)
{
    ptx::griddep_wait();
    const int64_t c = (int64_t)blockIdx.x * kLnThreads + threadIdx.x;
    if (c >= a.dim) return;
    const X* x = static_cast<const X*>(a.x);
    const X* dy = static_cast<const X*>(a.dy);
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < a.rows; r += a.slices) {
        const float g = to_f32(dy[r * a.dy_stride + c]);
        db += g;
        dw = fmaf(g, (to_f32(x[r * a.x_stride + c]) - a.mean_in[r]) * a.rstd_in[r], dw);
    }
    float* p = a.part + (int64_t)blockIdx.y * 2 * a.dim;
    p[c] = dw;
    p[a.dim + c] = db;
}

template <typename X, typename W> __global__ void __launch_bounds__(kLnThreads) ln_backward_long_kernel(const LnArgs a)
{
    __shared__ float2 shared[kLnThreads / 32];
    ptx::griddep_wait();
    const int64_t row = blockIdx.x;
    const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
    const X* dy = static_cast<const X*>(a.dy) + row * a.dy_stride;
    X* dx = static_cast<X*>(a.dx) + row * a.dx_stride;
    const W* w = static_cast<const W*>(a.w);
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int64_t i = threadIdx.x; i < a.dim; i += kLnThreads) {
        const float g = to_f32(dy[i]) * to_f32(w[i]);
        s0 += g;
        s1 = fmaf(g, (to_f32(x[i]) - mean) * rstd, s1);
    }
    s0 = warp_sum(s0);
    s1 = warp_sum(s1);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = make_float2(s0, s1);
    __syncthreads();
    s0 = s1 = 0.0f;
    for (int i = 0; i < kLnThreads / 32; ++i) {
        s0 += shared[i].x;
        s1 += shared[i].y;
    }
    s0 /= (float)a.dim;
    s1 /= (float)a.dim;
    for (int64_t i = threadIdx.x; i < a.dim; i += kLnThreads) {
        const float h = (to_f32(x[i]) - mean) * rstd;
        dx[i] = from_f32<X>(rstd * (fmaf(to_f32(dy[i]), to_f32(w[i]), -s0) - h * s1));
    }
}

// ---------------------------------------------------------------- launches
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

// The threads of a row.
int row_group(int64_t dim, int n, int cols)
{
    const int64_t places = (dim + n - 1) / n;
    if (places <= 16) return group_of(places, 16);
    return 32 * group_of((dim + 32 * cols - 1) / (32 * cols), kLnBack / 32);
}

template <typename X, typename W, int N> cudaError_t ln_forward_n(LnArgs a, cudaStream_t stream)
{
    const dim3 one((unsigned)a.rows), threads(kLnThreads);
    if (a.dim > 64 * kLnThreads) return launch_after(ln_forward_long_kernel<X, W>, one, threads, 0, stream, a);
    // the elements of a piece: no more than four weights of 32 bits
    constexpr bool kWhole = Piece<X, N>::kBytes == 16;
    constexpr int M = kWhole && sizeof(W) == 4 ? 4 : N;
    const auto with = [&](auto kernel, int group, int threads) {
        a.group = group;
        const int each = threads / group;
        return launch_after(kernel, dim3((unsigned)((a.rows + each - 1) / each)), dim3(threads), 0, stream, a);
    };
    // Elements per thread and threads per row by measurement, us with the choice and with the
    // next best. Aligned rows want many elements for each of few threads (16384 x 2048 bf16: two
    // warps 25, one warp of 64 each 28, four of 16 each 27; 32768 x 1024 bf16: one warp 24, 64
    // each 32), fp32 rows of 2049 to 4096 less so (8192 x 4096: 41, four warps of 32 each 43).
    if (a.dim > 8192) return with(ln_forward_row_kernel<X, W, M, 64, 8>, 256, 256);
    if (a.dim > 4096) return with(ln_forward_row_kernel<X, W, M, 32, 8>, 256, 256);
    if (a.dim > 2048) {
        if constexpr (kWhole && sizeof(X) == 2) return with(ln_forward_row_kernel<X, W, M, 32, 4>, 128, 128);
        else return with(ln_forward_row_kernel<X, W, M, 16, 8>, 256, 256);
    }
    // Pieces of single elements are as many instructions, which wants more threads (32768 x 1001
    // fp32: four warps 46, one warp 63).
    if constexpr (N == 1) {
        if (a.dim > 1024) return with(ln_forward_row_kernel<X, W, 1, 16, 4>, 128, 128);
        if (a.dim > 512) return with(ln_forward_row_kernel<X, W, 1, 8, 4>, 128, 128);
    } else {
        if (a.dim > 1024) return with(ln_forward_row_kernel<X, W, M, 32, 2>, 64, 64);
        if (a.dim > 512) return with(ln_forward_row_kernel<X, W, M, 32, 1>, 32, 128);
    }
    // 65536 x 256 bf16: 16 lanes 16.5, a warp 18.5; x 254 (pieces of two): a warp 21, 16 lanes 27
    if (a.dim > (kWhole ? 256 : 128)) return with(ln_forward_row_kernel<X, W, M, 16, 1>, 32, 128);
    // 262144 x 64 bf16: 16 elements per lane 16, 8 per lane 20; x 63: 8 per lane 39, 4 per lane 47
    constexpr int kCols = M < 4 ? 8 : 16;
    return with(ln_forward_row_kernel<X, W, M, kCols, 0>, group_of((a.dim + kCols - 1) / kCols, 32), 128);
}

template <typename X, typename W> cudaError_t ln_forward(const LnArgs& a, cudaStream_t stream)
{
    const int n = piece_of(a, (int)sizeof(X), {a.x, a.y}, {a.x_stride, a.y_stride}, {a.w, a.b});
    if (n == 16 / (int)sizeof(X)) return ln_forward_n<X, W, 16 / sizeof(X)>(a, stream);
    if constexpr (sizeof(X) == 2)
        if (n == 2) return ln_forward_n<X, W, 2>(a, stream);
    return ln_forward_n<X, W, 1>(a, stream);
}

int ln_slices(int64_t rows, int64_t dim)
{
    // either way of the backward pass, as the call's alignment decides, within these
    const int64_t most = dim > kLnDim ? kLnWideSlices : kLnParts;
    return (int)(rows < 1 ? 1 : rows < most ? rows : most);
}

template <typename X, typename W, int N> cudaError_t ln_backward_n(LnArgs a, cudaStream_t stream)
{
    static bool set[64] = {};
    constexpr int sums = 2 * (int)kLnDim * 4, ring = LnRing<X, N>::kBytes, shared = ring > sums ? ring : sums;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e == cudaSuccess && !set[dev]) {
        e = cudaFuncSetAttribute(ln_backward_kernel<X, W, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
        set[dev] = e == cudaSuccess;
    }
    if (e != cudaSuccess) return e;
    a.group = row_group(a.dim, N, LnRing<X, N>::kCols);
    const int64_t per = kLnBack / a.group, need = (a.rows + per - 1) / per;
    const int64_t most = sms < kLnParts ? sms : kLnParts;
    a.slices = (int)(need < most ? need : most);
    e = launch_after(ln_backward_kernel<X, W, N>, dim3((unsigned)a.slices), dim3(kLnBack), shared, stream, a);
    if (e != cudaSuccess) return e;
    return launch_after(ln_join_kernel<W>, dim3((unsigned)((2 * a.dim + 31) / 32)), dim3(kLnJoin), 0, stream, a);
}

template <typename X, typename W> cudaError_t ln_backward(LnArgs a, cudaStream_t stream)
{
    if (a.rows == 0) {
        a.slices = 0;
        return launch_after(ln_join_kernel<W>, dim3((unsigned)((2 * a.dim + 31) / 32)), dim3(kLnJoin), 0, stream, a);
    }
    {
        const int n = piece_of(a, (int)sizeof(X), {a.x, a.dy, a.dx}, {a.x_stride, a.dy_stride, a.dx_stride}, {a.w});
        if (a.dim <= kLnDim) {
            if (n == 16 / (int)sizeof(X)) return ln_backward_n<X, W, 16 / sizeof(X)>(a, stream);
            if (n == 4 / (int)sizeof(X)) return ln_backward_n<X, W, 4 / sizeof(X)>(a, stream);
        }
        if constexpr (sizeof(X) == 2)
            if (n == 1 && a.dim <= kLnDim / 2) return ln_backward_n<X, W, 1>(a, stream);
    }
    a.slices = (int)(a.rows < kLnWideSlices ? a.rows : kLnWideSlices);
    const unsigned cols = (unsigned)((a.dim + kLnThreads - 1) / kLnThreads);
    cudaError_t e = launch_after(ln_columns_kernel<X>, dim3(cols, (unsigned)a.slices), dim3(kLnThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_after(ln_join_kernel<W>, dim3((unsigned)((2 * a.dim + 31) / 32)), dim3(kLnJoin), 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_after(ln_backward_long_kernel<X, W>, dim3((unsigned)a.rows), dim3(kLnThreads), 0, stream, a);
}

}  // namespace
}  // namespace adacomp

using adacomp::is_aligned;

extern "C" {

adacomp_status adacomp_layer_norm_init(adacomp_layer_norm_t* out, int64_t dim, adacomp_dtype x_dtype,
                                       adacomp_dtype w_dtype, float eps)
{
    if (!out) return ADACOMP_ERR_INVALID_ARG;
    *out = nullptr;
    if (dim < 1 || dim > (int64_t)1 << 30 || !adacomp::known_dtype(x_dtype) || !adacomp::known_dtype(w_dtype) ||
        !(eps >= 0.0f) || !std::isfinite(eps))
        return ADACOMP_ERR_INVALID_ARG;
    adacomp_layer_norm* h = new (std::nothrow) adacomp_layer_norm;
    if (!h) return ADACOMP_ERR_INVALID_ARG;
    h->dim = dim;
    h->x_dtype = x_dtype;
    h->w_dtype = w_dtype;
    h->eps = eps;
    *out = h;
    return ADACOMP_OK;
}

adacomp_status adacomp_layer_norm_forward(adacomp_layer_norm_t h, int64_t rows, const void* x, int64_t x_stride,
                                          const void* w, const void* b, void* y, int64_t y_stride, float* mean,
                                          float* rstd, cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_layer_norm_forward");
    if (!h || rows < 0 || rows >= (int64_t)1 << 31) return ADACOMP_ERR_INVALID_ARG;
    if (rows == 0) return ADACOMP_OK;
    if (!x || !w || !y || x_stride < 0 || (rows > 1 && y_stride < h->dim)) return ADACOMP_ERR_INVALID_ARG;
    const uintptr_t ex = adacomp::dtype_bytes(h->x_dtype), ew = adacomp::dtype_bytes(h->w_dtype);
    if (!is_aligned(x, ex) || !is_aligned(y, ex) || !is_aligned(w, ew) || !is_aligned(b, ew) || !is_aligned(mean, 4) ||
        !is_aligned(rstd, 4))
        return ADACOMP_ERR_ALIGNMENT;
    adacomp::LnArgs a = {};
    a.x = x;
    a.w = w;
    a.b = b;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.dim = h->dim;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.eps = h->eps;
    const bool xb = h->x_dtype == ADACOMP_BF16, wb = h->w_dtype == ADACOMP_BF16;
    using adacomp::bf16;
    const cudaError_t e = xb ? (wb ? adacomp::ln_forward<bf16, bf16>(a, stream) : adacomp::ln_forward<bf16, float>(a, stream))
                             : (wb ? adacomp::ln_forward<float, bf16>(a, stream) : adacomp::ln_forward<float, float>(a, stream));
    return adacomp::launch_result(e, stream);
}

size_t adacomp_layer_norm_backward_ws_bytes(adacomp_layer_norm_t h, int64_t rows)
{
    if (!h || rows < 0) return 0;
    return (size_t)adacomp::ln_slices(rows, h->dim) * 2 * (size_t)h->dim * 4;
}

adacomp_status adacomp_layer_norm_backward(adacomp_layer_norm_t h, int64_t rows, const void* dy, int64_t dy_stride,
                                           const void* x, int64_t x_stride, const void* w, const float* mean,
                                           const float* rstd, void* dx, int64_t dx_stride, void* dw, void* db,
                                           void* ws, size_t ws_bytes, cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_layer_norm_backward");
    if (!h || rows < 0 || rows >= (int64_t)1 << 31 || !w || !dw || !ws) return ADACOMP_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx || dy_stride < 0 || x_stride < 0 ||
                     (rows > 1 && dx_stride < h->dim)))
        return ADACOMP_ERR_INVALID_ARG;
    const uintptr_t ex = adacomp::dtype_bytes(h->x_dtype), ew = adacomp::dtype_bytes(h->w_dtype);
    if (!is_aligned(dy, ex) || !is_aligned(x, ex) || !is_aligned(dx, ex) || !is_aligned(w, ew) || !is_aligned(dw, ew) ||
        !is_aligned(db, ew) || !is_aligned(mean, 4) || !is_aligned(rstd, 4) || !is_aligned(ws, 16))
        return ADACOMP_ERR_ALIGNMENT;
    if (ws_bytes < adacomp_layer_norm_backward_ws_bytes(h, rows)) return ADACOMP_ERR_WORKSPACE;
    adacomp::LnArgs a = {};
    a.x = x;
    a.dy = dy;
    a.w = w;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.part = static_cast<float*>(ws);
    a.rows = rows;
    a.dim = h->dim;
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.dx_stride = dx_stride;
    const bool xb = h->x_dtype == ADACOMP_BF16, wb = h->w_dtype == ADACOMP_BF16;
    using adacomp::bf16;
    const cudaError_t e = xb ? (wb ? adacomp::ln_backward<bf16, bf16>(a, stream) : adacomp::ln_backward<bf16, float>(a, stream))
                             : (wb ? adacomp::ln_backward<float, bf16>(a, stream) : adacomp::ln_backward<float, float>(a, stream));
    return adacomp::launch_result(e, stream);
}

void adacomp_layer_norm_free(adacomp_layer_norm_t h) { delete h; }

}  // extern "C"
