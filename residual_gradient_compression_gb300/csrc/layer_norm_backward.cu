// Layer norm: the backward pass's kernels, with the gradients of the weight and the bias.
#include "layer_norm.cuh"

namespace adacomp {
namespace {

constexpr int kLnCols = 16;      // columns of a thread
constexpr int kLnThreads = 512;  // a CTA's
constexpr int kLnParts = 152;    // CTAs at most (one per SM), each with partial sums of dw and db
constexpr int64_t kLnDim = (int64_t)kLnThreads * kLnCols;

__device__ __forceinline__ void group_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Copies a piece of 16 bytes to shared memory, or zeros where it is not `there`.
__device__ __forceinline__ void copy_piece(uint32_t to, const void* from, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

// The rows of x and dy that a thread has on their way, and the shared memory for them. Pieces of
// 16 bytes are copied there; shorter ones are loaded to registers one row ahead, half as many
// columns at a time (65536 x 127 fp32: 22 us, copied four bytes at a time 44; 32768 x 1002 bf16:
// 51 and 49).
template <typename X, int N> struct LnRing {
    static constexpr bool kRing = Piece<X, N>::kBytes == 16;
    static constexpr int kCols = kRing ? kLnCols : kLnCols / 2;
    static constexpr int kRow = (kCols / N) * 2 * kLnThreads * Piece<X, N>::kBytes;
    static constexpr int kStages = sizeof(X) == 2 ? 6 : 3;
    static constexpr int kBytes = kRing ? kStages * kRow : 0;
};

// With xh = (x - mean) * rstd and g = dy * w:
//   dx = rstd * (g - sum(g) / n - xh * sum(g * xh) / n),  dw = sum over rows of dy * xh,  db = of dy.
// Bound by memory: dy and x are read once and dx written. A row is had by kWarps warps, or by
// a.group lanes (kWarps 0), 16 columns per thread, which go from row to row with the weights and
// the sums for dw and db in registers; so much state leaves a CTA of 16 warps per SM, and what
// hides the loads are the rows to come, copied to shared memory (every thread its own pieces,
// zeros where it has none: no barrier). The two sums of a row take one tree of shuffles for both,
// and one barrier of the row's warps. At the end the CTA's groups add their column sums in
// order, and a second kernel adds the CTAs' (2.4 us).
//
// With 32-bit weights, all in us, both kernels: 16384 x 2048 bf16 42 (4.8 TB/s; 65536 rows 132,
// 6.1 TB/s), fp32 66 (6.1 TB/s); 8192 x 8192 bf16 79, fp32 128 (6.3 TB/s); 32768 x 1001 fp32 75
// (5.2 TB/s), bf16 56. Short runs are bound by the start, the column sums and the join, and bf16
// rows by latency: at four warps per scheduler half of the issue slots are used (49.5 % at 16384 x
// 2048) and 56 % of the DRAM's rate.
template <typename X, typename W, int N, int kWarps>
__global__ void __launch_bounds__(kLnThreads, 1) ln_backward_kernel(const LnArgs a)
{
    using Ring = LnRing<X, N>;
    constexpr int kCols = Ring::kCols, kPieces = kCols / N, kPairs = kCols / 2;
    constexpr int kBytes = Piece<X, N>::kBytes, kStages = Ring::kStages;
    constexpr bool kRing = Ring::kRing;
    using Raw = typename Piece<X, N>::Raw;
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    __shared__ __align__(16) float2 sums[2][kLnThreads / 32];  // read two at a time
    ptx::griddep_wait();
    const int group = kWarps ? 32 * kWarps : a.group, place = threadIdx.x & (group - 1), dim = (int)a.dim;
    const int groups = kLnThreads / group, which = threadIdx.x / group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_n = 1.0f / (float)dim;
    const auto column = [&](int k) { return (k * group + place) * N; };
    Pair w[kPairs], dw[kPairs], db[kPairs];
    {
        float v[kCols] = {};
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            if (column(k) < dim)
                weights<N>(static_cast<const W*>(a.w) + column(k), *reinterpret_cast<float(*)[N]>(v + k * N));
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            w[i] = pair(v[2 * i], v[2 * i + 1]);
            dw[i] = db[i] = pair(0.0f);
        }
    }
    // the ring: [stage][piece][x, dy][thread]
    const Raw* const ring = reinterpret_cast<const Raw*>(shared_bytes) + threadIdx.x;
    const uint32_t ring_to = (uint32_t)__cvta_generic_to_shared(ring);
    const int64_t stride = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups + which;
    const auto row_of = [&](const void* p, int64_t row, int64_t step) { return static_cast<const X*>(p) + row * step; };
    int64_t row = first;
    const X *x = row_of(a.x, row, a.x_stride) + place * N, *dy = row_of(a.dy, row, a.dy_stride) + place * N;
    const int64_t x_step = stride * a.x_stride, dy_step = stride * a.dy_stride;
    int64_t ahead = row;  // the row that x and dy are at
    const auto stage_row = [&](int stage) {
        if constexpr (kRing) {
            const uint32_t to = ring_to + stage * Ring::kRow;
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const bool there = ahead < a.rows && column(k) < dim;
                copy_piece(to + (2 * k) * kLnThreads * kBytes, there ? x + k * group * N : a.x, there);
                copy_piece(to + (2 * k + 1) * kLnThreads * kBytes, there ? dy + k * group * N : a.dy, there);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        x += x_step, dy += dy_step, ahead += stride;
    };
    Piece<X, N> px[kPieces], pd[kPieces], next_x[kPieces], next_d[kPieces];
    const auto load_next = [&]() {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            next_x[k].zero();
            next_d[k].zero();
            if (ahead < a.rows && column(k) < dim) {
                next_x[k].load(x + k * group * N);
                next_d[k].load(dy + k * group * N);
            }
        }
        x += x_step, dy += dy_step, ahead += stride;
    };
    float mean = 0.0f, rstd = 0.0f;
    if (row < a.rows) mean = a.mean_in[row], rstd = a.rstd_in[row];
    if (kRing) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) stage_row(i);
    } else {
        load_next();
    }
    X* dx = static_cast<X*>(a.dx) + row * a.dx_stride + place * N;
    const int64_t dx_step = stride * a.dx_stride;
    // every lane of a warp takes part as long as the warp's first group has a row
    const int64_t lead = kWarps ? row : (int64_t)blockIdx.x * groups + warp * (32 / group);
    int stage = 0, turn = 0;
    for (int64_t at = lead; at < a.rows; at += stride, row += stride, dx += dx_step) {
        float mean_next = 0.0f, rstd_next = 0.0f;
        if (row + stride < a.rows) mean_next = a.mean_in[row + stride], rstd_next = a.rstd_in[row + stride];
        if (kRing) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                px[k].q = ring[(stage * kPieces + k) * 2 * kLnThreads];
                pd[k].q = ring[((stage * kPieces + k) * 2 + 1) * kLnThreads];
            }
            stage_row(stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
        } else {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) px[k] = next_x[k], pd[k] = next_d[k];
            load_next();
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
        if (kWarps == 0) {
            s0 = group_sum(s0, group);
            s1 = group_sum(s1, group);
        } else {
            // both sums in one tree: the lower half of the lanes goes on with s0, the upper with s1
            const bool low = lane < 16;
            float s = (low ? s0 : s1) + __shfl_xor_sync(0xffffffffu, low ? s1 : s0, 16);
#pragma unroll
            for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (kWarps == 1) {
                const float t = __shfl_xor_sync(0xffffffffu, s, 16);
                s0 = low ? s : t;
                s1 = low ? t : s;
            } else {
                if ((lane & 15) == 0) reinterpret_cast<float*>(&sums[turn][warp])[lane >> 4] = s;
                group_barrier(1 + which, group);
                const float2* from = sums[turn] + which * kWarps;
                s0 = s1 = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; i += 2) {
                    const float4 q = *reinterpret_cast<const float4*>(from + i);
                    s0 += q.x + q.z;
                    s1 += q.y + q.w;
                }
                turn ^= 1;
            }
        }
        if (kWarps || row < a.rows) {
            // dx = rstd * (g - s0 / n - xh * s1 / n)
            const Pair scale = pair(rstd), k0 = pair(-(s0 * inv_n) * rstd), k1 = pair(-(s1 * inv_n) * rstd * rstd);
            float v[kCols];
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                split(fma2(g[i], scale, fma2(d[i], k1, k0)), v[2 * i], v[2 * i + 1]);
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                if (column(k) < dim) put_piece<N>(dx + k * group * N, *reinterpret_cast<const float(*)[N]>(v + k * N));
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
    if (kWarps == 0) {  // the warp's groups first
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            for (int o = group; o < 32; o <<= 1) {
                sw[i] += __shfl_xor_sync(0xffffffffu, sw[i], o);
                sb[i] += __shfl_xor_sync(0xffffffffu, sb[i], o);
            }
    }
    const int owners = kWarps ? groups : kLnThreads / 32, mine = kWarps ? which : warp;
    if (kWarps || lane < group) {
        float* const to = total + mine * 2 * dim;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int c = column(k);
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
    for (int i = threadIdx.x; i < 2 * dim; i += kLnThreads) {
        float v = total[i];
        for (int o = 1; o < owners; ++o) v += total[o * 2 * dim + i];
        part[i] = v;
    }
}

constexpr int kLnStrip = 256;        // threads of a CTA where rows are too wide for registers
template <int N> constexpr int kLnStripCols = N == 1 ? 4 : 8;      // columns of a thread there
constexpr int kLnStripCtas = 3;      // per SM
constexpr int kLnStripSlices = 128;  // of the rows, at most
constexpr int64_t kLnSpan = 2 * kLnRun * kLnStrip;  // elements of a row that its threads add in one run (two sums each)

// The rows' two sums, behind the column sums.
__device__ __forceinline__ float2* row_sums(const LnArgs& a)
{
    return reinterpret_cast<float2*>(a.part + (a.rows < kLnStripSlices ? a.rows : kLnStripSlices) * 2 * a.dim);
}

// Adds the partial sums: 32 columns per CTA, 32 rows of threads that each add every 32nd. Bound by
// latency: the sums were just written, 152 times 16 KB at 2048 columns.
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

// Rows too wide for that: the two sums of every row by a CTA each, then strips of columns, whose
// CTAs go from row to row with their weights and column sums in registers, in one wave. Bound by
// memory: x and dy are read twice, the second time from the last row upwards, of which L2 has
// the more the fewer there are (4096 x 12288 bf16: 99 us, downwards 106; 5.1 TB/s of the five
// passes). fp32 4096 x 16000: 195 us (6.7 TB/s). Pieces of two bytes: 4096 x 12289 148 us.
// kRuns: rows of more than kLnSpan elements.
template <typename X, typename W, int N, bool kRuns>
__global__ void __launch_bounds__(kLnStrip) ln_sums_kernel(const LnArgs a)
{
    __shared__ float2 shared[kLnStrip / 32];
    ptx::griddep_wait();
    constexpr int M = N == 1 ? 32 / (int)sizeof(X) : 8;  // elements of a turn
    static_assert(2 * kLnRun % M == 0, "whole turns");
    const int64_t row = blockIdx.x;
    const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
    const X* dy = static_cast<const X*>(a.dy) + row * a.dy_stride;
    const W* w = static_cast<const W*>(a.w);
    const float mean = a.mean_in[row];
    Pair t0 = pair(0.0f), t1 = pair(0.0f);
    const auto turn = [&](int64_t c) {
        Piece<X, N> px[M / N], pd[M / N];
        float wv[M] = {};
#pragma unroll
        for (int k = 0; k < M / N; ++k) {
            px[k].zero();
            pd[k].zero();
            if (c + k * kLnStrip * N < a.dim) {
                px[k].load(x + c + k * kLnStrip * N);
                pd[k].load(dy + c + k * kLnStrip * N);
                weights<N>(w + c + k * kLnStrip * N, *reinterpret_cast<float(*)[N]>(wv + k * N));
            }
        }
#pragma unroll
        for (int i = 0; i < M / 2; ++i) {
            const Pair g = pair_of(pd, i) * pair(wv[2 * i], wv[2 * i + 1]);
            t0 = t0 + g;
            t1 = fma2(g, pair_of(px, i) + pair(-mean), t1);
        }
    };
    RunSum r0, r1;
    if constexpr (!kRuns) {
        for (int64_t c = threadIdx.x * N; c < a.dim; c += kLnStrip * M) turn(c);
    } else {
        for (int64_t c = threadIdx.x * N; c < a.dim;) {
            for (int i = 0; i < kLnSpan / (kLnStrip * M) && c < a.dim; ++i, c += kLnStrip * M) turn(c);
            r0.add(both(t0));
            r1.add(both(t1));
            t0 = t1 = pair(0.0f);
        }
    }
    float s0 = warp_sum(kRuns ? r0.value() : both(t0)), s1 = warp_sum(kRuns ? r1.value() : both(t1));
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = make_float2(s0, s1);
    __syncthreads();
    if (threadIdx.x) return;
    s0 = s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < kLnStrip / 32; ++i) {
        s0 += shared[i].x;
        s1 += shared[i].y;
    }
    const float rstd = a.rstd_in[row], inv_n = 1.0f / (float)a.dim;
    // dx = rstd * (g - s0 / n - xh * s1 / n), with s1 of xh = rstd * d
    row_sums(a)[row] = make_float2(-(s0 * inv_n) * rstd, -(s1 * rstd * inv_n) * rstd * rstd);
}

template <typename X, typename W, int N> __global__ void __launch_bounds__(kLnStrip, kLnStripCtas)
    ln_strip_kernel(const LnArgs a)
{
    constexpr int kCols = kLnStripCols<N>, kPieces = kCols / N, kPairs = kCols / 2;
    constexpr int kRows = sizeof(X) == 2 && N > 1 ? 4 : 2;  // on their way
    ptx::griddep_wait();
    const int64_t first = (int64_t)blockIdx.x * (kLnStrip * kCols) + threadIdx.x * N;
    const X* x = static_cast<const X*>(a.x) + first;
    const X* dy = static_cast<const X*>(a.dy) + first;
    X* dx = static_cast<X*>(a.dx) + first;
    bool there[kPieces];
    Pair w[kPairs], dw[kPairs], db[kPairs];
    {
        float v[kCols] = {};
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            there[k] = first + k * kLnStrip * N < a.dim;
            if (there[k])
                weights<N>(static_cast<const W*>(a.w) + first + k * kLnStrip * N, *reinterpret_cast<float(*)[N]>(v + k * N));
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            w[i] = pair(v[2 * i], v[2 * i + 1]);
            dw[i] = db[i] = pair(0.0f);
        }
    }
    // upwards from the last row, which L2 has still from the first kernel
    for (int64_t last = a.rows - 1 - blockIdx.y; last >= 0; last -= (int64_t)kRows * a.slices) {
        Piece<X, N> px[kRows][kPieces], pd[kRows][kPieces];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t r = last - (int64_t)k * a.slices;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                px[k][i].zero();
                pd[k][i].zero();
                if (r >= 0 && there[i]) {
                    px[k][i].load(x + r * a.x_stride + i * kLnStrip * N);
                    pd[k][i].load(dy + r * a.dy_stride + i * kLnStrip * N);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t r = last - (int64_t)k * a.slices;
            if (r < 0) break;
            const Pair minus = pair(-a.mean_in[r]), rstd = pair(a.rstd_in[r]);
            const float2 s = row_sums(a)[r];
            const Pair k0 = pair(s.x), k1 = pair(s.y);
            float v[kCols];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const Pair d = pair_of(px[k], i) + minus, g = pair_of(pd[k], i);
                db[i] = db[i] + g;
                dw[i] = fma2(g * rstd, d, dw[i]);
                split(fma2(g * w[i], rstd, fma2(d, k1, k0)), v[2 * i], v[2 * i + 1]);
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                if (there[i])
                    put_piece<N>(dx + r * a.dx_stride + i * kLnStrip * N, *reinterpret_cast<const float(*)[N]>(v + i * N));
        }
    }
    float* p = a.part + (int64_t)blockIdx.y * 2 * a.dim + first;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        if (!there[k]) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float w0, w1, b0, b1;
            split(dw[(k * N + j) / 2], w0, w1);
            split(db[(k * N + j) / 2], b0, b1);
            p[k * kLnStrip * N + j] = (k * N + j) % 2 ? w1 : w0;
            p[a.dim + k * kLnStrip * N + j] = (k * N + j) % 2 ? b1 : b0;
        }
    }
}

// ---------------------------------------------------------------- launches
template <typename W> cudaError_t ln_join(const LnArgs& a, cudaStream_t stream)
{
    return launch_after(ln_join_kernel<W>, dim3((unsigned)((2 * a.dim + 31) / 32)), dim3(kLnJoin), 0, stream, a);
}

template <typename X, typename W, int N, int kWarps> cudaError_t ln_backward_group(LnArgs a, cudaStream_t stream)
{
    constexpr int sums = 2 * (int)kLnDim * 4, ring = LnRing<X, N>::kBytes, shared = ring > sums ? ring : sums;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) e = allow<ln_backward_kernel<X, W, N, kWarps>>(shared);
    if (e != cudaSuccess) return e;
    const int64_t per = kLnThreads / a.group, need = (a.rows + per - 1) / per;
    const int64_t most = sms < kLnParts ? sms : kLnParts;
    a.slices = (int)(need < most ? need : most);
    e = launch_after(ln_backward_kernel<X, W, N, kWarps>, dim3((unsigned)a.slices), dim3(kLnThreads), shared, stream, a);
    return e == cudaSuccess ? ln_join<W>(a, stream) : e;
}

template <typename X, typename W, int N> cudaError_t ln_backward_n(LnArgs a, cudaStream_t stream)
{
    constexpr int cols = LnRing<X, N>::kCols;
    const int64_t places = (a.dim + N - 1) / N;
    a.group = places <= 16 ? group_of(places, 16) : 32 * group_of((a.dim + 32 * cols - 1) / (32 * cols), kLnThreads / 32);
    switch (a.group / 32) {
    case 0: return ln_backward_group<X, W, N, 0>(a, stream);
    case 1: return ln_backward_group<X, W, N, 1>(a, stream);
    case 2: return ln_backward_group<X, W, N, 2>(a, stream);
    case 4: return ln_backward_group<X, W, N, 4>(a, stream);
    case 8: return ln_backward_group<X, W, N, 8>(a, stream);
    default: return ln_backward_group<X, W, N, 16>(a, stream);
    }
}

template <typename X, typename W, int N> cudaError_t ln_backward_wide(LnArgs a, cudaStream_t stream)
{
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t strips = (a.dim + kLnStrip * kLnStripCols<N> - 1) / (kLnStrip * kLnStripCols<N>);
    int64_t most = kLnStripCtas * sms / strips;  // one wave
    most = most < 1 ? 1 : most < kLnStripSlices ? most : kLnStripSlices;
    a.slices = (int)(a.rows < most ? a.rows : most);
    e = launch_after(a.dim > kLnSpan ? ln_sums_kernel<X, W, N, true> : ln_sums_kernel<X, W, N, false>,
                     dim3((unsigned)a.rows), dim3(kLnStrip), 0, stream, a);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)strips, (unsigned)a.slices);
    e = launch_after(ln_strip_kernel<X, W, N>, grid, dim3(kLnStrip), 0, stream, a);
    return e == cudaSuccess ? ln_join<W>(a, stream) : e;
}

}  // namespace

size_t ln_backward_bytes(int64_t rows, int64_t dim)
{
    // whichever way a call's alignment takes
    const size_t sums = (size_t)dim * 2 * 4;
    const auto parts = [&](int64_t most) { return (size_t)(rows < 1 ? 1 : rows < most ? rows : most) * sums; };
    const size_t group = dim <= kLnDim ? parts(kLnParts) : sums;
    const size_t wide = dim > kLnDim / 2 ? parts(kLnStripSlices) + (size_t)rows * sizeof(float2) : sums;
    return group > wide ? group : wide;
}

template <typename X, typename W> cudaError_t ln_backward(const LnArgs& a, cudaStream_t stream)
{
    if (a.rows == 0) {
        LnArgs none = a;
        none.slices = 0;
        return ln_join<W>(none, stream);
    }
    const int n = piece_of(a, (int)sizeof(X), {a.x, a.dy, a.dx}, {a.x_stride, a.dy_stride, a.dx_stride}, {a.w});
    if (n == 16 / (int)sizeof(X)) {
        constexpr int N = 16 / sizeof(X);
        return a.dim <= kLnDim ? ln_backward_n<X, W, N>(a, stream) : ln_backward_wide<X, W, N>(a, stream);
    }
    if constexpr (sizeof(X) == 2)
        if (n == 2) return a.dim <= kLnDim / 2 ? ln_backward_n<X, W, 2>(a, stream) : ln_backward_wide<X, W, 2>(a, stream);
    return a.dim <= kLnDim / 2 ? ln_backward_n<X, W, 1>(a, stream) : ln_backward_wide<X, W, 1>(a, stream);
}

template cudaError_t ln_backward<float, float>(const LnArgs&, cudaStream_t);
template cudaError_t ln_backward<float, bf16>(const LnArgs&, cudaStream_t);
template cudaError_t ln_backward<bf16, float>(const LnArgs&, cudaStream_t);
template cudaError_t ln_backward<bf16, bf16>(const LnArgs&, cudaStream_t);

}  // namespace adacomp
