// Layer norm: the forward pass's kernels, and the C entry points (adacomp.h).
#include <new>

#include "layer_norm.cuh"

struct adacomp_layer_norm {
    int64_t dim = 0;
    int32_t x_dtype = ADACOMP_F32, w_dtype = ADACOMP_F32;
    float eps = 0.0f;
};

namespace adacomp {
namespace {

constexpr int kLnThreads = 256;  // a CTA's where rows are too wide for registers

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
// from L2). kRuns: of more than a run's elements per thread.
template <typename X, typename W, bool kRuns>
__global__ void __launch_bounds__(kLnThreads) ln_forward_long_kernel(const LnArgs a)
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
    const auto runs = [&](auto&& add) {
        if constexpr (!kRuns) {
            float s = 0.0f;
            for (int64_t i = threadIdx.x; i < a.dim; i += kLnThreads) s = add(to_f32(x[i]), s);
            return s;
        }
        RunSum r;
        for (int64_t i = threadIdx.x; i < a.dim;) {
            const int64_t end = i + kLnRun * kLnThreads < a.dim ? i + kLnRun * kLnThreads : a.dim;
            float s = 0.0f;
            for (; i < end; i += kLnThreads) s = add(to_f32(x[i]), s);
            r.add(s);
        }
        return r.value();
    };
    const float mean = sum(runs([](float v, float s) { return s + v; }), 0) / (float)a.dim;
    const float squares = runs([mean](float v, float s) { return fmaf(v - mean, v - mean, s); });
    const float rstd = 1.0f / sqrtf(sum(squares, 1) / (float)a.dim + a.eps);
    for (int64_t i = threadIdx.x; i < a.dim; i += kLnThreads)
        y[i] = from_f32<X>(fmaf((to_f32(x[i]) - mean) * rstd, to_f32(w[i]), b ? to_f32(b[i]) : 0.0f));
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// ---------------------------------------------------------------- launches
template <typename X, typename W, int N> cudaError_t ln_forward_n(LnArgs a, cudaStream_t stream)
{
    const dim3 one((unsigned)a.rows), threads(kLnThreads);
    if (a.dim > kLnRun * kLnThreads) return launch_after(ln_forward_long_kernel<X, W, true>, one, threads, 0, stream, a);
    if (a.dim > 64 * kLnThreads) return launch_after(ln_forward_long_kernel<X, W, false>, one, threads, 0, stream, a);
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
    // Few rows: as many threads as there can be, for the loads' latency (one row of 12745 fp32, caches
    // cold: 15, eight warps 33; of 16384: 11 and 17), and so wide rows of two-byte pieces (4000 x
    // 16383 bf16: 146 and 166, but fp32 169 and 150).
    constexpr bool kShort = Piece<X, N>::kBytes == 2;
    if (a.dim > 2048 && (a.rows <= 152 || (kShort && a.dim > 8192)))
        return with(ln_forward_row_kernel<X, W, M, 16, 32>, 1024, 1024);
    if constexpr (!kShort) {
        if (a.dim > 8192) return with(ln_forward_row_kernel<X, W, M, 64, 8>, 256, 256);
    }
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
    return adacomp::ln_backward_bytes(rows, h->dim);
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
