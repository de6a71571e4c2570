// Layer norm, forward and backward with the gradients of the weight and the bias:
// kernels and C entry points (adacomp.h).
#include <new>

#include "train_common.cuh"

struct adacomp_layer_norm {
    int64_t dim = 0;
    int32_t x_dtype = ADACOMP_F32, w_dtype = ADACOMP_F32;
    float eps = 0.0f;
};

namespace adacomp {
namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;

struct LnArgs {
    const void *x, *dy, *w, *b;
    void *y, *dx, *dw, *db;
    float *mean, *rstd;          // outputs of the forward pass
    const float *mean_in, *rstd_in;
    float* part;                 // [slices][2][dim] partial sums of dw and db
    int64_t rows, dim, x_stride, y_stride, dy_stride, dx_stride;
    int32_t slices;
    float eps;
};

// One warp per row, three passes over it (the second and third from L1 or L2).
template <typename X, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_forward_kernel(const LnArgs a)
{
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kLnWarps + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
    X* y = static_cast<X*>(a.y) + row * a.y_stride;
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    const float n = (float)a.dim;
    float s = 0.0f;
    for (int64_t i = lane; i < a.dim; i += 32) s += to_f32(x[i]);
    const float mean = warp_sum(s) / n;
    s = 0.0f;
    for (int64_t i = lane; i < a.dim; i += 32) {
        const float d = to_f32(x[i]) - mean;
        s += d * d;
    }
    const float rstd = 1.0f / sqrtf(warp_sum(s) / n + a.eps);
    for (int64_t i = lane; i < a.dim; i += 32)
        y[i] = from_f32<X>((to_f32(x[i]) - mean) * rstd * to_f32(w[i]) + (b ? to_f32(b[i]) : 0.0f));
    if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <typename X, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_backward_kernel(const LnArgs a)
{
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kLnWarps + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
    const X* dy = static_cast<const X*>(a.dy) + row * a.dy_stride;
    X* dx = static_cast<X*>(a.dx) + row * a.dx_stride;
    const W* w = static_cast<const W*>(a.w);
    const float mean = a.mean_in[row], rstd = a.rstd_in[row], n = (float)a.dim;
    float s0 = 0.0f, s1 = 0.0f;
    for (int64_t i = lane; i < a.dim; i += 32) {
        const float g = to_f32(dy[i]) * to_f32(w[i]);
        s0 += g;
        s1 += g * (to_f32(x[i]) - mean) * rstd;
    }
    s0 = warp_sum(s0) / n;
    s1 = warp_sum(s1) / n;
    for (int64_t i = lane; i < a.dim; i += 32) {
        const float g = to_f32(dy[i]) * to_f32(w[i]);
        dx[i] = from_f32<X>(rstd * (g - s0 - (to_f32(x[i]) - mean) * rstd * s1));
    }
}

// Column sums: a slice of the rows per blockIdx.y, one column per thread. Runs before
// dx is written, which may be in place of dy or x.
template <typename X>
__global__ void __launch_bounds__(kLnThreads) ln_columns_kernel(const LnArgs a)
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
        dw += g * (to_f32(x[r * a.x_stride + c]) - a.mean_in[r]) * a.rstd_in[r];
    }
    float* p = a.part + (int64_t)blockIdx.y * 2 * a.dim;
    p[c] = dw;
    p[a.dim + c] = db;
}

template <typename W>
__global__ void __launch_bounds__(kLnThreads) ln_join_kernel(const LnArgs a)
{
    ptx::griddep_wait();
    const int64_t c = (int64_t)blockIdx.x * kLnThreads + threadIdx.x;
    if (c >= a.dim) return;
    float dw = 0.0f, db = 0.0f;
    for (int s = 0; s < a.slices; ++s) {
        dw += a.part[(int64_t)s * 2 * a.dim + c];
        db += a.part[(int64_t)s * 2 * a.dim + a.dim + c];
    }
    static_cast<W*>(a.dw)[c] = from_f32<W>(dw);
    if (a.db) static_cast<W*>(a.db)[c] = from_f32<W>(db);
}

int ln_slices(int64_t rows) { return (int)(rows < 1 ? 1 : rows < 128 ? rows : 128); }

template <typename X, typename W> cudaError_t ln_forward(const LnArgs& a, cudaStream_t stream)
{
    return launch_after(ln_forward_kernel<X, W>, dim3((unsigned)((a.rows + kLnWarps - 1) / kLnWarps)), dim3(kLnThreads),
                        0, stream, a);
}

template <typename X, typename W> cudaError_t ln_backward(const LnArgs& a, cudaStream_t stream)
{
    const unsigned cols = (unsigned)((a.dim + kLnThreads - 1) / kLnThreads);
    cudaError_t e = launch_after(ln_columns_kernel<X>, dim3(cols, (unsigned)a.slices), dim3(kLnThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_after(ln_join_kernel<W>, dim3(cols), dim3(kLnThreads), 0, stream, a);
    if (e != cudaSuccess || a.rows == 0) return e;
    return launch_after(ln_backward_kernel<X, W>, dim3((unsigned)((a.rows + kLnWarps - 1) / kLnWarps)),
                        dim3(kLnThreads), 0, stream, a);
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
    if (dim < 1 || dim > (int64_t)1 << 31 || !adacomp::known_dtype(x_dtype) || !adacomp::known_dtype(w_dtype) ||
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
    return (size_t)adacomp::ln_slices(rows) * 2 * (size_t)h->dim * 4;
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
    a.slices = adacomp::ln_slices(rows);
    const bool xb = h->x_dtype == ADACOMP_BF16, wb = h->w_dtype == ADACOMP_BF16;
    using adacomp::bf16;
    const cudaError_t e = xb ? (wb ? adacomp::ln_backward<bf16, bf16>(a, stream) : adacomp::ln_backward<bf16, float>(a, stream))
                             : (wb ? adacomp::ln_backward<float, bf16>(a, stream) : adacomp::ln_backward<float, float>(a, stream));
    return adacomp::launch_result(e, stream);
}

void adacomp_layer_norm_free(adacomp_layer_norm_t h) { delete h; }

}  // extern "C"
