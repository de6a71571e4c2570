// Linear layers: the forward and backward pass and their C entry points (adacomp.h).
#include <initializer_list>
#include <new>

#include "product_few.cuh"
#include "product_tc.cuh"

struct adacomp_linear {
    int64_t in = 0, out = 0;
    int32_t dtype = ADACOMP_F32, act = ADACOMP_ACT_NONE;
    adacomp::TcWaits waits;
};

namespace adacomp {
namespace {

constexpr int kDzCols = 256, kDzRows = 8;  // of a CTA: a warp has 256 columns of a row
constexpr int kDzFew = 32;                 // columns of one for few rows, of which it has 64 at a time
constexpr int kDzSlices = 152;             // partial sums of db: one per slice of the rows
constexpr int kDbCols = 32, kDbRows = 16;
constexpr int64_t kOneSlice = 128;         // rows that one slice has, without a second kernel

struct LinearArgs {
    int64_t rows, in, out;
    int32_t act;
    const void *x, *w, *bias, *residual, *dy, *pre_in;
    void *y, *pre, *dx, *dw, *db;
    int64_t x_stride, w_stride, residual_stride, dy_stride, pre_in_stride, y_stride, pre_stride, dx_stride, dw_stride;
    TcWaits waits;
};

struct LinearParts {  // of a pass's workspace
    float* sums;            // backward: of dz, over slices of the rows
    bf16 *dz, *x, *w;       // copies of what cannot be read as it lies
    float* parts;           // of products whose terms are split
};

// Which products are for the kernel of small matrices, by what its whole tiles of 32 x 32 and 128 terms compute.
// us with it and without: fp32 256 x 512 x 512 12 and 17, 512 x 512 x 512 17 and 17, 2048 x 2048 of one term 66
// and 14; bf16 256 x 256 x 256 7 and 10, 128 x 512 x 512 12 and 9.
template <typename T> bool is_small(int64_t m, int64_t n, int64_t k)
{
    constexpr int64_t most = (int64_t)1 << (sizeof(T) == 4 ? 27 : 24);
    const auto at_least = [](int64_t x, int64_t least) { return x > least ? x : least; };
    m = at_least(m, kSmallTile);
    n = at_least(n, kSmallTile);
    k = at_least(k, kSmallDepth);
    return m <= most / n && m * n <= most / k;
}
template <typename T> bool both_small(int64_t rows, int64_t in, int64_t out) { return is_small<T>(rows, in, out) && is_small<T>(out, in, rows); }
template <typename T> constexpr int64_t few_of() { return sizeof(T) == 2 ? kFewBf16 : kFewF32; }

// What the kernels of few rows and of small matrices do not use is not in it: of fewer rows a pass takes those if it
// does of more, so that a workspace for more rows is enough for fewer.
template <typename T> LinearParts linear_parts(Carve& c, int64_t rows, int64_t in, int64_t out, bool backward)
{
    constexpr int bytes = sizeof(T);
    LinearParts p = {};
    if (backward) {
        p.sums = c.take<float>(kDzSlices * out);
        // in two parts, or as fp32 numbers, of few rows
        const int64_t few = packed_elements(2 * (rows < kFewRows ? rows : kFewRows), out, bytes), all = packed_elements(rows, out, bytes);
        p.dz = c.take<bf16>(few > all ? few : all);
        if (both_small<T>(rows, in, out)) return p;
    } else if (rows <= few_of<T>() || is_small<T>(rows, out, in)) {
        c.take<float>(1);  // sizes are not 0
        return p;
    }
    p.x = c.take<bf16>(packed_elements(rows, in, bytes));
    p.w = c.take<bf16>(packed_elements(out, in, bytes));
    p.parts = c.take<float>(backward ? parts_elements(rows, in) + parts_elements(out, in) : parts_elements(rows, out));
    return p;
}

inline size_t linear_bytes(int32_t dtype, int64_t rows, int64_t in, int64_t out, bool backward)
{
    Carve c;
    if (dtype == ADACOMP_BF16) linear_parts<bf16>(c, rows, in, out, backward);
    else linear_parts<float>(c, rows, in, out, backward);
    return c.at;
}

struct DzArgs {
    const void *dy, *pre;
    void* dz;       // planes of bf16 numbers, or (plain) T's
    void* db;       // of one slice alone
    float* sums;
    int64_t rows, n, dy_stride, pre_stride, dz_stride, dz_plane;
    int32_t act, slices;
    bool plain, two, dy_whole, pre_whole;  // two: parts; with plain, fp32 numbers
};

// Eight columns of a row as they lie in memory, until they are used.
template <typename T> struct Eight {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T* p, int64_t left, bool whole)
    {
        if (whole && left >= 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                const uint4 q = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
            }
            return;
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = i < left ? __float_as_uint(p[i]) : 0u;
        } else {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (2 * i < left ? q[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)q[2 * i + 1] << 16 : 0u);
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return i & 1 ? bf16_high(w[i / 2]) : bf16_low(w[i / 2]);
    }
};

// dz = dy * act'(pre), and its sums over slices of the rows. Bound by memory: a thread has eight columns of every
// kRowsOfCta-th row of a slice, several rows under way at a time; the CTA's sums meet in shared memory, the slices' in a
// second kernel, in a fixed order.
template <typename T, int kAct, int kRowsOfCta> __device__ __forceinline__ void dz_rows(const DzArgs& a, int32_t c, float (&sum)[8])
{
    constexpr int kAhead = sizeof(T) == 2 ? 3 : 2;
    const T *dy = static_cast<const T*>(a.dy) + c, *pre = static_cast<const T*>(a.pre) + c;
    const int64_t left = a.n - c, step = (int64_t)a.slices * kRowsOfCta;
    for (int64_t r0 = blockIdx.y * kRowsOfCta + threadIdx.y; r0 < a.rows; r0 += kAhead * step) {
        Eight<T> v[kAhead], z[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t r = r0 + i * step, here = r < a.rows ? left : 0;
            v[i].load(dy + r * a.dy_stride, here, a.dy_whole);
            if constexpr (kAct != ADACOMP_ACT_NONE) z[i].load(pre + r * a.pre_stride, here, a.pre_whole);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t r = r0 + i * step;
            if (r >= a.rows) break;
            float d[8], s[8];
            if constexpr (kAct != ADACOMP_ACT_NONE) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = z[i].get(j);
                slope_all<T, kAct>(s);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = v[i].get(j);
                // one rounding whatever is asked for: db is the sum of what dz would be rounded from
                if constexpr (kAct != ADACOMP_ACT_NONE) d[j] = __fmul_rn(d[j], s[j]);
                sum[j] += d[j];
            }
            if (kAct == ADACOMP_ACT_NONE || !a.dz) continue;
            if (a.plain && a.two) put_chunk(static_cast<float*>(a.dz) + r * a.dz_stride + c, d, left, true);
            else if (a.plain) put_chunk(static_cast<T*>(a.dz) + r * a.dz_stride + c, d, left, true);
            else put_parts<T>(static_cast<bf16*>(a.dz) + r * a.dz_stride + c, a.dz_plane, d, left, a.two);
        }
    }
}

template <typename T, int kColsOfCta, int kRowsOfCta>
__global__ void __launch_bounds__(kColsOfCta / 8 * kRowsOfCta, sizeof(T) == 2 ? 4 : 3) linear_dz_kernel(const DzArgs a)
{
    __shared__ float sums[kRowsOfCta][kColsOfCta];
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int32_t c = blockIdx.x * kColsOfCta + threadIdx.x * 8;
    float sum[8] = {};
    if (c < a.n) switch (a.act) {
        case ADACOMP_ACT_RELU: dz_rows<T, ADACOMP_ACT_RELU, kRowsOfCta>(a, c, sum); break;
        case ADACOMP_ACT_GELU: dz_rows<T, ADACOMP_ACT_GELU, kRowsOfCta>(a, c, sum); break;
        case ADACOMP_ACT_GELU_TANH: dz_rows<T, ADACOMP_ACT_GELU_TANH, kRowsOfCta>(a, c, sum); break;
        case ADACOMP_ACT_SILU: dz_rows<T, ADACOMP_ACT_SILU, kRowsOfCta>(a, c, sum); break;
        default: dz_rows<T, ADACOMP_ACT_NONE, kRowsOfCta>(a, c, sum);
        }
    if (!a.sums && !a.db) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[threadIdx.y][threadIdx.x * 8 + j] = sum[j];
    __syncthreads();
    const int i = threadIdx.y * (kColsOfCta / 8) + threadIdx.x;
    const int64_t at = (int64_t)blockIdx.x * kColsOfCta + i;
    if (i >= kColsOfCta || at >= a.n) return;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kRowsOfCta; ++j) s += sums[j][i];
    if (a.db) static_cast<T*>(a.db)[at] = from_f32<T>(s);
    else a.sums[blockIdx.y * a.n + at] = s;
}

template <typename T> __global__ void __launch_bounds__(kDbCols * kDbRows) linear_db_kernel(const float* part, T* db, int64_t n, int32_t slices)
{
    __shared__ float sums[kDbRows][kDbCols];
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int64_t c = (int64_t)blockIdx.x * kDbCols + threadIdx.x;
    float s = 0.0f;
    if (c < n)
#pragma unroll 4
        for (int i = threadIdx.y; i < slices; i += kDbRows) s += part[i * n + c];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= n) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kDbRows; ++i) s += sums[i][threadIdx.x];
    db[c] = from_f32<T>(s);
}

template <typename T> cudaError_t linear_forward(const LinearArgs& a, void* ws, cudaStream_t stream)
{
    EpiLinear<T> epi = {};
    epi.y = static_cast<T*>(a.y);
    epi.pre = static_cast<T*>(a.pre);
    epi.bias = static_cast<const T*>(a.bias);
    epi.residual = static_cast<const T*>(a.residual);
    epi.y_stride = a.y_stride;
    epi.pre_stride = a.pre_stride;
    epi.residual_stride = a.residual_stride;
    epi.n = (int32_t)a.out;
    epi.act = a.act;
    epi.whole = whole_rows(a.y, a.y_stride, a.rows, sizeof(T)) && whole_rows(a.pre, a.pre_stride, a.rows, sizeof(T)) &&
                is_aligned(a.bias, 16) && whole_rows(a.residual, a.residual_stride, a.rows, sizeof(T));
    if (a.rows <= few_of<T>())
        return product_few<T>(FewArgs{a.x, a.w, a.x_stride, a.w_stride, (int32_t)a.rows, (int32_t)a.out, (int32_t)a.in}, epi, stream);
    if (is_small<T>(a.rows, a.out, a.in))
        return product_small<T, T>(SmallArgs{{a.x, a.x_stride, 1}, {a.w, a.w_stride, 1}, (int32_t)a.rows, (int32_t)a.out, (int32_t)a.in}, epi, stream);
    Carve carve{static_cast<char*>(ws)};
    const LinearParts p = linear_parts<T>(carve, a.rows, a.in, a.out, false);
    Matrix x, w;
    cudaError_t e = take_matrix<T>(&x, a.x, a.x_stride, a.rows, a.in, p.x, stream);
    if (e == cudaSuccess) e = take_matrix<T>(&w, a.w, a.w_stride, a.out, a.in, p.w, stream);
    if (e != cudaSuccess) return e;
    const TcProduct product = {x, w, false, false, a.rows, a.out, a.in, nullptr, nullptr, 1, a.waits};
    return product_tc<T>(product, p.parts, epi, stream);
}

template <typename T> cudaError_t linear_backward(const LinearArgs& a, void* ws, cudaStream_t stream)
{
    Carve carve{static_cast<char*>(ws)};
    const LinearParts p = linear_parts<T>(carve, a.rows, a.in, a.out, true);
    const bool act = a.act != ADACOMP_ACT_NONE, products = a.dx || a.dw, small = both_small<T>(a.rows, a.in, a.out);
    const bool two = sizeof(T) == 2 && act && a.rows <= kFewRows;
    cudaError_t e = cudaSuccess;
    Matrix dz = {p.dz, a.rows, a.out, pitch_of(a.out), a.rows * pitch_of(a.out)}, x, w;
    if ((act && products) || a.db) {
        DzArgs d = {};
        d.dy = a.dy;
        d.pre = a.pre_in;
        d.dz = products ? p.dz : nullptr;
        d.sums = a.db ? p.sums : nullptr;
        d.rows = a.rows;
        d.n = a.out;
        d.dy_stride = a.dy_stride;
        d.pre_stride = a.pre_in_stride;
        d.dz_stride = dz.stride;
        d.dz_plane = dz.plane;
        d.act = a.act;
        d.plain = small;
        d.two = two;
        d.dy_whole = whole_rows(a.dy, a.dy_stride, a.rows, sizeof(T));
        d.pre_whole = whole_rows(a.pre_in, a.pre_in_stride, a.rows, sizeof(T));
        // CTAs for eight on each SM, of no fewer than two rows a thread
        const int64_t blocks = (a.out + kDzCols - 1) / kDzCols, most = (a.rows + 2 * kDzRows - 1) / (2 * kDzRows);
        int64_t slices = 8 * kDzSlices / blocks;
        slices = slices < 1 ? 1 : slices < kDzSlices ? slices : kDzSlices;
        d.slices = (int32_t)(a.rows <= kOneSlice ? 1 : slices < most ? slices : most);
        if (d.slices == 1 || a.rows == 0) {
            d.db = a.db;
            d.sums = nullptr;
        }
        e = d.slices == 1 ? launch_after(linear_dz_kernel<T, kDzFew, 64>, dim3((unsigned)((a.out + kDzFew - 1) / kDzFew)), dim3(kDzFew / 8, 64), 0, stream, d)
                          : launch_after(linear_dz_kernel<T, kDzCols, kDzRows>, dim3((unsigned)blocks, d.slices), dim3(kDzCols / 8, kDzRows), 0, stream, d);
        if (e == cudaSuccess && a.db && !d.db)
            e = launch_after(linear_db_kernel<T>, dim3((unsigned)((a.out + kDbCols - 1) / kDbCols)), dim3(kDbCols, kDbRows), 0, stream,
                             (const float*)p.sums, static_cast<T*>(a.db), a.out, d.slices);
    }
    if (e != cudaSuccess) return e;
    const auto store = [&](void* out, int64_t stride, int64_t rows) {
        EpiStore<T> epi = {};
        epi.out = static_cast<T*>(out);
        epi.stride = stride;
        epi.n = (int32_t)a.in;
        epi.first = epi.last = true;
        epi.whole = whole_rows(out, stride, rows, sizeof(T));
        return epi;
    };
    const EpiStore<T> to_dx = store(a.dx, a.dx_stride, a.rows), to_dw = store(a.dw, a.dw_stride, a.out);
    if (a.rows == 0) return a.dw ? product_none(a.out, a.in, to_dw, stream) : cudaSuccess;
    const int32_t rows = (int32_t)a.rows, in = (int32_t)a.in, out = (int32_t)a.out;
    if (small) {
        const Operand by_row = act ? Operand{p.dz, dz.stride, 1} : Operand{a.dy, a.dy_stride, 1};
        const SmallArgs to_x = {by_row, {a.w, 1, a.w_stride}, rows, in, out}, to_w = {{by_row.p, 1, by_row.row}, {a.x, 1, a.x_stride}, out, in, rows};
        if (a.dx) e = two ? product_small<float, T>(to_x, to_dx, stream) : product_small<T, T>(to_x, to_dx, stream);
        if (a.dw && e == cudaSuccess) e = two ? product_small<float, T>(to_w, to_dw, stream) : product_small<T, T>(to_w, to_dw, stream);
        return e;
    }
    if (!act && products) e = take_matrix<T>(&dz, a.dy, a.dy_stride, a.rows, a.out, p.dz, stream);
    if (a.dx && e == cudaSuccess) e = take_matrix<T>(&w, a.w, a.w_stride, a.out, a.in, p.w, stream);
    if (a.dw && e == cudaSuccess) e = take_matrix<T>(&x, a.x, a.x_stride, a.rows, a.in, p.x, stream);
    if (e != cudaSuccess) return e;
    const TcProduct dx = {dz, w, false, true, a.rows, a.in, a.out, nullptr, nullptr, two ? 2 : 1, a.waits};
    const TcProduct dw = {dz, x, true, true, a.out, a.in, a.rows, nullptr, nullptr, two ? 2 : 1, a.waits};
    return product_tc_both<T>(dx, to_dx, a.dx, dw, to_dw, a.dw, p.parts, stream);
}

constexpr int64_t kMostDim = (int64_t)1 << 30, kMostRows = ((int64_t)1 << 30) + 1;

}  // namespace
}  // namespace adacomp

using adacomp::is_aligned;

extern "C" {

adacomp_status adacomp_linear_init(adacomp_linear_t* out, int64_t in_dim, int64_t out_dim, adacomp_dtype dtype,
                                   adacomp_activation activation)
{
    if (!out) return ADACOMP_ERR_INVALID_ARG;
    *out = nullptr;
    if (in_dim < 1 || in_dim > adacomp::kMostDim || out_dim < 1 || out_dim > adacomp::kMostDim ||
        !adacomp::known_dtype(dtype) || (int)activation < ADACOMP_ACT_NONE || (int)activation > ADACOMP_ACT_SILU)
        return ADACOMP_ERR_INVALID_ARG;
    adacomp_linear* h = new (std::nothrow) adacomp_linear;
    if (!h) return ADACOMP_ERR_INVALID_ARG;
    h->in = in_dim;
    h->out = out_dim;
    h->dtype = dtype;
    h->act = activation;
    *out = h;
    return ADACOMP_OK;
}

size_t adacomp_linear_forward_ws_bytes(adacomp_linear_t h, int64_t rows)
{
    return h && rows >= 0 && rows < adacomp::kMostRows ? adacomp::linear_bytes(h->dtype, rows, h->in, h->out, false) : 0;
}

size_t adacomp_linear_backward_ws_bytes(adacomp_linear_t h, int64_t rows)
{
    return h && rows >= 0 && rows < adacomp::kMostRows ? adacomp::linear_bytes(h->dtype, rows, h->in, h->out, true) : 0;
}

adacomp_status adacomp_linear_forward(adacomp_linear_t h, int64_t rows, const void* x, int64_t x_stride, const void* w,
                                      int64_t w_stride, const void* bias, const void* residual, int64_t residual_stride,
                                      void* y, int64_t y_stride, void* pre, int64_t pre_stride, void* ws,
                                      size_t ws_bytes, cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_linear_forward");
    if (!h || rows < 0 || rows >= adacomp::kMostRows) return ADACOMP_ERR_INVALID_ARG;
    if (rows == 0) return ADACOMP_OK;
    if (!x || !w || !y || !ws || x_stride < 0 || w_stride < 0 || (residual && residual_stride < 0) ||
        (rows > 1 && (y_stride < h->out || (pre && pre_stride < h->out))))
        return ADACOMP_ERR_INVALID_ARG;
    const uintptr_t e = adacomp::dtype_bytes(h->dtype);
    if (!is_aligned(x, e) || !is_aligned(w, e) || !is_aligned(bias, e) || !is_aligned(residual, e) || !is_aligned(y, e) ||
        !is_aligned(pre, e) || !is_aligned(ws, 16))
        return ADACOMP_ERR_ALIGNMENT;
    if (ws_bytes < adacomp_linear_forward_ws_bytes(h, rows)) return ADACOMP_ERR_WORKSPACE;
    adacomp::LinearArgs a = {};
    a.rows = rows;
    a.in = h->in;
    a.out = h->out;
    a.act = h->act;
    a.waits = h->waits;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.residual = residual;
    a.y = y;
    a.pre = pre;
    a.x_stride = x_stride;
    a.w_stride = w_stride;
    a.residual_stride = residual_stride;
    a.y_stride = y_stride;
    a.pre_stride = pre_stride;
    const cudaError_t err = h->dtype == ADACOMP_BF16 ? adacomp::linear_forward<adacomp::bf16>(a, ws, stream)
                                                     : adacomp::linear_forward<float>(a, ws, stream);
    return adacomp::launch_result(err, stream);
}

adacomp_status adacomp_linear_backward(adacomp_linear_t h, int64_t rows, const void* dy, int64_t dy_stride,
                                       const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                                       const void* pre, int64_t pre_stride, void* dx, int64_t dx_stride, void* dw,
                                       int64_t dw_stride, void* db, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_linear_backward");
    if (!h || rows < 0 || rows >= adacomp::kMostRows) return ADACOMP_ERR_INVALID_ARG;
    if ((!dx && !dw && !db) || !ws) return ADACOMP_ERR_INVALID_ARG;
    if (dw && h->out > 1 && dw_stride < h->in) return ADACOMP_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || dy_stride < 0 || (h->act != ADACOMP_ACT_NONE && (!pre || pre_stride < 0)) ||
                     (dw && (!x || x_stride < 0)) || (dx && (!w || w_stride < 0 || (rows > 1 && dx_stride < h->in)))))
        return ADACOMP_ERR_INVALID_ARG;
    const uintptr_t e = adacomp::dtype_bytes(h->dtype);
    for (const void* p : {dy, x, w, pre, (const void*)dx, (const void*)dw, (const void*)db})
        if (!is_aligned(p, e)) return ADACOMP_ERR_ALIGNMENT;
    if (!is_aligned(ws, 16)) return ADACOMP_ERR_ALIGNMENT;
    if (ws_bytes < adacomp_linear_backward_ws_bytes(h, rows)) return ADACOMP_ERR_WORKSPACE;
    adacomp::LinearArgs a = {};
    a.rows = rows;
    a.in = h->in;
    a.out = h->out;
    a.act = h->act;
    a.waits = h->waits;
    a.dy = dy;
    a.x = x;
    a.w = w;
    a.pre_in = pre;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.dy_stride = dy_stride;
    a.x_stride = x_stride;
    a.w_stride = w_stride;
    a.pre_in_stride = pre_stride;
    a.dx_stride = dx_stride;
    a.dw_stride = dw_stride;
    const cudaError_t err = h->dtype == ADACOMP_BF16 ? adacomp::linear_backward<adacomp::bf16>(a, ws, stream)
                                                     : adacomp::linear_backward<float>(a, ws, stream);
    return adacomp::launch_result(err, stream);
}

adacomp_status adacomp_linear_set_timeout_ns(adacomp_linear_t h, uint64_t timeout_ns)
{
    return h ? adacomp::set_timeout(h->waits, timeout_ns) : ADACOMP_ERR_INVALID_ARG;
}

adacomp_status adacomp_linear_set_fault_injection(adacomp_linear_t h, uint32_t silent_cta)
{
    if (!h) return ADACOMP_ERR_INVALID_ARG;
    h->waits.silent = silent_cta;
    return ADACOMP_OK;
}

void adacomp_linear_free(adacomp_linear_t h) { delete h; }

}  // extern "C"
