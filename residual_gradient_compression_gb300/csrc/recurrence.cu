// The gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t, a_t = sigmoid(z_t),
// forward and backward: kernels and C entry points (adacomp.h).
#include <new>

#include "train_common.cuh"

struct adacomp_recurrence {
    int64_t channels = 0;
    int32_t dtype = ADACOMP_F32;
};

namespace adacomp {
namespace {

constexpr int kRecThreads = 128;
constexpr int kRecChunk = ADACOMP_RECURRENCE_CHUNK;

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

// a = sigmoid(z) and 1 - a = sigmoid(-z), neither formed by a subtraction.
__device__ __forceinline__ void gate(float z, float* a, float* b)
{
    const float e = __expf(-fabsf(z));
    const float r = __fdividef(1.0f, 1.0f + e);
    const float s = e * r;
    *a = z >= 0.0f ? r : s;
    *b = z >= 0.0f ? s : r;
    if (z != z) *a = *b = z;
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

// One thread per channel, step after step.
template <typename T> __global__ void __launch_bounds__(kRecThreads) rec_forward_kernel(const RecArgs p)
{
    ptx::griddep_wait();
    const int64_t i = (int64_t)blockIdx.x * kRecThreads + threadIdx.x;
    if (i >= p.batch * p.channels) return;
    const int64_t b = i / p.channels, c = i - b * p.channels, len = length_of(p, b);
    float h = p.h0 ? p.h0[i] : 0.0f;
    for (int64_t t = 0; t < p.steps; ++t) {
        if (p.carry && t % kRecChunk == 0) p.carry[(b * p.chunks + t / kRecChunk) * p.channels + c] = h;
        if (t < len) {
            float a, r;
            gate(to_f32(*at<T>(p.z, b, t, c)), &a, &r);
            h = a * h + r * to_f32(*at<T>(p.x, b, t, c));
        }
        *at<T>(p.y, b, t, c) = from_f32<T>(t < len ? h : 0.0f);
    }
    if (p.h_last) p.h_last[i] = h;
}

template <typename T> __global__ void __launch_bounds__(kRecThreads) rec_backward_kernel(const RecArgs p)
{
    ptx::griddep_wait();
    const int64_t i = (int64_t)blockIdx.x * kRecThreads + threadIdx.x;
    if (i >= p.batch * p.channels) return;
    const int64_t b = i / p.channels, c = i - b * p.channels, len = length_of(p, b);
    float g = p.dh_last ? p.dh_last[i] : 0.0f;  // the gradient that reaches h_t from the steps after it
    float before[kRecChunk];
    for (int64_t k = p.chunks - 1; k >= 0; --k) {
        const int64_t t0 = k * kRecChunk, t1 = t0 + kRecChunk < p.steps ? t0 + kRecChunk : p.steps;
        float h = p.carry[(b * p.chunks + k) * p.channels + c];
        for (int64_t t = t0; t < t1; ++t) {
            before[t - t0] = h;
            if (t < len) {
                float a, r;
                gate(to_f32(*at<T>(p.z, b, t, c)), &a, &r);
                h = a * h + r * to_f32(*at<T>(p.x, b, t, c));
            }
        }
        for (int64_t t = t1 - 1; t >= t0; --t) {
            float dz = 0.0f, dx = 0.0f;
            if (t < len) {
                float a, r;
                gate(to_f32(*at<T>(p.z, b, t, c)), &a, &r);
                g += to_f32(*at<T>(p.dy, b, t, c));
                dx = r * g;
                dz = a * dx * (before[t - t0] - to_f32(*at<T>(p.x, b, t, c)));
                g *= a;
            }
            *at<T>(p.dz, b, t, c) = from_f32<T>(dz);
            *at<T>(p.dx, b, t, c) = from_f32<T>(dx);
        }
    }
    if (p.dh0) p.dh0[i] = g;
}

bool rec_seq_ok(const RecSeq& s, int64_t batch, int64_t steps, int64_t channels, bool written)
{
    if (!s.p || s.batch < 0 || s.step < 0) return false;
    if (!written) return true;
    return (steps < 2 || s.step >= channels) && (batch < 2 || s.batch >= channels);
}

}  // namespace
}  // namespace adacomp

using adacomp::is_aligned;

extern "C" {

adacomp_status adacomp_recurrence_init(adacomp_recurrence_t* out, int64_t channels, adacomp_dtype dtype)
{
    if (!out) return ADACOMP_ERR_INVALID_ARG;
    *out = nullptr;
    if (channels < 1 || channels > (int64_t)1 << 31 || !adacomp::known_dtype(dtype)) return ADACOMP_ERR_INVALID_ARG;
    adacomp_recurrence* h = new (std::nothrow) adacomp_recurrence;
    if (!h) return ADACOMP_ERR_INVALID_ARG;
    h->channels = channels;
    h->dtype = dtype;
    *out = h;
    return ADACOMP_OK;
}

size_t adacomp_recurrence_carry_bytes(adacomp_recurrence_t h, int64_t batch, int64_t steps)
{
    if (!h || batch < 0 || steps < 0) return 0;
    return (size_t)batch * (size_t)((steps + adacomp::kRecChunk - 1) / adacomp::kRecChunk) * (size_t)h->channels * 4;
}

static adacomp_status rec_sizes(const adacomp_recurrence* h, int64_t batch, int64_t steps)
{
    if (!h || batch < 0 || steps < 0 || batch > 0x7fffffff || steps > 0x7fffffff) return ADACOMP_ERR_INVALID_ARG;
    return ADACOMP_OK;
}

adacomp_status adacomp_recurrence_forward(adacomp_recurrence_t h, int64_t batch, int64_t steps, const void* z,
                                          int64_t z_batch, int64_t z_step, const void* x, int64_t x_batch,
                                          int64_t x_step, const float* h0, const int32_t* lengths, void* y,
                                          int64_t y_batch, int64_t y_step, float* h_last, float* carry,
                                          cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_recurrence_forward");
    const adacomp_status st = rec_sizes(h, batch, steps);
    if (st != ADACOMP_OK || batch == 0) return st;
    adacomp::RecArgs p = {};
    p.z = {const_cast<void*>(z), z_batch, z_step};
    p.x = {const_cast<void*>(x), x_batch, x_step};
    p.y = {y, y_batch, y_step};
    if (steps > 0 && (!adacomp::rec_seq_ok(p.z, batch, steps, h->channels, false) ||
                      !adacomp::rec_seq_ok(p.x, batch, steps, h->channels, false) ||
                      !adacomp::rec_seq_ok(p.y, batch, steps, h->channels, true)))
        return ADACOMP_ERR_INVALID_ARG;
    const uintptr_t e = adacomp::dtype_bytes(h->dtype);
    if (!is_aligned(z, e) || !is_aligned(x, e) || !is_aligned(y, e) || !is_aligned(h0, 4) || !is_aligned(lengths, 4) ||
        !is_aligned(h_last, 4) || !is_aligned(carry, 4))
        return ADACOMP_ERR_ALIGNMENT;
    p.h0 = h0;
    p.lengths = lengths;
    p.h_last = h_last;
    p.carry = carry;
    p.batch = batch;
    p.steps = steps;
    p.channels = h->channels;
    p.chunks = (steps + adacomp::kRecChunk - 1) / adacomp::kRecChunk;
    const int64_t n = batch * h->channels;
    const dim3 grid((unsigned)((n + adacomp::kRecThreads - 1) / adacomp::kRecThreads));
    const cudaError_t err =
        adacomp::launch_after(h->dtype == ADACOMP_BF16 ? adacomp::rec_forward_kernel<adacomp::bf16>
                                                       : adacomp::rec_forward_kernel<float>,
                              grid, dim3(adacomp::kRecThreads), 0, stream, p);
    return adacomp::launch_result(err, stream);
}

adacomp_status adacomp_recurrence_backward(adacomp_recurrence_t h, int64_t batch, int64_t steps, const void* z,
                                           int64_t z_batch, int64_t z_step, const void* x, int64_t x_batch,
                                           int64_t x_step, const void* dy, int64_t dy_batch, int64_t dy_step,
                                           const float* carry, const int32_t* lengths, const float* dh_last,
                                           void* dz, int64_t dz_batch, int64_t dz_step, void* dx, int64_t dx_batch,
                                           int64_t dx_step, float* dh0, cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_recurrence_backward");
    const adacomp_status st = rec_sizes(h, batch, steps);
    if (st != ADACOMP_OK || batch == 0) return st;
    adacomp::RecArgs p = {};
    p.z = {const_cast<void*>(z), z_batch, z_step};
    p.x = {const_cast<void*>(x), x_batch, x_step};
    p.dy = {const_cast<void*>(dy), dy_batch, dy_step};
    p.dz = {dz, dz_batch, dz_step};
    p.dx = {dx, dx_batch, dx_step};
    if (steps > 0 && (!carry || !adacomp::rec_seq_ok(p.z, batch, steps, h->channels, false) ||
                      !adacomp::rec_seq_ok(p.x, batch, steps, h->channels, false) ||
                      !adacomp::rec_seq_ok(p.dy, batch, steps, h->channels, false) ||
                      !adacomp::rec_seq_ok(p.dz, batch, steps, h->channels, true) ||
                      !adacomp::rec_seq_ok(p.dx, batch, steps, h->channels, true)))
        return ADACOMP_ERR_INVALID_ARG;
    const uintptr_t e = adacomp::dtype_bytes(h->dtype);
    if (!is_aligned(z, e) || !is_aligned(x, e) || !is_aligned(dy, e) || !is_aligned(dz, e) || !is_aligned(dx, e) ||
        !is_aligned(carry, 4) || !is_aligned(lengths, 4) || !is_aligned(dh_last, 4) || !is_aligned(dh0, 4))
        return ADACOMP_ERR_ALIGNMENT;
    p.carry = const_cast<float*>(carry);
    p.lengths = lengths;
    p.dh_last = dh_last;
    p.dh0 = dh0;
    p.batch = batch;
    p.steps = steps;
    p.channels = h->channels;
    p.chunks = (steps + adacomp::kRecChunk - 1) / adacomp::kRecChunk;
    const int64_t n = batch * h->channels;
    const dim3 grid((unsigned)((n + adacomp::kRecThreads - 1) / adacomp::kRecThreads));
    const cudaError_t err =
        adacomp::launch_after(h->dtype == ADACOMP_BF16 ? adacomp::rec_backward_kernel<adacomp::bf16>
                                                       : adacomp::rec_backward_kernel<float>,
                              grid, dim3(adacomp::kRecThreads), 0, stream, p);
    return adacomp::launch_result(err, stream);
}

void adacomp_recurrence_free(adacomp_recurrence_t h) { delete h; }

}  // extern "C"
