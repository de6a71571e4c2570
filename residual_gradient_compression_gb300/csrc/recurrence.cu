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
constexpr int kRecFew = 4;  // steps up to which a thread takes all of them
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

// ---------------------------------------------------------------- few steps
// One thread per column (a channel of a sequence), step after step.
template <typename T> __global__ void __launch_bounds__(kRecThreads) rec_forward_few_kernel(const RecArgs p)
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
            h = fmaf(a, h, r * to_f32(*at<T>(p.x, b, t, c)));
        }
        *at<T>(p.y, b, t, c) = from_f32<T>(t < len ? h : 0.0f);
    }
    if (p.h_last) p.h_last[i] = h;
}

// ---------------------------------------------------------------- many steps
// The steps are split: a warp has 32 columns and S consecutive steps, a CTA one chunk of
// 128 steps, a cluster of up to eight CTAs consecutive chunks, and where the sequence is
// longer than that the cluster goes on in rounds. Each warp forms what its steps do to a
// state, h -> A h + H with A the product of its gates; the CTA's warps exchange these
// through shared memory and the cluster's CTAs through each other's; then each warp knows
// the state before its first step and goes through its steps again, from registers. So
// every element is read once, and no CTA waits for one that may not be running. The split
// depends on the number of steps alone.
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A float2 of this CTA's shared memory, as it lies in the CTA `rank` of the cluster.
__device__ __forceinline__ float2 remote(const float2* p, uint32_t rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

struct Column {
    bool on;
    int64_t i, b, c;
    int64_t len;

    __device__ __forceinline__ Column(const RecArgs& p, uint32_t tile)
    {
        i = (int64_t)tile * 32 + (threadIdx.x & 31);
        on = i < p.batch * p.channels;
        if (!on) i = 0;
        b = i / p.channels;
        c = i - b * p.channels;
        len = on ? length_of(p, b) : 0;
    }
};

constexpr int kForwardSteps = 16, kForwardCtas = 3;

template <typename T, int S>
__global__ void __launch_bounds__(32 * kRecChunk / S, kForwardCtas) rec_forward_kernel(const RecArgs p, const uint32_t ranks)
{
    constexpr int kWarpsPer = kRecChunk / S;
    __shared__ float2 part[2][kWarpsPer][32];  // a warp's (A, H), by the round's parity
    __shared__ float2 total[2][32];            // and the CTA's
    ptx::griddep_wait();
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Column col(p, blockIdx.x / ranks);
    float h0 = p.h0 && col.on ? p.h0[col.i] : 0.0f;  // before the round's first step
    int par = 0;
    for (int64_t t0 = 0; t0 < p.steps; t0 += (int64_t)ranks * kRecChunk, par ^= 1) {
        const int64_t ts = t0 + rank * kRecChunk + warp * S;
        const int live = (int)(col.len - ts < 0 ? 0 : col.len - ts > S ? S : col.len - ts);
        const int whole = !col.on || p.steps <= ts ? 0 : (int)(p.steps - ts > S ? S : p.steps - ts);
        T zr[S], xr[S];
        {
            const T* z = at<T>(p.z, col.b, ts, col.c);
            const T* x = at<T>(p.x, col.b, ts, col.c);
#pragma unroll
            for (int k = 0; k < S; ++k, z += p.z.step, x += p.x.step)
                if (k < live) {
                    zr[k] = *z;
                    xr[k] = *x;
                }
        }
        float a[S], u[S], A = 1.0f, H = 0.0f;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            a[k] = 1.0f;
            u[k] = 0.0f;
            if (k < live) {
                float r;
                gate(to_f32(zr[k]), &a[k], &r);
                u[k] = r * to_f32(xr[k]);
            }
            H = fmaf(a[k], H, u[k]);
            A *= a[k];
        }
        part[par][warp][lane] = make_float2(A, H);
        __syncthreads();
        A = 1.0f;
        H = 0.0f;
        for (int w = 0; w < warp; ++w) {
            const float2 q = part[par][w][lane];
            H = fmaf(q.x, H, q.y);
            A *= q.x;
        }
        float hc = h0;  // before the CTA's first step
        if (ranks > 1) {
            if (warp == kWarpsPer - 1) {
                const float2 q = part[par][warp][lane];
                total[par][lane] = make_float2(A * q.x, fmaf(q.x, H, q.y));
            }
            cluster_sync();
            for (uint32_t r = 0; r < ranks; ++r) {
                if (r == rank) hc = h0;
                const float2 q = remote(&total[par][lane], r);
                h0 = fmaf(q.x, h0, q.y);
            }
        } else {
            float e = h0;
            for (int w = 0; w < kWarpsPer; ++w) {
                const float2 q = part[par][w][lane];
                e = fmaf(q.x, e, q.y);
            }
            h0 = e;
        }
        float h = fmaf(A, hc, H);
        if (p.carry && warp == 0 && whole > 0)
            p.carry[(col.b * p.chunks + ts / kRecChunk) * p.channels + col.c] = h;
        T* y = at<T>(p.y, col.b, ts, col.c);
#pragma unroll
        for (int k = 0; k < S; ++k, y += p.y.step) {
            h = fmaf(a[k], h, u[k]);
            if (k < whole) *y = from_f32<T>(k < live ? h : 0.0f);
        }
    }
    if (p.h_last && col.on && rank == 0 && warp == 0) p.h_last[col.i] = h0;
    if (ranks > 1) cluster_sync();  // the others may still read this CTA's totals
}

// The reverse of it: p, the gradient that reaches a state from the steps after it, goes
// through a warp's steps as p -> A p + P, P = sum of dy_k times the gates up to and with
// step k. The states are formed again from the chunk's first one, which the forward pass
// kept: that is less to read than y, and not rounded.
constexpr int kBackwardSteps = 16, kBackwardCtas = 2;

template <typename T, int S>
__global__ void __launch_bounds__(32 * kRecChunk / S, kBackwardCtas) rec_backward_kernel(const RecArgs p, const uint32_t ranks)
{
    constexpr int kWarpsPer = kRecChunk / S;
    __shared__ float2 part[2][kWarpsPer][32];  // a warp's (A, H), by the round's parity
    __shared__ float grad[2][kWarpsPer][32];   // its P
    __shared__ float2 total[2][32];            // the CTA's (A, P)
    ptx::griddep_wait();
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Column col(p, blockIdx.x / ranks);
    float p0 = p.dh_last && col.on ? p.dh_last[col.i] : 0.0f;  // after the round's last step
    const int64_t span = (int64_t)ranks * kRecChunk;
    int par = 0;
    for (int64_t t0 = (p.steps - 1) / span * span; t0 >= 0; t0 -= span, par ^= 1) {
        const int64_t tc = t0 + rank * kRecChunk, ts = tc + warp * S;
        const int live = (int)(col.len - ts < 0 ? 0 : col.len - ts > S ? S : col.len - ts);
        const int whole = !col.on || p.steps <= ts ? 0 : (int)(p.steps - ts > S ? S : p.steps - ts);
        T zr[S], xr[S], dr[S];
        {
            const T* z = at<T>(p.z, col.b, ts, col.c);
            const T* x = at<T>(p.x, col.b, ts, col.c);
            const T* d = at<T>(p.dy, col.b, ts, col.c);
#pragma unroll
            for (int k = 0; k < S; ++k, z += p.z.step, x += p.x.step, d += p.dy.step)
                if (k < live) {
                    zr[k] = *z;
                    xr[k] = *x;
                    dr[k] = *d;
                }
        }
        float hc = col.on && tc < p.steps ? p.carry[(col.b * p.chunks + tc / kRecChunk) * p.channels + col.c] : 0.0f;
        float a[S], b[S], x[S], g[S], A = 1.0f, H = 0.0f, P = 0.0f;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            a[k] = 1.0f;
            b[k] = x[k] = g[k] = 0.0f;
            if (k < live) {
                gate(to_f32(zr[k]), &a[k], &b[k]);
                x[k] = to_f32(xr[k]);
                g[k] = to_f32(dr[k]);
            }
            H = fmaf(a[k], H, b[k] * x[k]);
            A *= a[k];
            P = fmaf(A, g[k], P);
        }
        part[par][warp][lane] = make_float2(A, H);
        grad[par][warp][lane] = P;
        __syncthreads();
        float h = hc;
        for (int w = 0; w < warp; ++w) {
            const float2 q = part[par][w][lane];
            h = fmaf(q.x, h, q.y);
        }
        float Pa = 1.0f, Pp = 0.0f;  // from after the CTA's last step to after the warp's
        for (int w = kWarpsPer - 1; w > warp; --w) {
            const float q = part[par][w][lane].x;
            Pp = fmaf(q, Pp, grad[par][w][lane]);
            Pa *= q;
        }
        float pc = p0;  // after the CTA's last step
        if (ranks > 1) {
            if (warp == 0) total[par][lane] = make_float2(A * Pa, fmaf(A, Pp, P));
            cluster_sync();
            for (uint32_t r = ranks; r-- > 0;) {
                if (r == rank) pc = p0;
                const float2 q = remote(&total[par][lane], r);
                p0 = fmaf(q.x, p0, q.y);
            }
        } else {
            float e = p0;
            for (int w = kWarpsPer - 1; w >= 0; --w) e = fmaf(part[par][w][lane].x, e, grad[par][w][lane]);
            p0 = e;
        }
        float before[S];
#pragma unroll
        for (int k = 0; k < S; ++k) {
            before[k] = h;
            h = fmaf(a[k], h, b[k] * x[k]);
        }
        float q = fmaf(Pa, pc, Pp);
        T* dz = at<T>(p.dz, col.b, ts + (S - 1), col.c);
        T* dx = at<T>(p.dx, col.b, ts + (S - 1), col.c);
#pragma unroll
        for (int k = S - 1; k >= 0; --k, dz -= p.dz.step, dx -= p.dx.step) {
            const float G = g[k] + q, d = b[k] * G;
            if (k < whole) {
                *dx = from_f32<T>(k < live ? d : 0.0f);
                *dz = from_f32<T>(k < live ? a[k] * d * (before[k] - x[k]) : 0.0f);
            }
            q = a[k] * G;
        }
    }
    if (p.dh0 && col.on && rank == 0 && warp == 0) p.dh0[col.i] = p0;
    if (ranks > 1) cluster_sync();  // the others may still read this CTA's totals
}

// Launches a kernel of clusters, behind the kernel ahead of it as launch_after does.
cudaError_t launch_ranks(void (*kern)(RecArgs, uint32_t), int threads, const RecArgs& p, cudaStream_t stream)
{
    uint32_t ranks = 1;
    while (ranks < 8 && (int64_t)ranks * kRecChunk < p.steps) ranks *= 2;
    const int64_t tiles = (p.batch * p.channels + 31) / 32;
    if (tiles > 0x7fffffff / ranks) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * ranks));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, ranks);
}

template <typename T> cudaError_t forward(const RecArgs& p, cudaStream_t stream)
{
    const int64_t n = p.batch * p.channels;
    if (p.steps <= kRecFew) {
        if (n > (int64_t)0x7fffffff * kRecThreads) return cudaErrorInvalidConfiguration;
        return launch_after(rec_forward_few_kernel<T>, dim3((unsigned)((n + kRecThreads - 1) / kRecThreads)),
                            dim3(kRecThreads), 0, stream, p);
    }
    return launch_ranks(rec_forward_kernel<T, kForwardSteps>, 32 * kRecChunk / kForwardSteps, p, stream);
}

template <typename T> cudaError_t backward(const RecArgs& p, cudaStream_t stream)
{
    return launch_ranks(rec_backward_kernel<T, kBackwardSteps>, 32 * kRecChunk / kBackwardSteps, p, stream);
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
    const cudaError_t err = h->dtype == ADACOMP_BF16 ? adacomp::forward<adacomp::bf16>(p, stream)
                                                     : adacomp::forward<float>(p, stream);
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
    const cudaError_t err = h->dtype == ADACOMP_BF16 ? adacomp::backward<adacomp::bf16>(p, stream)
                                                     : adacomp::backward<float>(p, stream);
    return adacomp::launch_result(err, stream);
}

void adacomp_recurrence_free(adacomp_recurrence_t h) { delete h; }

}  // extern "C"
