// The gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t, a_t = sigmoid(z_t),
// forward and backward: kernels and C entry points (adacomp.h).
#include <initializer_list>
#include <new>

#include "recurrence.cuh"

struct adacomp_recurrence {
    int64_t channels = 0;
    int32_t dtype = ADACOMP_F32;
    uint64_t timeout_ns = 2000000000ull;
    uint32_t inject_silent_cta = 0xffffffffu;  // test-only fault injection
};

namespace adacomp {
namespace {

constexpr int kRecThreads = 128;
// Steps up to which a thread takes all of a column's, and those up to which it does so where there
// are many columns; the backward pass keeps them in registers (300 x 20 x 1000 fp32: 35 us, by
// warps 50; but bf16 32 and 21).
constexpr int kRecFew = 4, kRecSome = 32;
template <typename T> constexpr int kRecSomeBack = sizeof(T) == 4 ? 32 : 16;
constexpr int64_t kRecColumns = 152 * 128;

// ---------------------------------------------------------------- few steps
// One thread per column (a channel of a sequence), step after step; bound by memory where there
// are many. A warp for 32 columns, as below, has a CTA of its own for so few steps, and the
// CTAs' starts are what that waits for. us with this and with that, forward and backward:
// 135 x 11 x 2833 fp32 10 and 15, 38 and 52; 1000 x 4 x 1024 fp32 13 and 13, backward 136;
// 100 x 16 x 4096 fp32 13 and 28, 22 and 60; forward 100 x 32 x 4096 fp32 34 and 36, 100 x 64 x
// 4096 63 and 58.
template <typename T> __global__ void __launch_bounds__(kRecThreads) rec_forward_few_kernel(const RecArgs p)
{
    ptx::griddep_wait();
    const int64_t i = (int64_t)blockIdx.x * kRecThreads + threadIdx.x;
    if (i >= p.batch * p.channels) return;
    const int64_t b = i / p.channels, c = i - b * p.channels, len = length_of(p, b);
    float h = p.h0 ? p.h0[i] : 0.0f;
    constexpr int S = 4;  // steps' loads on their way
    const T* z = at<const T>(p.z, b, 0, c);
    const T* x = at<const T>(p.x, b, 0, c);
    T* y = at<T>(p.y, b, 0, c);
    for (int64_t t0 = 0; t0 < p.steps; t0 += S) {
        T zv[S], xv[S];
#pragma unroll
        for (int k = 0; k < S; ++k)
            if (t0 + k < len) {
                zv[k] = z[(t0 + k) * p.z.step];
                xv[k] = x[(t0 + k) * p.x.step];
            }
        if (p.carry && t0 % kRecChunk == 0) p.carry[(b * p.chunks + t0 / kRecChunk) * p.channels + c] = h;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            if (t0 + k < len) {
                float a, r;
                gate(to_f32(zv[k]), &a, &r);
                h = fmaf(a, h, r * to_f32(xv[k]));
            }
            if (t0 + k < p.steps) y[(t0 + k) * p.y.step] = from_f32<T>(t0 + k < len ? h : 0.0f);
        }
    }
    if (p.h_last) p.h_last[i] = h;
}

template <typename T, int S> __global__ void __launch_bounds__(kRecThreads) rec_backward_few_kernel(const RecArgs p)
{
    ptx::griddep_wait();
    const int64_t i = (int64_t)blockIdx.x * kRecThreads + threadIdx.x;
    if (i >= p.batch * p.channels) return;
    const int64_t b = i / p.channels, c = i - b * p.channels;
    const int len = (int)length_of(p, b), steps = (int)p.steps;
    const T* z = at<const T>(p.z, b, 0, c);
    const T* x = at<const T>(p.x, b, 0, c);
    const T* dy = at<const T>(p.dy, b, 0, c);
    float h = p.carry[b * p.chunks * p.channels + c], q = p.dh_last ? p.dh_last[i] : 0.0f;
    T zv[S], xv[S], dv[S];
#pragma unroll
    for (int k = 0; k < S; ++k)
        if (k < len) {
            zv[k] = z[k * p.z.step];
            xv[k] = x[k * p.x.step];
            dv[k] = dy[k * p.dy.step];
        }
    float a[S], r[S], before[S];  // before: h_{t-1} - x_t
#pragma unroll
    for (int k = 0; k < S; ++k)
        if (k < len) {
            gate(to_f32(zv[k]), &a[k], &r[k]);
            const float v = to_f32(xv[k]);
            before[k] = h - v;
            h = fmaf(a[k], h, r[k] * v);
        }
    T* dz = at<T>(p.dz, b, 0, c);
    T* dx = at<T>(p.dx, b, 0, c);
#pragma unroll
    for (int k = S - 1; k >= 0; --k) {
        if (k >= steps) continue;
        float gx = 0.0f, gz = 0.0f;
        if (k < len) {
            const float G = __fadd_rn(q, to_f32(dv[k]));
            gx = r[k] * G;
            gz = a[k] * gx * before[k];
            q = __fmul_rn(a[k], G);
        }
        dx[k * p.dx.step] = from_f32<T>(gx);
        dz[k * p.dz.step] = from_f32<T>(gz);
    }
    if (p.dh0) p.dh0[i] = q;
}

// ---------------------------------------------------------------- many steps
// A warp has 32 or 64 columns and some consecutive steps, a chunk, and the warps of a CTA take
// the chunks of their columns in turn. Each forms from its elements alone what its steps do to
// a state, h -> A h + H with A the product of its gates; then it waits for the state before its
// first step from the warp that has the chunk before, hands A h + H on to the next at once, and
// goes through its steps again, from registers. So every element is read once, the chain
// through the sequence is one fused multiply-add and one hand-over per chunk, and no warp waits
// for one that may not be running. A hand-over is a named barrier of the two warps. The warp's
// next chunk is copied to shared memory meanwhile.
//
// Bound by memory and, in bf16, nearly as much by instructions (23 per element forward, 45
// backward). Measured over 16 sequences of 2048 steps and 1024 channels: forward 35 us in bf16
// (5.7 TB/s) and 65 in fp32 (6.2), backward 73 (4.6) and 104 (6.4). Rows that are not aligned
// to 16 bytes: with 1023 channels 59 and 112 us in bf16, 78 and 146 in fp32; there each row's
// place in its 16 bytes is found again for every tensor, and its results are written one by one.
constexpr int kWarps = 8;

__device__ __forceinline__ void hand_on(int barrier)
{
    __syncwarp();
    asm volatile("bar.arrive %0, 64;" ::"r"(barrier) : "memory");
}

__device__ __forceinline__ void take_over(int barrier)
{
    __syncwarp();
    asm volatile("bar.sync %0, 64;" ::"r"(barrier) : "memory");
}

// A column of a tile.
template <int kBytes, int kCols> struct Column {
    int64_t b, c;
    int32_t len;  // of its sequence; 0 past the last column
    bool on;

    __device__ __forceinline__ Column(const RecArgs& p, uint32_t tile, int j)
    {
        if (kApart<kBytes>) {
            const uint32_t blocks = (uint32_t)((p.channels + kCols - 1) / kCols);
            b = tile / blocks;
            c = (int64_t)(tile - (uint32_t)b * blocks) * kCols + j;
            on = c < p.channels;
        } else {
            const int64_t i = (int64_t)tile * kCols + j;
            on = i < p.batch * p.channels;
            b = on ? i / p.channels : 0;
            c = on ? i - b * p.channels : 0;
        }
        len = on ? (int32_t)length_of(p, b) : 0;
    }
    __device__ __forceinline__ int64_t state(const RecArgs& p) const { return b * p.channels + c; }
    __device__ __forceinline__ int64_t kept(const RecArgs& p, int32_t t) const
    {
        return (b * p.chunks + t / kRecChunk) * p.channels + c;
    }
};

// Copies a warp's chunk of kTensors tensors to shared memory, [tensor][step][column], kBytes
// at a time: every lane has one place in the rows and takes every kStride-th of them. What
// lies past a sequence's length or the last channel is not read, and what stands there not used.
template <typename T, int kBytes, int kCols, int kChunk, int kTensors> struct Copier {
    static constexpr int kPlaces = kCols * (int)sizeof(T) / kBytes;
    static constexpr int kStride = 32 / kPlaces < kChunk ? 32 / kPlaces : kChunk;
    static constexpr int kEach = kBytes / (int)sizeof(T);  // elements at a time
    static constexpr int kPitch = kCols;
    static constexpr int kElements = kChunk * kPitch;      // of one tensor
    static_assert(kPlaces <= 32 && kChunk % kStride == 0, "whole rows");
    const T* from[kTensors];
    Distance<kBytes> step[kTensors];
    int32_t len;
    uint32_t bytes;

    __device__ __forceinline__ Copier(const RecArgs& p, uint32_t tile, const RecSeq* const (&s)[kTensors])
    {
        const int lane = threadIdx.x & 31;
        const Column<kBytes, kCols> col(p, tile, lane % kPlaces * kEach);
        const int64_t rest = (p.channels - col.c) * (int)sizeof(T);
        bytes = !col.on ? 0u : rest < kBytes ? (uint32_t)rest : (uint32_t)kBytes;
        len = bytes == 0 ? 0 : col.len;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            from[i] = at<const T>(*s[i], col.b, 0, col.c);
            step[i] = (Distance<kBytes>)(s[i]->step * (int)sizeof(T));
        }
    }

    __device__ __forceinline__ void copy(T* to, int32_t t0) const
    {
        const int lane = threadIdx.x & 31, row0 = lane / kPlaces;
        const int left = row0 < kChunk ? len - t0 - row0 : 0;  // the other lanes have no place
        T* const place = to + row0 * kCols + lane % kPlaces * kEach;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            const T* const f = moved(from[i], (int64_t)(t0 + row0) * step[i]);
            T v[kChunk / kStride];
#pragma unroll
            for (int k = 0; k < kChunk / kStride; ++k)
                if (k * kStride < left) {
                    const T* const g = moved(f, (Distance<kBytes>)(k * kStride) * step[i]);
                    const uint32_t d = (uint32_t)__cvta_generic_to_shared(place + i * kElements + k * kStride * kCols);
                    if constexpr (kBytes == 2) v[k] = *g;
                    else if constexpr (kBytes == 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(g), "r"(bytes)
                                     : "memory");
                    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(g) : "memory");
                }
            if constexpr (kBytes == 2) {
#pragma unroll
                for (int k = 0; k < kChunk / kStride; ++k)
                    if (k * kStride < left) place[i * kElements + k * kStride * kCols] = v[k];
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

// Rows without alignment, by the aligned 16 bytes that hold them (a copy of four bytes costs as
// much as one of 16): the first and the last of these may hold a neighbour's elements too, and a
// row's first element lies `before` bytes into its place.
template <typename T, int kBytes, int kCols, int kChunk, int kTensors> struct CopierOff {
    static constexpr int kGranules = (kCols * (int)sizeof(T) + 16 - (int)sizeof(T) + 15) / 16;  // of a row, at most
    static constexpr int kPitch = kGranules * 16 / (int)sizeof(T);
    static constexpr int kElements = kChunk * kPitch;
    const T* from[kTensors];
    int32_t step[kTensors];
    int32_t len, bytes;

    __device__ __forceinline__ CopierOff(const RecArgs& p, uint32_t tile, const RecSeq* const (&s)[kTensors])
    {
        const Column<kBytes, kCols> col(p, tile, 0);
        const int64_t rest = p.channels - col.c;
        bytes = (rest < kCols ? (int32_t)rest : kCols) * (int)sizeof(T);
        len = col.len;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            from[i] = at<const T>(*s[i], col.b, 0, col.c);
            step[i] = (int32_t)s[i]->step * (int)sizeof(T);
        }
    }

    __device__ __forceinline__ void copy(T* to, int32_t t0) const
    {
        const int lane = threadIdx.x & 31, left = len - t0;
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(to) + lane * 16;
#pragma unroll
        for (int k = 0; k < (kChunk * kGranules + 31) / 32; ++k) {
            const int row = (k * 32 + lane) / kGranules, place = (k * 32 + lane - row * kGranules) * 16;
            if (row >= left || row >= kChunk) continue;
#pragma unroll
            for (int i = 0; i < kTensors; ++i) {
                const uintptr_t g = reinterpret_cast<uintptr_t>(from[i]) + (int64_t)(t0 + row) * step[i];
                const int before = (int)(g & 15), n = min(16, before + bytes - place);
                if (n > 0)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     d + i * kElements * (int)sizeof(T) + k * 512),
                                 "l"(g - before + place), "r"(n)
                                 : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

template <typename T, int kBytes, int kCols, int kChunk, int kTensors>
using CopierOf = typename std::conditional<kBytes < 0, CopierOff<T, kBytes, kCols, kChunk, kTensors>,
                                           Copier<T, kBytes < 0 ? 4 : kBytes, kCols, kChunk, kTensors>>::type;

// How many bytes lie before a row's first element in its place: none, but in rows without alignment.
template <int kBytes, typename Copy> __device__ __forceinline__ uint32_t before(const Copy& c, int tensor, int32_t t)
{
    if constexpr (kBytes < 0)
        return ((uint32_t)reinterpret_cast<uintptr_t>(c.from[tensor]) + (uint32_t)t * (uint32_t)c.step[tensor]) & 15;
    else return 0;
}

__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();  // the other lanes' too, and their reads of what is copied over next
}

// h -> A h + H, or the gradient's p -> A p + H.
struct Step {
    float A, H;
};

// kV neighbouring values of a row.
template <int kV> __device__ __forceinline__ void values(const float* p, float (&v)[kV])
{
    if constexpr (kV == 2) {
        const float2 q = *reinterpret_cast<const float2*>(p);
        v[0] = q.x, v[1] = q.y;
    } else {
        v[0] = *p;
    }
}

template <int kV> __device__ __forceinline__ void values(const bf16* p, float (&v)[kV])
{
    if constexpr (kV == 2) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(p);
        v[0] = bf16_low(q), v[1] = bf16_high(q);
    } else {
        v[0] = to_f32(*p);
    }
}

template <int kV> __device__ __forceinline__ void put(float* p, const float (&v)[kV])
{
    if constexpr (kV == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else *p = v[0];
}

template <int kV> __device__ __forceinline__ void put(bf16* p, const float (&v)[kV])
{
    if constexpr (kV == 2) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
    else *p = from_f32<bf16>(v[0]);
}

// kV: columns of a lane, two where rows are read 16 bytes at a time and there are many.
constexpr int kForward = 16;  // steps of a chunk

template <typename T, int kBytes, int kV>
__global__ void __launch_bounds__(32 * kWarps, kV == 2 ? 2 : 4) rec_forward_kernel(const __grid_constant__ RecArgs p)
{
    constexpr int kCols = 32 * kV, S = kForward;
    static_assert(kV == 1 || kBytes == 16, "neighbours lie in one row");
    using Copy = CopierOf<T, kBytes, kCols, S, 2>;
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    __shared__ __align__(8) float state[kWarps][kCols];  // after a warp's chunk; a lane's columns at a time
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, j = lane * kV;
    T* const ring = reinterpret_cast<T*>(shared_bytes) + warp * (4 * Copy::kElements);  // two chunks
    const Column<kBytes, kCols> col(p, blockIdx.x, j);
    const int on = !col.on ? 0 : kV == 2 && col.c + 1 < p.channels ? 2 : 1;  // of the lane's columns
    const Copy copier(p, blockIdx.x, {&p.z, &p.x});
    const Distance<kBytes> step = (Distance<kBytes>)(p.y.step * (int)sizeof(T));
    const int32_t steps = (int32_t)p.steps, turn = warps * S;
    const int prev = warp == 0 ? warps - 1 : warp - 1;
    int32_t t0 = warp * S;
    if (t0 < steps) copier.copy(ring, t0);
    for (int slot = 0; t0 < steps; t0 += turn, slot ^= 1) {
        copies_wait();
        if (t0 + turn < steps) copier.copy(ring + (slot ^ 1) * (2 * Copy::kElements), t0 + turn);
        const T* const first = ring + slot * (2 * Copy::kElements) + j;
        const auto place = [&](int tensor, int k) {  // step k's
            return moved(first + tensor * Copy::kElements + k * Copy::kPitch, before<kBytes>(copier, tensor, t0 + k));
        };
        const int32_t live = col.len - t0;
        const bool all = __all_sync(0xffffffffu, (live >= S && on == kV) || (kBytes < 0 && on == 0));
        float a[S][kV], u[S][kV], h[kV], after[kV];
        Step own[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) own[v] = {1.0f, 0.0f};
        const auto form = [&](auto masked) {
#pragma unroll
            for (int k = 0; k < S; ++k) {
                float zv[kV], xv[kV];
                values(place(0, k), zv);
                values(place(1, k), xv);
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    float r;
                    gate(zv[v], &a[k][v], &r);
                    u[k][v] = r * xv[v];
                    if (masked.value && k >= live) a[k][v] = 1.0f, u[k][v] = 0.0f;  // past the length the state stays
                    own[v].H = fmaf(a[k][v], own[v].H, u[k][v]);
                    own[v].A *= a[k][v];
                }
            }
        };
        if (all) form(std::false_type());
        else form(std::true_type());
#pragma unroll
        for (int v = 0; v < kV; ++v) {  // as product() of them all
            float least = kLeast;
#pragma unroll
            for (int k = 0; k < S; k += 2) least = least3(least, a[k][v], a[k + 1][v]);
            own[v].A = not_below(own[v].A, least);
        }
        if (t0 == 0) {
#pragma unroll
            for (int v = 0; v < kV; ++v) h[v] = p.h0 && v < on ? p.h0[col.state(p) + v] : 0.0f;
        } else {
            take_over(1 + prev);
            values(&state[prev][j], h);
        }
#pragma unroll
        for (int v = 0; v < kV; ++v) after[v] = fmaf(own[v].A, h[v], own[v].H);
        if (t0 + S < steps) {
            put(&state[warp][j], after);
            hand_on(1 + warp);
        } else if (p.h_last) {
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (v < on) p.h_last[col.state(p) + v] = after[v];
        }
        if (p.carry && t0 % kRecChunk == 0) {
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (v < on) p.carry[col.kept(p, t0) + v] = h[v];
        }
        T* const y = at<T>(p.y, col.b, t0, col.c);
        if (all) {
#pragma unroll
            for (int k = 0; k < S; ++k) {
#pragma unroll
                for (int v = 0; v < kV; ++v) h[v] = fmaf(a[k][v], h[v], u[k][v]);
                if (kBytes > 0 || on) put(moved(y, k * step), h);
            }
        } else {
#pragma unroll
            for (int k = 0; k < S; ++k)
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    h[v] = fmaf(a[k][v], h[v], u[k][v]);
                    if (v < on && t0 + k < steps) moved(y, k * step)[v] = from_f32<T>(k < live ? h[v] : 0.0f);
                }
        }
    }
}

// The reverse of it: p, the gradient that reaches a state from the steps after it, goes
// through a chunk as p -> A p + P, P = sum of dy_k times the gates up to and with step k. A
// CTA's warps have the chunks of a kept state at a time, and form the states again from it
// (handed on from the first to the last of them): that is less to read than y, and not rounded.
template <int kV> constexpr int kBackward = kV == 2 ? 8 : 16;  // steps of a chunk
template <int kV> constexpr int kBackWarps = kRecChunk / kBackward<kV>;
static_assert(kBackWarps<2> <= 8, "fifteen named barriers");

template <typename T, int kBytes, int kV>
__global__ void __launch_bounds__(32 * kBackWarps<kV>, kV == 2 ? 2 : kBytes == 16 ? 6 : 5) rec_backward_kernel(const __grid_constant__ RecArgs p)
{
    constexpr int kCols = 32 * kV, S = kBackward<kV>, W = kBackWarps<kV>;
    using Copy = CopierOf<T, kBytes, kCols, S, 3>;
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    __shared__ __align__(8) float state[W][kCols];  // after a warp's chunk; a lane's columns at a time
    __shared__ __align__(8) float grad[W][kCols];   // the gradient before it
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane * kV;
    T* const ring = reinterpret_cast<T*>(shared_bytes) + warp * (6 * Copy::kElements);  // two chunks
    const Column<kBytes, kCols> col(p, blockIdx.x, j);
    const int on = !col.on ? 0 : kV == 2 && col.c + 1 < p.channels ? 2 : 1;  // of the lane's columns
    const Copy copier(p, blockIdx.x, {&p.z, &p.x, &p.dy});
    const Distance<kBytes> step_z = (Distance<kBytes>)(p.dz.step * (int)sizeof(T));
    const Distance<kBytes> step_x = (Distance<kBytes>)(p.dx.step * (int)sizeof(T));
    const int32_t steps = (int32_t)p.steps;
    const int next = warp == W - 1 ? 0 : warp + 1;  // has the chunk after this warp's
    if (steps == 0) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (p.dh0 && warp == 0 && v < on) p.dh0[col.state(p) + v] = p.dh_last ? p.dh_last[col.state(p) + v] : 0.0f;
        return;
    }
    // the last of the warp's chunks, if it has one
    int32_t t0 = (steps - 1) / kRecChunk * kRecChunk + warp * S;
    if (t0 >= steps) t0 -= kRecChunk;
    if (t0 >= 0) copier.copy(ring, t0);
    for (int slot = 0; t0 >= 0; t0 -= kRecChunk, slot ^= 1) {
        float h[kV], q[kV];  // before the chunk's first step, and after its last
#pragma unroll
        for (int v = 0; v < kV; ++v) h[v] = warp == 0 && v < on ? p.carry[col.kept(p, t0) + v] : 0.0f;
        copies_wait();
        if (t0 >= kRecChunk) copier.copy(ring + (slot ^ 1) * (3 * Copy::kElements), t0 - kRecChunk);
        const T* const first = ring + slot * (3 * Copy::kElements) + j;
        const auto place = [&](int tensor, int k) {  // step k's
            return moved(first + tensor * Copy::kElements + k * Copy::kPitch, before<kBytes>(copier, tensor, t0 + k));
        };
        const int32_t live = col.len - t0;
        const bool all = __all_sync(0xffffffffu, (live >= S && on == kV) || (kBytes < 0 && on == 0));
        float a[S][kV], b[S][kV], from_x[S][kV];  // from_x: x_t, later h_{t-1} - x_t
        Step own[kV];
        float P[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) own[v] = {1.0f, 0.0f}, P[v] = 0.0f;
        const auto form = [&](auto masked) {
#pragma unroll
            for (int k = 0; k < S; ++k) {
                float zv[kV], dv[kV];
                values(place(0, k), zv);
                values(place(1, k), from_x[k]);
                values(place(2, k), dv);
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    gate(zv[v], &a[k][v], &b[k][v]);
                    if (masked.value && k >= live) a[k][v] = 1.0f, b[k][v] = from_x[k][v] = dv[v] = 0.0f;
                    own[v].H = fmaf(a[k][v], own[v].H, b[k][v] * from_x[k][v]);
                    own[v].A = product(own[v].A, a[k][v]);
                    P[v] = fmaf(own[v].A, dv[v], P[v]);
                }
            }
        };
        if (all) form(std::false_type());
        else form(std::true_type());
        // The gradient's hand-over comes first, so that the next kept state's last warp, which
        // starts from it, has it soon; a warp's next hand-overs wait for one that follows them.
        if (t0 + S >= steps) {
#pragma unroll
            for (int v = 0; v < kV; ++v) q[v] = p.dh_last && v < on ? p.dh_last[col.state(p) + v] : 0.0f;
        } else {
            take_over(8 + next);
            values(&grad[next][j], q);
        }
        float on_to[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) on_to[v] = fmaf(own[v].A, q[v], P[v]);
        if (t0 > 0) {
            put(&grad[warp][j], on_to);
            hand_on(8 + warp);
        } else if (p.dh0) {
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (v < on) p.dh0[col.state(p) + v] = on_to[v];
        }
        if (warp > 0) {
            take_over(warp);
            values(&state[warp - 1][j], h);
        }
        if (warp < W - 1 && t0 + S < steps) {
#pragma unroll
            for (int v = 0; v < kV; ++v) on_to[v] = fmaf(own[v].A, h[v], own[v].H);
            put(&state[warp][j], on_to);
            hand_on(1 + warp);
        }
        T* const dz = at<T>(p.dz, col.b, t0, col.c);
        T* const dx = at<T>(p.dx, col.b, t0, col.c);
        const auto finish = [&](auto masked) {
#pragma unroll
            for (int k = 0; k < S; ++k)
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const float xv = from_x[k][v];
                    from_x[k][v] = h[v] - xv;
                    h[v] = fmaf(a[k][v], h[v], b[k][v] * xv);
                }
#pragma unroll
            for (int k = S - 1; k >= 0; --k) {
                float dv[kV], gx[kV], gz[kV];
                values(place(2, k), dv);
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const float G = __fadd_rn(q[v], masked.value && k >= live ? 0.0f : dv[v]);
                    gx[v] = b[k][v] * G;
                    gz[v] = a[k][v] * gx[v] * from_x[k][v];
                    q[v] = __fmul_rn(a[k][v], G);
                }
                if (!masked.value) {
                    if (kBytes > 0 || on) {
                        put(moved(dx, k * step_x), gx);
                        put(moved(dz, k * step_z), gz);
                    }
                } else if (t0 + k < steps) {
#pragma unroll
                    for (int v = 0; v < kV; ++v)
                        if (v < on) {
                            moved(dx, k * step_x)[v] = from_f32<T>(k < live ? gx[v] : 0.0f);
                            moved(dz, k * step_z)[v] = from_f32<T>(k < live ? gz[v] : 0.0f);
                        }
                }
            }
        };
        if (all) finish(std::false_type());
        else finish(std::true_type());
    }
}

// ---------------------------------------------------------------- launches
// How many bytes at a time the rows of all given tensors can be copied: 16, 4 or 2.
int row_bytes(const RecArgs& p, int e, std::initializer_list<const RecSeq*> seqs)
{
    int64_t bits = 0;
    bool near = true;  // a chunk's steps span less than 2^31 bytes
    for (const RecSeq* s : seqs) {
        bits |= (int64_t)reinterpret_cast<uintptr_t>(s->p) | s->batch * e | s->step * e;
        near = near && s->step < (int64_t)1 << 22;
    }
    if (bits % 16 == 0 && near && p.channels >= 32) return 16;
    return e == 4 || ((bits | p.channels * e) % 4 == 0) ? 4 : 2;
}

// A kernel with a CTA of `warps` per tile of `cols` columns; per_warp: shared bytes of a warp.
template <void (*kern)(RecArgs)>
cudaError_t launch_tiles(const RecArgs& p, bool apart, int cols, int most, int warps, int per_warp, cudaStream_t stream)
{
    const int64_t tiles = apart ? p.batch * ((p.channels + cols - 1) / cols) : (p.batch * p.channels + cols - 1) / cols;
    if (tiles > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const cudaError_t e = allow<kern>(most * per_warp);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3((unsigned)tiles), dim3(32 * (unsigned)warps), (size_t)(warps * per_warp), stream, p);
}

template <typename T, int kBytes, int kV> cudaError_t forward_v(const RecArgs& p, cudaStream_t stream)
{
    const int64_t chunks = (p.steps + kForward - 1) / kForward;
    return launch_tiles<rec_forward_kernel<T, kBytes, kV>>(
        p, kApart<kBytes>, 32 * kV, kWarps, chunks < kWarps ? (int)chunks : kWarps,
        2 * 2 * CopierOf<T, kBytes, 32 * kV, kForward, 2>::kElements * (int)sizeof(T), stream);
}

template <typename T, int kBytes, int kV> cudaError_t backward_v(const RecArgs& p, cudaStream_t stream)
{
    // no warps without a chunk (135 x 11 x 2833 fp32: 52 us, and 74 with the others)
    const int64_t chunks = (p.steps + kBackward<kV> - 1) / kBackward<kV>;
    const int warps = chunks < 1 ? 1 : chunks < kBackWarps<kV> ? (int)chunks : kBackWarps<kV>;
    return launch_tiles<rec_backward_kernel<T, kBytes, kV>>(
        p, kApart<kBytes>, 32 * kV, kBackWarps<kV>, warps,
        2 * 3 * CopierOf<T, kBytes, 32 * kV, kBackward<kV>, 3>::kElements * (int)sizeof(T), stream);
}

// How a call is split, by the columns n = batch * channels, in us with the choice and without. Many
// columns: a CTA for 64 or 32 of them, if that makes one for every SM; otherwise, if there are
// steps to split, clusters (4x4096x1001 bf16: forward 35 with clusters, 41 without, backward 69
// and 124). The backward pass, whose chain from one kept state to the next is longer, wants
// clusters also where there are up to twice as many columns and the chain is long (5x4096x1000
// bf16 74 and 143, 6x1500x1024 fp32 42 and 49; but 8x1000x1024 fp32 41 and 36), fewer where rows
// are off alignment (5x4096x1001 fp32 102 and 147; but 9x4096x1001 167 and 148).
constexpr int64_t kManyColumns = 152 * 32;
constexpr int64_t kSplitSteps = 128;
constexpr int64_t kLongSteps = 1200;
// A CTA for 64 columns, two per lane, saves instructions and halves the CTAs (forward: 16x2048x1024
// fp32 65, with 32 columns 69; but 12x2048x1024 58 and 47).
constexpr int64_t kTwoColumns = 3 * kManyColumns;

// Rows without alignment (forward and backward us by 16 bytes, and by four or two): 16 x 2048 x 1023
// fp32 78 and 146, 142 and 209; bf16 59 and 112, 81 and 174. But rows of pairs of bf16 elements
// take as many copies of four bytes as there are lanes: 16 x 2048 x 1022 58 and 114, 55 and 96.
template <typename T> constexpr int kPairs = sizeof(T) == 2 ? 4 : 0;

template <typename T> cudaError_t forward(const RecArgs& p, cudaStream_t stream)
{
    const int64_t n = p.batch * p.channels;
    if (p.steps <= kRecFew || (p.steps <= kRecSome && n >= kRecColumns)) {
        if (n > (int64_t)0x7fffffff * kRecThreads) return cudaErrorInvalidConfiguration;
        return launch_after(rec_forward_few_kernel<T>, dim3((unsigned)((n + kRecThreads - 1) / kRecThreads)),
                            dim3(kRecThreads), 0, stream, p);
    }
    const int by = row_bytes(p, (int)sizeof(T), {&p.z, &p.x, &p.y});
    if (n < kManyColumns && p.steps > kSplitSteps) return rec_split_forward<T>(p, by, stream);
    if (by == 16) return n >= kTwoColumns ? forward_v<T, 16, 2>(p, stream) : forward_v<T, 16, 1>(p, stream);
    if (by != kPairs<T> && by_granules(p, 32, 32, 0, {&p.z, &p.x, &p.y})) return forward_v<T, -(int)sizeof(T), 1>(p, stream);
    if constexpr (sizeof(T) == 2)
        if (by == 2) return forward_v<T, 2, 1>(p, stream);
    return forward_v<T, 4, 1>(p, stream);
}

template <typename T> cudaError_t backward(const RecArgs& p, cudaStream_t stream)
{
    const int64_t n = p.batch * p.channels;
    if (p.steps >= 1 && (p.steps <= kRecFew || (p.steps <= kRecSomeBack<T> && n >= kRecColumns))) {
        if (n > (int64_t)0x7fffffff * kRecThreads) return cudaErrorInvalidConfiguration;
        const dim3 grid((unsigned)((n + kRecThreads - 1) / kRecThreads));
        const auto kern = p.steps <= kRecFew ? rec_backward_few_kernel<T, kRecFew>
                          : p.steps <= 16    ? rec_backward_few_kernel<T, 16>
                                             : rec_backward_few_kernel<T, kRecSomeBack<T>>;
        return launch_after(kern, grid, dim3(kRecThreads), 0, stream, p);
    }
    const int by = row_bytes(p, (int)sizeof(T), {&p.z, &p.x, &p.dy, &p.dz, &p.dx});
    const int64_t many = p.steps < kLongSteps ? kManyColumns : by == 16 ? 2 * kManyColumns : kManyColumns * 3 / 2;
    if (n < many && p.steps > kSplitSteps) return rec_split_backward<T>(p, by, stream);
    if constexpr (sizeof(T) == 2) {
        // two columns per lane save instructions (16x2048x1024 bf16: 73 us against 86); with fp32
        // tensors, which are bound by memory, one is faster (104 us against 115)
        if (by == 16 && n >= kTwoColumns) return backward_v<T, 16, 2>(p, stream);
    }
    if (by == 16) return backward_v<T, 16, 1>(p, stream);
    if (by != kPairs<T> && by_granules(p, 32, 32, 0, {&p.z, &p.x, &p.dy, &p.dz, &p.dx}))
        return backward_v<T, -(int)sizeof(T), 1>(p, stream);
    if constexpr (sizeof(T) == 2)
        if (by == 2) return backward_v<T, 2, 1>(p, stream);
    return backward_v<T, 4, 1>(p, stream);
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
    if (!h || batch < 0 || steps < 0 || batch > 0x7fffffff || steps > 0x7fff0000) return ADACOMP_ERR_INVALID_ARG;
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
    p.timeout = (uint32_t)(h->timeout_ns < (uint64_t)1 << 41 ? (h->timeout_ns + 1023) >> 10 : 1u << 31);
    p.silent = h->inject_silent_cta;
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
    p.timeout = (uint32_t)(h->timeout_ns < (uint64_t)1 << 41 ? (h->timeout_ns + 1023) >> 10 : 1u << 31);
    p.silent = h->inject_silent_cta;
    const cudaError_t err = h->dtype == ADACOMP_BF16 ? adacomp::backward<adacomp::bf16>(p, stream)
                                                     : adacomp::backward<float>(p, stream);
    return adacomp::launch_result(err, stream);
}

adacomp_status adacomp_recurrence_set_timeout_ns(adacomp_recurrence_t h, uint64_t timeout_ns)
{
    if (!h || timeout_ns == 0) return ADACOMP_ERR_INVALID_ARG;
    h->timeout_ns = timeout_ns;
    return ADACOMP_OK;
}

adacomp_status adacomp_recurrence_set_fault_injection(adacomp_recurrence_t h, uint32_t silent_cta)
{
    if (!h) return ADACOMP_ERR_INVALID_ARG;
    h->inject_silent_cta = silent_cta;
    return ADACOMP_OK;
}

void adacomp_recurrence_free(adacomp_recurrence_t h) { delete h; }

}  // extern "C"
