// The recurrence where there are few columns: the steps split over warps, CTAs and clusters.
#include <cmath>

#include "recurrence.cuh"

namespace adacomp {
namespace {

// A lane's two columns. (Two values per instruction, add.f32x2 and its like, need fewer
// instructions here but have longer latencies, and the chains are what is waited for:
// backward 88 us with them, 77 without, at 16 sequences of 2048 steps of 1024 bf16 channels.)
struct Two {
    float x, y;
};
__device__ __forceinline__ Two two_of(float x, float y) { return {x, y}; }
__device__ __forceinline__ Two two_of(float x) { return {x, x}; }
__device__ __forceinline__ Two operator*(Two a, Two b) { return {__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)}; }
__device__ __forceinline__ Two operator+(Two a, Two b) { return {__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)}; }
__device__ __forceinline__ Two operator-(Two a, Two b) { return {__fsub_rn(a.x, b.x), __fsub_rn(a.y, b.y)}; }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) { return {fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }
__device__ __forceinline__ Two product(Two A, Two a) { return {product(A.x, a.x), product(A.y, a.y)}; }

// ---------------------------------------------------------------- many steps
// The steps are split: a warp has 64 columns (two per lane) and eight consecutive steps, a
// CTA 64 steps, a cluster of up to 16 CTAs up to 1024, and where the sequence is longer the
// cluster goes on in rounds. Each warp forms what its steps do to a state, h -> A h + H with
// A the product of its gates. The warps exchange these through shared memory, and the CTAs
// write theirs into every CTA of the cluster (one warp of each does); then each warp knows
// the state before its first step and goes through its steps again, from registers. So every element
// is read once, and no CTA waits for one that may not be running. The next round's elements
// are copied to shared memory meanwhile.
//
// Bound by the rounds' latency (some 3 us each: the gates, one exchange, the results), as a
// few columns leave an SM one or two CTAs. Measured: one sequence of 32768 steps of 1024 bf16
// channels 92 us forward (2.2 TB/s), 137 backward (2.5); four ragged ones of up to 20011 steps
// of 501 fp32 channels 116 (2.7 TB/s) and 179 (3.1).
constexpr int kCols = 64, kSteps = 8, kWarps = 8, kThreads = 32 * kWarps, kSpan = kSteps * kWarps;
constexpr int kTile = kSpan * kCols;  // elements of a tensor that a CTA has in a round
static_assert(kRecChunk == kSpan, "a kept state for every CTA");

// A tile's columns: of rows without alignment, as many as 64 elements hold wherever the row
// begins in the first 16 bytes.
template <int kBytes> constexpr int kTileCols = kBytes > 0 ? kCols : kCols + 1 + 16 / kBytes;

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

// Waits for the CTAs of the cluster without an order of memory: the results' stores need none.
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t shared_address(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ Two low(float4 v) { return two_of(v.x, v.y); }
__device__ __forceinline__ Two high(float4 v) { return two_of(v.z, v.w); }

__device__ __forceinline__ float4 quad(Two a, Two b) { return make_float4(a.x, a.y, b.x, b.y); }

// What the CTAs of a cluster write to each other in a round: each CTA's values, and the
// barrier that counts their bytes. Two of them take turns: a CTA that writes for the round
// after next has all others' values of the next one, so that they have read these.
// (A barrier of the whole cluster would have to wait for each round's stores of results.)
template <int kRanks> struct Exchange {
    float4 value[kRanks][32];
    unsigned long long barrier;
};

// CTAs of a cluster at most. Sixteen halve the rounds of few and long sequences; but for others
// than these the exchange's memory would cost an SM one of its CTAs.
template <typename T, int kBytes> constexpr int kRanks = sizeof(T) == 2 && kApart<kBytes> ? 16 : 8;

template <int R> __device__ __forceinline__ void exchange_init(Exchange<R>* x)
{
    if (threadIdx.x < 2)
        asm volatile("mbarrier.init.shared.b64 [%0], 1;" ::"r"(shared_address(&x[threadIdx.x].barrier)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

template <int R> __device__ __forceinline__ void exchange_expect(Exchange<R>* x, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(shared_address(&x->barrier)), "r"(bytes)
                 : "memory");
}

// Writes v to the place of `p` in the CTA `rank`, and counts it at that CTA's barrier.
template <int R> __device__ __forceinline__ void push(Exchange<R>* x, float4* p, uint32_t rank, float4 v)
{
    uint32_t a, b;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(shared_address(p)), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(shared_address(&x->barrier)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(b)
                 : "memory");
}

__device__ __forceinline__ uint32_t clock_1024ns() { return (uint32_t)(ptx::globaltimer() >> 10); }

// Whether a barrier's phase is complete; kSleep: the thread may be suspended until it is, for some
// microseconds.
template <bool kSleep, int R> __device__ __forceinline__ bool exchange_done(Exchange<R>* x, uint32_t phase)
{
    uint32_t done;
    if constexpr (kSleep)
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
            : "=r"(done)
            : "r"(shared_address(&x->barrier)), "r"(phase)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
            : "=r"(done)
            : "r"(shared_address(&x->barrier)), "r"(phase)
            : "memory");
    return done != 0;
}

// Waits for a barrier's phase: some hundred tries, and then for `timeout` times 1024 ns at most. The
// CTAs of a cluster run together and each writes before it waits, so the wait ends. Were it not
// to, the CTA exchanges nothing any more, as its barrier's phase is still open, and its results
// from there on are NaN: so each CTA runs into one timeout at most. (The lanes vote, so that the
// way past the tries is the warp's: with a timer in a lane's own loop 4x20011x501 takes 7 us more.)
template <int R> __device__ __forceinline__ bool exchange_wait(Exchange<R>* x, uint32_t phase, uint32_t timeout)
{
    bool done = false;
    for (uint32_t i = 0; i < 256 && !done; ++i) done = exchange_done<true>(x, phase);
    if (__all_sync(0xffffffffu, done)) return true;
    const uint32_t start = clock_1024ns();
    do {
        done = __all_sync(0xffffffffu, exchange_done<false>(x, phase));
    } while (!done && clock_1024ns() - start <= timeout);
    return __all_sync(0xffffffffu, done);
}

// The end of a cluster's kernel: no CTA ends while another may write to it. What a CTA that gave
// up was written by then and has not waited for lands within far less than a millisecond.
__device__ __forceinline__ void exchange_end(bool given_up)
{
    cluster_meet();
    if (!given_up) return;
    const uint32_t start = clock_1024ns();
    while (clock_1024ns() - start < 1024) {
    }
}

// The columns of a tile. Where a sequence's rows are read 16 bytes at a time, a tile is of one
// sequence's channels; otherwise the channels of all sequences are numbered through, so that
// few channels fill a tile too.
template <int kBytes> struct Column {
    int64_t b, c;
    int32_t len;  // of its sequence; 0 past the last column
    bool on;

    __device__ __forceinline__ Column(const RecArgs& p, uint32_t tile, int j)
    {
        if (kApart<kBytes>) {
            const uint32_t blocks = (uint32_t)((p.channels + kTileCols<kBytes> - 1) / kTileCols<kBytes>);
            b = tile / blocks;
            c = (int64_t)(tile - (uint32_t)b * blocks) * kTileCols<kBytes> + j;
            on = j < kTileCols<kBytes> && c < p.channels;
        } else {
            const int64_t i = (int64_t)tile * kCols + j;
            on = i < p.batch * p.channels;
            b = on ? i / p.channels : 0;
            c = on ? i - b * p.channels : 0;
        }
        len = on ? (int32_t)length_of(p, b) : 0;
    }
    __device__ __forceinline__ int64_t state(const RecArgs& p) const { return b * p.channels + c; }
};

// Copies a CTA's 64 steps of a tile to shared memory, [step][column], kBytes at a time:
// every thread has one place in the rows and takes every kStride-th of them. What lies past
// a sequence's length or the last channel is not read, and what stands there not used.
template <typename T, int kBytes, int kTensors> struct Copier {
    static constexpr int kCopy = kBytes < 0 ? 16 : kBytes;
    static constexpr int kPlaces = kCols * (int)sizeof(T) / kCopy;
    static constexpr int kStride = kThreads / kPlaces;
    static constexpr int kEach = kBytes < 0 ? 0 : kBytes / (int)sizeof(T);  // elements at a time
    const T* from[kTensors];
    Distance<kBytes> step[kTensors];
    int32_t len;
    uint32_t bytes;

    __device__ __forceinline__ Copier(const RecArgs& p, uint32_t tile, const RecSeq* const (&s)[kTensors])
    {
        const Column<kBytes> col(p, tile, (threadIdx.x % kPlaces) * kEach);
        const int64_t rest = (p.channels - col.c) * (int)sizeof(T);
        constexpr int most = kBytes < 0 ? kTileCols<kBytes> * (int)sizeof(T) : kBytes;  // of the row, or of a place in it
        bytes = !col.on ? 0u : rest < most ? (uint32_t)rest : (uint32_t)most;
        len = bytes == 0 ? 0 : col.len;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            from[i] = at<const T>(*s[i], col.b, 0, col.c);
            step[i] = (Distance<kBytes>)(s[i]->step * (int)sizeof(T));
        }
    }

    __device__ __forceinline__ void copy(T* to, int32_t t0) const
    {
        const int row0 = threadIdx.x / kPlaces, left = len - t0;
        if constexpr (kBytes < 0) {
            const int place = (threadIdx.x % kPlaces) * 16;
#pragma unroll
            for (int i = 0; i < kTensors; ++i) {
                const T* const f = moved(from[i], (int64_t)(t0 + row0) * step[i]);
                const uint32_t d0 = shared_address(to + i * kTile + row0 * kCols) + place;
#pragma unroll
                for (int k = 0; k < kSpan / kStride; ++k) {
                    const uintptr_t g = reinterpret_cast<uintptr_t>(f) + (int64_t)(k * kStride * step[i]);
                    const int before = (int)(g & 15), n = min(16, before + (int)bytes - place);
                    if (row0 + k * kStride < left && n > 0)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         d0 + k * kStride * kCols * (int)sizeof(T)),
                                     "l"(g - before + place), "r"(n)
                                     : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            return;
        }
        T* const place = to + row0 * kCols + (threadIdx.x % kPlaces) * kEach;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            const T* const f = moved(from[i], (int64_t)(t0 + row0) * step[i]);
            T v[kSpan / kStride];
#pragma unroll
            for (int k = 0; k < kSpan / kStride; ++k)
                if (row0 + k * kStride < left) {
                    const T* const g = moved(f, (Distance<kBytes>)(k * kStride) * step[i]);
                    const uint32_t d = shared_address(place + i * kTile + k * kStride * kCols);
                    if constexpr (kBytes == 2) v[k] = *g;
                    else if constexpr (kBytes == 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(g), "r"(bytes) : "memory");
                    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(g) : "memory");
                }
            if constexpr (kBytes == 2) {
#pragma unroll
                for (int k = 0; k < kSpan / kStride; ++k)
                    if (row0 + k * kStride < left) place[i * kTile + k * kStride * kCols] = v[k];
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // how many bytes are before step t's first element in its first 16 bytes
    __device__ __forceinline__ uint32_t before(int tensor, int32_t t) const
    {
        return ((uint32_t)reinterpret_cast<uintptr_t>(from[tensor]) + (uint32_t)t * (uint32_t)step[tensor]) & 15;
    }
};

__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// A lane's columns of a tile: two side by side where a row's elements are written two at a
// time, and otherwise half a tile apart, which puts a warp's writes side by side.
template <int kBytes> __device__ __forceinline__ int place_of(int lane, int j)
{
    return kBytes == 16 ? 2 * lane + j : lane + j * (kCols / 2);
}

// Their elements, from the first one's on.
template <int kBytes, typename T> __device__ __forceinline__ void two(const T* p, float& x, float& y)
{
    if constexpr (kBytes != 16) {
        x = to_f32(p[0]), y = to_f32(p[kCols / 2]);
    } else if constexpr (sizeof(T) == 4) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x = v.x, y = v.y;
    } else {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
        x = bf16_low(v), y = bf16_high(v);
    }
}

// Where a lane's two columns of a warp's steps go.
template <typename T, int kBytes> struct Writer {
    T* p[2];
    Distance<kBytes> step;

    __device__ __forceinline__ Writer(const RecSeq& s, const Column<kBytes> (&col)[2], int64_t t)
        : step((Distance<kBytes>)(s.step * (int)sizeof(T)))
    {
        p[0] = at<T>(s, col[0].b, t, col[0].c);
        p[1] = kBytes < 0 ? p[0] + kCols / 2 : at<T>(s, col[1].b, t, col[1].c);
    }
    // step k of both columns, as far as they are there (two side by side are)
    __device__ __forceinline__ void put(int k, Two v, bool on0, bool on1) const
    {
        T* const q = moved(p[0], k * step);
        if constexpr (kBytes == 16) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(q) = make_float2(v.x, v.y);
            else *reinterpret_cast<__nv_bfloat162*>(q) = __floats2bfloat162_rn(v.x, v.y);
        } else {
            if (on0) *q = from_f32<T>(v.x);
            if (on1) *moved(p[1], k * step) = from_f32<T>(v.y);
        }
    }
    __device__ __forceinline__ void put(int k, float x, float y, bool on0, bool on1) const
    {
        T* const q = moved(p[0], k * step);
        if (on0) *q = from_f32<T>(x);
        if (on1) *(kBytes == 16 ? q + 1 : moved(p[1], k * step)) = from_f32<T>(y);
    }
};

// What a warp has to mind in a round: how many of its steps lie within each column's length
// and within the tensors, and whether all do.
struct Live {
    int live0, live1, whole;
    bool all;

    template <int kBytes>
    __device__ __forceinline__ Live(const RecArgs& p, const Column<kBytes> (&col)[2], int32_t ts)
        : live0(max(0, min(kSteps, col[0].len - ts))), live1(max(0, min(kSteps, col[1].len - ts))),
          whole(max(0, min(kSteps, (int32_t)p.steps - ts))),
          all(__all_sync(0xffffffffu, (live0 == kSteps || (kBytes != 16 && !col[0].on)) &&
                                          (live1 == kSteps || (kBytes != 16 && !col[1].on))))
    {
    }
};

template <int kBytes>
__device__ __forceinline__ Two load_state(const float* p, const RecArgs& a, const Column<kBytes> (&col)[2], int64_t more = 0)
{
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (p && col[j].on) v[j] = p[col[j].state(a) + more];
    return two_of(v[0], v[1]);
}

template <int kBytes>
__device__ __forceinline__ void store_state(float* p, const RecArgs& a, const Column<kBytes> (&col)[2], Two s)
{
    if (p && col[0].on) p[col[0].state(a)] = s.x;
    if (p && col[1].on) p[col[1].state(a)] = s.y;
}

// The address of a column's kept state: [batch][chunks][channels].
template <int kBytes> __device__ __forceinline__ float* kept(const RecArgs& p, const Column<kBytes>& col, int32_t t)
{
    return p.carry + (col.b * p.chunks + t / kRecChunk) * p.channels + col.c;
}

// ---------------------------------------------------------------- chunks at once
// Few columns of many steps leave most SMs without work even so. There every chunk of 64 steps
// has a CTA of its own, in three kernels: what each chunk does to a state; the states before the
// chunks (the gradients after them), by the columns; and each chunk's results from these, for
// which the inputs are read again, mostly from L2. The first two hand on through the rows of
// the chunk's own outputs, which the third writes last: no workspace is needed for them.
template <typename T> struct Place {  // of an fp32 value in two rows, of which fp32 rows need one
    T *high, *low;
    __device__ __forceinline__ void put(float v) const
    {
        if constexpr (sizeof(T) == 4) {
            *high = v;
        } else {
            *reinterpret_cast<uint16_t*>(high) = (uint16_t)(__float_as_uint(v) >> 16);
            *reinterpret_cast<uint16_t*>(low) = (uint16_t)__float_as_uint(v);
        }
    }
    __device__ __forceinline__ float get() const
    {
        if constexpr (sizeof(T) == 4) return *high;
        else
            return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(high) << 16 |
                                   *reinterpret_cast<const uint16_t*>(low));
    }
};

// The places of values at a chunk's first steps: the two that the first kernel leaves, and the one
// that the third begins with, apart from them, as the second writes it while it reads them; but
// the last chunk may be short, and has one place for both. The forward pass has them in the rows of
// y, the backward pass in those of dz and dx, where one of each holds a value.
__device__ __forceinline__ int begin_place(bool last) { return last ? 0 : 2; }

template <typename T, bool kBack> __device__ __forceinline__ Place<T> place_at(const RecArgs& p, int64_t b, int64_t c, int64_t t, int i)
{
    if constexpr (kBack) {
        if constexpr (sizeof(T) == 4) return {at<T>(i & 1 ? p.dx : p.dz, b, t + i / 2, c), nullptr};
        else return {at<T>(p.dz, b, t + i, c), at<T>(p.dx, b, t + i, c)};
    } else {
        if constexpr (sizeof(T) == 4) return {at<T>(p.y, b, t + i, c), nullptr};
        else return {at<T>(p.y, b, t + 2 * i, c), at<T>(p.y, b, t + 2 * i + 1, c)};
    }
}

template <typename T, bool kBack, int kBytes>
__device__ __forceinline__ Two begin_of(const RecArgs& p, const Column<kBytes> (&col)[2], int32_t t, bool last)
{
    const int place = begin_place(last);
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (col[j].on) v[j] = place_at<T, kBack>(p, col[j].b, col[j].c, t, place).get();
    return two_of(v[0], v[1]);
}

// The first kernel: a CTA's chunk, h -> A h + H (not of the last chunk), or p -> A p + P (not of
// the first; of the last, p itself).
template <typename T, int kBytes, bool kBack>
__global__ void __launch_bounds__(kThreads, 4) rec_totals_kernel(const __grid_constant__ RecArgs p, const uint32_t chunks)
{
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    __shared__ float4 part[kWarps][32];
    T* const tile_at = reinterpret_cast<T*>(shared_bytes);
    ptx::griddep_wait();
    const uint32_t tile = blockIdx.x / (chunks - 1);
    const int32_t tc = (int32_t)(blockIdx.x - tile * (chunks - 1) + (kBack ? 1 : 0)) * kSpan;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Column<kBytes> col[2] = {Column<kBytes>(p, tile, place_of<kBytes>(lane, 0)),
                                  Column<kBytes>(p, tile, place_of<kBytes>(lane, 1))};
    const Copier<T, kBytes, 2> copier(p, tile, {&p.z, kBack ? &p.dy : &p.x});
    copier.copy(tile_at, tc);
    copies_wait();
    __syncthreads();
    const int32_t ts = tc + warp * kSteps;
    const Live at_hand(p, col, ts);
    const T* const first = tile_at + warp * kSteps * kCols + place_of<kBytes>(lane, 0);
    Two A = two_of(1.0f), H = two_of(0.0f);
    const auto form = [&](auto masked) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            float v[2][2], a0, a1, b0, b1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const T* q = first + i * kTile + k * kCols;
                two<kBytes>(kBytes < 0 ? moved(q, copier.before(i, ts + k)) : q, v[i][0], v[i][1]);
            }
            gate(v[0][0], &a0, &b0);
            gate(v[0][1], &a1, &b1);
            if (masked.value) {
                if (k >= at_hand.live0) a0 = 1.0f, b0 = v[1][0] = 0.0f;
                if (k >= at_hand.live1) a1 = 1.0f, b1 = v[1][1] = 0.0f;
            }
            const Two a = two_of(a0, a1), u = two_of(v[1][0], v[1][1]);
            A = product(A, a);
            if (kBack) H = fma2(A, u, H);
            else H = fma2(a, H, two_of(b0, b1) * u);
        }
    };
    if (at_hand.all) form(std::false_type());
    else form(std::true_type());
    part[warp][lane] = quad(A, H);
    __syncthreads();
    if (warp != 0) return;
    A = two_of(1.0f), H = two_of(0.0f);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const float4 q = part[kBack ? kWarps - 1 - i : i][lane];
        H = fma2(low(q), H, high(q));
        A = product(A, low(q));
    }
    const bool last = kBack && tc + kSpan >= (int32_t)p.steps;
    if (last) A = fma2(A, load_state(p.dh_last, p, col), H);
    const float v[2][2] = {{A.x, H.x}, {A.y, H.y}};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!col[j].on) continue;
        place_at<T, kBack>(p, col[j].b, col[j].c, tc, 0).put(v[j][0]);
        if (!last) place_at<T, kBack>(p, col[j].b, col[j].c, tc, 1).put(v[j][1]);
    }
}

// The second: 32 columns per CTA, whose warps have consecutive chunks each.
constexpr int kStateWarps = 32;

template <typename T, bool kBack>
__global__ void __launch_bounds__(32 * kStateWarps) rec_states_kernel(const __grid_constant__ RecArgs p, const uint32_t chunks)
{
    __shared__ float2 part[kStateWarps][32];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane;
    const bool on = i < p.batch * p.channels;
    const int64_t b = on ? i / p.channels : 0, c = on ? i - b * p.channels : 0;
    // Turn k: the step from chunk k to k + 1, or back from chunk `chunks - 1 - k` (its gradient
    // is given) to the one before it.
    const int32_t turns = (int32_t)chunks - 1, each = (turns + kStateWarps - 1) / kStateWarps;
    const int32_t begin = min(turns, warp * each), end = min(turns, begin + each);
    const auto chunk_of = [&](int32_t k) { return kBack ? (int32_t)chunks - 1 - k : k; };
    const auto step_of = [&](int32_t k) {
        const int64_t t = (int64_t)chunk_of(k) * kSpan;
        float2 v = make_float2(1.0f, 0.0f);
        if (on) {
            v.x = place_at<T, kBack>(p, b, c, t, 0).get();
            if (kBack && k == 0) v = make_float2(0.0f, v.x);
            else v.y = place_at<T, kBack>(p, b, c, t, 1).get();
        }
        return v;
    };
    float2 own = make_float2(1.0f, 0.0f);
#pragma unroll 8
    for (int32_t k = begin; k < end; ++k) {
        const float2 v = step_of(k);
        own.y = fmaf(v.x, own.y, v.y);
        own.x = product(own.x, v.x);
    }
    part[warp][lane] = own;
    __syncthreads();
    float h = !kBack && p.h0 && on ? p.h0[i] : 0.0f;
    const auto hand = [&](int32_t chunk, float v) {
        if (!kBack && p.carry) p.carry[(b * p.chunks + chunk) * p.channels + c] = v;
        else place_at<T, kBack>(p, b, c, (int64_t)chunk * kSpan, begin_place(chunk + 1 == (int32_t)chunks)).put(v);
    };
    if (!kBack && on && warp == 0) hand(0, h);
    for (int w = 0; w < warp; ++w) h = fmaf(part[w][lane].x, h, part[w][lane].y);
    for (int32_t k0 = begin; k0 < end; k0 += 8) {
        float2 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j < end) v[j] = step_of(k0 + j);
        if (!on) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t k = k0 + j;
            if (k >= end) break;
            h = fmaf(v[j].x, h, v[j].y);
            // (where dh0 is dh_last itself, the third kernel cannot read it)
            if (kBack && k == 0) hand((int32_t)chunks - 1, p.dh_last ? p.dh_last[i] : 0.0f);
            hand(chunk_of(k) + (kBack ? -1 : 1), h);
        }
    }
}

// ranks: the CTAs of a cluster, or (kChunks) the chunks of a sequence, with their states at hand.
template <typename T, int kBytes, bool kChunks>
__global__ void __launch_bounds__(kThreads, 4) rec_forward_kernel(const __grid_constant__ RecArgs p, const uint32_t ranks)
{
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    __shared__ float4 part[kWarps][32];   // a warp's (A, H) of the lane's columns
    __shared__ Two begin[kWarps][32];  // the state before its first step
    __shared__ Exchange<kRanks<T, kBytes>> exchange[2];
    const auto tile_of = [&](int i) { return reinterpret_cast<T*>(shared_bytes) + i * (2 * kTile); };
    ptx::griddep_wait();
    if constexpr (!kChunks) {
        exchange_init(exchange);
        cluster_sync();  // all CTAs run, and their barriers are there, before one writes to another
    }
    const uint32_t tile = blockIdx.x / ranks, rank = kChunks ? blockIdx.x - tile * ranks : cluster_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Column<kBytes> col[2] = {Column<kBytes>(p, tile, place_of<kBytes>(lane, 0)),
                                  Column<kBytes>(p, tile, place_of<kBytes>(lane, 1))};
    const Copier<T, kBytes, 2> copier(p, tile, {&p.z, &p.x});
    const int32_t steps = (int32_t)p.steps, span = (int32_t)ranks * kSpan;
    int32_t tc = (int32_t)rank * kSpan;
    Two h0;  // before the round's first step (the joining warp's)
    if (!kChunks) h0 = load_state(p.h0, p, col);
    else if (p.carry) h0 = two_of(col[0].on ? *kept(p, col[0], tc) : 0.0f, col[1].on ? *kept(p, col[1], tc) : 0.0f);
    else if (warp == 0) h0 = begin_of<T, false>(p, col, tc, rank + 1 == ranks);
    bool given_up = false;
    copier.copy(tile_of(0), tc);
    for (int32_t t0 = 0, round = 0; t0 < steps; t0 += span, tc += span, ++round) {
        const int par = round & 1;
        copies_wait();
        __syncthreads();
        if (!kChunks && t0 + span < steps) copier.copy(tile_of(par ^ 1), tc + span);
        const int32_t ts = tc + warp * kSteps;
        const Live at_hand(p, col, ts);
        const T* const first = tile_of(par) + warp * kSteps * kCols + place_of<kBytes>(lane, 0);
        const auto place = [&](int tensor, int k) {  // step k's
            const T* q = first + tensor * kTile + k * kCols;
            return kBytes < 0 ? moved(q, copier.before(tensor, ts + k)) : q;
        };
        Two a[kSteps], u[kSteps], A = two_of(1.0f), H = two_of(0.0f);
        const auto form = [&](auto masked) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                float z0, z1, x0, x1, a0, a1, b0, b1;
                two<kBytes>(place(0, k), z0, z1);
                two<kBytes>(place(1, k), x0, x1);
                gate(z0, &a0, &b0);
                gate(z1, &a1, &b1);
                if (masked.value) {  // past the length the state stays as it is
                    if (k >= at_hand.live0) a0 = 1.0f, b0 = x0 = 0.0f;
                    if (k >= at_hand.live1) a1 = 1.0f, b1 = x1 = 0.0f;
                }
                a[k] = two_of(a0, a1);
                u[k] = two_of(b0, b1) * two_of(x0, x1);
                H = fma2(a[k], H, u[k]);
                A = A * a[k];
            }
        };
        if (at_hand.all) form(std::false_type());
        else form(std::true_type());
        Two least = two_of(kLeast);  // as product() of them all
#pragma unroll
        for (int k = 0; k < kSteps; k += 2)
            least = two_of(least3(least.x, a[k].x, a[k + 1].x), least3(least.y, a[k].y, a[k + 1].y));
        A = two_of(not_below(A.x, least.x), not_below(A.y, least.y));
        part[warp][lane] = quad(A, H);
        __syncthreads();
        if (warp == 0) {
            Two h = h0;  // before the CTA's first step
            if constexpr (!kChunks) {
                Exchange<kRanks<T, kBytes>>& x = exchange[par];
                if (!given_up) {
                    if (lane == 0) exchange_expect(&x, ranks * 512);
                    Two tA = two_of(1.0f), tH = two_of(0.0f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float4 q = part[w][lane];
                        tH = fma2(low(q), tH, high(q));
                        tA = product(tA, low(q));
                    }
                    if (rank != p.silent)
                        for (uint32_t r = 0; r < ranks; ++r) push(&x, &x.value[rank][lane], r, quad(tA, tH));
                    given_up = !exchange_wait(&x, (round >> 1) & 1, p.timeout);
                }
                for (uint32_t r = 0; r < ranks; ++r) {
                    if (r == rank) h = h0;
                    const float4 q = x.value[r][lane];
                    h0 = fma2(low(q), h0, high(q));
                }
                if (given_up) h = h0 = two_of(NAN);
            }
            if (!kChunks && p.carry && tc < steps) {
                const Two v = h;
                if (col[0].on) *kept(p, col[0], tc) = v.x;
                if (col[1].on) *kept(p, col[1], tc) = v.y;
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                begin[w][lane] = h;
                const float4 q = part[w][lane];
                h = fma2(low(q), h, high(q));
            }
            if (kChunks) h0 = h;
        }
        __syncthreads();
        Two h = begin[warp][lane];
        const Writer<T, kBytes> y(p.y, col, ts);
        if (at_hand.all) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                h = fma2(a[k], h, u[k]);
                y.put(k, h, col[0].on, col[1].on);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                h = fma2(a[k], h, u[k]);
                const Two v = h;
                if (k < at_hand.whole)
                    y.put(k, k < at_hand.live0 ? v.x : 0.0f, k < at_hand.live1 ? v.y : 0.0f, col[0].on, col[1].on);
            }
        }
        if (kChunks) break;  // one round (the next one's first step may not be a 32-bit number)
    }
    if (rank == (kChunks ? ranks - 1 : 0) && warp == 0) store_state(p.h_last, p, col, h0);
    if constexpr (!kChunks) exchange_end(given_up);
}

// The reverse of it: p, the gradient that reaches a state from the steps after it, goes
// through a warp's steps as p -> A p + P, P = sum of dy_k times the gates up to and with
// step k. The states are formed again from the one that the forward pass kept for the CTA's
// steps: that is less to read than y, and not rounded.
template <typename T, int kBytes, bool kChunks>
__global__ void __launch_bounds__(kThreads, kBytes == 16 ? 3 : 2)
    rec_backward_kernel(const __grid_constant__ RecArgs p, const uint32_t ranks)
{
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    __shared__ float4 part[kWarps][32];  // a warp's (A, H)
    __shared__ Two grad[kWarps][32];  // its P
    __shared__ float4 begin[32];         // the state before the CTA's first step, and p after its last
    __shared__ Exchange<kRanks<T, kBytes>> exchange[2];
    const auto tile_of = [&](int i) { return reinterpret_cast<T*>(shared_bytes) + i * (3 * kTile); };
    ptx::griddep_wait();
    if constexpr (!kChunks) {
        exchange_init(exchange);
        cluster_sync();  // all CTAs run, and their barriers are there, before one writes to another
    }
    const uint32_t tile = blockIdx.x / ranks, rank = kChunks ? blockIdx.x - tile * ranks : cluster_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Column<kBytes> col[2] = {Column<kBytes>(p, tile, place_of<kBytes>(lane, 0)),
                                  Column<kBytes>(p, tile, place_of<kBytes>(lane, 1))};
    const int32_t steps = (int32_t)p.steps, span = (int32_t)ranks * kSpan;
    int32_t t0 = (steps - 1) / span * span, tc = t0 + (int32_t)rank * kSpan;
    const Copier<T, kBytes, 3> copier(p, tile, {&p.z, &p.x, &p.dy});
    Two p0;  // after the round's last step (the joining warp's)
    if (!kChunks) p0 = load_state(p.dh_last, p, col);
    else if (warp == kWarps - 1) p0 = begin_of<T, true>(p, col, tc, rank + 1 == ranks);
    bool given_up = false;
    copier.copy(tile_of(0), tc);
    for (int32_t round = 0; t0 >= 0; t0 -= span, tc -= span, ++round) {
        const int par = round & 1;
        Two h = two_of(0.0f);  // before the CTA's first step
        if (warp == kWarps - 1 && tc < steps)
            h = two_of(col[0].on ? *kept(p, col[0], tc) : 0.0f, col[1].on ? *kept(p, col[1], tc) : 0.0f);
        copies_wait();
        __syncthreads();
        if (!kChunks && t0 > 0) copier.copy(tile_of(par ^ 1), tc - span);
        const int32_t ts = tc + warp * kSteps;
        const Live at_hand(p, col, ts);
        const T* const first = tile_of(par) + warp * kSteps * kCols + place_of<kBytes>(lane, 0);
        const auto place = [&](int tensor, int k) {  // step k's
            const T* q = first + tensor * kTile + k * kCols;
            return kBytes < 0 ? moved(q, copier.before(tensor, ts + k)) : q;
        };
        Two a[kSteps], b[kSteps], A = two_of(1.0f), H = two_of(0.0f), P = two_of(0.0f);
        const auto inputs = [&](auto masked, int tensor, int k) {  // x or dy
            float v0, v1;
            two<kBytes>(place(tensor, k), v0, v1);
            if (masked.value) {
                if (k >= at_hand.live0) v0 = 0.0f;
                if (k >= at_hand.live1) v1 = 0.0f;
            }
            return two_of(v0, v1);
        };
        const auto form = [&](auto masked) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                float z0, z1, a0, a1, b0, b1;
                two<kBytes>(place(0, k), z0, z1);
                gate(z0, &a0, &b0);
                gate(z1, &a1, &b1);
                if (masked.value) {
                    if (k >= at_hand.live0) a0 = 1.0f, b0 = 0.0f;
                    if (k >= at_hand.live1) a1 = 1.0f, b1 = 0.0f;
                }
                a[k] = two_of(a0, a1);
                b[k] = two_of(b0, b1);
                H = fma2(a[k], H, b[k] * inputs(masked, 1, k));
                A = product(A, a[k]);
                P = fma2(A, inputs(masked, 2, k), P);
            }
        };
        if (at_hand.all) form(std::false_type());
        else form(std::true_type());
        part[warp][lane] = quad(A, H);
        grad[warp][lane] = P;
        __syncthreads();
        A = two_of(1.0f), H = two_of(0.0f);  // from the CTA's first step to the warp's
        for (int w = 0; w < warp; ++w) {
            const float4 v = part[w][lane];
            H = fma2(low(v), H, high(v));
            A = product(A, low(v));
        }
        Two B = two_of(1.0f);  // and from the CTA's end back to the warp's
        P = two_of(0.0f);
        for (int w = kWarps - 1; w > warp; --w) {
            const Two v = low(part[w][lane]);
            P = fma2(v, P, grad[w][lane]);
            B = product(B, v);
        }
        if (warp == kWarps - 1) {
            const float4 own = part[warp][lane];
            const Two tA = product(A, low(own));
            Two tP = two_of(0.0f), q = p0;  // q: after the CTA's last step
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w)
                tP = fma2(low(part[w][lane]), tP, grad[w][lane]);
            if constexpr (!kChunks) {
                Exchange<kRanks<T, kBytes>>& x = exchange[par];
                if (!given_up) {
                    if (lane == 0) exchange_expect(&x, ranks * 512);
                    if (rank != p.silent)
                        for (uint32_t r = 0; r < ranks; ++r) push(&x, &x.value[rank][lane], r, quad(tA, tP));
                    given_up = !exchange_wait(&x, (round >> 1) & 1, p.timeout);
                }
                for (uint32_t r = ranks; r-- > 0;) {
                    if (r == rank) q = p0;
                    const float4 v = x.value[r][lane];
                    p0 = fma2(low(v), p0, high(v));
                }
                if (given_up) h = q = p0 = two_of(NAN);
            } else {
                p0 = fma2(tA, p0, tP);
            }
            begin[lane] = quad(h, q);
        }
        __syncthreads();
        h = fma2(A, low(begin[lane]), H);
        Two q = fma2(B, high(begin[lane]), P);
        const Writer<T, kBytes> dz(p.dz, col, ts), dx(p.dx, col, ts);
        const auto finish = [&](auto masked) {
            Two before[kSteps];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const Two x = inputs(masked, 1, k);
                before[k] = h - x;  // h_{t-1} - x_t
                h = fma2(a[k], h, b[k] * x);
            }
#pragma unroll
            for (int k = kSteps - 1; k >= 0; --k) {
                const Two G = q + inputs(masked, 2, k), g = b[k] * G;
                q = a[k] * G;
                const Two v = a[k] * g * before[k];
                if (!masked.value) {
                    dx.put(k, g, col[0].on, col[1].on);
                    dz.put(k, v, col[0].on, col[1].on);
                } else if (k < at_hand.whole) {
                    const Two e = g, f = v;
                    const bool l0 = k < at_hand.live0, l1 = k < at_hand.live1;
                    dx.put(k, l0 ? e.x : 0.0f, l1 ? e.y : 0.0f, col[0].on, col[1].on);
                    dz.put(k, l0 ? f.x : 0.0f, l1 ? f.y : 0.0f, col[0].on, col[1].on);
                }
            }
        };
        if (at_hand.all) finish(std::false_type());
        else finish(std::true_type());
        if (kChunks) break;
    }
    if (rank == 0 && warp == kWarps - 1) store_state(p.dh0, p, col, p0);
    if constexpr (!kChunks) exchange_end(given_up);
}

// Launches a kernel of clusters, behind the kernel ahead of it as launch_after does.
template <int kRanks, void (*kern)(RecArgs, uint32_t)>
cudaError_t launch_ranks(int cols, int shared, const RecArgs& p, cudaStream_t stream)
{
    const int64_t tiles = cols ? p.batch * ((p.channels + cols - 1) / cols) : (p.batch * p.channels + kCols - 1) / kCols;
    // a CTA more in a cluster is worth its exchange where the GPU is not full without it; more
    // than eight where all clusters still run at once
    const uint32_t most = tiles <= 19 ? (uint32_t)kRanks : 8;
    uint32_t ranks = 2;  // at least, as there are more than 128 steps and less than 512 tiles
    while (ranks < most && (int64_t)ranks * kSpan < p.steps && tiles * ranks < 1024) ranks *= 2;
    const cudaError_t e = allow<kern, (kRanks > 8)>(shared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * ranks));
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.dynamicSmemBytes = (size_t)shared;
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

// Rows without alignment (a training step's us by 16 bytes and by four or two): 4 x 20011 x 501
// fp32 295 and 440, 4 x 4096 x 1001 bf16 104 and 159; 32 x 4096 x 33 fp32, twice as many tiles but
// all running at once, 56 and 72; 32 x 4096 x 62 fp32, more than that, 115 and 94.
constexpr int64_t kAtOnce = 38;

// Whether every chunk has a CTA of its own, which costs their number, and three launches, where
// clusters cost the number of their rounds: forward and backward us with it and without, 1 x 9918
// x 3 fp32 13 and 22, 45 and 56; 233 x 1500 x 1 15 and 22, 20 and 34; 1 x 32768 x 1024 122 and
// 170, 152 and 222 (bf16, with clusters of 16, 101 and 145, 92 and 137); 16 x 9656 x 133 bf16 106
// and 168, 94 and 121; 1 x 1000000 x 8 382 and 682, 4162 and 5191. The numbers in by_chunks lie
// between such pairs.
template <typename T, int kBytes> bool by_chunks(const RecArgs& p, int64_t tiles, int64_t chunks)
{
    // the last chunk's beginning needs two rows of bf16 elements, if it is not in the carry
    if (!p.carry && sizeof(T) == 2 && p.steps % kSpan == 1) return false;
    return kRanks<T, kBytes> > 8 ? tiles * chunks + 800 <= 15 * chunks : tiles * chunks + 400 <= 22 * chunks;
}

// Launches a kernel with a CTA for each of `chunks` chunks of every tile.
template <void (*kern)(RecArgs, uint32_t)>
cudaError_t launch_chunks(int64_t tiles, uint32_t grid, uint32_t chunks, int shared, const RecArgs& p, cudaStream_t stream)
{
    const cudaError_t e = allow<kern>(shared);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3((unsigned)(tiles * grid)), dim3(kThreads), (size_t)shared, stream, p, chunks);
}

template <typename T, int kBytes, bool kBack> cudaError_t run(const RecArgs& p, cudaStream_t stream)
{
    constexpr int cols = kApart<kBytes> ? kTileCols<kBytes> : 0, pad = kBytes < 0 ? 16 : 0;
    constexpr int one = kTile * (int)sizeof(T), tensors = kBack ? 3 : 2;
    const int64_t tiles = cols ? p.batch * ((p.channels + cols - 1) / cols) : (p.batch * p.channels + kCols - 1) / kCols;
    const int64_t chunks = (p.steps + kSpan - 1) / kSpan;
    if (by_chunks<T, kBytes>(p, tiles, chunks)) {
        const uint32_t n = (uint32_t)chunks;
        cudaError_t e =
            launch_chunks<rec_totals_kernel<T, kBytes, kBack>>(tiles, n - 1, n, 2 * one + pad, p, stream);
        if (e != cudaSuccess) return e;
        e = launch_after(rec_states_kernel<T, kBack>, dim3((unsigned)((p.batch * p.channels + 31) / 32)),
                         dim3(32 * kStateWarps), 0, stream, p, n);
        if (e != cudaSuccess) return e;
        if constexpr (kBack)
            return launch_chunks<rec_backward_kernel<T, kBytes, true>>(tiles, n, n, tensors * one + pad, p, stream);
        else return launch_chunks<rec_forward_kernel<T, kBytes, true>>(tiles, n, n, tensors * one + pad, p, stream);
    }
    if constexpr (kBack)
        return launch_ranks<kRanks<T, kBytes>, rec_backward_kernel<T, kBytes, false>>(cols, 2 * tensors * one + pad, p, stream);
    else return launch_ranks<kRanks<T, kBytes>, rec_forward_kernel<T, kBytes, false>>(cols, 2 * tensors * one + pad, p, stream);
}

}  // namespace

template <typename T> cudaError_t rec_split_forward(const RecArgs& p, int by, cudaStream_t stream)
{
    if (by == 16) return run<T, 16, false>(p, stream);
    if (by_granules(p, kTileCols<-(int)sizeof(T)>, kCols, kAtOnce, {&p.z, &p.x, &p.y}))
        return run<T, -(int)sizeof(T), false>(p, stream);
    if constexpr (sizeof(T) == 2)
        if (by == 2) return run<T, 2, false>(p, stream);
    return run<T, 4, false>(p, stream);
}

template <typename T> cudaError_t rec_split_backward(const RecArgs& p, int by, cudaStream_t stream)
{
    if (by == 16) return run<T, 16, true>(p, stream);
    if (by_granules(p, kTileCols<-(int)sizeof(T)>, kCols, kAtOnce, {&p.z, &p.x, &p.dy, &p.dz, &p.dx}))
        return run<T, -(int)sizeof(T), true>(p, stream);
    if constexpr (sizeof(T) == 2)
        if (by == 2) return run<T, 2, true>(p, stream);
    return run<T, 4, true>(p, stream);
}

template cudaError_t rec_split_forward<float>(const RecArgs&, int, cudaStream_t);
template cudaError_t rec_split_forward<bf16>(const RecArgs&, int, cudaStream_t);
template cudaError_t rec_split_backward<float>(const RecArgs&, int, cudaStream_t);
template cudaError_t rec_split_backward<bf16>(const RecArgs&, int, cudaStream_t);

}  // namespace adacomp
