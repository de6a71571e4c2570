// The norm of many gradients and an AdamW step over many tensors, with the moments in
// 32 or in 8 bits: kernels and C entry points (adacomp.h).
#include <memory>
#include <new>
#include <type_traits>
#include <vector>

#include <cuda_fp16.h>

#include "train_common.cuh"

namespace adacomp {
namespace {

constexpr int kAwThreads = 256;
constexpr int kAwWarps = kAwThreads / 32;
constexpr int kAwBlock = ADACOMP_ADAMW_BLOCK;      // elements per scale, and per warp and turn
constexpr int kAwTile = kAwWarps * kAwBlock;       // elements per CTA
constexpr int kAwTensors = 400;                    // tensors per launch (a by-value kernel parameter)
constexpr int kAwFew = 16;                         // and of its short form: 32 KB of parameters cost a launch 4 us
constexpr int kNormTensors = 1200;
constexpr int kNormFew = 64;
constexpr int kJumps = 1024, kJumpsFew = 64;       // see owner_of
constexpr int kNormGrid = 912;                     // CTAs per launch at most (six per SM), each with a partial sum
constexpr int kNormVectors = 4;                    // 16-byte vectors per thread and tile

// The step's constants.
struct Adam {
    float c, beta1, beta2, rest1, rest2, step, root, eps, one, half, minus, decay;
};

struct AwTensor {
    void *w, *m, *v, *copy;
    const void* g;
    float *ms, *vs;
    int64_t n;
    uint32_t tile_begin;
    float decay;  // 1 - lr * weight_decay
};

template <int N> struct Jumps {
    static constexpr int kCount = N;
    int32_t shift;
    uint16_t id[N];  // the tensor of tile k << shift
};

struct AwHead {
    int32_t count;
    uint32_t tiles;  // of this launch
    uint32_t ahead;  // tiles from a CTA's own to the one that it has brought into L2 (8-bit states)
    int32_t fast;    // eps and root lie where the step's own root and quotient are exact (adam_lane)
    Adam k;          // its c and decay are filled in by the kernel
    const float* coefficient;
};

template <int N, int J> struct AwTable : AwHead {
    AwTensor t[N];
    Jumps<J> jump;
};
using AwLong = AwTable<kAwTensors, kJumps>;
using AwShort = AwTable<kAwFew, kJumpsFew>;
static_assert(sizeof(AwLong) <= 32764, "kernel parameters");

struct NormTensor {
    const void* g;
    int64_t n;
    uint32_t tile_begin;
};

struct NormHead {
    int32_t count;
    uint32_t tiles;        // of this launch
    uint32_t first_part;   // where its partial sums start
    uint32_t all_parts;    // partial sums of all launches of the call
    float scale, max_norm;
    float* result;
    uint32_t* ticket;
    double* part;
};

template <int N, int J> struct NormTable : NormHead {
    NormTensor t[N];
    Jumps<J> jump;
};
using NormLong = NormTable<kNormTensors, kJumps>;
using NormShort = NormTable<kNormFew, kJumpsFew>;
static_assert(sizeof(NormLong) <= 32764, "kernel parameters");

// The last tensor whose first tile is at or before `tile`: from the first tile's of its
// stretch of 2^shift tiles on (a search by halves over hundreds of tensors is nine
// dependent reads).
template <typename Table> __device__ __forceinline__ int owner_of(const Table& tab, uint32_t tile)
{
    int id = tab.jump.id[tile >> tab.jump.shift];
    while (id + 1 < tab.count && tab.t[id + 1].tile_begin <= tile) ++id;
    return id;
}

template <typename Table> void fill_jumps(Table* tab)
{
    int shift = 0, id = 0;
    while ((tab->tiles - 1) >> shift >= (uint32_t)decltype(tab->jump)::kCount) ++shift;
    tab->jump.shift = shift;
    for (uint32_t k = 0; k <= (tab->tiles - 1) >> shift; ++k) {
        while (id + 1 < tab->count && tab->t[id + 1].tile_begin <= k << shift) ++id;
        tab->jump.id[k] = (uint16_t)id;
    }
}

// ---------------------------------------------------------------- e4m3
// Two values as two e4m3 numbers, the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t c)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ---------------------------------------------------------------- step
// One element's root u of v, and its weight, by the scalar operations.
__device__ __forceinline__ void root_and_weight(const Adam& k, float m, float v, float& u, float& w)
{
    u = __fsqrt_rn(v);
    const float q = __fdiv_rn(m, __fadd_rn(__fmul_rn(u, k.root), k.eps));
    w = __fsub_rn(__fmul_rn(k.decay, w), __fmul_rn(k.step, q));
}

// The sum of two products, each rounded before it: `one` is 1, which the compiler does not
// know. It fuses add.rn.f32x2 with mul.rn.f32x2 (seen with CUDA 13.0), but not this.
__device__ __forceinline__ Pair sum2(Pair x, Pair y, Pair one) { return fma2(x, one, y); }

// The correctly rounded root of two values within 2^+-60: s = v * rsqrt(v), and one Newton
// step with the residual v - s * s from a fused multiply-add (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990). That the step rounds
// as sqrt does was checked for every significand of both parities of the exponent.
__device__ __forceinline__ Pair root2(Pair v, const Adam& k)
{
    float x, y;
    split(v, x, y);
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(x));
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(y));
    const Pair r = pair(x, y);
    const Pair s = v * r, minus = s * pair(k.minus);
    return fma2(fma2(minus, s, v), r * pair(k.half), s);
}

// The correctly rounded quotients -a / b of values within 2^+-60 (or a = 0): with n the
// correctly rounded -1 / b (one Newton step on the approximate one; checked for every
// significand) and q = a * n, the residual r = a + b * q is exact and q + r * n rounds as
// -a / b does (Markstein's theorem, same paper), a zero with its sign.
__device__ __forceinline__ Pair minus_quotient2(Pair a, Pair b, const Adam& k)
{
    float x, y;
    split(b, x, y);
    x = -x, y = -y;
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y));
    Pair n = pair(x, y);
    n = fma2(fma2(b, n, pair(k.one)), n, n);
    const Pair q = a * n;
    return fma2(fma2(b, q, a), n, q);
}

__device__ __forceinline__ float top3(float x, float y, float z)  // the largest magnitude; NaN if one is
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

__device__ __forceinline__ float low3(float x, float y, float z)  // the smallest magnitude
{
    float r;
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// Four consecutive elements as they lie in memory. Past a tensor's end they read as zero
// and are not written.
template <typename T> struct Four;
template <> struct Four<float> {
    uint4 q;
};
template <> struct Four<bf16> {
    uint2 q;
};
template <> struct Four<uint8_t> {
    uint32_t q;
};

template <bool kWhole, typename T> __device__ __forceinline__ Four<T> load4(const void* base, int64_t i, int64_t n)
{
    const T* p = static_cast<const T*>(base);
    Four<T> r = {};
    if (kWhole || i + 4 <= n) {
        r = *reinterpret_cast<const Four<T>*>(p + i);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) {
                if constexpr (sizeof(T) == 4) (&r.q.x)[j] = reinterpret_cast<const uint32_t*>(p)[i + j];
                else if constexpr (sizeof(T) == 2)
                    (&r.q.x)[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i + j] << (16 * (j & 1));
                else r.q |= (uint32_t)p[i + j] << (8 * j);
            }
    }
    return r;
}

__device__ __forceinline__ void widen(const Four<float>& r, float* v)
{
    v[0] = __uint_as_float(r.q.x), v[1] = __uint_as_float(r.q.y);
    v[2] = __uint_as_float(r.q.z), v[3] = __uint_as_float(r.q.w);
}

__device__ __forceinline__ void widen(const Four<bf16>& r, float* v)
{
    v[0] = __uint_as_float(r.q.x << 16), v[1] = __uint_as_float(r.q.x & 0xffff0000u);
    v[2] = __uint_as_float(r.q.y << 16), v[3] = __uint_as_float(r.q.y & 0xffff0000u);
}

template <bool kWhole> __device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, const float* v)
{
    if (kWhole || i + 4 <= n) {
        *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) p[i + j] = v[j];
    }
}

template <bool kWhole> __device__ __forceinline__ void store4(bf16* p, int64_t i, int64_t n, const float* v)
{
    if (kWhole || i + 4 <= n) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) p[i + j] = from_f32<bf16>(v[j]);
    }
}

template <bool kWhole> __device__ __forceinline__ void store4(uint8_t* p, int64_t i, int64_t n, uint32_t v)
{
    if (kWhole || i + 4 <= n) {
        *reinterpret_cast<uint32_t*>(p + i) = v;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) p[i + j] = (uint8_t)(v >> (8 * j));
    }
}

constexpr int kAwEach = kAwBlock / 32;  // elements of a lane
constexpr float kLow = 0x1p-60f, kHigh = 0x1p60f;

// The step on a lane's elements, two at a time. Where all of v and |m| lie in the range of
// root2 and minus_quotient2 (2^+-60, with the bounds that the host keeps on eps and root:
// `fast`), those are used; otherwise, also for zeros, the scalar operations are. v is left
// as its root when kRoot. Returns whether all of v is positive for sure.
template <bool kRoot>
__device__ __forceinline__ bool adam_lane(const Adam& k, bool fast, const float (&g)[kAwEach], float (&m)[kAwEach],
                                          float (&v)[kAwEach], float (&w)[kAwEach], float& mtop, float& vtop)
{
    float mlow = kHigh, vlow = kHigh;
    Pair m2[kAwEach / 2], v2[kAwEach / 2];
    mtop = vtop = 0.0f;
#pragma unroll
    for (int j = 0; j < kAwEach / 2; ++j) {
        const Pair d = pair(k.c) * pair(g[2 * j], g[2 * j + 1]);
        m2[j] = sum2(pair(k.beta1) * pair(m[2 * j], m[2 * j + 1]), pair(k.rest1) * d, pair(k.one));
        v2[j] = sum2(pair(k.beta2) * pair(v[2 * j], v[2 * j + 1]), pair(k.rest2) * (d * d), pair(k.one));
        float x, y, p, q;
        split(m2[j], x, y);
        split(v2[j], p, q);
        mtop = top3(mtop, x, y);
        vtop = top3(vtop, p, q);
        mlow = low3(mlow, x, y);
        vlow = low3(vlow, p, q);
    }
    if (fast && fminf(mlow, vlow) >= kLow && mtop <= kHigh && vtop <= kHigh) {
#pragma unroll
        for (int j = 0; j < kAwEach / 2; ++j) {
            const Pair u = root2(v2[j], k);
            const Pair q = minus_quotient2(m2[j], sum2(u * pair(k.root), pair(k.eps), pair(k.one)), k);
            const Pair x = sum2(pair(k.decay) * pair(w[2 * j], w[2 * j + 1]), pair(k.step) * q, pair(k.one));
            split(x, w[2 * j], w[2 * j + 1]);
            split(m2[j], m[2 * j], m[2 * j + 1]);
            split(kRoot ? u : v2[j], v[2 * j], v[2 * j + 1]);
        }
        return true;
    }
#pragma unroll
    for (int j = 0; j < kAwEach / 2; ++j) {
        split(m2[j], m[2 * j], m[2 * j + 1]);
        split(v2[j], v[2 * j], v[2 * j + 1]);
    }
#pragma unroll
    for (int j = 0; j < kAwEach; ++j) {  // unrolled: the elements are in registers
        float u;
        root_and_weight(k, m[j], v[j], u, w[j]);
        if (kRoot) v[j] = u;
    }
    return false;
}

struct Scales {
    float scale, inverse;
};

// The scale of a block whose largest magnitude is `top`, given as its bits (NaN is the
// largest of all). Below 2^-96, where 448 / top would come near overflow, there is none.
__device__ __forceinline__ Scales scales_of(float top, const Adam& k)
{
    Scales s = {0.0f, 0.0f};
    if (top >= kLow && top <= kHigh) {
        split(minus_quotient2(pair(-top, -448.0f), pair(448.0f, top), k), s.scale, s.inverse);
    } else if (!(top < 0x1p-96f)) {
        s.scale = __fdiv_rn(top, 448.0f);
        s.inverse = __fdiv_rn(448.0f, top);
    }
    return s;
}

// A lane's part of a block, as it lies in memory: four elements of either half, so that
// every access of a warp is contiguous.
template <typename W, typename G, bool kEight> struct Part {
    using S = typename std::conditional<kEight, uint8_t, float>::type;
    Four<W> w[2];
    Four<G> g[2];
    Four<S> m[2], v[2];
    float ms, vs;
};

// Where a block's results go.
template <typename W, typename S> struct Out {
    W* w;
    S *m, *v;
    bf16* copy;
    float *ms, *vs;
};

// `left`: elements from the block's start to the tensor's end; kWhole: at least a block.
template <bool kWhole, typename W, typename G, bool kEight>
__device__ __forceinline__ void adamw_block(const Out<W, typename Part<W, G, kEight>::S>& o, int64_t left,
                                            const Part<W, G, kEight>& r, const Adam& a, bool fast)
{
    const int lane4 = (threadIdx.x & 31) * 4;
    float wv[kAwEach], gv[kAwEach], mv[kAwEach], vv[kAwEach];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        widen(r.w[k], wv + 4 * k);
        widen(r.g[k], gv + 4 * k);
        if constexpr (kEight) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = 4 * k + 2 * j;
                const float2 m = from_e4m3x2(r.m[k].q >> (16 * j)), u = from_e4m3x2(r.v[k].q >> (16 * j));
                split(pair(m.x, m.y) * pair(r.ms), mv[e], mv[e + 1]);
                const Pair x = pair(u.x, u.y) * pair(r.vs);
                split(x * x, vv[e], vv[e + 1]);
            }
        } else {
            widen(r.m[k], mv + 4 * k);
            widen(r.v[k], vv + 4 * k);
        }
    }
    float mtop, vtop;
    const bool positive = adam_lane<kEight>(a, fast, gv, mv, vv, wv, mtop, vtop);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = lane4 + k * 128;
        store4<kWhole>(o.w, i, left, wv + 4 * k);
        if (o.copy) store4<kWhole>(o.copy, i, left, wv + 4 * k);
        if constexpr (!kEight) {
            store4<kWhole>(o.m, i, left, mv + 4 * k);
            store4<kWhole>(o.v, i, left, vv + 4 * k);
        }
    }
    if constexpr (kEight) {
        // magnitudes order as their bits do; the largest root is the root of the largest v
        const Scales p = scales_of(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop))), a);
        const Scales q =
            scales_of(__fsqrt_rn(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)))), a);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t m = 0, u = 0;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = 4 * k + 2 * j;
                float x, y;
                split(pair(mv[e], mv[e + 1]) * pair(p.inverse), x, y);
                m |= to_e4m3x2(x, y) << (16 * j);
                split(pair(vv[e], vv[e + 1]) * pair(q.inverse), x, y);
                if (positive || vv[e] > 0.0f) x = fmaxf(x, 0x1p-9f);  // the smallest e4m3: a positive root stays so
                if (positive || vv[e + 1] > 0.0f) y = fmaxf(y, 0x1p-9f);
                u |= to_e4m3x2(x, y) << (16 * j);
            }
            store4<kWhole>(o.m, lane4 + k * 128, left, m);
            store4<kWhole>(o.v, lane4 + k * 128, left, u);
        }
        if (lane4 == 0) {
            *o.ms = p.scale;
            *o.vs = q.scale;
        }
    }
}

// The tensor of consecutive tiles.
template <typename Table> struct Cursor {
    int id;
    uint32_t next;  // where the next tensor begins

    __device__ __forceinline__ Cursor(const Table& tab, uint32_t tile) : id(owner_of(tab, tile)) { bound(tab); }
    __device__ __forceinline__ void bound(const Table& tab)
    {
        next = id + 1 < tab.count ? tab.t[id + 1].tile_begin : 0xffffffffu;
    }
    __device__ __forceinline__ void to(const Table& tab, uint32_t tile)
    {
        if (tile < next) return;
        ++id;
        bound(tab);
    }
};

// Fills in what a kernel knows of the constants; false if the step is to be left out.
__device__ __forceinline__ bool step_constants(const AwHead& tab, Adam* a)
{
    *a = tab.k;
    if (tab.coefficient) a->c = *tab.coefficient;
    return isfinite(a->c);
}

// Asks for `bytes` from p on to be brought into L2 (whole 16-byte pieces).
__device__ __forceinline__ void prefetch(const void* p, int64_t bytes)
{
    if (bytes >= 16)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"((uint32_t)bytes & ~15u) : "memory");
}

// The step. Bound by memory: 28 bytes per element with fp32 weights, gradients and states,
// 14 with bf16 gradients and 8-bit states. One warp per block of 256 elements (one scale),
// a tile of eight blocks per CTA, no loop: the resident warps' loads keep the memory busy
// (134M elements, 32-bit states: 0.530 ms, 7.1 TB/s). With 8-bit states there are 2 KB of
// loads to a warp's 400 instructions; there one thread also has the tile `ahead` CTAs on
// (four per SM, less than run at once; 300 to 900 measure alike) brought into L2, so that
// its loads take an L2 access's time (1.3B elements: 2.58 ms, 7.2 TB/s; 2.80 without).
// Registers decide here: at 48 to 62 there are 40 or 32 warps per SM; with the scalar
// operations' inputs kept alive behind the test for them there were 24, and it took 3.4.
// Loading the next block ahead into registers (3.6) or shared memory (3.5) cost more warps
// than it gained. bf16 weights and gradients with 8-bit states (10 bytes per element) are
// bound by instructions: 134M elements 0.243 ms, 5.6 TB/s.
template <typename Table, typename W, typename G, bool kEight>
__global__ void __launch_bounds__(kAwThreads, kEight ? 5 : 4) adamw_kernel(const __grid_constant__ Table tab)
{
    using S = typename Part<W, G, kEight>::S;
    ptx::griddep_wait();
    if (kEight && threadIdx.x == kAwThreads - 32 && blockIdx.x + tab.ahead < tab.tiles) {
        const uint32_t tile = blockIdx.x + tab.ahead;
        const AwTensor& t = tab.t[owner_of(tab, tile)];
        const int64_t first = (int64_t)(tile - t.tile_begin) * kAwTile;
        const int64_t count = t.n - first < kAwTile ? t.n - first : kAwTile;
        prefetch(static_cast<const W*>(t.w) + first, count * (int)sizeof(W));
        prefetch(static_cast<const G*>(t.g) + first, count * (int)sizeof(G));
        prefetch(static_cast<const uint8_t*>(t.m) + first, count);
        prefetch(static_cast<const uint8_t*>(t.v) + first, count);
    }
    const AwTensor& t = tab.t[owner_of(tab, blockIdx.x)];
    const int64_t block = (int64_t)(blockIdx.x - t.tile_begin) * kAwWarps + (threadIdx.x >> 5);
    const int64_t first = block * kAwBlock, left = t.n - first;
    if (left <= 0) return;
    const Out<W, S> o = {static_cast<W*>(t.w) + first, static_cast<S*>(t.m) + first, static_cast<S*>(t.v) + first,
                         t.copy ? static_cast<bf16*>(t.copy) + first : nullptr, t.ms + block, t.vs + block};
    const G* g = static_cast<const G*>(t.g) + first;
    Part<W, G, kEight> r;
    const auto load = [&](auto whole) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = (threadIdx.x & 31) * 4 + k * 128;
            r.w[k] = load4<whole.value, W>(o.w, i, left);
            r.g[k] = load4<whole.value, G>(g, i, left);
            r.m[k] = load4<whole.value, S>(o.m, i, left);
            r.v[k] = load4<whole.value, S>(o.v, i, left);
        }
        if (kEight) {
            r.ms = *o.ms;
            r.vs = *o.vs;
        }
    };
    Adam a;
    if (left >= kAwBlock) {
        load(std::true_type());
        if (!step_constants(tab, &a)) return;
        a.decay = t.decay;
        adamw_block<true>(o, left, r, a, tab.fast != 0);
    } else {
        load(std::false_type());
        if (!step_constants(tab, &a)) return;
        a.decay = t.decay;
        adamw_block<false>(o, left, r, a, tab.fast != 0);
    }
}

// ---------------------------------------------------------------- norm
__device__ __forceinline__ double block_sum(double v, double* shared)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < kAwWarps; ++i) s += shared[i];
    return s;
}

// One 16-byte vector of a gradient, zeros past its end.
template <typename G> __device__ __forceinline__ uint4 load_vector(const G* g, int64_t i, int64_t n)
{
    constexpr int kPer = 16 / (int)sizeof(G);
    if (i + kPer <= n) return *reinterpret_cast<const uint4*>(g + i);
    uint32_t r[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (i + j < n) r[j * (int)sizeof(G) / 4] |= sizeof(G) == 4 ? reinterpret_cast<const uint32_t*>(g)[i + j]
                         : (uint32_t)reinterpret_cast<const uint16_t*>(g)[i + j] << (16 * (j & 1));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <typename G> __device__ __forceinline__ int values_of(uint32_t word, float (&v)[2])
{
    if (sizeof(G) == 4) {
        v[0] = __uint_as_float(word);
        return 1;
    }
    v[0] = __uint_as_float(word << 16);
    v[1] = __uint_as_float(word & 0xffff0000u);
    return 2;
}

// The sum of squares of all gradients. Bound by memory: each CTA (six per SM) reads a run of
// consecutive tiles, 64 bytes per thread in flight (1.3B bf16 elements: 0.366 ms, 7.2 TB/s).
// fp32 sums over the 16 or 32 elements of a thread's turn, fp64 from there on; a turn whose
// fp32 sum overflows, or is so small that squares may have vanished, is summed again in
// fp64. A CTA leaves one fp64 partial sum; the last CTA of the call adds the partial sums in
// their order.
template <typename Table, typename G>
__global__ void __launch_bounds__(kAwThreads, 6) grad_norm_kernel(const __grid_constant__ Table tab)
{
    constexpr int kPer = 16 / (int)sizeof(G);
    ptx::griddep_wait();
    __shared__ double shared[kAwWarps];
    __shared__ bool last;
    double sum = 0.0;
    uint32_t tile = (uint32_t)((uint64_t)tab.tiles * blockIdx.x / gridDim.x);
    const uint32_t end = (uint32_t)((uint64_t)tab.tiles * (blockIdx.x + 1) / gridDim.x);
    Cursor<Table> at(tab, tile);
    for (; tile < end; ++tile) {
        at.to(tab, tile);
        const NormTensor& t = tab.t[at.id];
        const G* g = static_cast<const G*>(t.g);
        const int64_t first = (int64_t)(tile - t.tile_begin) * (kNormVectors * kAwThreads * kPer) + threadIdx.x * kPer;
        uint32_t word[kNormVectors][4];
#pragma unroll
        for (int k = 0; k < kNormVectors; ++k) {
            const uint4 q = load_vector(g, first + k * (kAwThreads * kPer), t.n);
            word[k][0] = q.x, word[k][1] = q.y, word[k][2] = q.z, word[k][3] = q.w;
        }
        float s = 0.0f;
        uint32_t any = 0;
#pragma unroll
        for (int k = 0; k < kNormVectors * 4; ++k) {
            float v[2];
            const int c = values_of<G>(word[k / 4][k % 4], v);
            for (int j = 0; j < c; ++j) {
                s = fmaf(v[j], v[j], s);
                any |= __float_as_uint(v[j]) << 1;
            }
        }
        if (!(s >= 0x1p-90f && s < 0x1p+127f) && any != 0) {  // squares that overflow or vanish in fp32
#pragma unroll 1
            for (int k = 0; k < kNormVectors * kPer; ++k) {
                const int64_t i = first + k / kPer * (kAwThreads * kPer) + k % kPer;
                const double v = i < t.n ? (double)to_f32(g[i]) : 0.0;
                sum = fma(v, v, sum);
            }
        } else {
            sum += (double)s;
        }
    }
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0) {
        tab.part[tab.first_part + blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(tab.ticket, 1u) == tab.all_parts - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (uint32_t i = threadIdx.x; i < tab.all_parts; i += kAwThreads) sum += __ldcg(tab.part + i);
    __syncthreads();
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0) {
        const float norm = (float)(sqrt(sum) * (double)tab.scale);
        float k = 1.0f;
        if (tab.max_norm > 0.0f) k = fminf(__fdiv_rn(tab.max_norm, __fadd_rn(norm, 1e-6f)), 1.0f);
        tab.result[0] = norm;
        tab.result[1] = isfinite(norm) ? __fmul_rn(tab.scale, k) : __uint_as_float(0x7fc00000u);
        *tab.ticket = 0;
    }
}

uint32_t step_tiles(int64_t n) { return (uint32_t)((n + kAwTile - 1) / kAwTile); }

uint32_t norm_tiles(int64_t n, bool is_bf16)
{
    const int64_t per = (int64_t)kNormVectors * kAwThreads * (is_bf16 ? 8 : 4);
    return (uint32_t)((n + per - 1) / per);
}

}  // namespace
}  // namespace adacomp

struct adacomp_adamw {
    std::vector<int64_t> n;
    std::vector<uint8_t> w_bf16, g_bf16;
    std::vector<float> weight_decay;
    std::vector<int32_t> by_g[2];     // tensors by gradient type, as the norm's launches take them
    std::vector<int32_t> by_wg[4];    // and by weight and gradient type
    int32_t state_bits = 32;
    uint32_t norm_parts = 0;
    size_t norm_ws = 0;
};

namespace {

using namespace adacomp;

// The launches of one call: runs of at most `cap` tensors and 2^31 - 1 tiles.
template <typename T, typename F> adacomp_status for_runs(const std::vector<int32_t>& list, int cap, T&& tiles_of, F&& f)
{
    size_t i = 0;
    while (i < list.size()) {
        size_t j = i;
        uint64_t tiles = 0;
        while (j < list.size() && (int)(j - i) < cap) {
            const uint64_t more = tiles_of((size_t)list[j]);
            if (j > i && tiles + more > 0x7fffffffull) break;
            tiles += more;
            ++j;
        }
        const adacomp_status st = f(i, j, (uint32_t)tiles);
        if (st != ADACOMP_OK) return st;
        i = j;
    }
    return ADACOMP_OK;
}

// The pointers of a step, as the caller gave them.
struct StepPointers {
    void* const* weight;
    const void* const* grad;
    void *const *m, *const *v;
    float *const *m_scale, *const *v_scale;
    void* const* copy;
    float lr;
};

template <typename Table, typename W, typename G>
cudaError_t step_launch(const Table& tab, bool eight, cudaStream_t stream)
{
    return launch_after(eight ? adamw_kernel<Table, W, G, true> : adamw_kernel<Table, W, G, false>, dim3(tab.tiles),
                        dim3(kAwThreads), 0, stream, tab);
}

// One launch: tensors list[i .. j) of weight and gradient type `kind`.
template <typename Table>
adacomp_status step_run(const adacomp_adamw* h, const AwHead& head, const StepPointers& p,
                        const std::vector<int32_t>& list, size_t i, size_t j, int kind, cudaStream_t stream)
{
    const std::unique_ptr<Table> tab(new (std::nothrow) Table);
    if (!tab) return ADACOMP_ERR_INVALID_ARG;
    static_cast<AwHead&>(*tab) = head;
    const bool eight = h->state_bits == 8;
    uint32_t tile = 0;
    for (size_t q = i; q < j; ++q) {
        const size_t id = (size_t)list[q];
        AwTensor& t = tab->t[q - i];
        t.w = p.weight[id];
        t.g = p.grad[id];
        t.m = p.m[id];
        t.v = p.v[id];
        t.ms = eight ? p.m_scale[id] : nullptr;
        t.vs = eight ? p.v_scale[id] : nullptr;
        t.copy = p.copy ? p.copy[id] : nullptr;
        t.n = h->n[id];
        t.tile_begin = tile;
        t.decay = (float)(1.0 - (double)p.lr * (double)h->weight_decay[id]);
        tile += step_tiles(t.n);
    }
    tab->count = (int32_t)(j - i);
    tab->tiles = tile;
    fill_jumps(tab.get());
    const cudaError_t e = kind == 0   ? step_launch<Table, float, float>(*tab, eight, stream)
                          : kind == 1 ? step_launch<Table, float, bf16>(*tab, eight, stream)
                          : kind == 2 ? step_launch<Table, bf16, float>(*tab, eight, stream)
                                      : step_launch<Table, bf16, bf16>(*tab, eight, stream);
    return launch_result(e, stream);
}

// The same of the norm; *parts is where its partial sums start, and is moved past them.
template <typename Table>
adacomp_status norm_run(const adacomp_adamw* h, const NormHead& head, const void* const* grad,
                        const std::vector<int32_t>& list, size_t i, size_t j, bool is_bf16, uint32_t* parts,
                        cudaStream_t stream)
{
    const std::unique_ptr<Table> tab(new (std::nothrow) Table);
    if (!tab) return ADACOMP_ERR_INVALID_ARG;
    static_cast<NormHead&>(*tab) = head;
    uint32_t tile = 0;
    for (size_t q = i; q < j; ++q) {
        const size_t id = (size_t)list[q];
        tab->t[q - i] = {grad[id], h->n[id], tile};
        tile += norm_tiles(h->n[id], is_bf16);
    }
    const uint32_t grid = tile < (uint32_t)kNormGrid ? tile : (uint32_t)kNormGrid;
    tab->count = (int32_t)(j - i);
    tab->tiles = tile;
    tab->first_part = *parts;
    *parts += grid;
    fill_jumps(tab.get());
    return launch_result(launch_after(is_bf16 ? grad_norm_kernel<Table, bf16> : grad_norm_kernel<Table, float>,
                                      dim3(grid), dim3(kAwThreads), 0, stream, *tab), stream);
}

}  // namespace

extern "C" {

adacomp_status adacomp_adamw_init(adacomp_adamw_t* out, int32_t num_tensors, const int64_t* n,
                                  const int32_t* w_dtype, const int32_t* g_dtype, const float* weight_decay,
                                  int32_t state_bits, size_t* norm_ws_bytes)
{
    if (!out) return ADACOMP_ERR_INVALID_ARG;
    *out = nullptr;
    if (num_tensors < 1 || num_tensors > ADACOMP_MAX_TENSORS || !n || !w_dtype || !g_dtype ||
        (state_bits != 8 && state_bits != 32))
        return ADACOMP_ERR_INVALID_ARG;
    for (int32_t i = 0; i < num_tensors; ++i)
        if (n[i] < 1 || n[i] > (int64_t)1 << 40 || !known_dtype(w_dtype[i]) || !known_dtype(g_dtype[i]) ||
            (weight_decay && !std::isfinite(weight_decay[i])))
            return ADACOMP_ERR_INVALID_ARG;
    adacomp_adamw* h = nullptr;
    try {
        h = new adacomp_adamw;
        for (int32_t i = 0; i < num_tensors; ++i) {
            h->n.push_back(n[i]);
            h->w_bf16.push_back(w_dtype[i] == ADACOMP_BF16);
            h->g_bf16.push_back(g_dtype[i] == ADACOMP_BF16);
            h->weight_decay.push_back(weight_decay ? weight_decay[i] : 0.0f);
            h->by_g[h->g_bf16.back()].push_back(i);
            h->by_wg[h->w_bf16.back() * 2 + h->g_bf16.back()].push_back(i);
        }
    } catch (...) {
        delete h;
        return ADACOMP_ERR_INVALID_ARG;
    }
    h->state_bits = state_bits;
    for (int k = 0; k < 2; ++k)
        for_runs(h->by_g[k], kNormTensors, [&](size_t id) { return norm_tiles(h->n[id], k); },
                 [&](size_t, size_t, uint32_t tiles) {
                     h->norm_parts += tiles < (uint32_t)kNormGrid ? tiles : (uint32_t)kNormGrid;
                     return ADACOMP_OK;
                 });
    h->norm_ws = 16 + 8 * (size_t)h->norm_parts;
    if (norm_ws_bytes) *norm_ws_bytes = h->norm_ws;
    *out = h;
    return ADACOMP_OK;
}

adacomp_status adacomp_grad_norm(adacomp_adamw_t h, const void* const* grad, float grad_scale, float max_norm,
                                 float* result, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    TrainRange range("adacomp_grad_norm");
    if (!h || !grad || !result || !ws || !(grad_scale > 0.0f) || !std::isfinite(grad_scale) || std::isnan(max_norm))
        return ADACOMP_ERR_INVALID_ARG;
    if (!is_aligned(ws, 16) || !is_aligned(result, 4)) return ADACOMP_ERR_ALIGNMENT;
    if (ws_bytes < h->norm_ws) return ADACOMP_ERR_WORKSPACE;
    for (size_t i = 0; i < h->n.size(); ++i) {
        if (!grad[i]) return ADACOMP_ERR_INVALID_ARG;
        if (!is_aligned(grad[i], 16)) return ADACOMP_ERR_ALIGNMENT;
    }
    NormHead head = {};
    head.all_parts = h->norm_parts;
    head.scale = grad_scale;
    head.max_norm = max_norm;
    head.result = result;
    head.ticket = static_cast<uint32_t*>(ws);
    head.part = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 16);
    uint32_t parts = 0;
    adacomp_status st = ADACOMP_OK;
    for (int k = 0; k < 2 && st == ADACOMP_OK; ++k) {
        const std::vector<int32_t>& list = h->by_g[k];
        st = for_runs(list, kNormTensors, [&](size_t id) { return norm_tiles(h->n[id], k); },
                      [&](size_t i, size_t j, uint32_t) {
                          return j - i <= (size_t)kNormFew
                                     ? norm_run<NormShort>(h, head, grad, list, i, j, k, &parts, stream)
                                     : norm_run<NormLong>(h, head, grad, list, i, j, k, &parts, stream);
                      });
    }
    return st;
}

adacomp_status adacomp_adamw_step(adacomp_adamw_t h, void* const* weight, const void* const* grad, void* const* m,
                                  void* const* v, float* const* m_scale, float* const* v_scale, void* const* copy,
                                  float lr, float beta1, float beta2, float eps, float bias_correction1,
                                  float bias_correction2, float grad_scale, const float* coefficient,
                                  cudaStream_t stream)
{
    TrainRange range("adacomp_adamw_step");
    if (!h || !weight || !grad || !m || !v) return ADACOMP_ERR_INVALID_ARG;
    const bool eight = h->state_bits == 8;
    if (eight != (m_scale != nullptr) || eight != (v_scale != nullptr)) return ADACOMP_ERR_INVALID_ARG;
    if (!std::isfinite(lr) || !(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f) || !(eps > 0.0f) ||
        !std::isfinite(eps) || !(bias_correction1 > 0.0f) || !(bias_correction2 > 0.0f))
        return ADACOMP_ERR_INVALID_ARG;
    if (!is_aligned(coefficient, 4)) return ADACOMP_ERR_ALIGNMENT;
    for (size_t i = 0; i < h->n.size(); ++i) {
        if (!weight[i] || !grad[i] || !m[i] || !v[i] || (eight && (!m_scale[i] || !v_scale[i])))
            return ADACOMP_ERR_INVALID_ARG;
        if (!is_aligned(weight[i], 16) || !is_aligned(grad[i], 16) || !is_aligned(m[i], 16) || !is_aligned(v[i], 16) ||
            (eight && (!is_aligned(m_scale[i], 4) || !is_aligned(v_scale[i], 4))) || (copy && !is_aligned(copy[i], 16)))
            return ADACOMP_ERR_ALIGNMENT;
    }
    AwHead head = {};
    head.k.c = grad_scale;
    head.k.beta1 = beta1;
    head.k.beta2 = beta2;
    head.k.rest1 = 1.0f - beta1;
    head.k.rest2 = 1.0f - beta2;
    head.k.step = (float)((double)lr / (double)bias_correction1);
    head.k.root = (float)(1.0 / std::sqrt((double)bias_correction2));
    head.k.eps = eps;
    head.k.one = 1.0f;
    head.k.half = 0.5f;
    head.k.minus = -1.0f;
    // u <= 2^30 in adam_lane's range, so that u * root + eps lies within 2^+-40
    head.fast = eps >= 0x1p-40f && eps <= 0x1p30f && head.k.root <= 0x1p9f;
    head.coefficient = coefficient;
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return ADACOMP_ERR_CUDA;
    head.ahead = (uint32_t)(4 * sms);
    const StepPointers p = {weight, grad, m, v, m_scale, v_scale, copy, lr};
    adacomp_status st = ADACOMP_OK;
    for (int k = 0; k < 4 && st == ADACOMP_OK; ++k) {
        const std::vector<int32_t>& list = h->by_wg[k];
        st = for_runs(list, kAwTensors, [&](size_t id) { return step_tiles(h->n[id]); },
                      [&](size_t i, size_t j, uint32_t) {
                          return j - i <= (size_t)kAwFew ? step_run<AwShort>(h, head, p, list, i, j, k, stream)
                                                         : step_run<AwLong>(h, head, p, list, i, j, k, stream);
                      });
    }
    return st;
}

void adacomp_adamw_free(adacomp_adamw_t h) { delete h; }

}  // extern "C"
