// Products that are too small for tiles of the tensor cores' pairs: of a few rows, whose time is that of reading the
// weights once, and of small matrices, whose time is that of starting kernels.
#pragma once

#include "product.cuh"

namespace adacomp {
namespace {

// Four columns to an epilogue, one by one where its rows are not aligned.
template <typename Epi> __device__ __forceinline__ void put_piece(const Epi& epi, int32_t r, int32_t c, const Cols<4>& v)
{
    if (epi.whole) {
        epi.piece(r, c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < epi.n) epi.piece(r, c + i, Cols<1>{{v.v[i]}});
    }
}

// ---------------------------------------------------------------- few rows
constexpr int kFewBf16 = 16, kFewF32 = 8;  // rows, at most

struct FewArgs {
    const void *x, *w;
    int64_t x_stride, w_stride;
    int32_t rows, n, k;
};

// y of up to kTokens rows: bound by memory, the weights. A CTA has 16 of their rows, its warps a part of the
// terms each; a lane reads 16 bytes of two of them, and of a token's row, at a time, kAhead times before it
// computes. The terms of a product (mma of 16 x 8 x 16, of which the tokens are the columns) may come in any
// order, so a lane's eight consecutive ones are two pairs of two products. The tensor cores' own memory would
// add a round trip to each of these short sums. The warps' sums meet in shared memory.
template <typename Epi, int kTokens, int kWarps, bool kWhole>
__global__ void __launch_bounds__(kWarps * 32) few_bf16_kernel(const FewArgs g, const Epi epi)
{
    constexpr int kTiles = kTokens / 8, kAhead = kTokens == 8 ? 4 : 2;
    __shared__ __align__(16) float sums[kWarps][kTokens][20];
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, row = lane / 4, quad = lane & 3;
    const int32_t c0 = blockIdx.x * 16;
    const int32_t steps = (g.k + 31) / 32, each = (steps + kWarps - 1) / kWarps;
    const int32_t from = warp * each, to = from + each < steps ? from + each : steps;
    const bf16* w = static_cast<const bf16*>(g.w);
    const bf16* x = static_cast<const bf16*>(g.x);
    const auto load = [&](const bf16* p, int64_t stride, int32_t r, int32_t rows, int32_t k) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (r >= rows || k >= g.k) return q;
        p += r * stride + k;
        if (kWhole && k + 8 <= g.k) return *reinterpret_cast<const uint4*>(p);
        uint16_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = k + i < g.k ? reinterpret_cast<const uint16_t*>(p)[i] : (uint16_t)0;
        return make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
    };
    float d[kTiles][4] = {};
    for (int32_t s = from; s < to; s += kAhead) {
        uint4 a[kAhead][2], b[kAhead][kTiles];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int32_t k = s + i < to ? (s + i) * 32 + quad * 8 : g.k;
            a[i][0] = load(w, g.w_stride, c0 + row, g.n, k);
            a[i][1] = load(w, g.w_stride, c0 + row + 8, g.n, k);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) b[i][t] = load(x, g.x_stride, t * 8 + row, g.rows, k);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                    : "+f"(d[t][0]), "+f"(d[t][1]), "+f"(d[t][2]), "+f"(d[t][3])
                    : "r"(a[i][0].x), "r"(a[i][1].x), "r"(a[i][0].y), "r"(a[i][1].y), "r"(b[i][t].x), "r"(b[i][t].y));
                asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                    : "+f"(d[t][0]), "+f"(d[t][1]), "+f"(d[t][2]), "+f"(d[t][3])
                    : "r"(a[i][0].z), "r"(a[i][1].z), "r"(a[i][0].w), "r"(a[i][1].w), "r"(b[i][t].z), "r"(b[i][t].w));
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[warp][t * 8 + quad * 2 + (i & 1)][row + (i >> 1) * 8] = d[t][i];
    __syncthreads();
    if (threadIdx.x >= kTokens * 4) return;
    const int32_t r = threadIdx.x / 4, c = threadIdx.x % 4 * 4;
    if (r >= g.rows || c0 + c >= g.n) return;
    Cols<4> v = {};
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v = v + get<4>(&sums[i][r][c], 4);
    put_piece(epi, r, c0 + c, v);
}

// The same of fp32 numbers: a warp has four rows of the weights, its lanes four terms each at a time. (8 x 2048
// x 8192 32 us, bound by the tokens' loads from L1, of which there are two for one of the weights'; two rows a
// warp 44.)
template <typename Epi, int kTokens, bool kWhole>
__global__ void __launch_bounds__(256, 2) few_f32_kernel(const FewArgs g, const Epi epi)
{
    constexpr int kOut = 4;
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int lane = threadIdx.x & 31;
    const int32_t c0 = (blockIdx.x * 8 + threadIdx.x / 32) * kOut;
    if (c0 >= g.n) return;
    const float* w = static_cast<const float*>(g.w);
    const float* x = static_cast<const float*>(g.x);
    float d[kTokens][kOut] = {};
#pragma unroll(kTokens == 8 ? 1 : 2)
    for (int32_t k = lane * 4; k < g.k; k += 128) {
        const auto load = [&](const float* p, int32_t left) {
            if constexpr (kWhole) {
                return get<4>(p, left);
            } else {
                Cols<4> v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v.v[i] = i < left ? p[i] : 0.0f;
                return v;
            }
        };
        Cols<4> a[kOut];
#pragma unroll
        for (int i = 0; i < kOut; ++i) a[i] = load(w + (c0 + i) * g.w_stride + k, c0 + i < g.n ? g.k - k : 0);
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const Cols<4> b = load(x + t * g.x_stride + k, t < g.rows ? g.k - k : 0);
#pragma unroll
            for (int i = 0; i < kOut; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[t][i] = fmaf(a[i].v[j], b.v[j], d[t][i]);
        }
    }
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
        Cols<4> v = {};
#pragma unroll
        for (int i = 0; i < kOut; ++i) v.v[i] = warp_sum(d[t][i]);
        if (lane != t || t >= g.rows) continue;
        put_piece(epi, t, c0, v);
    }
}

template <typename T, typename Epi> cudaError_t product_few(const FewArgs& g, const Epi& epi, cudaStream_t stream)
{
    const bool whole = whole_rows(g.x, g.x_stride, g.rows, sizeof(T)) && whole_rows(g.w, g.w_stride, g.n, sizeof(T));
    if constexpr (sizeof(T) == 4) {
        const auto with = [&](auto kernel) { return launch_after(kernel, dim3((unsigned)((g.n + 31) / 32)), dim3(256), 0, stream, g, epi); };
        if (!whole) return with(few_f32_kernel<Epi, 8, false>);
        if (g.rows == 1) return with(few_f32_kernel<Epi, 1, true>);
        return g.rows <= 4 ? with(few_f32_kernel<Epi, 4, true>) : with(few_f32_kernel<Epi, 8, true>);
    } else {
        const auto with = [&](auto kernel, int warps) {
            return launch_after(kernel, dim3((unsigned)((g.n + 15) / 16)), dim3(warps * 32), 0, stream, g, epi);
        };
        if (!whole) return with(few_bf16_kernel<Epi, 16, 8, false>, 8);
        const bool many = g.n <= 16 * 304;  // few CTAs: more warps in each
        if (g.rows <= 8) return many ? with(few_bf16_kernel<Epi, 8, 16, true>, 16) : with(few_bf16_kernel<Epi, 8, 8, true>, 8);
        return many ? with(few_bf16_kernel<Epi, 16, 16, true>, 16) : with(few_bf16_kernel<Epi, 16, 8, true>, 8);
    }
}

// ---------------------------------------------------------------- small matrices
struct Operand {
    const void* p;
    int64_t row, term;  // distances of rows, and of terms; one of them is 1
};

struct SmallArgs {
    Operand a, b;
    int32_t m, n, k, parts;
};

constexpr int kSmallTile = 32, kSmallDepth = 128;

// A CTA has a tile of 32 x 32, 128 terms at a time in shared memory, of which a warp has 16; a thread has 4 x 8
// of the tile's sums, fp32, in its warp's terms; the warps' sums meet in shared memory. A block of terms takes
// over a microsecond, most of it waiting for loads, so where tiles are few the terms are split over the CTAs of
// a cluster, whose sums the first one reads from the others' shared memory.
template <typename A, typename B, typename Epi> __global__ void __launch_bounds__(256) product_small_kernel(const SmallArgs g, const Epi epi)
{
    constexpr int kPitch = kSmallTile + 4, kEach = kSmallTile * kSmallDepth / 256;
    __shared__ __align__(16) float tile[8 * kSmallTile * kPitch];  // both operands' terms; then the warps' sums
    float *sa = tile, *sb = tile + kSmallDepth * kPitch;
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, r = lane / 4 * 4, c = lane % 4 * 8;
    const int32_t place = blockIdx.x / g.parts, part = blockIdx.x % g.parts, tiles_n = (g.n + kSmallTile - 1) / kSmallTile;
    const int32_t m0 = place / tiles_n * kSmallTile, n0 = place % tiles_n * kSmallTile;
    const int32_t blocks = (g.k + kSmallDepth - 1) / kSmallDepth, each = (blocks + g.parts - 1) / g.parts;
    const int32_t first = part * each * kSmallDepth, end = g.k - first < each * kSmallDepth ? g.k : first + each * kSmallDepth;
    // A thread's elements of an operand's block are kEach places `step` apart, along its rows or its terms.
    struct Mine {
        const char* p;
        int64_t step, next;         // bytes between a block's elements, and to the next block
        int32_t term, row, left, each;  // its first element; how far the other coordinate may go, in elements of the block
        int32_t at, at_step;        // in shared memory
        bool by_terms;
    };
    const auto mine = [&](const Operand& o, int32_t r0, int32_t rows, int32_t bytes) {
        Mine m;
        m.by_terms = o.term == 1;
        m.term = m.by_terms ? threadIdx.x % kSmallDepth : threadIdx.x / kSmallTile;
        m.row = m.by_terms ? threadIdx.x / kSmallDepth : threadIdx.x % kSmallTile;
        m.each = m.by_terms ? 256 / kSmallDepth : 256 / kSmallTile;
        m.step = m.each * (m.by_terms ? o.row : o.term) * bytes;
        m.next = kSmallDepth * o.term * bytes;
        m.p = static_cast<const char*>(o.p) + ((r0 + m.row) * o.row + (int64_t)(first + m.term) * o.term) * bytes;
        m.left = rows - r0 - m.row;
        m.at = m.term * kPitch + m.row;
        m.at_step = m.each * (m.by_terms ? 1 : kPitch);
        return m;
    };
    const auto load = [&](auto type, Mine& m, int32_t k0, float (&v)[kEach]) {
        const int32_t terms = end - k0 - m.term;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const bool there = m.by_terms ? terms > 0 && i * m.each < m.left : m.left > 0 && i * m.each < terms;
            v[i] = there ? to_f32(*reinterpret_cast<const decltype(type)*>(m.p + i * m.step)) : 0.0f;
        }
        m.p += m.next;
    };
    const auto store = [&](const Mine& m, float* s, const float (&v)[kEach]) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) s[m.at + i * m.at_step] = v[i];
    };
    float va[kEach], vb[kEach], d[4][8] = {};
    Mine ma = mine(g.a, m0, g.m, sizeof(A)), mb = mine(g.b, n0, g.n, sizeof(B));
    load(A{}, ma, first, va);
    load(B{}, mb, first, vb);
    for (int32_t k0 = first; k0 < end; k0 += kSmallDepth) {
        store(ma, sa, va);
        store(mb, sb, vb);
        __syncthreads();
        if (k0 + kSmallDepth < end) {
            load(A{}, ma, k0 + kSmallDepth, va);
            load(B{}, mb, k0 + kSmallDepth, vb);
        }
#pragma unroll
        for (int i = 0; i < kSmallDepth / 8; ++i) {
            const int k = warp * (kSmallDepth / 8) + i;
            const float4 a = *reinterpret_cast<const float4*>(sa + k * kPitch + r);
            const float4 b0 = *reinterpret_cast<const float4*>(sb + k * kPitch + c), b1 = *reinterpret_cast<const float4*>(sb + k * kPitch + c + 4);
            const float x[4] = {a.x, a.y, a.z, a.w}, y[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int q = 0; q < 8; ++q) d[p][q] = fmaf(x[p], y[q], d[p][q]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 8; q += 4)
            *reinterpret_cast<float4*>(tile + (warp * kSmallTile + r + p) * kPitch + c + q) = make_float4(d[p][q], d[p][q + 1], d[p][q + 2], d[p][q + 3]);
    __syncthreads();
    const int row = threadIdx.x / 8, col = threadIdx.x % 8 * 4;
    Cols<4> v = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) v = v + get<4>(tile + (i * kSmallTile + row) * kPitch + col, 4);
    if (g.parts > 1) {
        float* mine_at = tile + row * kPitch + col;
        __syncthreads();
        put(mine_at, v, 4);
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
        if (part == 0) {
            for (int i = 1; i < g.parts; ++i) {
                uint32_t at;
                Cols<4> more;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_addr(mine_at)), "r"(i));
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(more.v[0]), "=f"(more.v[1]), "=f"(more.v[2]), "=f"(more.v[3])
                             : "r"(at)
                             : "memory");
                v = v + more;
            }
        }
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    }
    if (part == 0 && m0 + row < g.m && n0 + col < g.n) put_piece(epi, m0 + row, n0 + col, v);
}

template <typename A, typename B, typename Epi> cudaError_t product_small(SmallArgs g, const Epi& epi, cudaStream_t stream)
{
    const int64_t tiles = (int64_t)((g.n + kSmallTile - 1) / kSmallTile) * ((g.m + kSmallTile - 1) / kSmallTile);
    // up to two CTAs an SM, of no fewer than a block of terms
    for (g.parts = 1; g.parts < 8 && tiles * g.parts * 2 <= 304 && g.k >= g.parts * 2 * kSmallDepth;) g.parts *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)g.parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * g.parts));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = g.parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, product_small_kernel<A, B, Epi>, (const SmallArgs)g, epi);
}

}  // namespace
}  // namespace adacomp
