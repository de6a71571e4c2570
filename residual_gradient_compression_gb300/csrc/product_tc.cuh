// Products on the tensor cores: C(m, n) = sum over k of A(m, k) B(n, k), bf16 operands, fp32 sums.
//
// A pair of CTAs (a cluster of two SMs) has tiles of 256 rows and up to 256 columns; each loads its 128 rows of
// A and its half of B's rows for 64 terms at a time, by TMA, into a ring of stages; one thread of the first CTA
// issues the products (tcgen05.mma, cta_group::2) on both CTAs' shared memory; the sums lie in tensor memory,
// 128 rows in each CTA, in two buffers. Eight warps take them over into registers, 128 columns of a row per
// thread, and hand them to the epilogue while the next tile is computed (sixteen with 64 columns each were
// slower, by the stores that they have under way at once). Where results are held in fp32 they do so every `run`
// blocks of terms and add the runs up: tensor memory's sums are truncated at every step, all in one direction,
// which over 2048 terms is 8e-7 of a sum. Each operand lies by rows of terms ("k major") or by terms of rows
// ("mn major", the transposed operands of the gradients): both are copied as they lie and told apart by the
// matrix descriptors.
//
// fp32 operands are four planes of bf16 numbers (split_parts), and their product is the sum of six products of
// planes, the smallest first.
#pragma once

#include <cuda.h>

#include "product.cuh"

namespace adacomp {
namespace {

constexpr int kTcThreads = 384;      // warps 0..3: copies, products, tensor memory, none; 4..11: epilogue
constexpr int kTcEpilogue = 4;       // the epilogue's first warp
constexpr int kTcDepth = 64;         // terms of a stage: 128 bytes of bf16
constexpr int kTcM = 256;            // rows of a pair's tile
constexpr int kTcN = 256;            // and columns, at most: a multiple of 32

// How long a wait goes on after its first tries (some 17 ms), and a CTA of every pair that makes no copies
// (0 or 1; tests only).
struct TcWaits {
    uint64_t limit_ns = 2000000000ull;
    uint32_t silent = 0xffffffffu;
};

constexpr int kTcStageA = 128 * kTcDepth * 2, kTcStageB = kTcN / 2 * kTcDepth * 2;  // bytes of a CTA's stage
constexpr int kTcStages = 196608 / (kTcStageA + kTcStageB);
constexpr int kTcStage = 4096;  // of an epilogue warp
constexpr int kTcShared = kTcStages * (kTcStageA + kTcStageB) + 8 * kTcStage + 1024;  // 1024: to begin on such a boundary

// ---------------------------------------------------------------- operands
// A matrix as a product takes it: rows of `cols` bf16 numbers that are contiguous, 16-byte aligned rows `stride`
// apart, and planes `plane` apart.
struct Matrix {
    const bf16* p;
    int64_t rows, cols, stride, plane;
};

struct TcArgs {
    int64_t m, n, k;
    const int32_t *m_count, *k_count;  // how many of the rows m, or terms k, there are; NULL: all
    int32_t passes;                    // products of planes that are summed: 1, two of a bf16 A in two parts, or kSix
    int32_t splits;                    // of the terms, each a product of its own
    int32_t a_mn, b_mn;                // operands that lie by terms
    int32_t run;                       // blocks of terms whose sums are formed in tensor memory
    int32_t width;                     // columns of a tile
    int32_t group;                     // tiles of rows that are taken before the next column's
    int32_t least;                     // blocks of terms whose time a tile's end takes
};

struct PackArgs {
    const void* from;
    bf16* to;
    const int32_t *map, *count;  // which rows, and how many; NULL: all
    int64_t rows, cols, from_stride, to_stride, plane;
    bool whole;  // rows that can be read 16 bytes at a time
};

// A matrix of any layout by rows of contiguous elements as aligned rows of bf16 numbers (planes of them for
// fp32); with `count`, zeros from there to a whole tile. A thread takes eight elements at a time.
constexpr int kTcPack = 256;
template <typename T>
__device__ __forceinline__ void pack_rows(const PackArgs& a, const int32_t* map, int64_t count, int64_t rows)
{
    const int64_t each = (a.cols + 7) / 8, all = rows * each;
    for (int64_t i = (int64_t)blockIdx.x * kTcPack + threadIdx.x; i < all; i += (int64_t)gridDim.x * kTcPack) {
        const int64_t r = i / each, c = (i - r * each) * 8;
        const T* from = static_cast<const T*>(a.from) + (r < count ? (map ? (int64_t)map[r] : r) * a.from_stride : 0) + c;
        float x[8];
        get_chunk(from, x, r < count ? a.cols - c : 0, a.whole);
        __align__(16) bf16 v[sizeof(T) == 4 ? kPlanes : 1][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(T) == 4) {
                bf16 part[kPlanes];
                split_parts(x[j], part);
#pragma unroll
                for (int p = 0; p < kPlanes; ++p) v[p][j] = part[p];
            } else {
                v[0][j] = __float2bfloat16_rn(x[j]);
            }
        }
        bf16* to = a.to + r * a.to_stride + c;
#pragma unroll
        for (int p = 0; p < (sizeof(T) == 4 ? kPlanes : 1); ++p)
            *reinterpret_cast<uint4*>(to + p * a.plane) = *reinterpret_cast<const uint4*>(v[p]);
    }
}

template <typename T> __global__ void __launch_bounds__(kTcPack) pack_kernel(const PackArgs a)
{
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int64_t count = a.count ? *a.count : a.rows;
    pack_rows<T>(a, a.map, count, a.count ? (count + kRows - 1) / kRows * kRows : count);
}

// ---------------------------------------------------------------- instructions
namespace tc {

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// One lane of a converged warp. The instructions that a single thread issues take their operands from uniform
// registers, and under this predicate, in loops of the whole warp, the compiler keeps them there (with a branch for
// one lane they are moved there each time: 8192 x 2048 x 16384 bf16 took 369 us, and 287 so).
__device__ __forceinline__ bool elect()
{
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t map_shared(const void* p, uint32_t rank)  // where p is in a CTA of the cluster
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_addr(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ void arrive_at(uint32_t bar)  // an address of the cluster
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A wait bounded in time; false when it ran out, here or in another warp (dead). A try that fails takes 4 us, and the
// clock is looked at after many tries only.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* dead, uint64_t limit)
{
    const uint64_t from = ptx::globaltimer();
    while (!*dead && ptx::globaltimer() - from <= limit) {
        for (int i = 0; i < 64; ++i)
            if (ptx::mbar_try_wait(bar, parity)) return true;
    }
    *dead = 1;
    return false;
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* dead, uint64_t limit)
{
#pragma unroll 1
    for (int i = 0; i < 4096; ++i)
        if (ptx::mbar_try_wait(bar, parity)) return true;
    return wait_long(bar, parity, dead, limit);
}

__device__ __forceinline__ void load(uint32_t to, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Of a tile in shared memory, in the 128-byte swizzle that TMA writes: where it begins, and the distances (bytes) of
// 64-element blocks along the rows (mn major only) and of groups of eight 128-byte lines.
__device__ __forceinline__ uint64_t descriptor(uint32_t at, uint32_t block, uint32_t group)
{
    return (uint64_t)((at & 0x3ffff) >> 4) | (uint64_t)(block >> 4) << 16 | (uint64_t)(group >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}

// Arrives at the barrier in both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void read_chunk(uint32_t at, uint32_t (&v)[16])  // 32 lanes' rows, 16 columns each
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void read_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

}  // namespace tc

constexpr double kTcBlock = 0.32;  // us, by estimate: a block of terms and 256 columns, per pass
// A tile's end, which goes on while the next one's sums are formed: where pairs have several units, none is counted as
// shorter than that (64 rows' gradients of 2048 x 8192 bf16 85 us without this, a few pairs having most of dw's tiles, and
// 31 so; the gradients of 32 rows against 50304 tokens 540 and 286).
constexpr double kTcEnd = 4.0;

// The pairs of planes of fp32 operands whose products are summed, the smallest first. Of a bf16 product A may
// have two planes, of which the second is what the first leaves of it.
constexpr int kSix = 6;
__device__ __forceinline__ int plane_a(int pass) { return (0x231130 >> 4 * (5 - pass)) & 15; }
__device__ __forceinline__ int plane_b(int pass) { return (0x321310 >> 4 * (5 - pass)) & 15; }

// ---------------------------------------------------------------- kernel
// One product, or two at once, of which the first has the longer sums.
struct TcMaps {
    CUtensorMap a[2], b[2];
};

template <typename Epi> struct TcParams {
    TcArgs g[2];
    Epi epi[2];
    TcWaits waits;
};

// What each pair of CTAs does when two products are computed at once: of the first one's units (tiles, or parts
// of their sums) every pairs-th; then of the second one's so many that all pairs have about as much to do: those
// with a unit more of the first (the first `more` pairs) `few` of them, the others `many`. Also on the host,
// which compares ways to split the sums by it.
struct TcShares {
    int64_t more, each, few, many, blocks;  // blocks: what the busiest pair has to do
    __host__ __device__ TcShares(int64_t pairs, int64_t units_a, int64_t a, int64_t units_b, int64_t b)
    {
        each = units_a / pairs;
        more = units_a - each * pairs;
        b = b > 0 ? b : 1;
        for (blocks = (a * units_a + b * units_b + pairs - 1) / pairs;; blocks += b) {
            few = blocks > a * (each + 1) ? (blocks - a * (each + 1)) / b : 0;
            many = blocks > a * each ? (blocks - a * each) / b : 0;
            if (more * few + (pairs - more) * many >= units_b) break;
        }
        if (more && blocks < a * (each + 1)) blocks = a * (each + 1);
    }
};

struct TcUnit {
    int32_t m0, n0, from, count, split, which;
};

// (Counts of units fit in 32 bits: 2^31 tiles would be a result of 2^47 elements.)
template <bool kBoth> struct TcSchedule {
    int32_t m[2], tiles_m[2], tiles_n[2], blocks[2], per_split[2], tiles[2], units[2], more, few, many, mine;

    __device__ __forceinline__ TcSchedule(const TcArgs (&g)[2])
    {
        const int32_t pairs = gridDim.x / 2, pair = blockIdx.x / 2;
#pragma unroll
        for (int i = 0; i < (kBoth ? 2 : 1); ++i) {
            m[i] = (int32_t)(g[i].m_count ? *g[i].m_count : g[i].m);
            const int32_t terms = (int32_t)(g[i].k_count ? *g[i].k_count : g[i].k);
            tiles_m[i] = (m[i] + kTcM - 1) / kTcM;
            tiles_n[i] = ((int32_t)g[i].n + g[i].width - 1) / g[i].width;
            blocks[i] = (terms + kTcDepth - 1) / kTcDepth;
            per_split[i] = (blocks[i] + g[i].splits - 1) / g[i].splits;
            tiles[i] = tiles_m[i] * tiles_n[i];
            units[i] = tiles[i] * g[i].splits;
        }
        if constexpr (kBoth) {
            int64_t unit[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t least = units[0] + units[1] > pairs ? g[i].least : 0;
                unit[i] = (int64_t)(per_split[i] > least ? per_split[i] : least) * g[i].width;
            }
            const TcShares shares(pairs, units[0], unit[0], units[1], unit[1]);
            more = (int32_t)shares.more;
            few = (int32_t)shares.few;
            many = (int32_t)shares.many;
            mine = (int32_t)shares.each + (pair < more);  // of the first product
        }
    }

    __device__ __forceinline__ bool at(const TcArgs (&g)[2], int32_t i, TcUnit& t) const
    {
        const int32_t pairs = gridDim.x / 2, pair = blockIdx.x / 2;
        int32_t unit = pair + i * pairs;
        bool second = false;
        if (kBoth && i >= mine) {
            const int32_t j = i - mine;
            second = true;
            if (j >= (pair < more ? few : many)) return false;
            unit = pair < more ? j * more + pair : more * few + j * (pairs - more) + (pair - more);
        }
        if (unit >= (second ? units[1] : units[0])) return false;
        t.which = second;
        const int32_t tm = second ? tiles_m[1] : tiles_m[0], tn = second ? tiles_n[1] : tiles_n[0], gr = g[second].group;
        const int32_t all = second ? blocks[1] : blocks[0], part = second ? per_split[1] : per_split[0];
        const int32_t count = second ? tiles[1] : tiles[0];
        t.split = unit / count;
        const int32_t tile = unit - t.split * count, whole = gr * tn, band = tile / whole, in = tile - band * whole;
        const int32_t rows = tm - band * gr < gr ? tm - band * gr : gr;
        t.n0 = in / rows * g[second].width;
        t.m0 = (band * gr + in % rows) * kTcM;
        t.from = t.split * part;
        t.count = all - t.from < part ? all - t.from : part;
        if (t.count < 0) t.count = 0;
        return true;
    }
};

template <bool kBoth, typename Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    product_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcParams<Epi> params)
{
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ __align__(8) uint64_t full[kTcStages], empty[kTcStages], sums_full[2], sums_empty[2], drained;
    __shared__ uint32_t tmem_at;
    __shared__ int dead_flag;
    volatile int* dead = &dead_flag;
    const uint64_t limit = params.waits.limit_ns;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const uint32_t base = (ptx::smem_addr(raw) + 1023) & ~1023u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kTcStages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sums_full[i], 1);
            ptx::mbar_init(&sums_empty[i], 2 * 8);  // a thread of each of both CTAs' epilogue warps
        }
        ptx::mbar_init(&drained, 1);
        dead_flag = 0;
        ptx::fence_mbar_init();
#pragma unroll
        for (int i = 0; i < (kBoth ? 2 : 1); ++i) {
            tc::prefetch(&maps.a[i]);
            tc::prefetch(&maps.b[i]);
        }
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_addr(&tmem_at)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        tc::fence_before();
    }
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = tmem_at;
    ptx::griddep_wait();
    const TcSchedule<kBoth> schedule(params.g);
    TcUnit t;

    // 384 threads of 168 registers: 128 with 40 and 256 with 232 are as many
    if (warp < kTcEpilogue) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {  // copies
            uint32_t at_stage = 0, turn = 0, issued = 0;
            const uint32_t full_at = tc::map_shared(full, 0);  // the first CTA's
            bool alive = rank != params.waits.silent;
            for (int32_t u = 0; alive && schedule.at(params.g, u, t); ++u) {
                const TcArgs& g = params.g[kBoth ? t.which : 0];
                const CUtensorMap *map_a = &maps.a[kBoth ? t.which : 0], *map_b = &maps.b[kBoth ? t.which : 0];
                const int passes = g.passes;
                const int32_t ma = t.m0 + (int32_t)rank * 128, nb = t.n0 + (int32_t)rank * (g.width / 2);
                const uint32_t bytes = kTcStageA + (g.b_mn ? (g.width + 127) / 128 * 8192 : g.width * kTcDepth);
                for (int32_t from = 0; from < t.count && alive; from += g.run) {
                    const int32_t end = t.count - from < g.run ? t.count : from + g.run;
                    for (int pass = 0; pass < passes && alive; ++pass) {
                        const int pa = passes == kSix ? plane_a(pass) : passes - 1 - pass, pb = passes == kSix ? plane_b(pass) : 0;
                        for (int32_t k = from; k < end; ++k) {
                            alive = __all_sync(0xffffffffu, tc::wait(&empty[at_stage], turn ^ 1, dead, limit));
                            if (!alive) break;
                            const uint32_t bar = full_at + at_stage * 8, at = base + at_stage * (kTcStageA + kTcStageB);
                            const int32_t k0 = (t.from + k) * kTcDepth;
                            if (tc::elect()) {
                                if (rank == 0) ptx::mbar_arrive_expect_tx(&full[at_stage], 2 * bytes);
                                if (g.a_mn) {
#pragma unroll
                                    for (int i = 0; i < 2; ++i) tc::load(at + i * 8192, map_a, ma + 64 * i, k0, pa, bar);
                                } else {
                                    tc::load(at, map_a, k0, ma, pa, bar);
                                }
                                if (g.b_mn) {
                                    tc::load(at + kTcStageA, map_b, nb, k0, pb, bar);
                                    if (g.width > 128) tc::load(at + kTcStageA + 8192, map_b, nb + 64, k0, pb, bar);
                                } else {
                                    tc::load(at + kTcStageA, map_b, k0, nb, pb, bar);
                                }
                            }
                            ++issued;
                            if (++at_stage == kTcStages) at_stage = 0, turn ^= 1;
                        }
                    }
                }
            }
            if (!alive) {  // the copies in flight end before the CTA does: each stage's last one
                int none = 0;
                if (rank == 0) {
                    for (uint32_t i = issued > kTcStages ? issued - kTcStages : 0; i < issued; ++i)
                        tc::wait(&full[i % kTcStages], i / kTcStages & 1, &none, limit);
                } else {  // their barrier is the other CTA's: 10 ms
                    const uint64_t from = ptx::globaltimer();
                    while (ptx::globaltimer() - from < 10000000ull) {}
                }
            }
        } else if (warp == 1 && rank == 0) {  // products
            uint32_t at_stage = 0, turn = 0, done = 0;
            bool alive = true;
            for (int32_t u = 0; alive && schedule.at(params.g, u, t); ++u) {
                const TcArgs& g = params.g[kBoth ? t.which : 0];
                const int passes = g.passes;
                const uint32_t kind = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(g.a_mn != 0) << 15 | (uint32_t)(g.b_mn != 0) << 16 |
                                      (uint32_t)(g.width / 8) << 17 | (uint32_t)(kTcM / 16) << 24;
                // 16 terms further: 32 bytes along a line, or 16 lines
                const uint32_t step_a = (g.a_mn ? 2048 : 32) >> 4, step_b = (g.b_mn ? 2048 : 32) >> 4;
                const uint64_t first_a = tc::descriptor(base, g.a_mn ? 8192 : 16, 1024);
                const uint64_t first_b = tc::descriptor(base + kTcStageA, g.b_mn ? 8192 : 16, 1024);
                for (int32_t from = 0; from < t.count && alive; from += g.run) {
                    const int buffer = (int)(done & 1);
                    alive = __all_sync(0xffffffffu, tc::wait(&sums_empty[buffer], (done / 2 & 1) ^ 1, dead, limit));
                    if (!alive) break;
                    tc::fence_after();
                    const uint32_t d = tmem + buffer * 256;
                    const int32_t all = (t.count - from < g.run ? t.count - from : g.run) * passes;
                    for (int32_t i = 0; i < all; ++i) {
                        alive = __all_sync(0xffffffffu, tc::wait(&full[at_stage], turn, dead, limit));
                        if (!alive) break;
                        tc::fence_after();
                        const uint32_t at = at_stage * ((kTcStageA + kTcStageB) >> 4);
                        if (tc::elect()) {
#pragma unroll
                            for (int j = 0; j < kTcDepth / 16; ++j)
                                tc::mma(d, first_a + at + j * step_a, first_b + at + j * step_b, kind, i > 0 || j > 0);
                            tc::commit(&empty[at_stage]);
                        }
                        if (++at_stage == kTcStages) at_stage = 0, turn ^= 1;
                    }
                    if (!alive) break;
                    if (tc::elect()) tc::commit(&sums_full[buffer]);
                    ++done;
                }
            }
            if (!alive) {  // the products in flight end before the tensor memory is given back
                int none = 0;
                if (tc::elect()) tc::commit(&drained);
                tc::wait(&drained, 0, &none, limit);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int quarter = warp & 3, strip = (warp - kTcEpilogue) / 4;
        const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + strip * kStrip;
        const Stage stage = {reinterpret_cast<float4*>(raw + (base - ptx::smem_addr(raw)) + kTcStages * (kTcStageA + kTcStageB) +
                                                       (warp - kTcEpilogue) * kTcStage)};
        const uint32_t freed[2] = {tc::map_shared(&sums_empty[0], 0), tc::map_shared(&sums_empty[1], 0)};
        uint32_t done = 0;
        bool alive = true;
        for (int32_t u = 0; schedule.at(params.g, u, t); ++u) {
            const TcArgs& g = params.g[kBoth ? t.which : 0];
            const Epi& epi = params.epi[kBoth ? t.which : 0];
            const int32_t m = kBoth && t.which ? schedule.m[1] : schedule.m[0], n = t.n0 + g.width < g.n ? t.n0 + g.width : (int32_t)g.n;
            const int32_t r = t.m0 + (int32_t)rank * 128 + quarter * 32 + lane, c0 = t.n0 + strip * kStrip;
            typename Epi::State state = {};
            if (r < m && c0 < n) state = epi.begin(r, c0);
            float v[kStrip];
#pragma unroll
            for (int i = 0; i < kStrip; ++i) v[i] = 0.0f;
            Fetched ahead;
            bool fetches = false;
            if constexpr (Epi::kFetches) {
                fetches = c0 < n && g.splits == 1 && epi.fetches();
                if (fetches) epi.fetch(ahead, r - lane, m, c0);
            }
#pragma unroll 1
            for (int32_t from = 0; from < t.count; from += g.run, ++done) {
                const int buffer = (int)(done & 1);
                alive = __all_sync(0xffffffffu, alive && tc::wait(&sums_full[buffer], done / 2 & 1, dead, limit));
                if (!alive) break;
                tc::fence_after();
#pragma unroll
                for (int c = 0; c < kStrip; c += 16) {
                    uint32_t w[16];
                    tc::read_chunk(mine + buffer * 256 + c, w);
                    tc::read_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[c + i] += __uint_as_float(w[i]);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::arrive_at(freed[buffer]);
            }
            if (!alive) {
#pragma unroll
                for (int i = 0; i < kStrip; ++i) v[i] = NAN;
            }
            if (c0 >= n) continue;
            epi.rows(stage, state, r, c0, n, t.n0 / g.width * ((g.width + kStrip - 1) / kStrip) + strip, r < m, v);
            __syncwarp();
            if constexpr (Epi::kChunks) {
#pragma unroll(Epi::kUnroll)
                for (int c = 0; c < kStrip; c += 32) {
                    if (c0 + c >= n) break;
                    const Fetched now = ahead;
                    put_chunk_of(stage, v, c / 32);
                    if constexpr (Epi::kFetches) {
                        if (fetches && c + 32 < kStrip && c0 + c + 32 < n) epi.fetch(ahead, r - lane, m, c0 + c + 32);
                    }
                    if constexpr (Epi::kPatches) {
                        if (r < m) epi.patch(stage, state, c0 + c);
                    }
                    __syncwarp();
                    if constexpr (Epi::kParts) {
                        if (g.splits > 1) {
                            epi.part(stage, t.split, r - lane, m, c0 + c);
                            __syncwarp();
                            continue;
                        }
                    }
                    epi.chunk(stage, state, now, r - lane, m, c0 + c);
                    __syncwarp();
                }
            }
        }
    }
    __syncwarp();  // lanes that left a wait one by one
    __syncthreads();
    tc::cluster_sync();
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    tc::cluster_sync();
}

// ---------------------------------------------------------------- host
// The sums of the parts that the terms were split into, one after the other, handed to an epilogue. A thread has
// four of a row's columns, or one.
struct JoinPartsArgs {
    const float* part;  // [splits][m][stride]
    int64_t m, n, stride;
    const int32_t* m_count;
    int32_t splits;
};

template <int N, typename Epi> __global__ void __launch_bounds__(kRows) join_parts_kernel(const JoinPartsArgs a, const Epi epi)
{
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int64_t m = a.m_count ? *a.m_count : a.m;
    const int64_t chunks = (a.n + N - 1) / N, i = (int64_t)blockIdx.x * kRows + threadIdx.x;
    if (i >= chunks * m) return;
    const int64_t r = i / chunks, c = (i - r * chunks) * N;
    Cols<N> v = {};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) v = v + get<N>(a.part + ((int64_t)s * a.m + r) * a.stride + c, 4);
    epi.piece((int32_t)r, (int32_t)c, v);
}

template <typename Epi> cudaError_t join_parts(const JoinPartsArgs& j, const Epi& epi, cudaStream_t stream)
{
    const int64_t all = (j.n + (epi.whole ? 3 : 0)) / (epi.whole ? 4 : 1) * j.m;
    return launch_after(epi.whole ? join_parts_kernel<4, Epi> : join_parts_kernel<1, Epi>, dim3((unsigned)((all + kRows - 1) / kRows)),
                        dim3(kRows), 0, stream, j, epi);
}

// A product of no terms: the epilogue of zeros.
template <typename Epi> cudaError_t product_none(int64_t m, int64_t n, const Epi& epi, cudaStream_t stream)
{
    return join_parts(JoinPartsArgs{nullptr, m, n, 0, nullptr, 0}, epi, stream);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled()
{
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled f = known.load(std::memory_order_acquire);
    if (!f) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeTiled>(p);
        known.store(f, std::memory_order_release);
    }
    return f;
}

// How TMA reads a matrix: 64 numbers of each of `box` rows at a time; zeros past its ends.
inline cudaError_t tensor_map(CUtensorMap* map, const Matrix& a, int planes, int box)
{
    const EncodeTiled f = encode_tiled();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)a.cols, (cuuint64_t)a.rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)a.stride * 2, (cuuint64_t)(planes > 1 ? a.plane : a.stride) * 2};
    const cuuint32_t boxes[3] = {(cuuint32_t)kTcDepth, (cuuint32_t)box, 1}, ones[3] = {1, 1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16*>(a.p), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// Whether a bf16 matrix can be read as it lies.
inline bool as_it_lies(const void* p, int64_t stride, int64_t rows, int64_t cols)
{
    return is_aligned(p, 16) && (rows < 2 || (stride % 8 == 0 && stride >= cols && stride < (int64_t)1 << 38));
}

inline Matrix matrix_of(const void* p, int64_t stride, int64_t rows, int64_t cols)
{
    return {static_cast<const bf16*>(p), rows, cols, rows < 2 ? pitch_of(cols) : stride, 0};
}

inline int64_t packed_elements(int64_t rows, int64_t cols, int bytes)  // of a workspace
{
    return rows * pitch_of(cols) * (bytes == 4 ? kPlanes : 1);
}

// A matrix of T's as a product takes it: as it lies, or copied to `room` (packed_elements).
template <typename T>
cudaError_t take_matrix(Matrix* out, const void* p, int64_t stride, int64_t rows, int64_t cols, bf16* room, cudaStream_t stream,
                        const int32_t* map = nullptr, const int32_t* count = nullptr, int64_t out_rows = 0)
{
    if (sizeof(T) == 2 && !count && as_it_lies(p, stride, rows, cols)) {
        *out = matrix_of(p, stride, rows, cols);
        return cudaSuccess;
    }
    const int64_t to_rows = count ? out_rows : rows;
    *out = {room, to_rows, cols, pitch_of(cols), to_rows * pitch_of(cols)};
    PackArgs a = {p, room, map, count, rows, cols, stride, out->stride, out->plane, whole_rows(p, stride, rows, sizeof(T))};
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t need = (to_rows * ((cols + 7) / 8) + kTcPack - 1) / kTcPack, most = (int64_t)sms * 16;
    if (need == 0) return cudaSuccess;
    return launch_after(pack_kernel<T>, dim3((unsigned)(need < most ? need : most)), dim3(kTcPack), 0, stream, a);
}

template <bool kBoth, typename Epi>
cudaError_t launch_tc(const TcMaps& maps, const TcParams<Epi>& p, cudaStream_t stream)
{
    cudaError_t e = allow<product_tc_kernel<kBoth, Epi>>(kTcShared);
    int sms = 0;
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    int64_t units = 0;
    for (int i = 0; i < (kBoth ? 2 : 1); ++i)
        units += (p.g[i].m + kTcM - 1) / kTcM * ((p.g[i].n + p.g[i].width - 1) / p.g[i].width) * p.g[i].splits;
    const int64_t pairs = sms / 2;
    return launch_after(product_tc_kernel<kBoth, Epi>, dim3((unsigned)(2 * (units < pairs ? units : pairs))), dim3(kTcThreads),
                        kTcShared, stream, maps, p);
}

// A product's operands. a_mn, b_mn: the matrix lies by terms (its rows are terms).
struct TcProduct {
    Matrix a, b;
    bool a_mn, b_mn;
    int64_t m, n, k;
    const int32_t *m_count, *k_count;
    int parts = 1;  // bf16: of A
    TcWaits waits = {};
};

inline adacomp_status set_timeout(TcWaits& waits, uint64_t timeout_ns)
{
    if (timeout_ns == 0 || timeout_ns > 60000000000ull) return ADACOMP_ERR_INVALID_ARG;
    waits.limit_ns = timeout_ns;
    return ADACOMP_OK;
}

template <typename T, typename Epi>
cudaError_t set_tc(TcMaps& maps, TcParams<Epi>& p, int i, const TcProduct& x, int width, int splits, const Epi& epi)
{
    TcArgs g = {};
    g.m = x.m;
    g.n = x.n;
    g.k = x.k;
    g.m_count = x.m_count;
    g.k_count = x.k_count;
    const int planes_a = sizeof(T) == 4 ? kPlanes : x.parts, planes_b = sizeof(T) == 4 ? kPlanes : 1;
    g.passes = sizeof(T) == 4 ? kSix : x.parts;
    g.splits = splits;
    g.width = width;
    g.a_mn = x.a_mn;
    g.b_mn = x.b_mn;
    g.group = 8;
    g.least = (int32_t)(kTcEnd / (kTcBlock * g.passes)) + 1;
    g.run = sizeof(T) == 4 ? 4 : Epi::kExact ? 8 : 1 << 30;
    p.g[i] = g;
    p.epi[i] = epi;
    p.waits = x.waits;
    const cudaError_t e = tensor_map(&maps.a[i], x.a, planes_a, x.a_mn ? kTcDepth : 128);
    return e == cudaSuccess ? tensor_map(&maps.b[i], x.b, planes_b, x.b_mn ? kTcDepth : width / 2) : e;
}

// ---------------------------------------------------------------- which way
// How wide the tiles are, and into how many parts the terms are split (which a kernel of its own joins), so that
// the last tiles leave few SMs idle. By estimate, us: a block of 64 terms and 256 columns takes a pair kTcBlock
// (six times that in fp32), a narrower one more than its share, as the rows of A are loaded all the same (tiles
// of 32 blocks, bf16: 256 columns 11.2, 224 9.7, 192 8.7, 160 7.8, 128 7.2, 96 6.7); the last tile's end 2 more,
// which nothing covers; the parts' sums are written and read, and the joining kernel begins 3 later. With it,
// and with 256 columns and whole sums: the logits of 512 rows over 50304 tokens 75 and 84; a layer's gradients
// 3001 x 1001 x 777 fp32 102 and 111.
constexpr int64_t kPairs = 76, kMostParts = 2 * kPairs;  // tiles x splits are at most kMostParts, if split
struct TcWay {
    int width, splits;
};

struct TcSize {
    int64_t m, n, k;
    int passes;
    bool may_split;
    int64_t tiles(int width) const { return (m + kTcM - 1) / kTcM * ((n + width - 1) / width); }
    int64_t blocks(int s) const { return ((k + kTcDepth - 1) / kTcDepth + s - 1) / s; }
    bool may(TcWay w) const { return w.splits == 1 || (may_split && tiles(w.width) * w.splits <= kMostParts && blocks(1) >= 4 * w.splits); }
    double join(TcWay w) const { return w.splits == 1 ? 0.0 : 3.0 + (double)w.splits * m * n * 8 / 5e6; }
    double unit(TcWay w) const
    {
        const double share = w.width / 256.0, least = 0.45 + 0.38 * share;
        return blocks(w.splits) * kTcBlock * passes * (share > least ? share : least);
    }
    double cost(TcWay w) const
    {
        const int64_t waves = (tiles(w.width) * w.splits + kPairs - 1) / kPairs;
        return waves * unit(w) + 2.0 + join(w);
    }
    // the narrowest that gives as few tiles as 256 columns
    int even() const { return (int)round_up((n + (n + 255) / 256 - 1) / ((n + 255) / 256), 32); }
    TcWay best() const
    {
        TcWay best = {even(), 1};
        for (int width = even(); width >= 32 && (width >= 96 || width == even()); width -= 32)
            for (TcWay w = {width, 1}; may(w); ++w.splits)
                if (cost(w) < 0.97 * cost(best)) best = w;
        return best;
    }
    TcWay split(int splits) const  // the terms in so many parts: how wide
    {
        TcWay best = {even(), splits};
        for (TcWay w = best; w.width >= 96; w.width -= 32)
            if (may(w) && cost(w) < 0.97 * cost(best)) best = w;
        return best;
    }
};

// The ways of two products, neither of which needs the other, in one launch, and whether the second has the longer sums.
struct TcBoth {
    TcWay way[2];
    bool turned;
};

inline TcBoth best_of_both(const TcSize (&size)[2])
{
    const int width[2] = {size[0].even(), size[1].even()};
    int alone[2];
    for (int i = 0; i < 2; ++i) {
        TcWay best = {width[i], 1};
        for (TcWay w = best; size[i].may(w); ++w.splits)
            if (size[i].cost(w) < 0.97 * size[i].cost(best)) best = w;
        alone[i] = best.splits;
    }
    TcBoth best = {};
    double least = -1.0;
    for (int i = 0; i < 9; ++i) {  // each whole, as it would be alone, and half of that
        const TcWay way[2] = {{width[0], i % 3 == 0 ? 1 : (alone[0] + i % 3 - 1) / (i % 3)},
                              {width[1], i / 3 == 0 ? 1 : (alone[1] + i / 3 - 1) / (i / 3)}};
        const int64_t units[2] = {size[0].tiles(width[0]) * way[0].splits, size[1].tiles(width[1]) * way[1].splits};
        double unit[2] = {size[0].unit(way[0]), size[1].unit(way[1])};
        for (double& u : unit)
            if (units[0] + units[1] > kPairs && u < kTcEnd) u = kTcEnd;
        const int a = unit[1] > unit[0], b = !a;  // the longer sums first
        const TcShares shares(kPairs, units[a], (int64_t)(unit[a] * 1000), units[b], (int64_t)(unit[b] * 1000));
        const double cost = shares.blocks / 1000.0 + 2.0 + size[0].join(way[0]) + size[1].join(way[1]);
        if (least < 0.0 || cost < 0.98 * least) least = cost, best = {{way[0], way[1]}, a != 0};
    }
    return best;
}

inline int64_t parts_elements(int64_t m, int64_t n)  // of a workspace
{
    const int64_t whole = kMostParts * kTcM * 256, all = kMostParts * m * round_up(n, 4);
    return all < whole ? all : whole;
}

template <typename T, typename Epi> TcSize size_of(const TcProduct& x) { return {x.m, x.n, x.k, sizeof(T) == 4 ? kSix : x.parts, Epi::kPieces}; }

// The epilogue of a product whose terms are split: its parts' sums.
template <typename T> EpiStore<T> to_parts(EpiStore<T> epi, float* parts, const TcProduct& x)
{
    epi.first = true;
    epi.acc = parts;
    epi.acc_stride = round_up(x.n, 4);
    epi.split_stride = x.m * epi.acc_stride;
    epi.n = (int32_t)x.n;
    return epi;
}

inline JoinPartsArgs joining(float* parts, const TcProduct& x, int splits)
{
    return {parts, x.m, x.n, round_up(x.n, 4), x.m_count, splits};
}

// A product of matrices of T's planes. parts: room for parts_elements.
template <typename T, typename Epi>
cudaError_t product_tc(const TcProduct& x, TcWay way, float* parts, const Epi& epi, cudaStream_t stream)
{
    if (x.m <= 0 || x.n <= 0) return cudaSuccess;
    TcMaps maps = {};
    if constexpr (Epi::kPieces) {
        if (way.splits > 1) {
            TcParams<EpiStore<T>> p = {};
            cudaError_t e = set_tc<T>(maps, p, 0, x, way.width, way.splits, to_parts(EpiStore<T>{}, parts, x));
            if (e == cudaSuccess) e = launch_tc<false>(maps, p, stream);
            return e == cudaSuccess ? join_parts(joining(parts, x, way.splits), epi, stream) : e;
        }
    }
    TcParams<Epi> p = {};
    const cudaError_t e = set_tc<T>(maps, p, 0, x, way.width, 1, epi);
    return e == cudaSuccess ? launch_tc<false>(maps, p, stream) : e;
}

template <typename T, typename Epi> cudaError_t product_tc(const TcProduct& x, float* parts, const Epi& epi, cudaStream_t stream)
{
    return product_tc<T>(x, size_of<T, Epi>(x).best(), parts, epi, stream);
}

// Two products, neither of which needs the other, in one launch, so that the units of one fill the SMs that the
// other's last ones leave idle; or the one of them that is wanted (the other's operands may be missing), whose terms are
// split as beside the other, so that its sums are the same. parts: room for both's parts_elements, the first's first.
template <typename T, typename Epi>
cudaError_t product_tc_both(const TcProduct& x, const Epi& epi_x, bool want_x, const TcProduct& y, const Epi& epi_y, bool want_y,
                            float* parts, cudaStream_t stream)
{
    const TcProduct* const product[2] = {&x, &y};
    const Epi* const epi[2] = {&epi_x, &epi_y};
    const TcSize size[2] = {size_of<T, Epi>(x), size_of<T, Epi>(y)};
    float* const room[2] = {parts, parts + parts_elements(x.m, x.n)};
    const TcBoth best = best_of_both(size);
    if (!want_x || !want_y) {
        const int i = want_y;
        return want_x || want_y ? product_tc<T>(*product[i], size[i].split(best.way[i].splits), room[i], *epi[i], stream) : cudaSuccess;
    }
    TcMaps maps = {};
    TcParams<Epi> p = {};
    for (int i = 0; i < 2; ++i) {
        const TcProduct& g = *product[i];
        const TcWay way = best.way[i];
        const cudaError_t e = set_tc<T>(maps, p, best.turned ? !i : i, g, way.width, way.splits, way.splits > 1 ? to_parts(*epi[i], room[i], g) : *epi[i]);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_tc<true>(maps, p, stream);
    for (int i = 0; i < 2 && e == cudaSuccess; ++i)
        if (best.way[i].splits > 1) e = join_parts(joining(room[i], *product[i], best.way[i].splits), *epi[i], stream);
    return e;
}

}  // namespace
}  // namespace adacomp
