// Losses over a vocabulary (softmax cross entropy, distillation from a teacher's top logits): forward and
// backward passes and their C entry points (adacomp.h).
#include <new>

#include "product_tc.cuh"

struct adacomp_vocab {
    int64_t dim = 0, vocab = 0;
    int32_t dtype = ADACOMP_F32;
    adacomp::TcWaits waits;
};

namespace adacomp {
namespace {

constexpr int kListThreads = 256;
constexpr int kScanThreads = 256, kScanRows = 1024;
constexpr int kScanMost = 1024;            // CTAs that have a run of the rows each
constexpr int64_t kScanAlone = 16384;   // rows up to which each CTA counts those before its own by itself
constexpr int kJoinThreads = 1024;
constexpr int kZeroThreads = 256;

struct VocabArgs {
    int64_t rows, dim, vocab;
    const void *x, *w;
    int64_t x_stride, w_stride;
    const void *target;            // cross entropy; or
    int32_t target_bytes;
    const int32_t* index;          // a teacher's lists
    const void* logit;
    int64_t index_stride, logit_stride;
    int32_t logit_dtype, k;
    float temperature;
    float *loss, *lse_out;         // forward
    const float *lse, *dloss;      // backward
    int64_t dloss_stride;
    void *dx, *dw;
    int64_t dx_stride, dw_stride;
    TcWaits waits;
};

struct VocabParts {
    int32_t *index, *map, *count;
    float *q, *given;      // weights; sum of q log q: -inf for a row without a loss, NaN for one without a value
    float2* part;          // forward
    float* picked;
    float* acc;            // backward: dx so far
    bf16 *x, *w, *dz;      // the rows that have a loss, one behind the other; a copy of w; a piece's gradient
    float* parts;          // of products whose terms are split
    int64_t padded, dz_stride, piece;
};

// Columns of a piece: so many that the piece's gradient, of whole tiles of rows, has up to 2^27 elements, and no
// fewer than 2048; and the most elements that one of up to `rows` rows has.
constexpr int64_t kPieceElements = (int64_t)1 << 27, kLeastPiece = 2048;
int64_t piece_of(int64_t rows, int64_t vocab)
{
    const int64_t padded = round_up(rows < 1 ? 1 : rows, kRows);
    if (padded * pitch_of(vocab) <= kPieceElements) return vocab;
    int64_t n = kPieceElements / padded / kStrip * kStrip;
    if (n < kLeastPiece) n = kLeastPiece;
    return n < vocab ? n : vocab;
}
int64_t piece_elements(int64_t rows, int64_t vocab)
{
    const int64_t padded = round_up(rows < 1 ? 1 : rows, kRows), all = padded * pitch_of(vocab);
    const int64_t least = padded * pitch_of(vocab < kLeastPiece ? vocab : kLeastPiece);
    return all <= kPieceElements ? all : least > kPieceElements ? least : kPieceElements;
}

// Strips of a row's logits, in tiles of `width` columns; and at most, whatever the tiles (of which all but narrow
// vocabularies' have 96 columns or more).
int64_t strips_of(int64_t vocab, int width)
{
    const int64_t tiles = (vocab + width - 1) / width, rest = vocab - (tiles - 1) * width;
    return (tiles - 1) * ((width + kStrip - 1) / kStrip) + (rest + kStrip - 1) / kStrip;
}
int64_t most_strips(int64_t vocab) { return vocab / 80 + 2; }

VocabParts vocab_parts(Carve& c, int64_t rows, int64_t dim, int64_t vocab, int bytes, int32_t k, bool backward)
{
    VocabParts p = {};
    p.index = c.take<int32_t>(rows * k);
    p.q = c.take<float>(rows * k);
    p.given = c.take<float>(rows);
    p.map = c.take<int32_t>(rows);
    p.count = c.take<int32_t>(1 + kScanMost);  // and of the runs
    p.padded = round_up(rows, kRows);
    p.x = c.take<bf16>(packed_elements(p.padded, dim, bytes));
    p.w = c.take<bf16>(packed_elements(vocab, dim, bytes));
    if (backward) {
        p.piece = piece_of(rows, vocab);
        p.dz_stride = pitch_of(p.piece);
        const int64_t few = 2 * piece_elements(rows < kFewRows ? rows : kFewRows, vocab), all = piece_elements(rows, vocab);
        p.dz = c.take<bf16>(bytes == 4 ? kPlanes * all : few > all ? few : all);
        p.acc = c.take<float>(rows * round_up(dim, 4));
        p.parts = c.take<float>(parts_elements(rows, dim) + parts_elements(vocab, dim));
    } else {
        p.part = c.take<float2>(rows * most_strips(vocab));
        p.picked = c.take<float>(rows * k);
    }
    return p;
}

// ---------------------------------------------------------------- rows
struct ListArgs {
    const void* target;
    const int32_t* index;
    const void* logit;
    int64_t rows, vocab, index_stride, logit_stride;
    int32_t target_bytes, k;
    float scale;
    int32_t* to_index;
    float *to_q, *given;
};

// A teacher's list of a row by a warp: softmax of its logits, and the tokens in ascending order (each place is
// the number of places before it, so equal tokens keep their order).
template <typename L> __global__ void __launch_bounds__(kListThreads) vocab_teacher_kernel(const ListArgs a)
{
    __shared__ int32_t keys[kListThreads / 32][ADACOMP_MAX_TEACHER];
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t r = (int64_t)blockIdx.x * (kListThreads / 32) + warp; r < a.rows;
         r += (int64_t)gridDim.x * (kListThreads / 32)) {
        const int32_t* index = a.index + r * a.index_stride;
        const L* logit = static_cast<const L*>(a.logit) + r * a.logit_stride;
        float u[ADACOMP_MAX_TEACHER / 32], top = -INFINITY;
        bool some = false, bad = false, none = false;  // none: a logit that is NaN
#pragma unroll
        for (int i = 0; i < ADACOMP_MAX_TEACHER / 32; ++i) {
            const int j = i * 32 + lane;
            u[i] = -INFINITY;
            if (j >= a.k) continue;
            const int32_t t = index[j];
            keys[warp][j] = t >= 0 ? t : INT32_MAX;
            if (t < 0) continue;
            some = true;
            bad = bad || t >= a.vocab;
            u[i] = to_f32(logit[j]) * a.scale;
            none = none || u[i] != u[i];
            top = fmaxf(top, u[i]);
        }
        some = __any_sync(0xffffffffu, some);
        bad = __any_sync(0xffffffffu, bad);
        none = __any_sync(0xffffffffu, none);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (bad || none || top == -INFINITY || top == INFINITY) {  // no list, or none that has a value
            for (int j = lane; j < a.k; j += 32) {
                a.to_index[r * a.k + j] = INT32_MAX;
                a.to_q[r * a.k + j] = 0.0f;
            }
            if (lane == 0) a.given[r] = some ? NAN : -INFINITY;
            __syncwarp();
            continue;
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < ADACOMP_MAX_TEACHER / 32; ++i) sum += u[i] > -INFINITY ? expf(u[i] - top) : 0.0f;
        sum = warp_sum(sum);
        const float log_sum = logf(sum);
        float given = 0.0f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < ADACOMP_MAX_TEACHER / 32; ++i) {
            const int j = i * 32 + lane;
            if (j >= a.k) continue;
            const float q = u[i] > -INFINITY ? expf(u[i] - top) / sum : 0.0f;
            if (q > 0.0f) given += q * (u[i] - top - log_sum);
            const int32_t key = keys[warp][j];
            int place = 0;
            for (int o = 0; o < a.k; ++o) place += keys[warp][o] < key || (keys[warp][o] == key && o < j);
            a.to_index[r * a.k + place] = key;
            a.to_q[r * a.k + place] = q;
        }
        given = warp_sum(given);
        if (lane == 0) a.given[r] = given;
        __syncwarp();
    }
}

__device__ __forceinline__ int64_t target_of(const ListArgs& a, int64_t r)
{
    return a.target_bytes == 8 ? static_cast<const int64_t*>(a.target)[r] : (int64_t) static_cast<const int32_t*>(a.target)[r];
}

template <bool kTarget> __device__ __forceinline__ bool has_loss(const ListArgs& a, int64_t r)
{
    return kTarget ? target_of(a, r) >= 0 : a.given[r] != -INFINITY;
}

// A thread's part of how many rows from `from` to `to` have a loss.
template <bool kTarget> __device__ __forceinline__ int32_t count_rows(const ListArgs& a, int64_t from, int64_t to)
{
    int32_t n = 0;
#pragma unroll 4
    for (int64_t r = from + threadIdx.x; r < to; r += kScanThreads) n += has_loss<kTarget>(a, r);
    return n;
}

// The rows that have a loss, in their order: put(place, row) for those of kScanRows rows from r0 on, by a CTA, whose
// threads' `before` add up to the number of those before them; and how many there are up to their end. kTarget: of one
// token each, which become lists of one, of weight 1, if `lists`.
template <bool kTarget, typename F>
__device__ __forceinline__ int32_t vocab_scan(const ListArgs& a, int64_t r0, int32_t before, bool lists, F put)
{
    constexpr int kEach = kScanRows / kScanThreads, kWarps = kScanThreads / 32;
    __shared__ int32_t sums[2][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t mine = 0;
    bool there[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t r = r0 + threadIdx.x * kEach + i;
        there[i] = r < a.rows && has_loss<kTarget>(a, r);
        mine += there[i];
        if (kTarget && lists && r < a.rows) {
            const int64_t t = target_of(a, r);
            a.to_index[r] = t >= 0 && t < a.vocab ? (int32_t)t : INT32_MAX;
            a.to_q[r] = 1.0f;
            a.given[r] = t < 0 ? -INFINITY : t < a.vocab ? 0.0f : NAN;
        }
    }
    int32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (lane == 31) {
        sums[0][warp] = sum;
        sums[1][warp] = before;
    }
    __syncthreads();
    int32_t at = sum - mine, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        at += sums[1][i] + (i < warp ? sums[0][i] : 0);
        all += sums[1][i] + sums[0][i];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (there[i]) put(at++, (int32_t)(r0 + threadIdx.x * kEach + i));
    return all;
}

template <bool kTarget>
__global__ void __launch_bounds__(kScanThreads) vocab_rows_kernel(const ListArgs a, int32_t* map, int32_t* count)
{
    ptx::griddep_wait();
    ptx::griddep_launch();
    const auto put = [&](int32_t at, int32_t row) { map[at] = row; };
    const int64_t r0 = (int64_t)blockIdx.x * kScanRows;
    const int32_t all = vocab_scan<kTarget>(a, r0, count_rows<kTarget>(a, 0, r0), true, put);
    if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) *count = all;
}

// Of many rows, a CTA has a run of `run` of them: how many of it have a loss (count[1 + its number]), and, in a second
// kernel, which. (A forward pass against 96 tokens of width 16, this way and with every CTA counting all rows before its
// own: 4096 rows 17.3 and 16.1 us, 16384 20.1 and 20.4, 131072 59 and 74, 4194304 1679 and 3805.)
template <bool kTarget> __global__ void __launch_bounds__(kScanThreads) vocab_count_kernel(const ListArgs a, int64_t run, int32_t* count)
{
    __shared__ int32_t sums[kScanThreads / 32];
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int64_t from = blockIdx.x * run, to = a.rows - from < run ? a.rows : from + run;
    int32_t n = count_rows<kTarget>(a, from, to);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = n;
    __syncthreads();
    if (threadIdx.x) return;
    n = 0;
    for (int i = 0; i < kScanThreads / 32; ++i) n += sums[i];
    count[1 + blockIdx.x] = n;
}

template <bool kTarget>
__global__ void __launch_bounds__(kScanThreads) vocab_runs_kernel(const ListArgs a, int64_t run, int32_t* map, int32_t* count)
{
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int64_t from = blockIdx.x * run, to = a.rows - from < run ? a.rows : from + run;
    const auto put = [&](int32_t at, int32_t row) { map[at] = row; };
    int32_t before = 0;
    for (int i = threadIdx.x; i < (int)blockIdx.x; i += kScanThreads) before += count[1 + i];
    for (int64_t r0 = from; r0 < to; r0 += kScanRows) {  // whole blocks of rows, but for the last run's last
        const int32_t all = vocab_scan<kTarget>(a, r0, before, true, put);
        before = threadIdx.x ? 0 : all;
        __syncthreads();
    }
    if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) *count = before;
}

// The same of up to kScanRows rows, and the rows' copies with it: each CTA scans all rows for itself, the first writes what
// later kernels read. One launch less (vocab_forward of 32 rows 49.5 -> 48.4 us, distill_train of 999 rows 251.1 -> 249.5).
template <typename T, bool kTarget>
__global__ void __launch_bounds__(kScanThreads) vocab_few_kernel(const ListArgs a, int32_t* map, int32_t* count,
                                                                const PackArgs pack)
{
    static_assert(kScanThreads == kTcPack, "pack_rows");
    __shared__ int32_t places[kScanRows];
    ptx::griddep_wait();
    ptx::griddep_launch();
    const bool first = blockIdx.x == 0;
    const int32_t all = vocab_scan<kTarget>(a, 0, 0, first, [&](int32_t at, int32_t row) {
        places[at] = row;
        if (first) map[at] = row;
    });
    if (first && threadIdx.x == 0) *count = all;
    __syncthreads();
    pack_rows<T>(pack, places, all, (all + kRows - 1) / kRows * kRows);
}

// The rows of dx without a loss, a warp each.
template <typename T>
__global__ void __launch_bounds__(kZeroThreads) vocab_zero_kernel(T* dx, int64_t stride, const float* given, int64_t rows, int64_t dim)
{
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int64_t warps = kZeroThreads / 32;
    for (int64_t r = blockIdx.x * warps + threadIdx.x / 32; r < rows; r += gridDim.x * warps) {
        if (given[r] != -INFINITY) continue;
        for (int64_t i = threadIdx.x & 31; i < dim; i += 32) dx[r * stride + i] = from_f32<T>(0.0f);
    }
}

struct JoinArgs {
    const float2* part;
    const float *picked, *q, *given;
    const int32_t *map, *count;
    float *loss, *lse;
    int64_t rows, strips;
    int32_t k;
    float temperature;
};

// Rows' strips joined, and their losses; rows without a loss are 0. A CTA has kJoinRows rows: a warp's lanes
// have a strip of each, or, where rows are few, four strips of eight rows; then a warp has a row, for its list.
template <int kJoinRows> __global__ void __launch_bounds__(kJoinThreads) vocab_join_kernel(const JoinArgs a)
{
    constexpr int kParts = kJoinThreads / kJoinRows;  // of a row's strips
    __shared__ float2 sums[kJoinRows][kParts + 1];
    ptx::griddep_wait();
    ptx::griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = threadIdx.x / kJoinRows, mine = threadIdx.x % kJoinRows;
    const int64_t count = *a.count;
    for (int64_t r0 = (int64_t)blockIdx.x * kJoinRows; r0 < count; r0 += (int64_t)gridDim.x * kJoinRows) {
        const int64_t r = r0 + mine;
        float top = -INFINITY, sum = 0.0f;
        if (r < count) {
#pragma unroll 4
            for (int64_t i = part; i < a.strips; i += kParts) {
                const float2 p = a.part[i * a.rows + r];
                const float more = fmaxf(top, p.x), less = more == -INFINITY ? 0.0f : more;
                sum = sum * expf(top - less) + p.y * expf(p.x - less);
                top = more;
            }
        }
        sums[mine][part] = make_float2(top, sum);
        __syncthreads();
        if (warp < kJoinRows && r0 + warp < count) {
            float2 p[kParts / 32];
            float most = -INFINITY, all = 0.0f;
#pragma unroll
            for (int i = 0; i < kParts / 32; ++i) {
                p[i] = sums[warp][i * 32 + lane];
                most = fmaxf(most, p[i].x);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
#pragma unroll
            for (int i = 0; i < kParts / 32; ++i) all += p[i].y * expf(p[i].x - (most == -INFINITY ? 0.0f : most));
            all = warp_sum(all);
            const float lse = most + logf(all);
            const int64_t row = a.map[r0 + warp];
            const float given = a.given[row];
            float mean = 0.0f;  // of the logits under q
            if (given == given)
                for (int j = lane; j < a.k; j += 32) {
                    const float q = a.q[row * a.k + j];
                    if (q > 0.0f) mean += q * a.picked[row * a.k + j];
                }
            mean = warp_sum(mean);
            if (lane == 0) {
                a.lse[row] = lse;
                a.loss[row] = a.temperature * a.temperature * (given + (lse - mean));
            }
        }
        __syncthreads();
    }
    for (int64_t r = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; r < a.rows; r += (int64_t)gridDim.x * kJoinThreads)
        if (a.given[r] == -INFINITY) a.loss[r] = a.lse[r] = 0.0f;
}

// ---------------------------------------------------------------- passes
unsigned blocks_of(int64_t n, int64_t each, int64_t most)
{
    const int64_t b = (n + each - 1) / each;
    return (unsigned)(b < 1 ? 1 : b < most ? b : most);
}

// The lists, the rows that have a loss, and the operands.
template <typename T> cudaError_t vocab_rows(const VocabArgs& a, const VocabParts& p, Matrix* x, Matrix* w, cudaStream_t stream)
{
    ListArgs l = {};
    l.target = a.target;
    l.index = a.index;
    l.logit = a.logit;
    l.rows = a.rows;
    l.vocab = a.vocab;
    l.index_stride = a.index_stride;
    l.logit_stride = a.logit_stride;
    l.target_bytes = a.target_bytes;
    l.k = a.k;
    l.scale = 1.0f / a.temperature;
    l.to_index = p.index;
    l.to_q = p.q;
    l.given = p.given;
    cudaError_t e = cudaSuccess;
    if (!a.target)
        e = launch_after(a.logit_dtype == ADACOMP_BF16 ? vocab_teacher_kernel<bf16> : vocab_teacher_kernel<float>,
                         dim3(blocks_of(a.rows, kListThreads / 32, 4096)), dim3(kListThreads), 0, stream, l);
    if (e != cudaSuccess) return e;
    if (a.rows <= kScanRows) {
        const int64_t pitch = pitch_of(a.dim);
        *x = {p.x, p.padded, a.dim, pitch, p.padded * pitch};
        const PackArgs pack = {a.x, p.x, nullptr, nullptr, a.rows, a.dim, a.x_stride, pitch, x->plane,
                               whole_rows(a.x, a.x_stride, a.rows, sizeof(T))};
        const dim3 grid(blocks_of(p.padded * ((a.dim + 7) / 8), kScanThreads, 304));
        e = launch_after(a.target ? vocab_few_kernel<T, true> : vocab_few_kernel<T, false>, grid, dim3(kScanThreads), 0,
                         stream, l, p.map, p.count, pack);
    } else {
        const int64_t blocks = (a.rows + kScanRows - 1) / kScanRows;
        if (a.rows <= kScanAlone) {
            e = launch_after(a.target ? vocab_rows_kernel<true> : vocab_rows_kernel<false>, dim3((unsigned)blocks), dim3(kScanThreads), 0,
                             stream, l, p.map, p.count);
        } else {
            const int64_t run = (blocks + kScanMost - 1) / kScanMost * kScanRows;
            const dim3 runs((unsigned)((a.rows + run - 1) / run));
            e = launch_after(a.target ? vocab_count_kernel<true> : vocab_count_kernel<false>, runs, dim3(kScanThreads), 0, stream, l, run, p.count);
            if (e == cudaSuccess)
                e = launch_after(a.target ? vocab_runs_kernel<true> : vocab_runs_kernel<false>, runs, dim3(kScanThreads), 0, stream, l, run,
                                 p.map, p.count);
        }
        if (e == cudaSuccess)
            e = take_matrix<T>(x, a.x, a.x_stride, a.rows, a.dim, p.x, stream, p.map, p.count, p.padded);
    }
    return e == cudaSuccess ? take_matrix<T>(w, a.w, a.w_stride, a.vocab, a.dim, p.w, stream) : e;
}

template <typename T> cudaError_t vocab_forward(const VocabArgs& a, void* ws, cudaStream_t stream)
{
    Carve carve{static_cast<char*>(ws)};
    const VocabParts p = vocab_parts(carve, a.rows, a.dim, a.vocab, sizeof(T), a.k, false);
    Matrix x, w;
    cudaError_t e = vocab_rows<T>(a, p, &x, &w, stream);
    if (e != cudaSuccess) return e;
    EpiSoftmax<T> epi = {};
    epi.part = p.part;
    epi.picked = p.picked;
    epi.lists = {p.index, p.q, p.map, a.k};
    epi.row_stride = a.rows;
    epi.scale = 1.0f / a.temperature;
    const TcProduct product = {x, w, false, false, a.rows, a.vocab, a.dim, p.count, nullptr, 1, a.waits};
    const TcWay way = size_of<T, EpiSoftmax<T>>(product).best();
    e = product_tc<T>(product, way, nullptr, epi, stream);
    if (e != cudaSuccess) return e;
    JoinArgs j = {};
    j.part = p.part;
    j.picked = p.picked;
    j.q = p.q;
    j.given = p.given;
    j.map = p.map;
    j.count = p.count;
    j.loss = a.loss;
    j.lse = a.lse_out;
    j.rows = a.rows;
    j.strips = strips_of(a.vocab, way.width);
    j.k = a.k;
    j.temperature = a.temperature;
    // few rows by more CTAs (512 rows of 50304 tokens: 8.2 us, and 12 by 32 rows each)
    if (a.rows <= 2048) return launch_after(vocab_join_kernel<8>, dim3(blocks_of(a.rows, 8, 4096)), dim3(kJoinThreads), 0, stream, j);
    return launch_after(vocab_join_kernel<32>, dim3(blocks_of(a.rows, 32, 4096)), dim3(kJoinThreads), 0, stream, j);
}

template <typename T> cudaError_t vocab_backward(const VocabArgs& a, void* ws, cudaStream_t stream)
{
    Carve carve{static_cast<char*>(ws)};
    const VocabParts p = vocab_parts(carve, a.rows, a.dim, a.vocab, sizeof(T), a.k, true);
    Matrix x, w;
    cudaError_t e = vocab_rows<T>(a, p, &x, &w, stream);
    if (a.dx && e == cudaSuccess)
        e = launch_after(vocab_zero_kernel<T>, dim3(blocks_of(a.rows, kZeroThreads / 32, 1216)), dim3(kZeroThreads), 0, stream, static_cast<T*>(a.dx),
                         a.dx_stride, (const float*)p.given, a.rows, a.dim);
    EpiGradient<T> grad = {};
    grad.dz = p.dz;
    grad.lists = {p.index, p.q, p.map, a.k};
    grad.lse = a.lse;
    grad.dloss = a.dloss;
    grad.given = p.given;
    grad.stride = p.dz_stride;
    grad.plane = p.padded * p.dz_stride;
    grad.room = (int32_t)p.padded;
    grad.dloss_stride = a.dloss_stride;
    grad.scale = 1.0f / a.temperature;
    grad.temperature = a.temperature;
    grad.two = sizeof(T) == 2 && a.rows <= kFewRows;
    for (int64_t at = 0; at < a.vocab && e == cudaSuccess; at += p.piece) {
        const int64_t n = a.vocab - at < p.piece ? a.vocab - at : p.piece;
        const Matrix here = {w.p + at * w.stride, n, a.dim, w.stride, w.plane}, dz = {p.dz, p.padded, n, p.dz_stride, grad.plane};
        grad.n = (int32_t)n;
        grad.first = (int32_t)at;
        const TcProduct logits = {x, here, false, false, a.rows, n, a.dim, p.count, nullptr, 1, a.waits};
        e = product_tc<T>(logits, nullptr, grad, stream);
        if (e != cudaSuccess) break;
        EpiStore<T> to_dx = {}, to_dw = {};
        to_dx.out = static_cast<T*>(a.dx);
        to_dx.acc = p.acc;
        to_dx.map = p.map;
        to_dx.stride = a.dx_stride;
        to_dx.acc_stride = round_up(a.dim, 4);
        to_dx.first = at == 0;
        to_dx.last = at + n == a.vocab;
        to_dx.whole = whole_rows(a.dx, a.dx_stride, a.rows, sizeof(T));
        to_dw.out = static_cast<T*>(a.dw) + (a.dw ? at * a.dw_stride : 0);
        to_dw.stride = a.dw_stride;
        to_dw.first = to_dw.last = true;
        to_dw.whole = whole_rows(a.dw, a.dw_stride, a.vocab, sizeof(T));
        to_dx.n = to_dw.n = (int32_t)a.dim;
        const TcProduct dx = {dz, here, false, true, a.rows, a.dim, n, p.count, nullptr, grad.two ? 2 : 1, a.waits};
        const TcProduct dw = {dz, x, true, true, n, a.dim, a.rows, nullptr, p.count, grad.two ? 2 : 1, a.waits};
        e = product_tc_both<T>(dx, to_dx, a.dx, dw, to_dw, a.dw, p.parts, stream);
    }
    return e;
}

template <typename T> cudaError_t zero_rows(const VocabArgs& a, cudaStream_t stream)  // dw of no rows
{
    if (!a.dw) return cudaSuccess;
    EpiStore<T> store = {};
    store.out = static_cast<T*>(a.dw);
    store.stride = a.dw_stride;
    store.n = (int32_t)a.dim;
    store.first = store.last = true;
    store.whole = whole_rows(a.dw, a.dw_stride, a.vocab, sizeof(T));
    return product_none(a.vocab, a.dim, store, stream);
}

constexpr int64_t kMostDim = (int64_t)1 << 30, kMostRows = ((int64_t)1 << 30) + 1;

// What both losses and both passes ask of their arguments.
adacomp_status vocab_check(adacomp_vocab_t h, const VocabArgs& a, const void* ws)
{
    if (!a.x || !a.w || !ws || a.x_stride < 0 || a.w_stride < 0) return ADACOMP_ERR_INVALID_ARG;
    const uintptr_t e = dtype_bytes(h->dtype);
    if (!is_aligned(a.x, e) || !is_aligned(a.w, e) || !is_aligned(a.loss, 4) || !is_aligned(a.lse_out, 4) ||
        !is_aligned(a.lse, 4) || !is_aligned(a.dloss, 4) || !is_aligned(a.dx, e) || !is_aligned(a.dw, e) ||
        (a.target && !is_aligned(a.target, a.target_bytes)) || !is_aligned(a.index, 4) ||
        (a.logit && !is_aligned(a.logit, dtype_bytes(a.logit_dtype))) || !is_aligned(ws, 16))
        return ADACOMP_ERR_ALIGNMENT;
    return ADACOMP_OK;
}

adacomp_status vocab_pass(adacomp_vocab_t h, VocabArgs& a, bool backward, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    a.dim = h->dim;
    a.vocab = h->vocab;
    a.waits = h->waits;
    if (a.rows > 0) {
        const adacomp_status s = vocab_check(h, a, ws);
        if (s != ADACOMP_OK) return s;
    }
    const bool narrow = h->dtype == ADACOMP_BF16;
    if (backward) {
        if ((!a.dx && !a.dw) || a.dloss_stride < 0 || (a.rows > 0 && (!a.lse || !a.dloss)) ||
            (a.dx && a.rows > 1 && a.dx_stride < a.dim) || (a.dw && a.vocab > 1 && a.dw_stride < a.dim))
            return ADACOMP_ERR_INVALID_ARG;
        if (!is_aligned(a.dw, dtype_bytes(h->dtype))) return ADACOMP_ERR_ALIGNMENT;
        if (a.rows == 0) return launch_result(narrow ? zero_rows<bf16>(a, stream) : zero_rows<float>(a, stream), stream);
    } else {
        if (a.rows == 0) return ADACOMP_OK;
        if (!a.loss || !a.lse_out) return ADACOMP_ERR_INVALID_ARG;
    }
    Carve need;
    vocab_parts(need, a.rows, a.dim, a.vocab, dtype_bytes(h->dtype), a.k, backward);
    if (ws_bytes < need.at) return ADACOMP_ERR_WORKSPACE;
    const cudaError_t e = backward ? (narrow ? vocab_backward<bf16>(a, ws, stream) : vocab_backward<float>(a, ws, stream))
                                   : (narrow ? vocab_forward<bf16>(a, ws, stream) : vocab_forward<float>(a, ws, stream));
    return launch_result(e, stream);
}

size_t vocab_bytes(adacomp_vocab_t h, int64_t rows, int32_t k, bool backward)
{
    if (!h || rows < 0 || rows >= kMostRows || k < 1 || k > ADACOMP_MAX_TEACHER) return 0;
    Carve c;
    vocab_parts(c, rows, h->dim, h->vocab, dtype_bytes(h->dtype), k, backward);
    return c.at;
}

// The entry points' arguments, those of each kind together.
VocabArgs vocab_args(int64_t rows, const void* x, int64_t x_stride, const void* w, int64_t w_stride)
{
    VocabArgs a = {};
    a.rows = rows;
    a.x = x;
    a.x_stride = x_stride;
    a.w = w;
    a.w_stride = w_stride;
    return a;
}

void set_target(VocabArgs& a, const void* target, int32_t target_bytes)
{
    a.target = target;
    a.target_bytes = target_bytes;
    a.k = 1;
    a.temperature = 1.0f;
}

void set_teacher(VocabArgs& a, int32_t k, const int32_t* index, int64_t index_stride, const void* logit, int64_t logit_stride,
                 int32_t logit_dtype, float temperature)
{
    a.k = k;
    a.index = index;
    a.index_stride = index_stride;
    a.logit = logit;
    a.logit_stride = logit_stride;
    a.logit_dtype = logit_dtype;
    a.temperature = temperature;
}

void set_gradients(VocabArgs& a, const float* lse, const float* dloss, int64_t dloss_stride, void* dx, int64_t dx_stride, void* dw,
                   int64_t dw_stride)
{
    a.lse = lse;
    a.dloss = dloss;
    a.dloss_stride = dloss_stride;
    a.dx = dx;
    a.dx_stride = dx_stride;
    a.dw = dw;
    a.dw_stride = dw_stride;
}

bool target_fits(const VocabArgs& a)
{
    return (a.target_bytes == 4 || a.target_bytes == 8) && (a.rows == 0 || a.target);
}

bool teacher_fits(const VocabArgs& a)
{
    return a.k >= 1 && a.k <= ADACOMP_MAX_TEACHER && known_dtype(a.logit_dtype) && a.temperature > 0.0f &&
           std::isfinite(a.temperature * a.temperature) && std::isfinite(1.0f / a.temperature) &&
           (a.rows == 0 || (a.index && a.logit && a.index_stride >= 0 && a.logit_stride >= 0));
}

}  // namespace
}  // namespace adacomp

extern "C" {

adacomp_status adacomp_vocab_init(adacomp_vocab_t* out, int64_t dim, int64_t vocab, adacomp_dtype dtype)
{
    if (!out) return ADACOMP_ERR_INVALID_ARG;
    *out = nullptr;
    if (dim < 1 || dim > adacomp::kMostDim || vocab < 1 || vocab > adacomp::kMostDim || !adacomp::known_dtype(dtype))
        return ADACOMP_ERR_INVALID_ARG;
    adacomp_vocab* h = new (std::nothrow) adacomp_vocab;
    if (!h) return ADACOMP_ERR_INVALID_ARG;
    h->dim = dim;
    h->vocab = vocab;
    h->dtype = dtype;
    *out = h;
    return ADACOMP_OK;
}

size_t adacomp_vocab_loss_forward_ws_bytes(adacomp_vocab_t h, int64_t rows) { return adacomp::vocab_bytes(h, rows, 1, false); }
size_t adacomp_vocab_loss_backward_ws_bytes(adacomp_vocab_t h, int64_t rows) { return adacomp::vocab_bytes(h, rows, 1, true); }
size_t adacomp_distill_forward_ws_bytes(adacomp_vocab_t h, int64_t rows, int32_t k) { return adacomp::vocab_bytes(h, rows, k, false); }
size_t adacomp_distill_backward_ws_bytes(adacomp_vocab_t h, int64_t rows, int32_t k) { return adacomp::vocab_bytes(h, rows, k, true); }

adacomp_status adacomp_vocab_loss_forward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride,
                                          const void* w, int64_t w_stride, const void* target, int32_t target_bytes,
                                          float* loss, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_vocab_loss_forward");
    if (!h || rows < 0 || rows >= adacomp::kMostRows) return ADACOMP_ERR_INVALID_ARG;
    adacomp::VocabArgs a = adacomp::vocab_args(rows, x, x_stride, w, w_stride);
    adacomp::set_target(a, target, target_bytes);
    a.loss = loss;
    a.lse_out = lse;
    if (!adacomp::target_fits(a)) return ADACOMP_ERR_INVALID_ARG;
    return adacomp::vocab_pass(h, a, false, ws, ws_bytes, stream);
}

adacomp_status adacomp_vocab_loss_backward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride,
                                           const void* w, int64_t w_stride, const void* target, int32_t target_bytes,
                                           const float* lse, const float* dloss, int64_t dloss_stride, void* dx,
                                           int64_t dx_stride, void* dw, int64_t dw_stride, void* ws, size_t ws_bytes,
                                           cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_vocab_loss_backward");
    if (!h || rows < 0 || rows >= adacomp::kMostRows) return ADACOMP_ERR_INVALID_ARG;
    adacomp::VocabArgs a = adacomp::vocab_args(rows, x, x_stride, w, w_stride);
    adacomp::set_target(a, target, target_bytes);
    adacomp::set_gradients(a, lse, dloss, dloss_stride, dx, dx_stride, dw, dw_stride);
    if (!adacomp::target_fits(a)) return ADACOMP_ERR_INVALID_ARG;
    return adacomp::vocab_pass(h, a, true, ws, ws_bytes, stream);
}

adacomp_status adacomp_distill_forward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride, const void* w,
                                       int64_t w_stride, int32_t k, const int32_t* index, int64_t index_stride,
                                       const void* logit, int64_t logit_stride, adacomp_dtype logit_dtype,
                                       float temperature, float* loss, float* lse, void* ws, size_t ws_bytes,
                                       cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_distill_forward");
    if (!h || rows < 0 || rows >= adacomp::kMostRows) return ADACOMP_ERR_INVALID_ARG;
    adacomp::VocabArgs a = adacomp::vocab_args(rows, x, x_stride, w, w_stride);
    adacomp::set_teacher(a, k, index, index_stride, logit, logit_stride, logit_dtype, temperature);
    a.loss = loss;
    a.lse_out = lse;
    if (!adacomp::teacher_fits(a)) return ADACOMP_ERR_INVALID_ARG;
    return adacomp::vocab_pass(h, a, false, ws, ws_bytes, stream);
}

adacomp_status adacomp_distill_backward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride, const void* w,
                                        int64_t w_stride, int32_t k, const int32_t* index, int64_t index_stride,
                                        const void* logit, int64_t logit_stride, adacomp_dtype logit_dtype,
                                        float temperature, const float* lse, const float* dloss, int64_t dloss_stride,
                                        void* dx, int64_t dx_stride, void* dw, int64_t dw_stride, void* ws,
                                        size_t ws_bytes, cudaStream_t stream)
{
    adacomp::TrainRange range("adacomp_distill_backward");
    if (!h || rows < 0 || rows >= adacomp::kMostRows) return ADACOMP_ERR_INVALID_ARG;
    adacomp::VocabArgs a = adacomp::vocab_args(rows, x, x_stride, w, w_stride);
    adacomp::set_teacher(a, k, index, index_stride, logit, logit_stride, logit_dtype, temperature);
    adacomp::set_gradients(a, lse, dloss, dloss_stride, dx, dx_stride, dw, dw_stride);
    if (!adacomp::teacher_fits(a)) return ADACOMP_ERR_INVALID_ARG;
    return adacomp::vocab_pass(h, a, true, ws, ws_bytes, stream);
}

adacomp_status adacomp_vocab_set_timeout_ns(adacomp_vocab_t h, uint64_t timeout_ns)
{
    return h ? adacomp::set_timeout(h->waits, timeout_ns) : ADACOMP_ERR_INVALID_ARG;
}

adacomp_status adacomp_vocab_set_fault_injection(adacomp_vocab_t h, uint32_t silent_cta)
{
    if (!h) return ADACOMP_ERR_INVALID_ARG;
    h->waits.silent = silent_cta;
    return ADACOMP_OK;
}

void adacomp_vocab_free(adacomp_vocab_t h) { delete h; }

}  // extern "C"
