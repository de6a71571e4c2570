/*
 * adacomp.h — C ABI of the GB300 (sm_103a) AdaComp library, libadacomp.so.
 *
 * AdaComp ("AdaComp (Adaptive Residual Gradient Compression)", summary paragraph and
 * Claims > Mechanism #r629-local-bin-soft-threshold-and-mean-gmax-quantization) is a
 * per-layer residual gradient compressor for data-parallel training. For one layer
 * with residue r and gradient dW (N elements):
 *     G = r + dW,  H = G + dW,  bins of length L_T over G,
 *     g_max(i) = max |G| over bin i,  s = (1/B) sum_i g_max(i),
 *     send every element with |H| >= g_max(i) as sign(G) * s,
 *     r = G - sign(G) * s for sent elements, r = G for the rest.
 * Codes are 8 bits when L_T < 64 and 16 bits otherwise (Claims > Application
 * #r629-conv-40x-and-fc-lstm-200x-compression-across-optimizers; Curated
 * Limitations). The pages leave open the points below; this library reads them so:
 *   - a partial last bin is a bin; its g_max covers its own elements;
 *   - only G != 0 is sent (sign(0) has no code); the tie |H| == g_max is sent;
 *   - H = fl32(G + dW) after G is rounded; IEEE fp32 adds, no contraction;
 *   - s = fl32( fl64(exact sum of the g_max) / B ), independent of summation order;
 *   - decoding adds sign * s_k into a dense fp32 buffer learner by learner,
 *     k = 0..K-1, with no averaging.
 *
 * Message format (little-endian, no padding), produced by adacomp_compress:
 *     offset 0      float32  s
 *     offset 4      uint32   B = ceil(N / L_T)
 *     offset 8      uint16   count[B]          codes sent from each bin
 *     offset 8+2B   codes, bin by bin, ascending offset within a bin;
 *                   code = (offset_in_bin << 1) | (G < 0); uint8 if L_T < 64 else uint16
 * Its length is 8 + 2B + w * nnz bytes (w = code bytes, nnz = elements sent); it never
 * exceeds max_msg_bytes = 8 + 2B + w * N.
 *
 * Conventions shared by every call:
 *   - Pointers named "device" are CUDA device pointers (e.g. torch tensor data_ptr());
 *     the caller owns every buffer. The library never allocates device memory.
 *   - residue, dW, dense and msg must be 16-byte aligned (ADACOMP_ERR_ALIGNMENT).
 *   - Work is enqueued on `stream` and returns before it runs; results, the message
 *     length and the device-side status are read back with adacomp_query /
 *     adacomp_decode_status. Every call is deterministic: same inputs, same bits.
 *   - A debug build of the library (compiled with ADACOMP_DEBUG_CHECKS defined)
 *     makes every compress, decode and materialise call wait for `stream` after its
 *     launches, unless the stream is being captured, and return ADACOMP_ERR_CUDA
 *     when its kernels raised an error, so that the error is reported by the call
 *     that caused it.
 *   - Argument errors are reported synchronously before anything is enqueued.
 *     ADACOMP_ERR_CUDA reports a failed launch (cudaGetLastError).
 *   - Workspaces: a compress workspace must be zero-filled before its first use
 *     (e.g. torch.zeros); every completed compress call leaves the parts that must
 *     start at zero zeroed again (the rest is written before it is read), so it can
 *     be reused by later calls and by other handles that fit in it. Calls that share a workspace must not overlap on the
 *     GPU (use one stream, or order the streams). After any device-side error
 *     status, zero the workspace again before reusing it.
 *   - Device-side waits (for the bulk copies into shared memory, and, for handles
 *     whose bin lengths are not all 16..509 or all 510..8189, the look-back between
 *     tiles) are bounded by a timeout
 *     (default 2 s, adacomp_set_timeout_ns); on expiry the kernel records
 *     ADACOMP_ERR_TIMEOUT in the workspace and returns. Nothing traps.
 *   - L_T (bin_len) is limited to 1..8192 by this implementation (the format itself
 *     would allow offsets up to 32767).
 */
#ifndef ADACOMP_H
#define ADACOMP_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ADACOMP_OK = 0,
    ADACOMP_ERR_INVALID_ARG = 1,  /* n < 1, bin_len outside 1..8192, B >= 2^32, K outside 1..256 ... */
    ADACOMP_ERR_ALIGNMENT = 2,    /* a buffer is not 16-byte aligned */
    ADACOMP_ERR_WORKSPACE = 3,    /* ws is NULL or smaller than the size init returned */
    ADACOMP_ERR_CAPACITY = 4,     /* msg_capacity < max_msg_bytes */
    ADACOMP_ERR_CUDA = 5,         /* a CUDA runtime call or launch failed */
    ADACOMP_ERR_TIMEOUT = 6,      /* device: a bounded wait (a copy, or the look-back between tiles) ran out */
    ADACOMP_ERR_BAD_MESSAGE = 7   /* device: a message's length, B, counts or offsets do not fit this layer */
} adacomp_status;

typedef enum { ADACOMP_F32 = 0, ADACOMP_BF16 = 1 } adacomp_dtype;

/* Opaque host-side handle: layer sizes, bin length, dW dtype and tile geometry. It
 * holds no device memory and may be used from one host thread at a time. */
typedef struct adacomp_layer* adacomp_layer_t;

/*
 * Describes one layer of n elements compressed with bins of bin_len elements and a
 * dW of type dw_dtype ("AdaComp ...", Claims > Mechanism #r629-local-bin-...: one
 * compressor per layer, with its own residue).
 * Out (each may be NULL):
 *   max_msg_bytes                 bytes a message buffer needs (8 + 2B + w*n)
 *   compress_ws_bytes             bytes of compress workspace
 *   decode_ws_bytes_per_learner   decode workspace = ADACOMP_DECODE_WS_FIXED + K * this
 * Host only: makes no CUDA call. Errors: ADACOMP_ERR_INVALID_ARG.
 */
adacomp_status adacomp_init_layer(adacomp_layer_t* out, int64_t n, int32_t bin_len,
                                  adacomp_dtype dw_dtype, size_t* max_msg_bytes,
                                  size_t* compress_ws_bytes,
                                  size_t* decode_ws_bytes_per_learner);

/*
 * A group of num_layers layers (1..ADACOMP_MAX_GROUP) compressed by one launch
 * sequence: layer l has n[l] elements, bin length bin_len[l] and dW type
 * dw_dtype[l]. Each layer keeps its own bins, s and message, exactly as if it were
 * compressed alone; grouping only removes per-layer launches. max_msg_bytes is an
 * array of num_layers entries (or NULL). Host only.
 */
adacomp_status adacomp_init_group(adacomp_layer_t* out, int32_t num_layers, const int64_t* n,
                                  const int32_t* bin_len, const int32_t* dw_dtype,
                                  size_t* max_msg_bytes, size_t* compress_ws_bytes,
                                  size_t* decode_ws_bytes_per_learner);

#define ADACOMP_MAX_GROUP 128
#define ADACOMP_MAX_LEARNERS 256
#define ADACOMP_DECODE_WS_FIXED 10240

/*
 * One AdaComp step for one layer (Algorithm 2 as restated in Claims > Mechanism
 * #r629-local-bin-soft-threshold-and-mean-gmax-quantization).
 *   residue   device fp32[n], in/out: the carried residue, updated in place
 *             (zeros before the first step)
 *   dW        device fp32[n] or bf16[n] (the dtype given at init), read only
 *   msg       device buffer of msg_capacity >= max_msg_bytes bytes; receives the
 *             message (format above)
 *   ws        device compress workspace of ws_bytes >= compress_ws_bytes (see
 *             Workspaces above)
 * residue and dW must not overlap msg or ws. Errors: INVALID_ARG (NULL handle or
 * pointer), ALIGNMENT, CAPACITY, WORKSPACE, CUDA. Device-side status via
 * adacomp_query.
 */
adacomp_status adacomp_compress(adacomp_layer_t h, float* residue, const void* dW, void* msg,
                                size_t msg_capacity, void* ws, size_t ws_bytes,
                                cudaStream_t stream);

/*
 * adacomp_compress for callers that cannot allocate device memory: plugins and
 * hooks of communication or training frameworks that are handed only their
 * gradient and message buffers, and that run where allocating is not allowed (the
 * host application's allocator owns all device memory, or a fixed memory budget
 * leaves no room for a separate workspace). The paper has no counterpart; this is
 * an interface convenience of this library.
 *
 * Same arguments, checks and results as adacomp_compress, but the compress
 * workspace is an array of ADACOMP_STATIC_WS_BYTES (1 MiB) inside the library (a
 * file-scope __device__ array that every GPU loading the library keeps until the
 * process exits). It therefore takes single-layer handles whose compress_ws_bytes
 * (from adacomp_init_layer) is at most ADACOMP_STATIC_WS_BYTES; compare the two to
 * know whether a layer fits (roughly 3.9M elements for 16 <= L_T <= 509, whose
 * workspace holds two bits per element, about 2M at L_T = 510, rising with L_T to
 * the block-sliced limit of 8189, and far more for other bin lengths). Larger
 * layers get ADACOMP_ERR_WORKSPACE.
 * The call allocates nothing: it zeroes the part of the array it uses
 * (cudaMemsetAsync) and runs the same kernels on `stream`.
 *   result_out  optional device buffer of 32 bytes, 8-byte aligned, that receives
 *               {float s; uint32 status; uint64 nnz; uint64 msg_bytes; uint64 pad}
 *               (the values adacomp_query reports for adacomp_compress); NULL skips it.
 * The first call on each device looks up the array's device address with that
 * device current and keeps it for the life of the process; make that first call
 * before capturing any stream. The kept address belongs to the device's context:
 * after cudaDeviceReset of that device, do not call this entry point again in the
 * same process. All calls share the one array, so calls that overlap on a GPU
 * (different streams, or several host threads) race and corrupt each other's
 * results: serialise them.
 */
#define ADACOMP_STATIC_WS_BYTES ((size_t)1 << 20)
adacomp_status adacomp_compress_static_ws(adacomp_layer_t h, float* residue, const void* dW,
                                          void* msg, size_t msg_capacity, void* result_out,
                                          cudaStream_t stream);

/* adacomp_compress for every layer of a group: arrays of num_layers device pointers
 * (host arrays) and capacities; one workspace for the whole group. */
adacomp_status adacomp_compress_group(adacomp_layer_t h, float* const* residue,
                                      const void* const* dW, void* const* msg,
                                      const size_t* msg_capacity, void* ws, size_t ws_bytes,
                                      cudaStream_t stream);

/*
 * Sums K learners' messages into a dense gradient: for k = 0..K-1 in order, every
 * code of msgs[k] adds sign * s_k to dense[bin * L_T + offset] (one fp32 add each).
 * The pages only say that learners' quantised gradients are combined in
 * data-parallel training (abstract; summary paragraph); the plain sum is this
 * library's reading, and the caller zeroes dense for a fresh sum.
 *   msgs       host array of K device pointers, each a message of this layer
 *              starting on a 16-byte boundary
 *   msg_bytes  host array of K lengths in bytes, the length of each message as
 *              received (messages are variable-length: "AdaComp (Adaptive Residual
 *              Gradient Compression)", Claims > Limitation
 *              #r629-minibatch-size-activity-and-variable-message-length). Nothing
 *              past a message's length is used; the library may read the rest of the
 *              16-byte block its last byte lies in.
 *   dense      device fp32[n], in/out
 *   ws         device decode workspace, ws_bytes >= ADACOMP_DECODE_WS_FIXED
 *              + K * decode_ws_bytes_per_learner; needs no initialisation
 * One CTA owns each range of bins, so no two threads ever add to one element and
 * no float atomics are used. Every message is checked before anything is added, and
 * a message that fails a check is skipped entirely (it adds nothing; the others are
 * summed as usual) and ADACOMP_ERR_BAD_MESSAGE is recorded (adacomp_decode_status).
 * The checks: the length is at least 8 + 2B, the header's B is the layer's B, no
 * count exceeds its bin's length, the length is exactly 8 + 2B + w * (sum of the
 * counts), and within every bin the code offsets rise strictly and stay below the
 * bin's length (a message gives each element at most one code). Errors:
 * INVALID_ARG (K outside 1..256, NULL pointers), ALIGNMENT (dense or a message not
 * 16-byte aligned), WORKSPACE, CUDA.
 */
adacomp_status adacomp_decode_accumulate(adacomp_layer_t h, const void* const* msgs,
                                         const uint64_t* msg_bytes, int32_t K, float* dense,
                                         void* ws, size_t ws_bytes, cudaStream_t stream);

/* Decode for every layer of a group: msgs and msg_bytes are host arrays of
 * num_layers * K entries, layer-major (msgs[l * K + k]); dense a host array of
 * num_layers device pointers. K <= ADACOMP_MAX_LEARNERS and K * num_layers <= 1024. */
adacomp_status adacomp_decode_accumulate_group(adacomp_layer_t h, const void* const* msgs,
                                               const uint64_t* msg_bytes, int32_t K,
                                               float* const* dense, void* ws, size_t ws_bytes,
                                               cudaStream_t stream);

/*
 * Waits for `stream` and reads the result of the last compress call that used `ws`
 * for layer `layer` (0 for a single layer): the message length in bytes, s, and the
 * device status (ADACOMP_OK, ADACOMP_ERR_TIMEOUT). Any output may be NULL.
 */
adacomp_status adacomp_query(adacomp_layer_t h, const void* ws, int32_t layer,
                             cudaStream_t stream, uint64_t* msg_bytes, float* s,
                             int32_t* device_status);

/* Waits for `stream` and reads the device status of the last decode call that used
 * `ws` (ADACOMP_OK or ADACOMP_ERR_BAD_MESSAGE). */
adacomp_status adacomp_decode_status(adacomp_layer_t h, const void* ws, cudaStream_t stream,
                                     int32_t* device_status);

/*
 * Measurement hook (not part of the method): when set, every later compress call
 * on this handle records `before` on its stream before the streaming kernel, `mid`
 * between the streaming kernel and the kernels after it (scale, codes, fix-up), and
 * `after` once all are enqueued, so cudaEventElapsedTime gives the streaming
 * kernel's duration and that of the rest. The events are created and
 * owned by the caller; pass NULLs to stop recording.
 */
adacomp_status adacomp_set_timing_events(adacomp_layer_t h, cudaEvent_t before, cudaEvent_t mid,
                                         cudaEvent_t after);

/*
 * Fault injection for tests of the device-side timeout (not part of the method):
 * when skip_tile is a valid tile index of this handle's next compress calls, the
 * bulk copies of that tile are never started when every layer has 16 <= L_T <= 509
 * or every layer 510 <= L_T <= 8189 (its warps' waits run out), and otherwise the
 * tile never publishes its look-back
 * descriptor (the tiles after it in its layer wait for it); either way the layer
 * reports ADACOMP_ERR_TIMEOUT once the timeout has passed. Nothing faults or hangs. Pass 0xFFFFFFFF to switch it off (the default). After such a
 * call, zero the workspace before reusing it.
 */
adacomp_status adacomp_set_fault_injection(adacomp_layer_t h, uint32_t skip_tile);

/* Bound on each device-side wait, in nanoseconds (default 2e9). */
adacomp_status adacomp_set_timeout_ns(adacomp_layer_t h, uint64_t timeout_ns);

/* Decode fused with one momentum-SGD step (the optimisers the learners use:
 * "AdaComp (Adaptive Residual Gradient Compression)", Claims > Application
 * #r629-conv-40x-and-fc-lstm-200x-compression-across-optimizers; the update rule
 * itself is not on the pages and is read as the usual heavy-ball form without
 * dampening). For each element j of each layer, with g_j the learners' codes summed
 * from zero exactly as adacomp_decode_accumulate sums them (learner order, fp32):
 *     v_j = fl32( fl32(mu * v_j) + fl32(grad_scale * g_j) )
 *     w_j = fl32( w_j - fl32(lr * v_j) )
 * (no fused multiply-add). weights and momentum are fp32[n] per layer, in/out,
 * 16-byte aligned; grad_scale = 1/K averages instead of summing. The gradient is
 * never written to global memory: it lives only in the tile being updated. Same
 * messages, workspace and error reporting as adacomp_decode_accumulate (a rejected
 * message contributes nothing). */
adacomp_status adacomp_decode_sgd(adacomp_layer_t h, const void* const* msgs, const uint64_t* msg_bytes,
                                  int32_t K, float* weights, float* momentum, float lr, float mu,
                                  float grad_scale, void* ws, size_t ws_bytes, cudaStream_t stream);
adacomp_status adacomp_decode_sgd_group(adacomp_layer_t h, const void* const* msgs, const uint64_t* msg_bytes,
                                        int32_t K, float* const* weights, float* const* momentum, float lr,
                                        float mu, float grad_scale, void* ws, size_t ws_bytes,
                                        cudaStream_t stream);

/* Decode fused with one Adam step, the other optimiser the learners use
 * ("AdaComp (Adaptive Residual Gradient Compression)", Claims > Application
 * #r629-conv-40x-and-fc-lstm-200x-compression-across-optimizers; the update rule is
 * not on the pages and is read as Kingma and Ba's Adam with the bias corrections
 * written out). For each element j of each layer, with s_j the learners' codes summed
 * from zero exactly as adacomp_decode_accumulate sums them (learner order, fp32):
 *     g   = fl32(grad_scale * s_j)
 *     m_j = fl32( fl32(beta1 * m_j) + fl32(fl32(1 - beta1) * g) )
 *     v_j = fl32( fl32(beta2 * v_j) + fl32(fl32(1 - beta2) * fl32(g * g)) )
 *     w_j = fl32( w_j - fl32( lr * fl32( fl32(m_j / bias_correction1) /
 *                                        fl32( sqrt(fl32(v_j / bias_correction2)) + eps ) ) ) )
 * (IEEE fp32, correctly rounded division and square root, no fused multiply-add).
 * bias_correction1 = 1 - beta1^t and bias_correction2 = 1 - beta2^t for step t are
 * the caller's (both > 0; ADACOMP_ERR_INVALID_ARG otherwise). weights, m and v are
 * fp32[n] per layer, in/out, 16-byte aligned. The gradient lives only in the tile
 * being updated. Same messages, lengths, workspace and error reporting as
 * adacomp_decode_accumulate (a rejected message contributes nothing). */
adacomp_status adacomp_decode_adam(adacomp_layer_t h, const void* const* msgs, const uint64_t* msg_bytes,
                                   int32_t K, float* weights, float* m, float* v, float lr, float beta1,
                                   float beta2, float eps, float bias_correction1, float bias_correction2,
                                   float grad_scale, void* ws, size_t ws_bytes, cudaStream_t stream);
adacomp_status adacomp_decode_adam_group(adacomp_layer_t h, const void* const* msgs, const uint64_t* msg_bytes,
                                         int32_t K, float* const* weights, float* const* m, float* const* v,
                                         float lr, float beta1, float beta2, float eps, float bias_correction1,
                                         float bias_correction2, float grad_scale, void* ws, size_t ws_bytes,
                                         cudaStream_t stream);

/* Selection rule. ADACOMP_RULE_ADACOMP (the default) sends an element when
 * G != 0 and |fl32(G + dW)| >= g_max of its bin ("AdaComp (Adaptive Residual
 * Gradient Compression)", Claims > Mechanism
 * #r629-local-bin-soft-threshold-and-mean-gmax-quantization).
 * ADACOMP_RULE_LOCAL_SELECTION is the hard Local Selection rule that the same entry
 * contrasts with it (Claims > Mechanism
 * #r629-self-adjusting-sparsity-prevents-residual-explosion): no soft-threshold
 * probe, G != 0 and |G| >= g_max, i.e. only the bin maxima (all of them on a tie).
 * s, the codes, the message format, the residue update and decoding are the same
 * for both. Returns ADACOMP_ERR_INVALID_ARG for any other value. */
enum { ADACOMP_RULE_ADACOMP = 0, ADACOMP_RULE_LOCAL_SELECTION = 1 };
adacomp_status adacomp_set_selection_rule(adacomp_layer_t h, int32_t rule);

/* Deferred ("lazy") fix-up, the next step after the eager path
 * ("AdaComp (Adaptive Residual Gradient Compression)", Claims > Mechanism
 * #r629-local-bin-soft-threshold-and-mean-gmax-quantization: residue = G - G_q for
 * sent elements; the arithmetic is unchanged, only its time moves).
 *
 * With enable != 0, a compress call on this handle leaves the residue of the
 * elements it sent at G and records, in the compress workspace, one bit per such
 * element; the next compress call on the same workspace applies
 * residue = fl32(G - sign(G) * s_prev) to them as it loads them, before forming its
 * own G, and adacomp_materialize applies them on demand. Messages, s and every
 * later step are bit-identical to the eager path; the residue buffer holds the
 * eager residue only after adacomp_materialize. The fix-up is deferred for every
 * layer when all of the handle's layers have 16 <= L_T <= 509, or all have
 * 510 <= L_T <= 8189; in a handle that mixes the ranges or holds other bin lengths
 * it is deferred for the layers with 16 <= L_T <= 509 and the others are fixed up
 * eagerly as before.
 *
 * *compress_ws_bytes receives the workspace size in this mode (it grows by 512
 * bytes per tile unless all layers lie in one of the two ranges above, whose
 * workspaces hold the masks in both modes), and the workspace must be zero-filled before its first use. Consecutive
 * calls must use the same workspace; materialise before checkpointing the residue,
 * before switching the mode off, or after a call that reported an error (then also
 * zero the workspace). adacomp_compress_static_ws rejects such handles
 * (ADACOMP_ERR_INVALID_ARG): its workspace is not kept between calls. */
adacomp_status adacomp_set_lazy_fixup(adacomp_layer_t h, int32_t enable, size_t* compress_ws_bytes);

/* Applies every pending deferred correction to residue[] (layer order of the
 * handle) and clears it; asynchronous on `stream`. Does nothing when the handle
 * defers nothing. Same alignment and workspace rules as adacomp_compress. */
adacomp_status adacomp_materialize(adacomp_layer_t h, float* residue, void* ws, size_t ws_bytes,
                                   cudaStream_t stream);
adacomp_status adacomp_materialize_group(adacomp_layer_t h, float* const* residue, void* ws, size_t ws_bytes,
                                         cudaStream_t stream);

/* ------------------------------------------------------------------------------
 * Training operators around the compressor: what makes the gradients that are
 * compressed (layer norm, a gated linear recurrence) and what is done with the
 * decoded ones (their common norm, an AdamW step over all tensors). The pages name
 * the nets and the optimisers (Claims > Application
 * #r629-conv-40x-and-fc-lstm-200x-compression-across-optimizers) without giving these
 * operators; they are read as defined below.
 *
 * The conventions above hold, with these differences: tensors of layer norm and the
 * recurrence are strided (strides count elements; the last axis is contiguous) and
 * aligned to their element type only (ADACOMP_ERR_ALIGNMENT otherwise); aligned to
 * 16 bytes, with strides that keep every row so, they are read and written faster. What shares
 * 16 bytes, aligned to as many, with a row's elements may be read with them and is not used.
 * Outputs may not overlap inputs or each other unless a call says so, and hold
 * intermediate values while a call runs. Sums, statistics
 * and states are fp32 or wider; results are rounded to the output's type once. Calls
 * are deterministic. Non-finite inputs reach only the results that depend on them.
 * A handle holds sizes, types and settings only and may be used by several host threads.
 * ------------------------------------------------------------------------------ */

/* Layer norm over rows of dim elements (dim >= 1) of type x_dtype, with a weight and
 * a bias of type w_dtype (both dtypes ADACOMP_F32 or ADACOMP_BF16):
 *     mean = sum(x) / dim,  var = sum((x - mean)^2) / dim,  rstd = 1 / sqrt(var + eps),
 *     y = (x - mean) * rstd * w + b.
 * eps >= 0 and finite. Host only. */
typedef struct adacomp_layer_norm* adacomp_layer_norm_t;
adacomp_status adacomp_layer_norm_init(adacomp_layer_norm_t* out, int64_t dim, adacomp_dtype x_dtype,
                                       adacomp_dtype w_dtype, float eps);

/* y = norm of each of `rows` rows (0 does nothing). w and b are w_dtype[dim], b may be
 * NULL (no bias). mean and rstd, fp32[rows] each, are what the backward pass needs;
 * either may be NULL. y may be x itself with the same stride. x_stride >= 0 (0: one row
 * read for all), y_stride >= dim unless rows < 2. */
adacomp_status adacomp_layer_norm_forward(adacomp_layer_norm_t h, int64_t rows, const void* x, int64_t x_stride,
                                          const void* w, const void* b, void* y, int64_t y_stride, float* mean,
                                          float* rstd, cudaStream_t stream);

/* Workspace bytes of a backward pass over `rows` rows (partial sums; needs no
 * initialisation). */
size_t adacomp_layer_norm_backward_ws_bytes(adacomp_layer_norm_t h, int64_t rows);

/* From dy and the forward pass's x, mean and rstd, with xh = (x - mean) * rstd and g = dy * w:
 *     dx = rstd * (g - sum(g)/dim - xh * sum(g * xh)/dim),
 *     dw = sum over rows of dy * xh,   db = sum over rows of dy.
 * dw and db are w_dtype[dim] and are overwritten (zeros for 0 rows); db may be NULL. dx
 * may be dy or x itself with the same stride. ws: 16-byte aligned, of at least
 * adacomp_layer_norm_backward_ws_bytes(h, rows) bytes. */
adacomp_status adacomp_layer_norm_backward(adacomp_layer_norm_t h, int64_t rows, const void* dy, int64_t dy_stride,
                                           const void* x, int64_t x_stride, const void* w, const float* mean,
                                           const float* rstd, void* dx, int64_t dx_stride, void* dw, void* db,
                                           void* ws, size_t ws_bytes, cudaStream_t stream);
void adacomp_layer_norm_free(adacomp_layer_norm_t h);

/* A gated linear recurrence over `channels` independent channels (>= 1) of sequences
 * [batch, steps, channels] in `dtype`: with the gate a_t = 1 / (1 + exp(-z_t)),
 *     h_t = a_t * h_{t-1} + (1 - a_t) * x_t,   y_t = h_t,   t = 0 .. length-1.
 * The state is fp32 throughout; y is it rounded once. steps = 1 is the form for one new
 * token. The smaller of a_t and 1 - a_t has an error of up to 6 + 1.2 |z_t| units in its last
 * place, the larger of up to 6, and what is below 2^-126 (|z_t| > 87.3) is 0. Steps may be
 * composed, h -> A h + H, in an order that depends on the sizes. An infinite state, or gradient
 * in the backward pass, stays infinite through gates that are not 0; one of 0 makes it infinite
 * or NaN. Host only. */
typedef struct adacomp_recurrence* adacomp_recurrence_t;
adacomp_status adacomp_recurrence_init(adacomp_recurrence_t* out, int64_t channels, adacomp_dtype dtype);

/* Bytes of the fp32 states that a forward pass keeps for the backward pass: one every
 * ADACOMP_RECURRENCE_CHUNK steps, [batch][ceil(steps / chunk)][channels]. */
#define ADACOMP_RECURRENCE_CHUNK 64
size_t adacomp_recurrence_carry_bytes(adacomp_recurrence_t h, int64_t batch, int64_t steps);

/* The forward pass. z, x and y each have a stride between sequences and one between
 * steps (z and x may be the two halves of one buffer).
 *   h0       device fp32[batch][channels], the state before the first step; NULL: zeros
 *   lengths  device int32[batch], each sequence's steps, clamped to 0..steps; NULL: all
 *            of them. z and x past the length are not read (they may hold anything), and
 *            y is zero there.
 *   h_last   device fp32[batch][channels], the state after the last step (h0 for a
 *            sequence without steps); may be NULL, may be h0 itself
 *   carry    as adacomp_recurrence_carry_bytes; NULL when no backward pass follows
 * batch = 0 does nothing; steps = 0 copies the state. */
adacomp_status adacomp_recurrence_forward(adacomp_recurrence_t h, int64_t batch, int64_t steps, const void* z,
                                          int64_t z_batch, int64_t z_step, const void* x, int64_t x_batch,
                                          int64_t x_step, const float* h0, const int32_t* lengths, void* y,
                                          int64_t y_batch, int64_t y_step, float* h_last, float* carry,
                                          cudaStream_t stream);

/* The backward pass, from the gradients dy of y and dh_last of h_last (NULL: zeros), the
 * forward pass's inputs and its carry. With G_t = dy_t + a_{t+1} * G_{t+1} (dh_last in
 * place of the last product):
 *     dx_t = (1 - a_t) * G_t,  dz_t = a_t * (1 - a_t) * (h_{t-1} - x_t) * G_t,
 *     dh0 = a_0 * G_0.
 * h_{t-1} is computed again in fp32 from the carry. dz and dx are zero past a sequence's
 * length, where dy is not read; dh0 (fp32[batch][channels]) may be NULL or dh_last itself.
 * z, x, dz and dx: a stride pair each, as in the forward pass. */
adacomp_status adacomp_recurrence_backward(adacomp_recurrence_t h, int64_t batch, int64_t steps, const void* z,
                                           int64_t z_batch, int64_t z_step, const void* x, int64_t x_batch,
                                           int64_t x_step, const void* dy, int64_t dy_batch, int64_t dy_step,
                                           const float* carry, const int32_t* lengths, const float* dh_last,
                                           void* dz, int64_t dz_batch, int64_t dz_step, void* dx, int64_t dx_batch,
                                           int64_t dx_step, float* dh0, cudaStream_t stream);

/* Calls over few channels of many steps split a sequence over CTAs of a cluster that wait for
 * each other's totals. Such a wait is bounded by a timeout in nanoseconds (default 2e9, rounded up
 * to microseconds, and begun after some 250 tries). The CTAs run together and each writes before
 * it waits, so none is expected to run out. On expiry the call still ends as usual, with the
 * status ADACOMP_OK that it returned: what the CTA computes from there on, y, dz and dx of its
 * steps and the states, is NaN, as there is no workspace to record ADACOMP_ERR_TIMEOUT in.
 * Nothing traps. Not to be set while another host thread calls with the handle. */
adacomp_status adacomp_recurrence_set_timeout_ns(adacomp_recurrence_t h, uint64_t timeout_ns);

/* Fault injection for tests of that timeout (not part of the operator): the given CTA of every
 * cluster writes nothing to the others, so that all of the cluster's waits run out. 0xFFFFFFFF
 * switches it off (the default). Nothing faults or hangs. */
adacomp_status adacomp_recurrence_set_fault_injection(adacomp_recurrence_t h, uint32_t silent_cta);
void adacomp_recurrence_free(adacomp_recurrence_t h);

/* AdamW over many tensors at once, and the norm of their gradients. Tensor i has n[i]
 * elements (>= 1), weights of w_dtype[i], gradients of g_dtype[i] (ADACOMP_F32 or
 * ADACOMP_BF16) and a decoupled weight decay weight_decay[i] (the array may be NULL: none
 * decays). state_bits is 32 (m and v are fp32[n]) or 8: m and the root of v are then
 * e4m3[n] numbers, each block of ADACOMP_ADAMW_BLOCK elements with an fp32 scale, so that
 * the block's largest magnitude is 448 * scale. num_tensors is 1..ADACOMP_MAX_TENSORS.
 * norm_ws_bytes (may be NULL) receives the workspace size of adacomp_grad_norm. Host only. */
typedef struct adacomp_adamw* adacomp_adamw_t;
#define ADACOMP_ADAMW_BLOCK 256
#define ADACOMP_MAX_TENSORS 65536
adacomp_status adacomp_adamw_init(adacomp_adamw_t* out, int32_t num_tensors, const int64_t* n,
                                  const int32_t* w_dtype, const int32_t* g_dtype, const float* weight_decay,
                                  int32_t state_bits, size_t* norm_ws_bytes);

/* norm = grad_scale * sqrt(sum of the squares of all gradients), and the coefficient that
 * adacomp_adamw_step multiplies the gradients by:
 *     result[0] = norm,
 *     result[1] = grad_scale * min(1, max_norm / (norm + 1e-6))   (grad_scale if max_norm <= 0),
 * or NaN in result[1] when the norm is not finite. Squares whose fp32 sums would overflow
 * or vanish are summed in fp64. grad is a host array of num_tensors device pointers,
 * 16-byte aligned; result is device fp32[2]; ws is 16-byte aligned and zero-filled before
 * its first use (every call leaves it ready for the next). grad_scale must be finite and
 * positive. */
adacomp_status adacomp_grad_norm(adacomp_adamw_t h, const void* const* grad, float grad_scale, float max_norm,
                                 float* result, void* ws, size_t ws_bytes, cudaStream_t stream);

/* One AdamW step. With c = *coefficient (or grad_scale where that is NULL), every operation
 * fp32, rounded once, without fused multiply-adds:
 *     g = c * g_j,  m = beta1 * m + (1 - beta1) * g,  v = beta2 * v + (1 - beta2) * (g * g),
 *     u = sqrt(v),
 *     w = fl32(1 - lr * weight_decay) * w
 *         - fl32(lr / bias_correction1) * (m / (u * fl32(1 / sqrt(bias_correction2)) + eps)).
 * The three constants are formed in fp64 and rounded once. With 8-bit states m and v enter
 * as (e4m3 * scale) and (e4m3 * scale)^2, and leave as the block's new scale = max/448 and
 * the e4m3 nearest to value * (448/max) (to even; a positive u never becomes 0 but the
 * smallest e4m3; a block whose max is below 2^-96 has scale 0, and so stands for zeros). A value
 * that is not finite reaches its whole block through the scale.
 *   weight, grad, m, v   host arrays of num_tensors device pointers, 16-byte aligned;
 *                        weight, m and v are in/out. State starts as zeros.
 *   m_scale, v_scale     8-bit states: device fp32[ceil(n/256)] per tensor; otherwise NULL
 *   copy                 NULL, or per tensor a bf16[n] buffer that receives the new weight
 *                        rounded (for weights held in fp32 next to a bf16 model), 16-byte
 *                        aligned, or NULL for none
 *   coefficient          device fp32 (e.g. result + 1 of adacomp_grad_norm) or NULL. When it
 *                        is not finite the call leaves weights, states and copies as they are.
 * beta1, beta2 in [0, 1), eps > 0 and bias corrections > 0, or ADACOMP_ERR_INVALID_ARG. */
adacomp_status adacomp_adamw_step(adacomp_adamw_t h, void* const* weight, const void* const* grad, void* const* m,
                                  void* const* v, float* const* m_scale, float* const* v_scale, void* const* copy,
                                  float lr, float beta1, float beta2, float eps, float bias_correction1,
                                  float bias_correction2, float grad_scale, const float* coefficient,
                                  cudaStream_t stream);
void adacomp_adamw_free(adacomp_adamw_t h);

/* ------------------------------------------------------------------------------
 * Linear layers and losses over a vocabulary: the matrix products of a training step. The
 * conventions of the training operators above hold. Matrices are strided by rows: inputs
 * by any stride >= 0 (0: one row read for all), outputs by at least a row; up to 2^30 rows. Products of few rows and
 * small ones read them as they lie, larger ones bf16 matrices with 16-byte aligned pointers and rows that are multiples
 * of 16 bytes, and no less than a row, apart; others, and hidden states, are first copied into the workspace. Workspaces
 * are 16-byte aligned, need no initialisation, and serve one call at a time.
 *
 * bf16 products are exact and summed in fp32; the tensor cores cut off a partial sum's last bits every 16 terms, so where
 * results are fp32 they sum runs of up to 512 terms, which are added up. fp32 numbers are, but in small products, split
 * into three bf16 numbers that add up to them (what is below 2^-126 may be lost), and of the nine products of
 * parts the six largest are summed, which leaves out less than 2^-22 of a product. Sums add the terms
 * in an order that depends on sizes and alignment alone, not on which outputs are asked for (over a vocabulary the terms
 * of dw are the rows that have a loss, so there it depends on which they are), and round or truncate each partial sum.
 *
 * The kernels of larger products wait for their own copies and products. Such a wait is bounded (below); each is
 * ended by what its own pair of CTAs does, so none is expected to run out. On expiry the call still ends as usual,
 * with the status ADACOMP_OK that it returned, and the results that it had not computed are NaN. Nothing traps.
 * ------------------------------------------------------------------------------ */

/* A linear layer from in_dim to out_dim (each 1..2^30), all of its tensors of one dtype:
 *     z = x w^T + bias,  y = act(z) + residual,   w[out_dim][in_dim].
 * Activations, of fp32 z (of bf16 layers by quick functions, off by no more than 2^-12 of the value and 2^-20 of z):
 * relu(z) = max(z, 0) (slope 0 at 0); gelu(z) = z (1 + erf(z / sqrt 2)) / 2;
 * gelu_tanh(z) = z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2; silu(z) = z / (1 + exp(-z)).
 * Host only. */
typedef enum {
    ADACOMP_ACT_NONE = 0,
    ADACOMP_ACT_RELU = 1,
    ADACOMP_ACT_GELU = 2,
    ADACOMP_ACT_GELU_TANH = 3,
    ADACOMP_ACT_SILU = 4
} adacomp_activation;
typedef struct adacomp_linear* adacomp_linear_t;
adacomp_status adacomp_linear_init(adacomp_linear_t* out, int64_t in_dim, int64_t out_dim, adacomp_dtype dtype,
                                   adacomp_activation activation);

/* Workspace bytes of a forward or backward pass over up to `rows` rows, whatever their alignment. */
size_t adacomp_linear_forward_ws_bytes(adacomp_linear_t h, int64_t rows);
size_t adacomp_linear_backward_ws_bytes(adacomp_linear_t h, int64_t rows);

/* y of `rows` rows (0 does nothing; one row, or a few, is the form for new tokens). bias[out_dim]
 * and residual may be NULL; y may be residual itself with the same stride. pre (may be NULL)
 * receives z rounded to dtype, which the backward pass of an activation needs. */
adacomp_status adacomp_linear_forward(adacomp_linear_t h, int64_t rows, const void* x, int64_t x_stride, const void* w,
                                      int64_t w_stride, const void* bias, const void* residual, int64_t residual_stride,
                                      void* y, int64_t y_stride, void* pre, int64_t pre_stride, void* ws,
                                      size_t ws_bytes, cudaStream_t stream);

/* From dy, with dz = dy * act'(pre) (dy itself without an activation; pre may then be NULL):
 *     dx = dz w,  dw = dz^T x,  db = sum over rows of dz;   the residual's gradient is dy.
 * For the products dz is rounded to bf16 where dtype is bf16 (in calls of up to 32 rows, taken in two parts); db is summed
 * from the unrounded dz. dx, dw and db may each be NULL (not wanted; x is needed for dw only, w for dx only) and are overwritten
 * (dw and db with zeros for 0 rows). */
adacomp_status adacomp_linear_backward(adacomp_linear_t h, int64_t rows, const void* dy, int64_t dy_stride,
                                       const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                                       const void* pre, int64_t pre_stride, void* dx, int64_t dx_stride, void* dw,
                                       int64_t dw_stride, void* db, void* ws, size_t ws_bytes, cudaStream_t stream);

/* The bound of the waits, in nanoseconds (1 to 6e10, default 2e9), begun after some 17 ms of tries, of the calls made with the
 * handle from then on. Not to be set while another host thread calls with the handle. */
adacomp_status adacomp_linear_set_timeout_ns(adacomp_linear_t h, uint64_t timeout_ns);

/* Fault injection for tests of that bound (not part of the operator): the given CTA (0 or 1) of every pair copies
 * nothing, so that the pair's waits run out. 0xFFFFFFFF switches it off (the default). Nothing faults or hangs. */
adacomp_status adacomp_linear_set_fault_injection(adacomp_linear_t h, uint32_t silent_cta);
void adacomp_linear_free(adacomp_linear_t h);

/* A vocabulary of `vocab` tokens (1..2^30) with weights w[vocab][dim] (dim 1..2^30), and the losses of
 * hidden states x[rows][dim] against it, x, w, dx and dw of one dtype. The logits z = x w^T stay in
 * fp32 and are not kept: a backward pass forms them again, a piece of the vocabulary at a time. Host only. */
typedef struct adacomp_vocab* adacomp_vocab_t;
adacomp_status adacomp_vocab_init(adacomp_vocab_t* out, int64_t dim, int64_t vocab, adacomp_dtype dtype);

/* Workspace bytes over up to `rows` rows, whatever their alignment; k as below. */
size_t adacomp_vocab_loss_forward_ws_bytes(adacomp_vocab_t h, int64_t rows);
size_t adacomp_vocab_loss_backward_ws_bytes(adacomp_vocab_t h, int64_t rows);
size_t adacomp_distill_forward_ws_bytes(adacomp_vocab_t h, int64_t rows, int32_t k);
size_t adacomp_distill_backward_ws_bytes(adacomp_vocab_t h, int64_t rows, int32_t k);

/* Softmax cross entropy:  lse = log(sum over v of exp(z_v)),  loss = lse - z_target.
 *   target   device int32[rows] or int64[rows] (target_bytes 4 or 8). A row whose target is negative
 *            has no loss: its loss and lse are 0, its x is not used (it may hold anything), and
 *            takes no time in the products. One of vocab or more makes the row's loss NaN.
 *   loss     device fp32[rows];  lse  device fp32[rows], for the backward pass
 * rows = 0 does nothing. */
adacomp_status adacomp_vocab_loss_forward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride,
                                          const void* w, int64_t w_stride, const void* target, int32_t target_bytes,
                                          float* loss, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/* The gradients, from the gradient dloss of loss (device fp32; row r's is dloss[r * dloss_stride], so 0 is one
 * value for all rows; not used for rows without a loss):
 *     dz = (exp(z - lse) - [v = target]) * dloss,  dx = dz w,  dw = dz^T x.
 * For the products dz is rounded to bf16 where dtype is bf16 (in calls of up to 32 rows,
 * with a loss or without, taken in two parts). dx and dw may each be NULL (not both) and are overwritten: dx is 0
 * in rows without a loss, dw is 0 if no row has one. A target of vocab or more makes the row's
 * dx, and dw, NaN. */
adacomp_status adacomp_vocab_loss_backward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride,
                                           const void* w, int64_t w_stride, const void* target, int32_t target_bytes,
                                           const float* lse, const float* dloss, int64_t dloss_stride, void* dx,
                                           int64_t dx_stride, void* dw, int64_t dw_stride, void* ws, size_t ws_bytes,
                                           cudaStream_t stream);

/* Distillation from a teacher's k logits per row (1 <= k <= ADACOMP_MAX_TEACHER), of the tokens
 * index: with t = temperature, q = softmax(logit / t) over the row's listed tokens and
 * p = softmax(z / t) over the vocabulary,
 *     lse = log(sum over v of exp(z_v / t)),
 *     loss = t^2 * sum over the list of q * (log q - log p).
 *   index    device int32[rows][k], rows index_stride apart. A negative one is no token (a shorter
 *            list); a row without any has no loss, as above. One of vocab or more makes the row's loss NaN.
 *            A token that is listed twice counts twice.
 *   logit    device, of logit_dtype, [rows][k], rows logit_stride apart; not used where index is
 *            negative. -inf is a probability of 0; a row of nothing else has a loss of NaN.
 * temperature is positive, and it, its square and its inverse are finite. The vocabulary's gradients as above, with
 *     dz = t * (p - sum of q over the token's places in the list) * dloss. */
#define ADACOMP_MAX_TEACHER 256
adacomp_status adacomp_distill_forward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride, const void* w,
                                       int64_t w_stride, int32_t k, const int32_t* index, int64_t index_stride,
                                       const void* logit, int64_t logit_stride, adacomp_dtype logit_dtype,
                                       float temperature, float* loss, float* lse, void* ws, size_t ws_bytes,
                                       cudaStream_t stream);
adacomp_status adacomp_distill_backward(adacomp_vocab_t h, int64_t rows, const void* x, int64_t x_stride, const void* w,
                                        int64_t w_stride, int32_t k, const int32_t* index, int64_t index_stride,
                                        const void* logit, int64_t logit_stride, adacomp_dtype logit_dtype,
                                        float temperature, const float* lse, const float* dloss, int64_t dloss_stride,
                                        void* dx, int64_t dx_stride, void* dw, int64_t dw_stride, void* ws,
                                        size_t ws_bytes, cudaStream_t stream);

/* As adacomp_linear_set_timeout_ns and adacomp_linear_set_fault_injection. */
adacomp_status adacomp_vocab_set_timeout_ns(adacomp_vocab_t h, uint64_t timeout_ns);
adacomp_status adacomp_vocab_set_fault_injection(adacomp_vocab_t h, uint32_t silent_cta);
void adacomp_vocab_free(adacomp_vocab_t h);

/* Releases the handle. adacomp_free(NULL) does nothing. */
void adacomp_free(adacomp_layer_t h);

/* Static text for a status code. */
const char* adacomp_status_string(adacomp_status s);

#ifdef __cplusplus
}
#endif

#endif /* ADACOMP_H */
