/*
 * ar.h -- C ABI of the GB300 partial-sum reduction (libtps_ar.so).
 *
 * The operation is the reduction step of a tensor-parallel AllReduce, done
 * on one GPU: R partial tensors ("ranks") of one activation, each in its own
 * device allocation, are each rounded through a narrower wire type, summed
 * in float in ascending rank order, and the sum is cast back to the tensor
 * type and written to every destination buffer:
 *
 *   for every element i:
 *     acc = float(wire(src[0][i]))
 *     acc = acc + float(wire(src[r][i]))        r = 1 .. R-1, in this order
 *     dst[d][i] = T_dst(acc)                     d = 0 .. n_dsts-1
 *
 * wire(x) and T_dst(x) round to nearest, ties to even, keep subnormals and
 * overflow to infinity; float(x) is exact; the adds are float adds rounded
 * to nearest.  The result is bit-for-bit the same for every variant, grid
 * size and alignment (NaN payloads aside).
 *
 * Where this comes from:
 *   - ggml-cuda allreduce.cu (toy 0.8.0 vendored ggml), ggml_cuda_ar_kernel,
 *     phases 1 and 3, and ggml_cuda_ar_add_kernel: both operands are rounded
 *     through the wire type, widened to float, added in float and the sum is
 *     cast back to the tensor type, so that every rank computes identical
 *     bits; ggml_cuda_ar_allreduce picks the wire type (bf16 for f32 tensors)
 *     and the strategy by tensor size.
 *   - ggml-hexagon htp/allreduce-ops.c (char-fork/llama.cpp),
 *     DEFINE_ALLREDUCE_THREAD_DMA_1D: the ranks are folded left to right and
 *     the result is written to each of n_dsts destinations; validate_allreduce
 *     and op_allreduce return status codes instead of asserting.
 *   - The float accumulator for R > 2, the start from rank 0's operand (not
 *     from zero) and the rounding rules are this library's readings where the
 *     pages are silent.
 *
 * Conventions for every call below:
 *   - Device pointers are CUDA addresses the device that was current at
 *     ar_init can access: device memory, or pinned/managed host memory
 *     (which the kernel then reads or writes over the CPU-GPU link); host
 *     pointers are ordinary (ideally pinned) host memory.  The caller owns
 *     every buffer and the stream; the library keeps no pointer after a call
 *     returns and allocates nothing per call.
 *   - Calls that take a stream only enqueue work on it and return; results
 *     are ready when the stream reaches that point.  No call synchronizes
 *     (a host call given pageable memory waits for CUDA's synchronous
 *     pageable copies, see ar_reduce_host and ar_reduce_host_noalloc), so ar_reduce and
 *     ar_reduce_variant can be captured in a CUDA graph.
 *   - On any status other than AR_OK nothing has been enqueued or written,
 *     except AR_ERR_CUDA from a launch, after which the stream's state is
 *     whatever CUDA reports.
 *   - All calls are thread-safe; they share one process-wide context.
 */
#ifndef TPS_AR_H
#define TPS_AR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The CUDA runtime's stream handle (identical to its own typedef). */
typedef struct CUstream_st *cudaStream_t;

/* Element types.  Sources and destinations hold T_dst; T_wire is the type
 * every operand is rounded through before the float sum. */
typedef enum { AR_F32 = 0, AR_F16 = 1, AR_BF16 = 2 } ar_dtype;

typedef enum {
    AR_OK = 0,
    AR_ERR_INVALID_ARG = 1,     /* bad count, NULL pointer, wrong device, ... */
    AR_ERR_UNSUPPORTED = 2,     /* unknown dtype, or the GPU cannot run the kernels */
    AR_ERR_TOO_LARGE = 3,       /* nelem > max_elems given to ar_init */
    AR_ERR_NOT_INITIALIZED = 4, /* ar_init has not succeeded */
    AR_ERR_OVERLAP = 5,         /* a destination partly overlaps another buffer */
    AR_ERR_CUDA = 6             /* a CUDA call failed */
} ar_status;

/* Limits: at most 16 ranks and 16 destinations per call (the pages cap
 * their rank arrays at compile-time maxima of this order:
 * GGML_CUDA_MAX_DEVICES in allreduce.cu, HTP_ALLREDUCE_MAX_RANKS in
 * allreduce-ops.c). */
#define AR_MAX_RANKS 16
#define AR_MAX_DSTS 16

/* Kernel variants.  AUTO picks LATENCY or BANDWIDTH by the call's byte
 * count.  The vector variants want every source and destination at the same
 * offset from a 16-byte boundary (32 for BANDWIDTH's wide f32 vectors, else
 * 16): they then shift past the few elements before the boundary, which they
 * reduce one by one.  When the offsets differ AUTO takes SCALAR.  Every
 * variant computes the same bits. */
typedef enum {
    AR_VARIANT_AUTO = 0,
    AR_VARIANT_NAIVE = 1,     /* one element per thread, grid-stride: a cross-check */
    AR_VARIANT_LATENCY = 2,   /* one 16-byte vector per thread, 128-thread CTAs */
    AR_VARIANT_BANDWIDTH = 3, /* one 32-byte (f32) or 16-byte vector per thread, 256-thread
                                 CTAs; all loads of two or four ranks issued together */
    AR_VARIANT_SCALAR = 4,    /* element-wise path used when the buffers' offsets differ */
    AR_VARIANT_TMA = 5        /* shared-memory staging: a producer warp bulk-copies (cp.async.bulk)
                                 R source tiles per stage, sixteen warps fold them, one thread
                                 bulk-stores the result tile to every destination; two CTAs per SM.
                                 Needs 16-byte aligned buffers.  Never chosen by AUTO (an
                                 AR_VARIANT environment override with offset buffers takes
                                 BANDWIDTH, or SCALAR when the offsets differ).  Its internal waits are bounded: a wait
                                 that runs out sets bit 0 of AR_Q_DEVICE_STATUS and the call's
                                 results are then unspecified (the call still ends). */
} ar_variant;

/*
 * ar_init -- create the process-wide context on the current CUDA device.
 *   R          number of ranks (partials) every ar_reduce call sums, 1..16.
 *   max_elems  largest nelem any later call may pass (>= 1).
 * Reads the environment once: AR_VARIANT (auto|naive|latency|bandwidth|
 * scalar|tma), AR_LATENCY_MAX_BYTES (size switch, bytes of sources plus
 * destinations), AR_TMA_STAGES (2..8, default 3), AR_TMA_TILE (largest
 * tile in bytes, a multiple of 1024 up to 32768, default 16384),
 * AR_TMA_CTAS_PER_SM (1..4, default 2), AR_PDL (1 = default: on a created
 * stream, every kernel but NAIVE's launches as a programmatic dependent of
 * the kernel before it on the stream, which it waits for before touching
 * memory; launches on the default streams stay plain; 0 = plain launches
 * everywhere), AR_L2_PREFETCH (1 = default: the first wave of CTAs of the
 * LATENCY and BANDWIDTH kernels asks L2 for its source vectors before that
 * wait, so they load while the kernel ahead drains; 0 = off; results are the
 * same either way), AR_LOG=1 (one line per init to stderr).
 * Calling it again replaces the context.  Returns AR_OK, AR_ERR_INVALID_ARG,
 * AR_ERR_UNSUPPORTED (the device is not sm_103) or AR_ERR_CUDA (no device).
 */
int ar_init(int R, size_t max_elems);

/*
 * ar_reduce -- enqueue one reduction on `stream`.
 *   srcs       host array of R device pointers, each to nelem elements of
 *              dst_dtype (contiguous); read only.
 *   dsts       host array of n_dsts device pointers, each to nelem elements
 *              of dst_dtype; all receive the same bits.  A destination may
 *              be exactly one of the sources (in-place reduction) but may
 *              not partly overlap any source or other destination.
 *   n_dsts     1..16.
 *   nelem      elements per buffer, <= max_elems; 0 is a no-op (AR_OK).
 *   dst_dtype  ar_dtype of sources and destinations.
 *   wire_dtype ar_dtype every operand is rounded through (any of the three).
 *   stream     CUDA stream of the init device (0 = legacy default stream).
 * Any element-aligned pointer works; buffers that all share one offset from
 * a 16-byte boundary take the vector paths.  Returns an ar_status.
 */
int ar_reduce(const void *const *srcs, void *const *dsts, int n_dsts, size_t nelem,
              int dst_dtype, int wire_dtype, cudaStream_t stream);

/* ar_free -- drop the context.  Safe to call when not initialized. */
void ar_free(void);

/* Static English text for a status code (never NULL). */
const char *ar_status_string(int status);

/*
 * ar_check_args -- the host-side validation ar_reduce runs before any CUDA
 * call, on explicit R and max_elems instead of the context's.  Makes no CUDA
 * call and touches no device memory, so it runs without a GPU.
 */
int ar_check_args(int R, const void *const *srcs, void *const *dsts, int n_dsts,
                  size_t nelem, size_t max_elems, int dst_dtype, int wire_dtype);

/*
 * ar_reduce_variant -- ar_reduce with the kernel variant forced.
 *   variant     an ar_variant; AUTO behaves exactly like ar_reduce.
 *   grid_blocks CTAs to launch for BANDWIDTH/NAIVE/SCALAR (0 = the library's
 *               choice); ignored by LATENCY, whose grid covers the tensor.
 *               A BANDWIDTH grid smaller than the tensor needs is persistent:
 *               its CTAs sweep the tensors together in rounds.
 * The result bits do not depend on either argument.  LATENCY or BANDWIDTH
 * asked for with buffers at different offsets from a 16-byte boundary, or
 * TMA with any buffer off that boundary, returns AR_ERR_INVALID_ARG.
 */
int ar_reduce_variant(const void *const *srcs, void *const *dsts, int n_dsts, size_t nelem,
                      int dst_dtype, int wire_dtype, int variant, int grid_blocks,
                      cudaStream_t stream);

/* Keys for ar_query / ar_set_option. */
typedef enum {
    AR_Q_RANKS = 0,             /* R fixed at ar_init (query only) */
    AR_Q_MAX_ELEMS = 1,         /* max_elems (query only) */
    AR_Q_DEVICE = 2,            /* CUDA device ordinal (query only) */
    AR_Q_SM_COUNT = 3,          /* SMs on that device (query only) */
    AR_Q_LATENCY_MAX_BYTES = 4, /* AUTO uses LATENCY below this many bytes */
    AR_Q_FORCED_VARIANT = 5,    /* variant AUTO resolves to when nonzero */
    AR_Q_LAST_VARIANT = 6,      /* variant the last successful launch used (query only); after
                                   ar_reduce_ex or ar_wire_pack: BANDWIDTH for their vector
                                   kernel, SCALAR for their element-wise one */
    AR_Q_FAULT_INJECT = 7,      /* nonzero: the next launches fail with AR_ERR_CUDA
                                   before anything is enqueued (host-side test hook) */
    AR_Q_BW_BLOCKS_PER_SM = 8,  /* 0: the BANDWIDTH grid covers the tensor (default); n > 0: a
                                   persistent grid of n CTAs per SM (capped by occupancy) */
    AR_Q_HOST_CHUNK_BYTES = 9,  /* ar_reduce_host pipeline chunk, bytes per buffer (default 4 MiB;
                                   at most 64 chunks per call) */
    AR_Q_DEVICE_STATUS = 10,    /* device-side status word (bit 0: a bounded wait of the TMA
                                   variant ran out; bit 1: one of ar_vocab_loss or
                                   ar_vocab_loss_grad, after two seconds - the call's results are
                                   then unspecified and the context stays usable); reading it
                                   synchronises with the device; set it to 0 to clear it */
    AR_Q_TMA_DROP_TILE = 11     /* test hook for failure detection, -1 (default) = off: TMA
                                   launches never load tile n, so the CTA that owns it waits
                                   for data that never comes until its bound (100 ms) runs out,
                                   reports through AR_Q_DEVICE_STATUS and returns; the results of
                                   such a launch are unspecified and the context stays usable */
} ar_key;

/* Read one context value into *value.  AR_ERR_NOT_INITIALIZED before init. */
int ar_query(int key, int64_t *value);

/* Change one settable context value.  Not to be called while a stream
 * capture that uses the library is in progress. */
int ar_set_option(int key, int64_t value);

/*
 * ar_reduce_host -- the same reduction for callers whose partials live in
 * host memory; the results are written back to host memory.
 *   h_srcs, h_dsts  R and n_dsts host pointers, nelem elements each.
 * Two ways to move the data, chosen by the staging arguments:
 *   d_srcs, d_dsts  R and n_dsts device buffers of nelem elements: each host
 *                   source is copied into its staging buffer, the reduction
 *                   writes the staging destinations, and those are copied
 *                   back to the host.  The work is cut into chunks (see
 *                   AR_Q_HOST_CHUNK_BYTES) and pipelined over three streams
 *                   the context owns, so copies in, kernels and copies out of
 *                   different chunks overlap.  Pinned host memory makes the
 *                   copies asynchronous; pageable memory also works, but CUDA
 *                   copies it synchronously, so the call then waits for its
 *                   copies.  It waits without holding the library lock:
 *                   other threads' calls go on, except another staged
 *                   ar_reduce_host (the pipeline is one per context) and
 *                   ar_init / ar_free, which wait for this call to end.
 *   both NULL       no staging: the kernel itself loads the host partials and
 *                   stores the host results over the CPU-GPU link (NVLink-C2C
 *                   on GB300), with no copies at all.  Every host buffer must
 *                   be memory the GPU can reach (cudaHostAlloc /
 *                   cudaHostRegister pinned memory, or managed memory);
 *                   otherwise AR_ERR_INVALID_ARG.
 * Everything else as for ar_reduce, and the host buffers obey ar_reduce's
 * buffer rules too: element-aligned, and a host destination may be exactly
 * a host source but may not partly overlap any host source or other host
 * destination (AR_ERR_OVERLAP, nothing enqueued).  Either way the work
 * starts after what is already enqueued on `stream`, and `stream` reaches
 * the end of this call only when the host results are complete.  Results
 * are identical to one ar_reduce over device copies of the same tensors.
 */
int ar_reduce_host(const void *const *h_srcs, void *const *h_dsts, int n_dsts, size_t nelem,
                   int dst_dtype, int wire_dtype, void *const *d_srcs, void *const *d_dsts,
                   cudaStream_t stream);

/*
 * Layout of an extended reduction (ar_reduce_ex): a 2-D tensor of ne1 rows
 * of ne0 elements with per-buffer row strides, ranks that may be inactive,
 * and an optional residual or bias added after the rank fold.
 *
 * Where this comes from:
 *   - row strides: the 2-D DMA variant DEFINE_ALLREDUCE_THREAD_DMA_2D of
 *     ggml-hexagon htp/allreduce-ops.c walks every source and destination
 *     row by row through its nb[1] byte stride;
 *   - residual and bias: the ALLREDUCE_ADD variants of the same file add one
 *     more tensor after the ranks (add_bcast adds one row to every row);
 *   - inactive ranks: ggml_cuda_ar_allreduce in ggml-cuda allreduce.cu zeroes
 *     the data of shards that did not compute, so they contribute zeros.
 * Readings taken where the pages are silent: the residual is added in float
 * after the rank fold and before the one final cast, and is not rounded
 * through the wire type (it never crosses the wire); an inactive rank
 * contributes +0 to every element, which is not the same as leaving it out
 * (-0 + +0 = +0).
 */
typedef struct {
    size_t ne0;                   /* elements per row */
    size_t ne1;                   /* rows; ne0 * ne1 <= max_elems */
    const int64_t *src_row_bytes; /* R row strides in bytes (>= ne0 * element size, a multiple of
                                     the element size), or NULL: every source's rows are packed */
    const int64_t *dst_row_bytes; /* n_dsts row strides in bytes, or NULL: packed */
    const void *residual;         /* NULL, or a T_dst tensor added after the rank fold */
    int64_t residual_row_bytes;   /* residual row stride in bytes; 0: the residual is one row of
                                     ne0 elements added to every row (a bias) */
    uint32_t inactive_mask;       /* bit r set: rank r contributes +0 everywhere and srcs[r] is not
                                     read (it may be NULL); bits >= R must be clear */
} ar_layout;

/*
 * ar_reduce_ex -- the reduction over an ar_layout, enqueued on `stream`:
 *   dst[d][row][i] = T_dst( fold_r wire(src[r][row][i]) (+ residual[row][i]) )
 * with the fold, casts and rounding of ar_reduce.  srcs has R entries (NULL
 * allowed for inactive ranks), dsts has n_dsts.  A destination may be
 * exactly a source or exactly the residual (same pointer and same row
 * stride: an in-place update such as x = x + allreduce(partials)); any other
 * overlap of the buffers' row spans is AR_ERR_OVERLAP (the check is
 * conservative: interleaved rows that never touch are also refused).
 * When every buffer's start agrees modulo 16 bytes, and (with more than one
 * row) so does every row stride, every row of every buffer starts at one
 * common offset from a 16-byte boundary: the vector path runs, reducing each
 * row's few elements before that boundary one by one.  Any other
 * element-aligned layout works element by element with the same bits.
 * Statuses as for ar_reduce; nothing is enqueued unless AR_OK.
 */
int ar_reduce_ex(const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *layout,
                 int dst_dtype, int wire_dtype, cudaStream_t stream);

/* Host-only validation of an ar_reduce_ex call on explicit R and max_elems
 * (no CUDA call; runs without a GPU). */
int ar_check_layout(int R, const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *layout,
                    size_t max_elems, int dst_dtype, int wire_dtype);

/*
 * ar_wire_pack -- materialise the wire copy of one partial:
 *   wire[i] = T_wire(src[i]) for i < nelem,
 * the buffer a transport sends to the other ranks (phase 1 of
 * ggml_cuda_ar_kernel in ggml-cuda allreduce.cu writes exactly this; its
 * copy-engine path converts to bf16 into a temporary before copying).
 *   src   nelem elements of dst_dtype (device-accessible).
 *   wire  nelem elements of wire_dtype; may be src itself when both types
 *         have the same size, otherwise must not overlap it.
 * Vector kernel when skipping the same first few elements aligns both
 * buffers (they are then converted one by one), element-wise otherwise; the
 * bits are the same.  Needs ar_init (nelem <= max_elems).  Statuses as for
 * ar_reduce.
 */
int ar_wire_pack(const void *src, void *wire, size_t nelem, int dst_dtype, int wire_dtype,
                 cudaStream_t stream);

/*
 * ar_reduce_host_noalloc -- ar_reduce_host for callers that cannot allocate
 * device memory.  (The pages have no counterpart: this entry point exists
 * for callers of this library, not because of the method.)
 *
 * Who needs it: code that may not call cudaMalloc -- for example a plug-in
 * running inside a framework whose caching allocator owns the whole device
 * memory budget, or a latency-critical path that cannot afford cudaMalloc /
 * cudaFree and the device-wide synchronisation they can cause.  Such
 * callers cannot provide the device staging buffers ar_reduce_host wants.
 *
 * What it does: copies each host source into a fixed staging area built into
 * the library, reduces there, and copies every destination back to its host
 * buffer, all enqueued on `stream` (results are valid once `stream` reaches
 * the end of this call).  It allocates nothing: no cudaMalloc, no cudaFree,
 * no allocating library routine.  Same arguments, buffer rules (partial
 * overlap of host buffers is AR_ERR_OVERLAP) and results as ar_reduce_host
 * with NULL staging arrays, except that the host buffers may be ordinary
 * pageable memory.  CUDA copies pageable memory synchronously, so with
 * pageable buffers the call itself waits until `stream` has reached its
 * copies; it holds no library lock while it waits, so other threads' calls
 * go on.
 *
 * Limits and rules:
 *   - The staging area is AR_NOALLOC_SCRATCH_BYTES (64 MiB) of device
 *     memory that every GPU which loads the library holds until the process
 *     exits.  A call needs R + n_dsts buffers of nelem elements, each rounded
 *     up to 256 bytes; a call that needs more returns AR_ERR_TOO_LARGE and
 *     does nothing.
 *   - The first call on a device after each ar_init looks up the staging
 *     area's device address (once, with that device current); make that
 *     first call before any stream capture.  ar_init and ar_free forget the
 *     address, so a context created after cudaDeviceReset finds the area
 *     where the new device context holds it.  If another thread runs
 *     ar_init or ar_free while a call is under way, the call may return
 *     AR_ERR_NOT_INITIALIZED after its copies into the staging area were
 *     enqueued (the caller's buffers are then not written).
 *   - Every call on a GPU uses the same staging area, and each call leaves
 *     its data there: nothing in it has to start at zero, because every call
 *     writes its inputs before reading them.  Calls whose work overlaps on
 *     the GPU (two streams, or two threads) race on the staging area and may
 *     produce wrong results: serialise them, e.g. on one stream.
 */
#define AR_NOALLOC_SCRATCH_BYTES (64u << 20)
int ar_reduce_host_noalloc(const void *const *h_srcs, void *const *h_dsts, int n_dsts, size_t nelem,
                           int dst_dtype, int wire_dtype, cudaStream_t stream);

/* ---- training operators ---------------------------------------------------
 * What a tensor-parallel training step does directly behind and before the
 * reduction: dropout on the reduced sum, and the loss over a vocabulary that
 * is split into pieces, whose gradient is again a set of partials.  They
 * have no counterpart in the pages.  The conventions above hold for them too:
 * ar_init first, work is only enqueued, nothing is allocated (calls that need
 * scratch memory take a workspace from the caller and say how large it has to
 * be), AR_Q_LAST_VARIANT is left alone, and calls can be captured in a graph.
 */

/*
 * Dropout whose mask is a function of its arguments and is never stored.
 * Element (row, col) owns word col % 4 of Philox4x32-10 (Salmon, Moraes, Dror
 * and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) under the key
 * (seed low, seed high) and the counter (col / 4, row, offset low, offset
 * high).  It is kept when that word is at least floor(p * 2^32), and a kept
 * element is multiplied by 1 / (1 - p) in float; p = 1 keeps nothing.  Strides, variants and
 * grids do not enter, so the backward pass sees the forward pass's mask.  Two
 * calls have independent masks when their offsets (or seeds) differ.
 */
typedef struct {
    uint64_t seed;
    uint64_t offset;  /* which call of the step and which step: the counter's upper half */
    float p;          /* probability that an element is dropped, 0 <= p <= 1 */
    const void *bias; /* NULL, or one row of ne0 T_dst elements added to the sum before dropout */
} ar_dropout;

/*
 * ar_reduce_dropout -- ar_reduce_ex with bias and dropout between the rank
 * fold and the residual:
 *   a = fold_r wire(src[r][row][i]);  a = a + bias[i];
 *   a = keep(row, i) ? a * scale : 0;  a = a + residual[row][i];
 *   dst[d][row][i] = T_dst(a)
 * each step rounded to float.  A dropped element is 0 whatever the sum holds
 * (infinities and NaN included).  Layout, in-place and overlap rules as for
 * ar_reduce_ex (a residual row broadcast with stride 0 is allowed); bias may
 * not overlap a destination.  ne1 must fit 32 bits and ne0 34 bits
 * (AR_ERR_TOO_LARGE).  Every layout and alignment gives the same bits.
 */
int ar_reduce_dropout(const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *layout,
                      const ar_dropout *dropout, int dst_dtype, int wire_dtype, cudaStream_t stream);

/* Host-only validation of an ar_reduce_dropout call (no CUDA call). */
int ar_check_dropout(int R, const void *const *srcs, void *const *dsts, int n_dsts, const ar_layout *layout,
                     const ar_dropout *dropout, size_t max_elems, int dst_dtype, int wire_dtype);

/*
 * ar_reduce_dropout_grad -- the backward pass of ar_reduce_dropout:
 *   dx[d][row][i]  = T_dst(keep(row, i) ? dy[row][i] * scale : 0)   d = 0 .. n_dxs-1
 *   dbias[i]       = sum over rows of the same, in float, unrounded
 *   dresidual[i]   = sum over rows of dy[row][i], in float
 * Rounding through the wire type is differentiated as the identity, so every
 * active rank's partial has the same gradient; the gradient of a full
 * residual is dy itself.
 *   dy         T_dst, ne1 rows at layout->src_row_bytes[0] (NULL: packed).
 *   dxs        n_dxs destinations, 1..16, at layout->dst_row_bytes; one may be
 *              exactly dy (same stride).
 *   layout     ne0, ne1 and the strides; residual must be NULL and
 *              inactive_mask 0.
 *   dropout    as in the forward call; its bias is not read and may be NULL.
 *   dbias, dresidual  NULL, or ne0 floats.  dresidual is the gradient of a
 *              residual row broadcast with stride 0.
 *   workspace  16-byte aligned device memory of ar_reduce_dropout_grad_workspace
 *              bytes (NULL where that is 0); its contents do not matter.
 * Sums are taken in a fixed order: the same call gives the same bits.
 */
int ar_reduce_dropout_grad(const void *dy, void *const *dxs, int n_dxs, const ar_layout *layout,
                           const ar_dropout *dropout, float *dbias, float *dresidual, void *workspace,
                           size_t workspace_bytes, int dst_dtype, cudaStream_t stream);

/* Workspace of an ar_reduce_dropout_grad call with n_sums (0..2) of dbias and
 * dresidual given (host only, needs no context). */
int ar_reduce_dropout_grad_workspace(const ar_layout *layout, int n_sums, size_t *bytes);

/*
 * Softmax cross entropy against an output matrix whose vocabulary rows are
 * split into pieces (one per rank), without keeping the logits:
 *   z[t][v] = sum_i hidden[t][i] * W[v][i]        (W: the pieces one after another)
 *   lse[t]  = log sum_v exp(z[t][v])
 *   loss[t] = lse[t] - z[t][targets[t]]
 * A token whose target is ignore_index has loss 0 and adds nothing to any
 * gradient, whatever its hidden state holds (infinities and NaN included); a
 * target that is neither ignore_index nor a row of the vocabulary gives the
 * loss NaN and no gradient.
 * Products of 16-bit types are exact and summed in float: the logits in
 * runs of at most 512 terms, which are added rounded to nearest (the tensor cores'
 * own sums are not rounded but cut off, and drift over long reductions), and alike
 * in both calls; the gradients in one run, below their own rounding.
 * Float inputs are split into three bf16 parts each; six products of parts
 * give a float product to 2^-25.  The gradient of the logits is held in the
 * 16-bit type for one chunk of the vocabulary at a time, relative to the
 * largest finite |dloss|: one rounding more than the outputs' own (with 64 tokens or
 * fewer in two parts, float inputs in three: none).  Infinite float inputs
 * give NaN where the formula has an infinity.
 */
typedef struct {
    size_t rows;                      /* tokens; rows * dim <= max_elems */
    size_t dim;                       /* elements of a hidden state, >= 1 */
    const void *hidden;               /* rows x dim of dtype */
    int64_t hidden_row_bytes;         /* row stride (>= dim elements, whole elements); 0: packed */
    int n_pieces;                     /* 1..16 */
    const size_t *piece_rows;         /* n_pieces vocabulary row counts; some may be 0, their sum not */
    const void *const *weights;       /* n_pieces matrices, piece_rows[r] x dim of dtype */
    const int64_t *weight_row_bytes;  /* n_pieces row strides, or NULL: packed */
    const int64_t *targets;           /* device, rows global vocabulary rows (of the pieces in order) */
    int64_t ignore_index;
    int dtype;                        /* ar_dtype of hidden, weights and their gradients */
} ar_vocab;

/*
 * ar_vocab_loss -- enqueue the loss of every token.
 *   loss, lse   rows floats each (device); lse is what the gradient call needs.
 *   workspace   256-byte aligned device memory of at least ar_vocab_workspace
 *               bytes; its contents do not matter.
 * Outputs and workspace may overlap neither each other nor an input.
 */
int ar_vocab_loss(const ar_vocab *v, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream);

/*
 * ar_vocab_loss_grad -- the gradients, the logits computed anew:
 *   d[t][v]         = dloss[t] * (exp(z[t][v] - lse[t]) - [v == targets[t]])
 *   dhidden[r]      = d over piece r's columns times weights[r]     rows x dim
 *   dweights[r]     = (d over piece r's columns)^T times hidden     piece_rows[r] x dim
 * The dhidden[r] are partials: their sum over r, which ar_reduce takes, is the
 * gradient of the hidden states.
 *   lse       as ar_vocab_loss wrote it for the same hidden states and weights.
 *   dloss     rows floats (device), the gradient of each token's loss.
 *   dhidden   n_pieces matrices of dtype at dhidden_row_bytes (NULL: packed),
 *             or NULL: not wanted.
 *   dweights  n_pieces matrices of dtype at dweight_row_bytes (NULL: packed),
 *             or NULL: not wanted.
 * Every output is written whole.  The same call gives the same bits.
 */
int ar_vocab_loss_grad(const ar_vocab *v, const float *lse, const float *dloss, void *const *dhidden,
                       const int64_t *dhidden_row_bytes, void *const *dweights, const int64_t *dweight_row_bytes,
                       void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Host-only checks of an ar_vocab (no CUDA call). */
int ar_check_vocab(const ar_vocab *v, size_t max_elems);

/* Workspace of ar_vocab_loss (grad = 0) or ar_vocab_loss_grad (grad = 1) for
 * these arguments (host only; pointers are not read, their alignment and the
 * strides count).  What can be large in it: copies of the weights in rows that
 * the tiled copies can read (6 bytes an element of float weights, 2 of 16-bit
 * ones off 16-byte boundaries, none otherwise), at most 2 GiB at a time; for
 * the gradients a copy of the hidden states, the logits' gradient of one chunk
 * of the vocabulary (256 MiB at most, or 256 vocabulary rows where that is
 * more) and up to 64 MiB of partial sums (or one float copy of the hidden
 * states' gradient for each piece where that is more). */
int ar_vocab_workspace(const ar_vocab *v, int grad, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* TPS_AR_H */
