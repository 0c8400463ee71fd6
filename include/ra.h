/*
 * ra.h — C ABI of the GB300 ring all-reduce library (libra.so).
 *
 * N "virtual ranks" live in one GPU's memory; each rank r owns a send buffer
 * and a receive buffer (device pointers). The calls follow the shape of
 * ncclAllReduce(sendbuff, recvbuff, count, datatype, op, comm, stream) as the
 * arjunsriva.com page "AllReduce, All the Way Down" (section "The Contract:
 * What AllReduce Means") states it, with the communicator replaced by
 * `nranks` and one host array of N device pointers per side.
 *
 * What is computed (tirogla.com "Ring all-reduce", section "How it works"):
 * the buffer of `count` elements is cut into N chunks, chunk c covering
 * elements [c*count/N, (c+1)*count/N) with floor division (section "Code"), so
 * chunks may differ by one element and may be empty. Element i of chunk c is
 * reduced in ring order, left to right,
 *
 *     x_c (+) x_{c+1} (+) ... (+) x_{c+N-1}      (rank indices mod N)
 *
 * which is the order in which the reduce-scatter phase of the ring visits
 * chunk c (it starts at rank c and ends at rank c-1, which then owns it).
 * Every hop is rounded to the buffer dtype: fp32 hops are fp32 operations;
 * fp16/bf16 hops compute in fp32 and round to nearest even once; int32 sum and
 * prod wrap modulo 2^32. RA_AVG is the ring sum followed by one multiply by
 * 1.0f/N (fp32) rounded to the dtype (int32: wrapped sum / N, truncated).
 * RA_MIN / RA_MAX follow IEEE 754-2019 minimum / maximum (NaN propagates,
 * -0 < +0). Results are bit-identical on every rank (same page,
 * "Implementation notes").
 *
 * Common rules for the three collectives:
 *  - count is the FULL per-rank vector length L in every call (also for
 *    reduce-scatter and all-gather, whose compact side holds one chunk).
 *  - sendbufs / recvbufs are host arrays of `nranks` device pointers. The
 *    arrays are read during the call only; the device buffers belong to the
 *    caller and must stay alive until the work on `stream` has completed.
 *  - The library allocates no device memory and keeps no state between
 *    calls; calls are reentrant. Work is enqueued on `stream` (a
 *    cudaStream_t; NULL = the legacy default stream) and the call returns
 *    without waiting. The collective kernels are programmatic dependent
 *    launches: their CTAs may be placed on the GPU while the previous kernel
 *    on `stream` is finishing, but no thread reads or writes memory before
 *    that kernel has completed, so the stream's order holds as for any
 *    launch (a graph captured from the stream records programmatic edges).
 *  - Arguments are checked on the host before any launch; on any error
 *    nothing is enqueued. Every pointer must be aligned to the element size;
 *    a pointer to a zero-length buffer may be NULL. Any other alignment is
 *    accepted: the vector path is used when the buffers share their address
 *    modulo ra_vector_bytes(), a per-element path otherwise.
 *  - Buffers may be device memory or host memory the device can address
 *    (pinned host memory under unified addressing, or any host memory on
 *    systems whose GPU accesses system memory coherently): the kernels then
 *    read and write host memory directly over the host link, which replaces
 *    explicit copies for callers whose data lives on the host. Such calls
 *    launch one resident wave (it streams the host link faster than a CTA per
 *    trip) and the all-gather takes plain stores; the TMA-staged bulk engine
 *    and the tree / Rabenseifner orders take device memory only and return
 *    RA_ERR_UNSUPPORTED for a host buffer, before enqueuing anything.
 *  - Buffers must not overlap, except in the exact in-place layout named for
 *    each call (each element is then read and written by the same thread).
 *    Send buffers may overlap each other (they are only read).
 *  - count == 0 returns RA_SUCCESS and launches nothing. nranks == 1 copies.
 */
#ifndef RA_H_
#define RA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RA_MAX_RANKS 64
/* largest accepted count: keeps c*count (c <= 64) inside 63 bits */
#define RA_MAX_COUNT ((((uint64_t)1) << 57) - 1)

typedef enum {
  RA_SUCCESS = 0,
  RA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, nranks outside [1, 64], bad enum, count too big */
  RA_ERR_UNSUPPORTED = 2, /* a dtype/op/option combination the library does not provide */
  RA_ERR_ALIAS = 3,       /* buffers overlap other than in the allowed in-place layout */
  RA_ERR_CUDA = 4,        /* the CUDA launch failed; see ra_last_cuda_error() */
  RA_ERR_SCRATCH_LIMIT = 5 /* ra_allreduce_bulk_noalloc: nranks above RA_NOALLOC_STATUS_WORDS */
} ra_status_t;

typedef enum { RA_FLOAT32 = 0, RA_FLOAT16 = 1, RA_BFLOAT16 = 2, RA_INT32 = 3 } ra_dtype_t;

/* bitfern.com "AllReduce Explained", section "What Is AllReduce?": sum,
 * average, minimum, maximum and product reductions. */
typedef enum { RA_SUM = 0, RA_AVG = 1, RA_MIN = 2, RA_MAX = 3, RA_PROD = 4 } ra_op_t;

/*
 * All-reduce (tirogla.com "Ring all-reduce", "How it works": reduce-scatter
 * then all-gather). sendbufs[r]: count elements of rank r. recvbufs[r]: count
 * elements; on completion every recvbufs[r] holds the reduction of all ranks.
 * In place: recvbufs[r] == sendbufs[r].
 * HBM traffic: reads N*count*e bytes, writes N*count*e bytes, in one launch.
 */
ra_status_t ra_allreduce(const void* const* sendbufs, void* const* recvbufs, size_t count,
                         ra_dtype_t dtype, ra_op_t op, int nranks, void* stream);

/*
 * Reduce-scatter (infra-guide "Collective communication primitives", section
 * 3.5: rank i keeps reduced shard i). sendbufs[r]: count elements.
 * recvbufs[r]: chunk r only, (end_r - begin_r) elements, compact. The shard
 * is reduced in the same ring order as ra_allreduce, so the all-gather of
 * these shards equals ra_allreduce bit for bit (same page, section 3.8).
 * In place: recvbufs[r] == sendbufs[r] + begin_r elements.
 * HBM traffic: reads N*count*e, writes count*e.
 */
ra_status_t ra_reduce_scatter(const void* const* sendbufs, void* const* recvbufs, size_t count,
                              ra_dtype_t dtype, ra_op_t op, int nranks, void* stream);

/*
 * All-gather (ramchalamkr.github.io "NCCL Primitives Deep Dive", section 1;
 * infra-guide section 3.6). sendbufs[r]: chunk r, (end_r - begin_r) elements,
 * compact. recvbufs[r]: count elements; on completion each holds every chunk
 * at its place. `op` is ignored (no reduction happens).
 * In place: sendbufs[r] == recvbufs[r] + begin_r elements.
 * HBM traffic: reads count*e, writes N*count*e.
 */
ra_status_t ra_allgather(const void* const* sendbufs, void* const* recvbufs, size_t count,
                         ra_dtype_t dtype, ra_op_t op, int nranks, void* stream);

/* Reduction order (the algorithm whose association the result reproduces). */
typedef enum {
  RA_ORDER_RING = 0,         /* tirogla.com "Ring all-reduce", "How it works" (the default) */
  RA_ORDER_TREE = 1,         /* double binary tree (same page, cost model): in-order trees over ranks
                                0..N-1 (first N/2 chunks) and N-1..0 (the rest) */
  RA_ORDER_RABENSEIFNER = 2  /* recursive halving / doubling, power-of-two nranks (same page) */
} ra_order_t;

/* Precision of the partials travelling between ranks. */
typedef enum {
  RA_ACCUM_DTYPE = 0, /* every hop rounded to the buffer dtype (the default) */
  RA_ACCUM_FP32 = 1   /* fp16/bf16: partials kept in fp32, rounded once at the end (after the
                         avg multiply); tirogla.com "Ring all-reduce", "Implementation notes".
                         No effect on fp32 and int32 buffers. */
} ra_accum_t;

/* How the fused all-reduce moves its loads. */
typedef enum {
  RA_ENGINE_REGISTERS = 0, /* every thread keeps its loads in flight in registers (the default) */
  RA_ENGINE_BULK = 1       /* a producer thread per CTA streams tiles of all ranks into shared memory
                              with bulk copies (the Tensor Memory Accelerator) and the other warps fold
                              from there: several times the bytes in flight per SM, for runs confined
                              to a few SMs by max_sms. All-reduce with the ring order and dtype
                              accumulation, nranks <= 16; needs `status` */
} ra_engine_t;

/* Options of the extended calls; NULL means all defaults. */
typedef struct {
  ra_order_t order;   /* RA_ORDER_RING by default */
  ra_accum_t accum;   /* RA_ACCUM_DTYPE by default */
  int max_sms;        /* 0: the launch may fill every SM; k > 0: at most k SMs' worth of CTAs, leaving the
                         rest to work running beside the collective (arjunsriva.com "AllReduce, All the
                         Way Down": communication kernels compete with compute for SMs). The hardware
                         places the CTAs: the budget bounds the collective's share of CTA slots, not
                         which SMs it runs on, and a launch shape with several CTAs per SM may spread
                         over more than k SMs (the bulk engine runs one CTA per SM); a hard partition
                         of the SMs needs green contexts */
  ra_engine_t engine; /* RA_ENGINE_REGISTERS by default */
  int* status;        /* RA_ENGINE_BULK only: one int of device memory, owned by the caller, that the
                         kernel sets to a nonzero code if one of its bounded waits gives up (1: a
                         bulk copy did not land within 1 s; 2: a stage was not released within 1 s)
                         instead of hanging; it is never cleared by the library */
} ra_options_t;

/*
 * All-reduce / reduce-scatter with options: ra_allreduce(...) is
 * ra_allreduce_ex(..., NULL, stream). Same buffers, in-place rules and errors
 * as the plain calls, plus RA_ERR_UNSUPPORTED for RA_ORDER_RABENSEIFNER with a
 * nranks that is not a power of two, for RA_ACCUM_FP32 with an order other
 * than the ring, and for RA_ENGINE_BULK outside its range (reduce-scatter,
 * another order or accumulation, nranks > 16, buffers without a common
 * address phase), and RA_ERR_INVALID_ARG for an unknown order/accum/engine,
 * a negative max_sms or RA_ENGINE_BULK without a status word.
 */
ra_status_t ra_allreduce_ex(const void* const* sendbufs, void* const* recvbufs, size_t count, ra_dtype_t dtype,
                            ra_op_t op, int nranks, const ra_options_t* options, void* stream);
ra_status_t ra_reduce_scatter_ex(const void* const* sendbufs, void* const* recvbufs, size_t count,
                                 ra_dtype_t dtype, ra_op_t op, int nranks, const ra_options_t* options,
                                 void* stream);

/*
 * Gradient buckets (bitfern.com "AllReduce Explained", "PyTorch DDP and
 * Gradient Synchronization"; tirogla.com "Ring all-reduce", "Implementation
 * notes": DDP's default bucket is 25 MB). Host only, touches no GPU.
 * param_counts[nparams]: element counts of the parameters, laid out
 * contiguously in this order in the flat gradient buffer. Parameters are
 * visited in reverse (the order backward produces their gradients) and packed
 * into buckets of at most bucket_bytes (a parameter larger than that gets its
 * own bucket). Writes up to max_buckets contiguous element ranges
 * [bucket_begin[b], bucket_begin[b] + bucket_count[b]) in the order they
 * become ready, and the number of buckets to *nbuckets (also when max_buckets
 * is too small, which returns RA_ERR_INVALID_ARG; NULL arrays with
 * max_buckets 0 query the count).
 */
ra_status_t ra_bucket_plan(const size_t* param_counts, int nparams, size_t bucket_bytes, int elem_size,
                           size_t* bucket_begin, size_t* bucket_count, int max_buckets, int* nbuckets);

/*
 * Bucketed all-reduce: bucket b (an element range of every rank's buffer,
 * listed in ascending or descending order, disjoint) is all-reduced as an
 * all-reduce of its own (its own chunk bounds), after `stream` waits for
 * ready_events[b] (a cudaEvent_t the producer recorded when the bucket's
 * gradients were complete; NULL entries or a NULL array wait for nothing).
 * The waits and launches are enqueued on `stream` in bucket order, so buckets
 * overlap with work on other streams as soon as they are ready. A run of
 * buckets with no ready event of their own (NULL entries, or a NULL array)
 * goes out as one grouped launch of up to 64 buckets when the options are the
 * default engine and ring order; each bucket's result bits are still those of
 * an all-reduce of its own. Buffers, in-place rule and options as
 * ra_allreduce_ex.
 */
ra_status_t ra_allreduce_buckets(const void* const* sendbufs, void* const* recvbufs, size_t count,
                                 ra_dtype_t dtype, ra_op_t op, int nranks, int nbuckets, const size_t* bucket_begin,
                                 const size_t* bucket_count, void* const* ready_events,
                                 const ra_options_t* options, void* stream);

/*
 * The literal ring schedule, one kernel launch per ring step (tirogla.com
 * "Ring all-reduce", "How it works"): reduce-scatter step s = 0..N-2 has rank
 * r combine chunk (r-s-1) mod N arriving from rank r-1 with its own copy;
 * all-gather step s has rank r copy chunk (r-s) mod N from rank r-1. Every
 * message is a read of rank r-1's buffer in HBM. Same arguments, rounding,
 * in-place rule and final result (bit for bit) as ra_allreduce; it moves
 * about 5(N-1)*S bytes instead of 2N*S, which is what the fused kernel saves.
 * nsteps: run only the first nsteps of the 2(N-1) steps (negative = all);
 * after a partial run each rank's buffer holds the schedule's state for the
 * chunks the steps have touched and is undefined elsewhere.
 */
ra_status_t ra_allreduce_ringsteps(const void* const* sendbufs, void* const* recvbufs, size_t count,
                                   ra_dtype_t dtype, ra_op_t op, int nranks, int nsteps, void* stream);

/*
 * Chunk bounds (tirogla.com "Ring all-reduce", section "Code"):
 * *begin = c*count/nranks, *end = (c+1)*count/nranks, floor division, exact
 * for every count <= RA_MAX_COUNT. Host only; touches no GPU.
 */
ra_status_t ra_chunk_range(size_t count, int nranks, int c, size_t* begin, size_t* end);

/*
 * Planner introspection (host only, no GPU): how chunk c is split between the
 * vector path and the per-element path for buffers of `elem_size`-byte
 * elements that share their address phase `phase_bytes` modulo `align_bytes`
 * (a power of two from ra_vector_bytes() to 512; the library uses the largest
 * such alignment the buffers share). Writes [vec_begin, vec_end) (elements
 * moved as whole vectors, starting on the alignment grid; empty if vec_begin
 * == vec_end) inside [begin, end); the rest of the chunk takes the
 * per-element path.
 */
ra_status_t ra_plan_chunk(size_t count, int nranks, int c, int elem_size, int align_bytes, int phase_bytes,
                          size_t* begin, size_t* end, size_t* vec_begin, size_t* vec_end);

/* A static, human-readable name for a status code. */
const char* ra_status_string(ra_status_t status);

/* The cudaError_t of the last RA_ERR_CUDA returned on the calling thread (0 if none). */
int ra_last_cuda_error(void);

/*
 * Self-test of the bulk engine's bounded waits (host-visible failure
 * reporting without a GPU fault): runs the RA_ENGINE_BULK all-reduce with the
 * first tile of CTA (0, withhold_chunk) never copied in, so that CTA's
 * consumers wait for it in vain and give up after 1 s; the CTA records a
 * nonzero code (1 or 2, as for ra_options_t.status), waits (bounded) for its
 * other copies in flight and winds down. The launch completes and the context
 * stays usable. The receive buffers' contents are unspecified afterwards.
 * status: caller-owned device ints, 0 before the call. status_per_chunk 0:
 * every chunk reports into status[0] (one int); 1: chunk c reports into
 * status[c] (nranks ints), as ra_allreduce_bulk_noalloc's words do.
 * withhold_chunk in [0, nranks); count must give that chunk at least one
 * whole tile for the self-test to fire. Same other arguments as ra_allreduce.
 */
ra_status_t ra_selftest_bulk_timeout(const void* const* sendbufs, void* const* recvbufs, size_t count,
                                     ra_dtype_t dtype, ra_op_t op, int nranks, int withhold_chunk, int* status,
                                     int status_per_chunk, void* stream);

/* Bytes per vector access of the library's compiled kernels (16 or 32): the address
 * phase (address mod this) the buffers must share for the vector path. */
int ra_vector_bytes(void);

/* Status words held by the library for ra_allreduce_bulk_noalloc: one per chunk. */
#define RA_NOALLOC_STATUS_WORDS 16

/*
 * The RA_ENGINE_BULK all-reduce for a caller that cannot allocate device
 * memory. The web pages have no counterpart: this is an interface of this
 * library only. Result bits, buffers, in-place rules and other errors are
 * those of ra_allreduce_ex with RA_ENGINE_BULK; the difference is where the
 * status words live. ra_allreduce_ex wants a device int from the caller;
 * here the library keeps RA_NOALLOC_STATUS_WORDS ints of its own, a fixed
 * array inside libra.so's device image, and the call allocates nothing.
 *
 * Who needs this: a caller whose device memory is all held by another
 * allocator (a framework's caching pool), which has no device allocation
 * call of its own to use and would only fragment that pool with a stray
 * cudaMalloc; a caller between the kernels of a training step, where
 * cudaFree would make the host wait for the whole device, including the
 * compute that the bulk engine is meant to run beside; and a caller that
 * wants the per-chunk codes in pinned host memory (chunk_status may be host
 * memory). The buffers themselves must be device memory (RA_ERR_UNSUPPORTED
 * otherwise): a program whose buffers are pinned host memory calls
 * ra_allreduce, which reads and writes them over the host link.
 *
 * Set-up: every call looks up the array's device address in the current
 * context (cudaGetSymbolAddress) and keeps nothing between calls, so a call
 * after a context switch or a device reset uses that context's copy. A failed
 * lookup returns RA_ERR_CUDA. The first lookup in a context can load the
 * library's kernels into it, so make the first call there before any stream
 * capture begins.
 *
 * Each call enqueues on `stream`: a clear of words [0, nranks) of the array;
 * the kernel, whose CTAs for chunk c record in word c the code of a bounded
 * wait that gave up (1: a bulk copy did not land within 1 s; 2: a stage was
 * not released within 1 s); and, if chunk_status is not NULL, a copy of
 * those nranks words to chunk_status (device memory or host memory, nranks
 * ints, caller-owned; pageable host memory makes the call wait until the
 * kernel has finished). Read chunk_status once the stream has passed the
 * call: 0 everywhere means every chunk finished. max_sms as in ra_options_t.
 * count == 0 enqueues nothing and leaves chunk_status untouched.
 *
 * Limit: nranks must be at most RA_NOALLOC_STATUS_WORDS (16, the bulk
 * engine's own limit); a larger nranks (up to RA_MAX_RANKS) returns
 * RA_ERR_SCRATCH_LIMIT before anything is enqueued.
 *
 * Errors: every check, the plan and the kernel's shared-memory set-up come
 * before the first enqueue, so an error returned from them enqueues nothing.
 * Only a failure of one of the three enqueues itself (RA_ERR_CUDA) can leave
 * the earlier ones queued; they touch nothing but the library's words and,
 * for the copy, chunk_status.
 *
 * Concurrency: each context has one copy of the array (on the usual primary
 * context: one per device), shared by all calls there. Two calls in flight at
 * once in one context (on different streams, or from different threads) race
 * on it: one call's clear can erase the other's codes, and a copy can return
 * the other's codes. The reduced buffers are not affected. Calls on one
 * stream run one after the other and do not race.
 */
ra_status_t ra_allreduce_bulk_noalloc(const void* const* sendbufs, void* const* recvbufs, size_t count,
                                      ra_dtype_t dtype, ra_op_t op, int nranks, int max_sms, int* chunk_status,
                                      void* stream);

/* ==== operators on either side of the gradient all-reduce ====================
 *
 * A data-parallel step fills the gradient buffer (backward), reduces it (the
 * calls above), measures and clips it, and steps the optimiser. The calls
 * below are the parts of that step that stream memory: layer norm with the
 * reduction of its weight gradient, the global gradient norm, and AdamW.
 *
 * Common rules: as for the collectives. Arguments are checked on the host
 * before any launch and nothing is enqueued on an error; the library allocates
 * nothing and keeps no state; work is enqueued on `stream` (NULL = the legacy
 * default stream) as programmatic dependent launches and can be captured in a
 * graph. Buffers are device memory; scratch comes from the caller. dtypes: RA_FLOAT32, RA_FLOAT16,
 * RA_BFLOAT16 (RA_INT32: RA_ERR_UNSUPPORTED). All arithmetic is fp32, rounded
 * to nearest even once where a result is stored; quotients and square roots
 * inside a formula may be off by a few ulp of fp32. Results do not depend on
 * timing: no sum is taken in an order that varies from run to run on a device.
 * Pointers must be aligned to their element size; wider alignment is faster.
 */

/*
 * Layer norm of `rows` rows of `cols` elements:
 *   mean = sum x / cols, rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
 *   y = (x - mean) * rstd * weight + bias.
 * x, y: dtype, row r at x + r * x_stride elements (strides >= cols).
 * weight, bias: `cols` elements of weight_dtype (dtype itself or RA_FLOAT32);
 * NULL weight = ones, NULL bias = zeros. mean, rstd: `rows` floats, kept for
 * the backward pass; either may be NULL. y may be x (same stride); any other
 * overlap of an output with another buffer is RA_ERR_ALIAS. Column slices of
 * one matrix (one stride, rows side by side) do not overlap.
 * rows == 0 or cols == 0 enqueues nothing.
 * HBM traffic: reads and writes rows*cols*e.
 */
ra_status_t ra_layernorm_forward(const void* x, size_t x_stride, const void* weight, const void* bias, void* y,
                                 size_t y_stride, float* mean, float* rstd, size_t rows, size_t cols, double eps,
                                 ra_dtype_t dtype, ra_dtype_t weight_dtype, void* stream);

/*
 * Its backward pass. With xhat = (x - mean) * rstd and a = dy * weight,
 *   dx      = rstd * (a - avg_row(a) - xhat * avg_row(a * xhat)),
 *   dweight = sum over rows of dy * xhat,   dbias = sum over rows of dy.
 * mean, rstd: as ra_layernorm_forward stored them. dx: dtype; it may be dy or
 * x (same stride), and overlap is as there. dweight, dbias: `cols` elements of weight_dtype, anywhere
 * (slices of a flat gradient buffer); either may be NULL. accumulate != 0 adds
 * to what they hold (in fp32, rounded once), 0 overwrites. rows == 0 gives
 * zero sums. workspace: at least ra_layernorm_workspace(rows, cols) bytes of
 * device memory, 16-byte aligned, contents irrelevant before and after; only
 * read or written when dweight or dbias is given, and may be NULL otherwise.
 * HBM traffic: reads 2*rows*cols*e, writes rows*cols*e.
 */
ra_status_t ra_layernorm_backward(const void* dy, size_t dy_stride, const void* x, size_t x_stride,
                                  const void* weight, const float* mean, const float* rstd, void* dx,
                                  size_t dx_stride, void* dweight, void* dbias, int accumulate, size_t rows,
                                  size_t cols, ra_dtype_t dtype, ra_dtype_t weight_dtype, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Bytes of workspace ra_layernorm_backward needs for this shape. Host only. */
size_t ra_layernorm_workspace(size_t rows, size_t cols);

/*
 * Global norm of `ntensors` gradient tensors and the factor that clips it:
 *   out[0] = norm  = sqrt(sum over all elements of (prescale * g)^2),
 *   out[1] = scale = prescale * min(1, max_norm / (norm + 1e-6)),
 * or NaN in out[1] if the norm is not finite, which makes ra_adamw leave
 * everything as it is. prescale undoes a loss scale (1 otherwise); max_norm
 * may be infinity (no clipping). Squares and sums are fp32: a norm above
 * 1.8e19 may come out infinite, and a |prescale * g| below 1e-19 loses digits
 * or counts as 0. out: 2 device floats.
 * workspace: ra_grad_norm_workspace() bytes of device memory, 16-byte aligned,
 * set to zero before its first use; every call leaves it ready for the next.
 * Two calls that may run at once need one each. Tensors of count 0 may be
 * NULL; no elements at all give norm 0. HBM traffic: reads count*e.
 */
ra_status_t ra_grad_norm(const void* const* grads, const size_t* counts, int ntensors, ra_dtype_t dtype,
                         double prescale, double max_norm, float* out, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Bytes of workspace ra_grad_norm needs. Host only. */
size_t ra_grad_norm_workspace(void);

/* How the two moments of AdamW are held. */
typedef enum {
  RA_STATE_F32 = 0, /* exp_avg = m and exp_avg_sq = v, fp32 */
  RA_STATE_E4M3 = 1 /* 8 bits: exp_avg = m and exp_avg_sq = sqrt(v) as e4m3 values, one byte each, times one
                       fp32 scale per RA_ADAMW_BLOCK elements (counted from the tensor's start). The
                       square root halves the dynamic range v would need */
} ra_state_t;
#define RA_ADAMW_BLOCK 256

/* One tensor of an AdamW step. */
typedef struct {
  void* param;             /* count elements of param_dtype, updated in place */
  const void* grad;        /* count elements of grad_dtype */
  void* exp_avg;           /* count floats, or count e4m3 bytes; updated */
  void* exp_avg_sq;        /* the same */
  float* exp_avg_scale;    /* RA_STATE_E4M3: ceil(count / RA_ADAMW_BLOCK) floats; ignored otherwise */
  float* exp_avg_sq_scale; /* the same */
  void* copy;              /* the updated parameter once more in copy_dtype (NULL: none) */
  size_t count;            /* 0: the tensor is skipped and its pointers may be NULL */
  double weight_decay;     /* decoupled, per tensor */
} ra_adamw_tensor_t;

typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;            /* 1 for the first step: the bias corrections are 1 - beta^step */
  const float* grad_scale; /* device float the gradients are multiplied by (ra_grad_norm's out + 1); NULL = 1.
                              If it is not finite the step is skipped: nothing is written */
  ra_state_t state;
  ra_dtype_t copy_dtype;   /* type of the copies; ignored where there are none */
  uint64_t seed;           /* RA_STATE_E4M3: seeds the stochastic rounding of the moments */
} ra_adamw_options_t;

/*
 * One AdamW step over `ntensors` tensors. Per element, every operation fp32
 * (the moments' products and sums rounded one by one):
 *   g = grad * grad_scale
 *   m = beta1 * m + (1 - beta1) * g,   v = beta2 * v + (1 - beta2) * g * g
 *   param = param * (1 - lr * weight_decay)
 *           - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * param is rounded to param_dtype and to copy_dtype from the same fp32 value.
 * The step uses the fresh fp32 moments; only what is stored of them is 8 bits.
 *
 * RA_STATE_E4M3 stores a block's values x as round(x * (448 * (1 / amax))) with
 * scale amax * (1 / 448), amax the block's largest magnitude (a block whose amax is not
 * above 2^-100 is stored as zeros with scale 0). Rounding is stochastic: with
 * nearest rounding a second moment that changes by 0.1% a step would never
 * leave its 8-bit value. The random bits are a hash of (seed, step, place of
 * the tensor in the list, place of the element in the tensor), 16 for each
 * moment, so a step can be repeated exactly. Below e4m3's normal range (2^-15
 * of the block's amax) the value so rounded is rounded once more, to nearest,
 * and a v that is not zero is not stored as zero. A NaN or infinity in a block's moments makes the whole block
 * NaN (nearest what fp32 moments would do; grad_scale avoids it).
 *
 * Written buffers must not overlap each other or a gradient (RA_ERR_ALIAS);
 * gradients may overlap each other. RA_ERR_INVALID_ARG: step < 1, betas
 * outside [0, 1), eps or lr or weight_decay negative or not finite, eps
 * positive but below 2^-126 (with eps 0 an element that never had a gradient
 * becomes 0/0 = NaN).
 * RA_ERR_UNSUPPORTED: no host memory for the check of a long list. Lists of
 * more than 384 tensors go out as several launches.
 * HBM traffic per element: param and moments read and written, grad read.
 */
ra_status_t ra_adamw(const ra_adamw_tensor_t* tensors, int ntensors, ra_dtype_t param_dtype, ra_dtype_t grad_dtype,
                     const ra_adamw_options_t* options, void* stream);

/* ==== the two ends of a language model ========================================
 *
 * The embedding lookup and the loss, with their gradients: they share the
 * vocabulary's table, the largest tensor of the gradient buffer (with tied
 * weights ra_cross_entropy_backward writes its gradient there and
 * ra_embedding_backward adds the lookup's). Common rules as above.
 * tokens and targets: `rows` integers of index_size bytes (4: int32, 8:
 * int64), aligned to that. rows and vocab are at most 2^31 - 1024. Matrices
 * have a stride in elements (>= cols) from row to row and may start anywhere;
 * column slices of one matrix do not overlap. Two calls that may run at once
 * need a workspace each; its contents are irrelevant before and after.
 */

/*
 * Embedding lookup: out[t] = scale * table[tokens[t]], with accumulate != 0
 * out[t] = out[t] + scale * table[tokens[t]] (position embeddings on top of
 * token embeddings, for one). fp32, rounded once; a scale that fp32 does not
 * hold is refused. A token outside [0, vocab) makes its row NaN. out must not overlap the table or the tokens.
 * HBM traffic: reads the distinct rows, writes rows*cols*e.
 */
ra_status_t ra_embedding_forward(const void* table, size_t table_stride, const void* tokens, size_t index_size,
                                 void* out, size_t out_stride, int accumulate, size_t rows, size_t cols, size_t vocab,
                                 double scale, ra_dtype_t dtype, void* stream);

/*
 * Its gradient: dtable[v] = scale * sum over the t with tokens[t] == v of dy[t]
 * for every v in [0, vocab) (zero where there is none), with accumulate != 0
 * added to what dtable holds (rows without a token are then not touched).
 * Sums are fp32, rounded once, in an order that the call's arguments alone
 * decide (its sizes, tokens and whether it adds), never timing.
 * Tokens equal to `padding` and tokens outside [0, vocab) contribute nothing
 * (a padding outside [0, vocab), such as -1, is none). dy: dtype; dtable:
 * table_dtype (dtype itself or RA_FLOAT32). workspace:
 * ra_embedding_workspace(rows, cols, vocab) bytes, 16-byte aligned.
 * HBM traffic: reads rows*cols*e, writes vocab*cols*e (accumulate: reads and
 * writes the distinct rows).
 */
ra_status_t ra_embedding_backward(const void* dy, size_t dy_stride, const void* tokens, size_t index_size,
                                  int64_t padding, void* dtable, size_t dtable_stride, int accumulate, size_t rows,
                                  size_t cols, size_t vocab, double scale, ra_dtype_t dtype, ra_dtype_t table_dtype,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace ra_embedding_backward needs (0: a size it does not take). Fewer rows may need more than many: ask
 * for each size that is called. Host only. */
size_t ra_embedding_workspace(size_t rows, size_t cols, size_t vocab);

/*
 * Softmax cross entropy over the vocabulary, from the hidden states and the
 * head's weight; the logits are not stored. With logit[t][v] = sum over the
 * columns of hidden[t] * weight[v]:
 *   lse[t]  = log(sum over v of exp(logit[t][v])),
 *   loss[t] = lse[t] - logit[t][targets[t]].
 * hidden [rows, cols] and weight [vocab, cols]: RA_FLOAT16 or RA_BFLOAT16 (the
 * products run on the tensor cores, products exact, sums fp32; RA_FLOAT32:
 * RA_ERR_UNSUPPORTED). loss, lse: `rows` floats; lse is kept for the backward
 * pass. A row whose target is `ignore` has loss 0 and lse 0, costs no products,
 * and its hidden states are not read as numbers (they may be NaN). Any other
 * target outside [0, vocab) makes its row's loss and lse NaN, as does a logit
 * of +infinity or NaN. No output may overlap
 * another buffer. cols == 0, cols above 2^24 and vocab == 0 are
 * RA_ERR_INVALID_ARG (rows == 0 enqueues nothing). workspace: as ra_cross_entropy_workspace says, 16-byte
 * aligned.
 * Work: 2*rows*cols*vocab operations; HBM traffic: hidden and weight.
 */
ra_status_t ra_cross_entropy_forward(const void* hidden, size_t hidden_stride, const void* weight,
                                     size_t weight_stride, const void* targets, size_t index_size, int64_t ignore,
                                     float* loss, float* lse, size_t rows, size_t cols, size_t vocab,
                                     ra_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Its gradients. With g[t][v] = dloss[t] * (exp(logit[t][v] - lse[t]) -
 * [v == targets[t]]), the logits computed again, a piece of the vocabulary at
 * a time:
 *   dhidden[t] = sum over v of g[t][v] * weight[v],
 *   dweight[v] = sum over t of g[t][v] * hidden[t].
 * For these products g is rounded to dtype, which the products' operands have
 * (sums are fp32, rounded once): each g is off by half a step of dtype, 2^-8
 * of itself at most in bf16 and 2^-11 in fp16, and so is each term of a sum, whether
 * the sum is stored in 16 bits, where its own rounding hides that, or in an
 * fp32 dweight, where it does not. g is held relative to the largest finite
 * |dloss| of the call: bf16 loses nothing by that; fp16 rounds a g below 2^-28
 * of it to a multiple of 2^-38 of it, so that a row whose dloss is 2^-k of the
 * largest has k bits less of range for its small probabilities.
 * targets, ignore, lse: as of the forward pass; rows with
 * target `ignore` have dhidden 0 and add nothing; another target outside
 * [0, vocab) makes dhidden's row and dweight NaN. dloss: `rows` floats (NULL:
 * ones). dhidden: dtype; dweight: dweight_dtype (dtype itself or RA_FLOAT32), with
 * accumulate != 0 added to what it holds. Either may be NULL. No output may
 * overlap another buffer. rows == 0 gives a zero dweight.
 * Work: 6*rows*cols*vocab operations.
 */
ra_status_t ra_cross_entropy_backward(const void* hidden, size_t hidden_stride, const void* weight,
                                      size_t weight_stride, const void* targets, size_t index_size, int64_t ignore,
                                      const float* lse, const float* dloss, void* dhidden, size_t dhidden_stride,
                                      void* dweight, size_t dweight_stride, int accumulate, size_t rows, size_t cols,
                                      size_t vocab, ra_dtype_t dtype, ra_dtype_t dweight_dtype, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace the two calls need for these sizes (0: sizes they do not
 * take). backward: 0 for the forward pass, 1 for the backward pass. The weight
 * is read in place where it starts on a 16-byte boundary and its stride is a
 * multiple of 16 bytes; otherwise the workspace holds a copy of it, so the
 * answer depends on weight and weight_stride (the address alone is looked at).
 * The backward pass holds two pieces of g, each 192 MiB at most or 1024 columns;
 * the forward pass 16 bytes a row for each 256 words or less. Fewer rows may need
 * more than many: ask for each size that is called. Host only.
 */
size_t ra_cross_entropy_workspace(const void* weight, size_t weight_stride, size_t rows, size_t cols, size_t vocab,
                                  ra_dtype_t dtype, int backward);

/*
 * Self-test of the bounded waits inside the two calls' kernels. No wait takes
 * more than 4 s there; one that does gives up, its launch ends, and every
 * result of a row that counts, and dweight, is NaN (the call itself has
 * returned RA_SUCCESS long before). This runs the forward pass (dhidden and
 * dweight NULL) or the backward pass of dense operands, targets of 64 bits,
 * ignore -100 and dloss 1, with waits of 1 ms and a part of the work withheld
 * from the others, so that they run out. withhold: 1 the numbers of the tiles,
 * 2 the second operand, 3 the products, 4 the reading of the results (as far
 * as a pair of SMs has more than two tiles). workspace: as for the call.
 */
ra_status_t ra_selftest_cross_entropy_timeout(const void* hidden, const void* weight, const int64_t* targets,
                                              float* loss, float* lse, void* dhidden, void* dweight, size_t rows,
                                              size_t cols, size_t vocab, ra_dtype_t dtype, int withhold,
                                              void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RA_H_ */
