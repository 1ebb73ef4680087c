/*
 * ccl.h -- C ABI of the single-GPU ring-collective library (libccl.so).
 *
 * N "ranks" are simulated on one GPU: each rank is a buffer in device memory
 * (normally a slice of one arena allocation).  Every collective computes the
 * exact data semantics of the textbook ring algorithm on the device:
 *
 *   ReduceScatter phase, step s = 0..N-2: rank i sends chunk (i-s) mod N to
 *   rank i+1 and adds the chunk (i-1-s) mod N arriving from rank i-1 into its
 *   own copy; AllGather phase: rank i forwards chunk (i+1-s) mod N and stores
 *   chunk (i-s) mod N.  (Collectives and sharded matmul, "ring ReduceScatter"
 *   and "ring AllGather"; AllReduce survey, "Algorithm 1: Ring AllReduce",
 *   phase 1 and 2; Collective Communication, Algorithm 1.)
 *
 * Chunk c of a K-element buffer holds len_c = K/N + (c < K mod N) elements
 * starting at off_c = sum_{d<c} len_d (the pages split evenly; the first
 * K mod N chunks take the remainder).  Chunk c is therefore folded in the order
 * x_c, x_{c+1}, ..., x_{c-1} (ranks mod N): each hop is one IEEE fp32 operation
 * rounded to nearest-even, followed by a round to the buffer type (identity for
 * fp32, round-to-nearest-even for bf16).  A NaN result is the canonical quiet
 * NaN (fp32 0x7FFFFFFF, bf16 0x7FFF).  AVG sums around the ring, then divides
 * the finished chunk once by N in fp32 before the gather, so every rank gets
 * identical bits.  AVG_PREMUL is NCCL's pre-multiplied average (Collective
 * Communication, libraries section on NCCL): every contribution is first
 * multiplied in fp32 by the correctly rounded reciprocal of N and rounded to
 * the buffer type, the scaled values are summed around the ring as SUM does,
 * and nothing is divided at the end.  It differs from AVG in the last bits for
 * N not a power of two (the same bits for N a power of two, barring
 * subnormals); its partial sums stay near the inputs' magnitude, where the
 * plain sum that AVG divides can overflow first.  MAX is NaN if
 * either side is NaN, else the larger, and
 * +0 against -0 gives +0; MIN likewise takes the smaller, and -0 wins the tie
 * (the pages list sum, min and max as the reductions: Collective
 * Communication, table of the six core primitives).
 *
 * Common conventions
 *   - Pointer arrays (send[], recv[], ptrs[]) are HOST arrays of nranks DEVICE
 *     pointers.  The caller owns every buffer; the library never frees them.
 *     A pointer to zero elements may be NULL (a ReduceScatter or Scatter
 *     output, or an AllGather or Gather input, for an empty chunk when
 *     count < nranks; a zero-length bucket tensor; an empty AllToAllv
 *     buffer), as may the entries a call ignores (noted per call); every other
 *     pointer a call uses must not be NULL (CCL_ERR_INVALID_ARG).
 *   - All entry points that take a stream are asynchronous: they validate
 *     their arguments on the host, enqueue kernels on `stream` (0 = legacy
 *     default stream) and return.  Completion is stream completion
 *     (Collective Communication, section on correctness: a non-blocking return
 *     means work in flight, not work done).
 *   - Argument errors are returned before anything is enqueued: NULL pointers,
 *     nranks outside [1, CCL_MAX_RANKS], counts that overflow, unknown dtype,
 *     op or mode, root out of range, and buffers that partially overlap
 *     (CCL_ERR_OVERLAP).  A CUDA launch error is returned as CCL_ERR_CUDA.
 *     Nothing aborts or traps.
 *   - count == 0 is a no-op returning CCL_OK; nranks == 1 is a copy (or
 *     nothing, in place).
 *   - In-place: send[r] == recv[r] is allowed for every rank.  Any other
 *     overlap between two buffers that the same call writes and reads is an
 *     error, except the in-place forms noted per call.
 *   - CCL_MODE_FUSED computes the ring's end state in one pass over memory (one
 *     launch).  CCL_MODE_STEP executes the ring's 2(N-1) steps one launch per
 *     step, in stream order, for validating the schedule; it gives identical
 *     bits and is slower.
 *   - CUDA graphs.  Fused-mode collectives, ccl_allreduce_algo,
 *     ccl_allreduce_compressed and ccl_check_identical enqueue only kernels
 *     whose arguments travel by value and allocate nothing, so they may be
 *     captured; a graph replays them on the pointers it was captured with.
 *     ccl_allreduce_compressed sets up its kernel (shared-memory opt-in) on
 *     its first call on a device: make that call before capturing.  In step
 *     mode, AllReduce, AllGather, Broadcast, Gather, Scatter and AllToAll(v)
 *     allocate nothing either and may be captured.  Step-mode ReduceScatter,
 *     Reduce and bucket AllReduce use a library-cached device workspace that
 *     a first or larger call allocates (and frees the old one): capture them
 *     only after a call at least as large has run on that device outside the
 *     capture, and while the graph may still be replayed make no larger such
 *     call and no ccl_finalize (either frees the memory the graph uses).
 *     ccl_reduce_scatter_step_static may be captured after its set-up call
 *     (count = 0).  ccl_allreduce_host refuses capture.
 *   - That step-mode workspace is one per device, shared by every call:
 *     step-mode ReduceScatter, Reduce or bucket AllReduce calls whose work
 *     overlaps on the GPU (different streams, different host threads) race on
 *     it and must be serialised.  Fused calls share nothing.
 *   - The environment variable CCL_MODE (or ccl_set_mode_override) can force
 *     one mode on every call that takes a mode argument; a forced step mode
 *     brings the step-mode rules above with it.  See "Settings" below.
 */
#ifndef CCL_H
#define CCL_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CCL_MAX_RANKS 1024
#define CCL_DEFAULT_BUCKET_BYTES (25u * 1024u * 1024u)
/* Size of the fixed device working space of ccl_reduce_scatter_step_static. */
#define CCL_STATIC_SCRATCH_BYTES (32u * 1024u * 1024u)

typedef enum { CCL_FP32 = 0, CCL_BF16 = 1 } ccl_dtype_t;
typedef enum {
    CCL_SUM = 0,
    CCL_AVG = 1,
    CCL_MAX = 2,
    CCL_PROD = 3,
    CCL_MIN = 4,
    CCL_AVG_PREMUL = 5 /* AllReduce, ReduceScatter, Reduce, bucket and host-buffer calls; ring order only */
} ccl_op_t;
typedef enum { CCL_MODE_FUSED = 0, CCL_MODE_STEP = 1 } ccl_mode_t;
typedef enum {
    CCL_ALGO_RING = 0,
    CCL_ALGO_HALVING_DOUBLING = 1,
    CCL_ALGO_TREE = 2,
    CCL_ALGO_HIERARCHICAL = 3
} ccl_algo_t;
typedef enum { CCL_COMP_INT8_BLOCK = 0, CCL_COMP_THRESHOLD = 1, CCL_COMP_TOPK = 2 } ccl_compressor_t;
typedef enum {
    CCL_OK = 0,
    CCL_ERR_INVALID_ARG = 1,
    CCL_ERR_UNSUPPORTED = 2,
    CCL_ERR_OVERLAP = 3,
    CCL_ERR_CUDA = 4,
    CCL_ERR_NO_MEMORY = 5,
    CCL_ERR_TIMEOUT = 6,
    CCL_ERR_CHECK_FAILED = 7
} ccl_status_t;

/* ------------------------------------------------------------------ */
/* Collectives                                                         */
/* ------------------------------------------------------------------ */

/* AllReduce: every rank ends with the reduction of all ranks' buffers
 * (Collectives and sharded matmul, "Reduce and AllReduce"; Collective
 * Communication, table of the six core primitives: y_i = sum_j x_j for all i).
 * send[r], recv[r]: `count` elements each.  In place when send[r] == recv[r].
 * Result: the ring fold of chunk c starting at rank c, on every rank. */
ccl_status_t ccl_allreduce(const void *const *send, void *const *recv, int nranks, size_t count,
                           ccl_dtype_t dtype, ccl_op_t op, ccl_mode_t mode, cudaStream_t stream);

/* ReduceScatter: rank r receives chunk r of the reduction (Collectives and
 * sharded matmul, "Scatter and ReduceScatter": the sum of block r goes only to
 * rank r).  send[r]: `count` elements; recv[r]: len_r elements.  The fold
 * order is the AllReduce's (start at rank r), so ReduceScatter followed by
 * AllGather is bit-identical to AllReduce.  In place when
 * recv[r] == send[r] + off_r elements. */
ccl_status_t ccl_reduce_scatter(const void *const *send, void *const *recv, int nranks, size_t count,
                                ccl_dtype_t dtype, ccl_op_t op, ccl_mode_t mode, cudaStream_t stream);

/* AllGather: send[r] holds len_r elements (chunk r of a `count`-element
 * result); every recv[q] receives all `count` elements, chunks in rank order
 * (Collectives and sharded matmul, "Gather and AllGather").  In place when
 * send[r] == recv[r] + off_r elements. */
ccl_status_t ccl_allgather(const void *const *send, void *const *recv, int nranks, size_t count,
                           ccl_dtype_t dtype, ccl_mode_t mode, cudaStream_t stream);

/* Broadcast: every recv[q] receives root's `count` elements
 * (Collectives and sharded matmul, "Broadcast").  Only send[root] is read;
 * other send[] entries may be NULL.  Step mode chains root -> root+1 -> ...
 * one hop per launch. */
ccl_status_t ccl_broadcast(const void *const *send, void *const *recv, int nranks, int root, size_t count,
                           ccl_dtype_t dtype, ccl_mode_t mode, cudaStream_t stream);

/* AllToAll, uniform blocks: send[i] holds nranks blocks of `count` elements
 * ordered by destination; recv[j] receives nranks blocks ordered by source:
 * recv[j][i*count + t] = send[i][j*count + t] ("rank = row, block = column:
 * a transpose", Collectives and sharded matmul, "AllToAll"; Collective
 * Communication, Figure 5).  send and recv buffers must not overlap. */
ccl_status_t ccl_alltoall(const void *const *send, void *const *recv, int nranks, size_t count,
                          ccl_dtype_t dtype, ccl_mode_t mode, cudaStream_t stream);

/* AllToAllv: counts is a HOST array of nranks*nranks element counts,
 * counts[i*nranks + j] = elements rank i sends to rank j.  send[i] holds its
 * blocks ordered by destination, recv[j] its blocks ordered by source, both at
 * prefix-sum displacements (explicit per-destination counts and displacements,
 * Collective Communication, section on correctness).  Step mode follows the
 * pairwise schedule: at step k rank i sends to (i+k) mod N (Distributed LLM
 * collectives, "Pairwise algorithm"). */
ccl_status_t ccl_alltoallv(const void *const *send, void *const *recv, int nranks, const size_t *counts,
                           ccl_dtype_t dtype, ccl_mode_t mode, cudaStream_t stream);

/* Bucket-fused gradient AllReduce (Collective Communication, "Bucket fusion").
 * Each rank registers ntensors gradient tensors in forward order:
 * ptrs[r*ntensors + t] is rank r's tensor t (numels[t] elements, HOST array).
 * The tensors are laid end to end in REVERSE registration order, the stream is
 * cut into buckets of bucket_bytes (0 = the default bucket size: 25 MiB,
 * CCL_DEFAULT_BUCKET_BYTES, unless CCL_BUCKET_MB or
 * ccl_set_default_bucket_bytes changed it; the last bucket is partial and a
 * tensor may span buckets) and every bucket is
 * ring-AllReduced on its own, with its own N-chunk partition.  In place on the
 * tensors; nothing is copied into a staging bucket (the kernel reads and writes
 * the pieces where they are). */
ccl_status_t ccl_bucket_allreduce(void *const *ptrs, const size_t *numels, int ntensors, int nranks,
                                  size_t bucket_bytes, ccl_dtype_t dtype, ccl_op_t op, ccl_mode_t mode,
                                  cudaStream_t stream);

/* Reduce: only recv[root] receives the reduction, the other ranks' buffers
 * are not touched (Collectives and sharded matmul, "Reduce and AllReduce";
 * Lesson 3, core concepts: AllReduce equals a Reduce followed by a Broadcast).
 * The root receives exactly the AllReduce's bits.  send[r]: `count` elements;
 * recv[root]: `count` elements; recv[r] for r != root is ignored (may be
 * NULL).  In place when send[root] == recv[root].  Step mode runs the ring's
 * ReduceScatter phase through a cached workspace, then brings each finished
 * chunk to the root. */
ccl_status_t ccl_reduce(const void *const *send, void *const *recv, int nranks, int root, size_t count,
                        ccl_dtype_t dtype, ccl_op_t op, ccl_mode_t mode, cudaStream_t stream);

/* Gather: recv[root] receives every rank's slice concatenated in rank order
 * (Lesson 3, core concepts: "Gather"; Collectives and sharded matmul, "Gather
 * and AllGather").  send[r] holds len_r elements (chunk r of `count`);
 * recv[r] for r != root is ignored.  In place when
 * send[root] == recv[root] + off_root elements; more generally, any send[r]
 * may already sit at its own place, recv[root] + off_r elements (its chunk is
 * then copied onto itself). */
ccl_status_t ccl_gather(const void *const *send, void *const *recv, int nranks, int root, size_t count,
                        ccl_dtype_t dtype, ccl_mode_t mode, cudaStream_t stream);

/* Scatter: send[root]'s `count` elements are split into the N chunks and
 * chunk r goes to recv[r] (len_r elements) (Lesson 3, core concepts: "Scatter",
 * the inverse of Gather; Collectives and sharded matmul, "Scatter and
 * ReduceScatter").  send[r] for r != root is ignored.  In place when
 * recv[root] == send[root] + off_root elements; more generally, any recv[r]
 * may already sit at its own place, send[root] + off_r elements (its chunk is
 * then copied onto itself). */
ccl_status_t ccl_scatter(const void *const *send, void *const *recv, int nranks, int root, size_t count,
                         ccl_dtype_t dtype, ccl_mode_t mode, cudaStream_t stream);

/* Bucket AllReduce overlapped with the backward pass (Collective
 * Communication, "Layer-wise overlap": a gradient hook per parameter starts a
 * bucket's AllReduce as soon as the bucket is full, while the backward pass
 * goes on).  ccl_bucketer_create takes the same tensors, layout and bucket
 * size as ccl_bucket_allreduce and plans the buckets once (the tensors stay
 * owned by the caller and must outlive the bucketer).  Each step, the caller
 * calls ccl_bucketer_mark_ready for every tensor once its gradient is final
 * on every rank, with an event recorded after it on the compute stream (or
 * NULL if comm_stream is already ordered after that work).  The call makes
 * comm_stream wait for that event (so the event need only be valid during the
 * call; mark tensors in the order they are produced, or a later wait delays
 * an earlier-filled bucket), and when all the tensors a bucket touches are
 * ready it enqueues the bucket's fused ring reduction on comm_stream.  Results
 * are bit-identical to ccl_bucket_allreduce.  ccl_bucketer_reset starts the
 * next step. */
typedef struct ccl_bucketer ccl_bucketer_t;
/* max_ctas > 0 caps each bucket kernel's grid so the reduction, which is
 * bound by memory bandwidth, runs beside the backward pass's compute-bound
 * kernels on part of the GPU instead of claiming every SM; 0 launches one CTA
 * per tile.  The bits do not depend on it. */
ccl_status_t ccl_bucketer_create(void *const *ptrs, const size_t *numels, int ntensors, int nranks,
                                 size_t bucket_bytes, ccl_dtype_t dtype, ccl_op_t op, int max_ctas,
                                 ccl_bucketer_t **out);
ccl_status_t ccl_bucketer_mark_ready(ccl_bucketer_t *b, int tensor, cudaEvent_t ready, cudaStream_t comm_stream);
ccl_status_t ccl_bucketer_reset(ccl_bucketer_t *b);
/* Buckets planned and buckets enqueued so far in this step. */
ccl_status_t ccl_bucketer_status(ccl_bucketer_t *b, size_t *nbuckets, size_t *launched);
ccl_status_t ccl_bucketer_destroy(ccl_bucketer_t *b);

/* AllReduce under another schedule's summation order, in one pass (fused).
 * Each schedule adds the contributions in its own order, so each gives its own
 * rounded bits; this call reproduces them exactly.
 *   CCL_ALGO_RING: the ring of ccl_allreduce (identical result).
 *   CCL_ALGO_HALVING_DOUBLING: round k pairs rank i with i XOR 2^k, k = 0, 1,
 *     ... (Collective Communication, "Recursive halving-doubling (butterfly)");
 *     for N not a power of two the first 2r ranks, r = N - 2^floor(log2 N), are
 *     first added pairwise (2v, 2v+1) (Distributed LLM collectives, "Recursive
 *     Halving-Doubling").  Per element: a balanced tree, adjacent leaves first.
 *   CCL_ALGO_TREE: binomial tree to rank 0, level k adding rank i + 2^k into
 *     rank i, then broadcast (Collective Communication, "Tree AllReduce").
 *   CCL_ALGO_HIERARCHICAL: ring ReduceScatter inside groups of group_size
 *     consecutive ranks, ring AllReduce among the groups' representatives,
 *     ring AllGather inside the groups (AllReduce survey, two-level table);
 *     group_size must divide nranks (1 or nranks gives the flat ring).
 * AVG divides the finished sum once by N; CCL_AVG_PREMUL is accepted with
 * CCL_ALGO_RING only (CCL_ERR_UNSUPPORTED otherwise).  Buffers as
 * ccl_allreduce (in place when send[r] == recv[r]).  group_size is ignored
 * except for CCL_ALGO_HIERARCHICAL. */
ccl_status_t ccl_allreduce_algo(const void *const *send, void *const *recv, int nranks, size_t count,
                                ccl_dtype_t dtype, ccl_op_t op, ccl_algo_t algo, int group_size,
                                cudaStream_t stream);

/* Compressed AllReduce with error feedback (Collective Communication,
 * "Gradient compression": blockwise INT8 quantization, and "Error feedback and
 * residual accumulation", Definition 1.4).  grads[r]: `count` elements of
 * dtype, in place; residuals[r]: `count` fp32 per rank, zero before the first
 * step, carried by the caller from step to step.  Each rank compresses
 * u = g + e and keeps e' = u - v:
 *   CCL_COMP_INT8_BLOCK (block = 64 or 128): s = max|u| / 127 over each
 *     block, q = round(u / s) (ties to even), v = q * s;
 *   CCL_COMP_THRESHOLD (the greedy 1-bit compressor of the pages' Tables 3
 *     and 4): v = 1 when u >= threshold, else 0.
 * The transmitted v are AllReduced in ring order in fp32 (op CCL_SUM, or
 * CCL_AVG dividing once by N; CCL_AVG_PREMUL returns CCL_ERR_UNSUPPORTED) and
 * rounded once to dtype, written to every grads[r].  Up to 16 ranks; grads
 * and residuals must not overlap.  CCL_COMP_TOPK needs k and a work buffer:
 * it is ccl_allreduce_topk's (CCL_ERR_INVALID_ARG here).  One launch, two
 * with a partial last block. */
ccl_status_t ccl_allreduce_compressed(void *const *grads, float *const *residuals, int nranks, size_t count,
                                      ccl_dtype_t dtype, ccl_op_t op, ccl_compressor_t comp, int block,
                                      float threshold, cudaStream_t stream);

/* Top-k sparsified AllReduce with error feedback (Collective Communication,
 * "Top-k sparsification", and "Error feedback and residual accumulation",
 * Definition 1.4).  grads[r]: `count` elements of dtype, in place;
 * residuals[r]: `count` fp32 per rank, zero before the first step, carried by
 * the caller.  Each rank forms u = g + e (fp32) and sends v = u where |u| is
 * at least its k-th largest magnitude |u|_(k), else 0 -- every value tied
 * with the k-th is sent, so a rank may send more than k -- and keeps
 * e' = u - v.  Magnitudes are ordered as the bit patterns of |u|, so a NaN
 * counts as the largest and is always sent.  k = 0 sends nothing; k >= count
 * sends everything.  The sent values are AllReduced in ring order in fp32
 * (CCL_SUM, or CCL_AVG dividing once by N; CCL_AVG_PREMUL returns
 * CCL_ERR_UNSUPPORTED) and rounded once to dtype, written to every grads[r].
 * The threshold is found on the device by a radix select, with no host round
 * trip: a sample (one 256-element run in 16; in 32, 64 or 128 when the
 * sparser sample still expects 4096 keys at or above the k-th and the
 * standard deviation of its estimate of that key's rank, sqrt(k * 128) for
 * one run in 128, is at most count / 2048) places a window of one to four top-12-bit bins, one full pass
 * over g and e counts every key's top bits and the low 19 bits of the keys
 * in the window, and a second full pass runs only when the k-th key's top
 * bin fell outside the window.  One more pass then sends, keeps the
 * residuals and reduces.  work: device memory of ccl_plan_topk_work_bytes
 * bytes (about 10 MiB per rank), 16-byte aligned,
 * owned by the caller, not shared with a concurrent call; its contents need
 * no initialisation.  Up to 16 ranks and count < 2^32; grads, residuals and
 * work must not overlap (CCL_ERR_OVERLAP).  Launches: one to reset the work
 * buffer; when 0 < k < count the sample and its scan (large aligned inputs),
 * the full pass and its scan, the two fallback launches (which return at once
 * when the window held the bin), and the low histogram's two scans; and the
 * compressed pass (one launch, two with a partial last block of 128). */
ccl_status_t ccl_allreduce_topk(void *const *grads, float *const *residuals, int nranks, size_t count,
                                ccl_dtype_t dtype, ccl_op_t op, size_t k, void *work, size_t work_bytes,
                                cudaStream_t stream);

/* Bytes of the work buffer ccl_allreduce_topk needs for nranks ranks. */
ccl_status_t ccl_plan_topk_work_bytes(int nranks, size_t *bytes);

/* The sample ccl_allreduce_topk takes for count elements per rank and this
 * k, when every gradient and residual is 16-byte aligned (others are never
 * sampled): *every = f when the sample reads one 256-element run in f (16,
 * 32, 64 or 128, by the rule in ccl_allreduce_topk's description), 0 when it
 * takes none -- k = 0, k >= count, or too few elements for the sample to
 * place a window (the select then counts the k-th key's top bin in a second
 * full pass).  Host only; CCL_ERR_INVALID_ARG for a null every or
 * count >= 2^32. */
ccl_status_t ccl_plan_topk_sample(size_t count, size_t k, uint32_t *every);

/* Bytes one rank would put on a link for Top-k with fp32 values and int32
 * indices: 8 * min(k, count), a ratio of 4 count / bytes = count / (2k) over
 * dense fp32 (Collective Communication, "Top-k sparsification": 500x, not
 * 1000x, for k = 0.001 count).  Host only. */
ccl_status_t ccl_plan_topk_bytes(size_t count, size_t k, size_t *bytes);

/* Step-by-step ReduceScatter that allocates nothing.  The pages have no
 * counterpart: this exists for callers that cannot let a library call
 * cudaMalloc -- a process whose framework has already reserved the GPU's
 * memory in its own caching pool (a raw cudaMalloc then fails or fragments
 * what is left), code that must not stall other streams on the device
 * synchronisation cudaMalloc/cudaFree can imply, or hosts that forbid driver
 * allocations after start-up.
 * Same arguments, result and error checks as ccl_reduce_scatter in
 * CCL_MODE_STEP (identical bits; the checks are the same code), but the
 * working copies of the N inputs live in one fixed array of
 * CCL_STATIC_SCRATCH_BYTES (32 MiB) in device memory, held by every GPU that
 * reserves it until the process exits.  nranks * round_up(count * element
 * size, 256) must not exceed CCL_STATIC_SCRATCH_BYTES: larger calls return
 * CCL_ERR_INVALID_ARG before anything is enqueued.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.
 *   - Set-up, once per device: a call with count = 0 (valid nranks, dtype and
 *     op, non-NULL pointer arrays whose entries are not read) looks up the
 *     array's device address (cudaGetSymbolAddress, with that device current),
 *     loads every kernel this entry launches, caches the address and enqueues
 *     nothing; it returns CCL_ERR_CUDA if that fails.  Under CUDA's lazy module
 *     loading (the default since CUDA 12.2) this lookup is when the driver
 *     reserves the array, so make this call at start-up, before a caching
 *     pool takes the GPU's memory and before any stream capture.  A first
 *     call with count > 0 does the same set-up itself.
 *   - Every call on a device shares the array and leaves its contents behind.
 *     Each call overwrites every byte it later reads, so nothing needs
 *     clearing, but calls whose work overlaps on the GPU (other streams, other
 *     host threads) race on it: serialise them.
 *   - ccl_finalize forgets the cached address of the current device; call it
 *     after a cudaDeviceReset, before the next call on that device. */
ccl_status_t ccl_reduce_scatter_step_static(const void *const *send, void *const *recv, int nranks, size_t count,
                                            ccl_dtype_t dtype, ccl_op_t op, cudaStream_t stream);

/* Device working space that lets ccl_allreduce_host run at the host link's
 * speed: three stages of 64 MiB. */
#define CCL_HOST_WORK_BYTES_DEFAULT (192u * 1024u * 1024u)

/* AllReduce of rank buffers that live in HOST memory: the same result, bit for
 * bit, as ccl_allreduce on the same data (the ring fold of chunk c starting at
 * rank c of the count-element partition).  send[r], recv[r]: `count` elements
 * each, any memory the GPU can copy from and to (cudaMemcpyDefault); page-
 * locked host memory (cudaHostAlloc, cudaHostRegister) is what makes the
 * copies asynchronous and overlapped.  In place when send[r] == recv[r].
 * Two paths give the same bits:
 *   - in place over the host link, when CCL_HOST_PATH=direct (or
 *     ccl_set_host_path(CCL_HOST_PATH_DIRECT)) and every send[r] and recv[r]
 *     is page-locked host memory that the current device can address: one
 *     fused AllReduce launch on `stream` reads and writes them directly
 *     (both link directions busy at once, nothing staged; `work` is
 *     validated but not used);
 *   - staged, the default, and for any other memory:
 * the vector moves through `work` (DEVICE memory, caller-owned, 16-byte
 * aligned, work_bytes >= 3 * nranks * 256 * element size; larger is faster,
 * up to CCL_HOST_WORK_BYTES_DEFAULT) in slices: copies in and out run on two
 * library-owned streams so that both directions of the host link are busy at
 * once, and each slice is reduced on `stream` (the link is the bottleneck:
 * Collective Communication, Table 1, GPU<->CPU row; the overlap is the
 * pipelining of the section on NCCL).  Ordering: the call starts after the
 * work already enqueued on `stream`, and work enqueued on `stream` afterwards
 * sees every result in recv[].  Calls that share `work` must be ordered (one
 * stream, or events); the library orders its own stage reuse across calls.
 * Returns CCL_ERR_UNSUPPORTED while `stream` is being captured into a CUDA
 * graph, CCL_ERR_INVALID_ARG for a work buffer that is too small or
 * misaligned, and the common argument errors otherwise. */
ccl_status_t ccl_allreduce_host(const void *const *send, void *const *recv, int nranks, size_t count,
                                ccl_dtype_t dtype, ccl_op_t op, void *work, size_t work_bytes,
                                cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* Operators of a training step                                        */
/* ------------------------------------------------------------------ */

/* What one rank computes between the collectives: the embedding lookup, the
 * loss and their gradients, whose outputs are buffers that the collectives
 * above reduce.  Unlike the collectives these calls take one rank's buffers.
 * The common conventions hold: device buffers owned by the caller, work
 * enqueued on `stream`, argument errors returned before anything is enqueued,
 * CCL_ERR_OVERLAP where a written buffer overlaps another one of the call
 * (except in the in-place forms noted), nothing allocated, so that every call
 * may be captured in a CUDA graph (after one call of its kind on the device,
 * which sets its kernels up).  Sums are held in fp32 and each output is
 * rounded once to its type.  Strides are in elements, from one row to the
 * next, and at least the row's length; buffers need only their element's
 * alignment (without it: CCL_ERR_INVALID_ARG; 16-byte aligned rows of whole
 * 16-byte vectors run at full bandwidth).  No value is added by an atomic: the same inputs give the same
 * bits. */

/* Embedding lookup: out[t] = round(scale * table[ids[t] - first_row]), t <
 * ntokens, rows of `dim` elements.  An id outside [first_row, first_row +
 * rows) -- a padding id, or a row of another rank's shard of the vocabulary --
 * gives a row of zeros, so that ccl_allreduce (CCL_SUM) over the ranks' outputs
 * completes a lookup in a table whose rows are sharded.  rows, ntokens < 2^31;
 * dim <= 2^24. */
ccl_status_t ccl_embedding(const void *table, size_t rows, size_t dim, size_t table_stride, ccl_dtype_t dtype,
                           const int64_t *ids, size_t ntokens, int64_t first_row, float scale, void *out,
                           size_t out_stride, cudaStream_t stream);

/* Its gradient: grad_table[v] = round([grad_table[v] +] scale * sum of
 * grad_out[t] over the tokens with ids[t] == first_row + v).  The tokens are
 * sorted by row, stably, and each row's are added in fp32 in runs of
 * consecutive sorted tokens, joined in order.  accumulate = 0 writes every
 * row (zeros where no token names it); accumulate != 0 adds to the rows that
 * a token names and leaves the others untouched (a tied output projection's
 * gradient, a further micro-batch).  work: device memory of
 * ccl_plan_embedding_grad_work_bytes bytes (fewer tokens may need more: for
 * several batch sizes the largest of their plans), 16-byte aligned, not shared
 * with a concurrent call; its contents need no initialisation.  Launches: the zero
 * rows (accumulate = 0), the sort (one launch for both up to 4096 tokens), the
 * sums, and the join when the tokens fill more than one run (of 8 to 32). */
ccl_status_t ccl_embedding_grad(const void *grad_out, size_t grad_out_stride, const int64_t *ids, size_t ntokens,
                                int64_t first_row, size_t rows, size_t dim, ccl_dtype_t dtype, float scale,
                                int accumulate, void *grad_table, size_t grad_table_stride, void *work,
                                size_t work_bytes, cudaStream_t stream);
ccl_status_t ccl_plan_embedding_grad_work_bytes(size_t ntokens, size_t rows, size_t dim, size_t *bytes);

/* Gated feed-forward block on ntokens rows of `dim` values:
 *   g = x w_gate^T, u = x w_up^T, h = act(g) * u, out = h w_down^T
 * with w_gate, w_up [ffn][dim] and w_down [dim][ffn] (an output unit's weights
 * are a row).  All matrices are contiguous and bf16 (CCL_FP32:
 * CCL_ERR_UNSUPPORTED); the products accumulate in fp32 and h is rounded to
 * bf16 once.  saved != NULL keeps g and u for the backward pass, fp32,
 * [2][ntokens][ffn].  work: device memory of ccl_plan_gated_ffn_work_bytes
 * bytes, 256-byte aligned, not shared with a concurrent call, contents
 * irrelevant.  dim and ffn <= 2^24. */
typedef enum { CCL_ACT_SILU = 0, CCL_ACT_GELU_TANH = 1 } ccl_act_t;
ccl_status_t ccl_gated_ffn(const void *x, const void *w_gate, const void *w_up, const void *w_down, size_t ntokens,
                           size_t dim, size_t ffn, ccl_dtype_t dtype, ccl_act_t act, void *out, float *saved, void *work,
                           size_t work_bytes, cudaStream_t stream);

/* Its gradients, from grad_out and the saved g and u (h is made again):
 *   dh = grad_out w_down, du = dh * act(g), dg = dh * u * act'(g)
 *   grad_x = dg w_gate + du w_up, grad_w_gate = dg^T x, grad_w_up = du^T x,
 *   grad_w_down = grad_out^T h
 * dg and du are rounded to bf16 once.  A NULL gradient is not computed.
 * accumulate != 0 adds to the weight gradients (grad_x is always written):
 * round(old + sum), one rounding.  work: as above, planned with backward = 1. */
ccl_status_t ccl_gated_ffn_grad(const void *grad_out, const void *x, const void *w_gate, const void *w_up,
                                const void *w_down, const float *saved, size_t ntokens, size_t dim, size_t ffn,
                                ccl_dtype_t dtype, ccl_act_t act, int accumulate, void *grad_x, void *grad_w_gate,
                                void *grad_w_up, void *grad_w_down, void *work, size_t work_bytes, cudaStream_t stream);

/* Bytes of the work buffer.  aligned != 0: every input matrix is 16-byte
 * aligned (else, or where a width is no multiple of 8, room for padded copies
 * of the inputs is included: the copy engine that feeds the tensor cores
 * addresses whole 16-byte vectors).  backward != 0: for ccl_gated_ffn_grad, and
 * enough for ccl_gated_ffn of the same sizes.  Fewer tokens may need more bytes
 * (their sums are cut into more parts): a buffer for several batch sizes has the
 * largest of their plans. */
ccl_status_t ccl_plan_gated_ffn_work_bytes(size_t ntokens, size_t dim, size_t ffn, int backward, int aligned, size_t *bytes);

/* How often a wait of a gated feed-forward kernel (ccl_expert_ffn's too) on the
 * current device for its own copies or products ran out: 0 on a sound machine.  What such a kernel
 * could not compute it writes as NaN, and so is every output that depends on
 * it.  Waits for the device. */
ccl_status_t ccl_gated_ffn_timeouts(unsigned long long *count);
/* The longest such wait, in ns, of calls made from now on (4 s by default).  0
 * gives up at once, without a copy or product that another one waits for: every
 * output is NaN, so that a program can try what it does then. */
ccl_status_t ccl_set_gated_ffn_wait_limit(unsigned long long ns);

/* Distillation loss from a teacher's top logits.  Row t's teacher
 * distribution p is the softmax of teacher_logits[t][0..top) / temperature
 * over the entries whose id teacher_ids[t][j] is in [0, vocab) (others do not
 * count, whatever their logit holds; an id may come twice); the student's q
 * is the softmax of logits[t] / temperature over the whole vocabulary.
 *   loss[t]    = weights[t] * sum_j p_j (log p_j - log q_{id_j})
 *   grad[t][v] = weights[t] / temperature * (q_v - sum over {j: id_j = v} p_j),
 * the derivative of the sum of the losses by logits[t][v].  A row without a
 * teacher (no valid id, or only -inf logits) and a row of weight 0 have loss 0
 * and gradient 0; weights == NULL means 1.  (The customary factor
 * temperature^2 belongs in the weights.)  A logit of -inf leaves that entry
 * out of the vocabulary.  teacher_ids and teacher_logits are contiguous
 * [nrows][top] arrays, top <= CCL_MAX_TEACHER_TOP.
 *
 * ccl_distill_loss writes the losses, with stats != NULL also every row's
 * (m, Z) -- its largest logit and sum_v exp((logits[v] - m) / temperature) --
 * as stats[2t], stats[2t+1], and with grad != NULL also the gradient, the row
 * then being read from memory once for both (rows of up to 512 KiB).
 * ccl_distill_grad computes the gradient later from the kept stats, with
 * weights of its own (weights times the incoming gradient of loss[t]).  In
 * place: grad == logits with the same stride.  One launch each. */
#define CCL_MAX_TEACHER_TOP 1024
ccl_status_t ccl_distill_loss(const void *logits, size_t nrows, size_t vocab, size_t logits_stride, ccl_dtype_t dtype,
                              const int64_t *teacher_ids, const float *teacher_logits, size_t top, float temperature,
                              const float *weights, float *loss, float *stats, void *grad, size_t grad_stride,
                              cudaStream_t stream);
ccl_status_t ccl_distill_grad(const void *logits, size_t nrows, size_t vocab, size_t logits_stride, ccl_dtype_t dtype,
                              const int64_t *teacher_ids, const float *teacher_logits, size_t top, float temperature,
                              const float *weights, const float *stats, void *grad, size_t grad_stride,
                              cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* Operators of an expert-parallel step                                */
/* ------------------------------------------------------------------ */

/* What a rank computes around ccl_alltoallv when a layer's feed-forward block
 * is a mixture of experts: the router with its balance loss, the tokens in
 * expert order (the exchange's send buffer and, from the offsets, its counts),
 * the experts' blocks over them, the weighted sum back, and the gradients, with
 * the activations kept in 8 bits in between.  The conventions of the operators
 * of a training step hold.  experts <= CCL_MAX_EXPERTS, choices of one token
 * (top) <= CCL_MAX_EXPERT_TOP, tokens * top < 2^31. */
#define CCL_MAX_EXPERTS 1024
#define CCL_MAX_EXPERT_TOP 32

/* Router.  Over each token's logits z (1 <= top <= experts of them are chosen):
 *   p = softmax(z); ids[t][0..top) = the experts of the largest logits, largest
 *   first, ties to the lower expert; weights[t][s] = p at ids[t][s], divided by
 *   the sum of the chosen ones when normalize != 0; lse[t] = log sum exp z
 *   counts[e] = tokens that chose e, counts[experts] = n, the tokens routed
 *   load[e] = counts[e] / all choices, importance[e] = (sum over tokens of p_e) / n
 *   losses[0] = experts * sum_e load[e] importance[e] (the balance loss: 1 when
 *   both are even), losses[1] = (sum over tokens of lse^2) / n (the z loss)
 * A logit of -inf is an expert that the token cannot choose; a slot left without
 * an expert has id -1 and weight 0.  A token with valid[t] == 0 (valid == NULL:
 * none), or without any expert, is not routed: ids -1, weights 0, lse 0, and it
 * counts nowhere.  A NaN or +inf makes its token's weights NaN (the ids stay in
 * range, NaN being the largest).  work: ccl_plan_route_work_bytes bytes, 256-byte
 * aligned, not shared with a concurrent call, contents irrelevant (0 bytes for
 * few tokens, and never fewer for more).  One launch, or two. */
ccl_status_t ccl_route(const void *logits, size_t ntokens, size_t experts, size_t logits_stride, ccl_dtype_t dtype,
                       const uint8_t *valid, size_t top, int normalize, int32_t *ids, float *weights, float *lse,
                       int32_t *counts, float *load, float *importance, float *losses, void *work, size_t work_bytes,
                       cudaStream_t stream);
ccl_status_t ccl_plan_route_work_bytes(size_t ntokens, size_t experts, size_t *bytes);

/* Its gradient by the logits, of sum grad_weights * weights + balance *
 * losses[0] + z * losses[1] (the choices and load are constants):
 *   grad[t][j] = p_j (G_j - sum_i G_i p_i + 2 z lse[t] / n),
 *   G_j = balance * experts * load[j] / n + [j chosen] (by its weight)
 * from what ccl_route left in ids, lse, counts (only counts[experts] is read) and
 * load, which may have been averaged over the ranks by ccl_allreduce in between.
 * grad_weights where the id is -1 does not count, whatever it holds.  Tokens that
 * are not routed have gradient 0.  In place: grad_logits == logits with the same
 * stride. */
ccl_status_t ccl_route_grad(const void *logits, size_t ntokens, size_t experts, size_t logits_stride, ccl_dtype_t dtype,
                            const int32_t *ids, size_t top, int normalize, const float *lse, const int32_t *counts,
                            const float *load, const float *grad_weights, float balance, float z, void *grad_logits,
                            size_t grad_stride, cudaStream_t stream);

/* The tokens' copies in expert order: place[t][s] = the row of token t's s-th
 * choice, rows being ordered by expert, then token, then choice; expert
 * first_expert + e has rows [offsets[e], offsets[e + 1]), offsets[0] = 0.  An id outside [first_expert, first_expert + experts)
 * (-1, or an expert of another rank) has place -1.  work:
 * ccl_plan_expert_order_work_bytes bytes (0 up to 16384 choices, and never fewer
 * for more tokens), 256-byte aligned, not shared with a concurrent call.  One
 * launch, or three. */
ccl_status_t ccl_expert_order(const int32_t *ids, size_t ntokens, size_t top, int32_t first_expert, size_t experts,
                              int32_t *offsets, int32_t *place, void *work, size_t work_bytes, cudaStream_t stream);
ccl_status_t ccl_plan_expert_order_work_bytes(size_t ntokens, size_t top, size_t experts, size_t *bytes);

/* rows[place[t][s]] = x[t].  A place outside [0, nrows) is skipped; rows that no
 * place names are left as they were.  No two places may name the same row.  Its
 * gradient is ccl_combine without weights. */
ccl_status_t ccl_dispatch(const void *x, size_t ntokens, size_t dim, size_t x_stride, ccl_dtype_t dtype,
                          const int32_t *place, size_t top, void *rows, size_t nrows, size_t rows_stride,
                          cudaStream_t stream);

/* out[t] = round(sum over s of weights[t][s] rows[place[t][s]]), the sum in fp32
 * in the order of s.  A place outside [0, nrows) adds nothing, whatever its
 * weight; a token without any gives zeros.  weights == NULL means 1. */
ccl_status_t ccl_combine(const void *rows, size_t nrows, size_t dim, size_t rows_stride, ccl_dtype_t dtype,
                         const int32_t *place, const float *weights, size_t ntokens, size_t top, void *out,
                         size_t out_stride, cudaStream_t stream);

/* Its gradients: grad_rows[place[t][s]] = round(weights[t][s] grad_out[t]) and
 * grad_weights[t][s] = <grad_out[t], rows[place[t][s]]> in fp32, 0 where there is
 * no row.  A NULL gradient is not computed, and rows is read for grad_weights
 * only.  Rows that no place names are left as they were; no two places may name
 * the same row.  In place: grad_rows == rows with the same stride. */
ccl_status_t ccl_combine_grad(const void *grad_out, size_t grad_out_stride, const void *rows, size_t nrows, size_t dim,
                              size_t rows_stride, ccl_dtype_t dtype, const int32_t *place, const float *weights,
                              size_t ntokens, size_t top, void *grad_rows, size_t grad_rows_stride, float *grad_weights,
                              cudaStream_t stream);

/* Activations in 8 bits, kept for the backward pass.  Each row is cut into blocks
 * of 32 values (the last one may be shorter); a block's step is 2^e, the least
 * power of two with |x| <= 127 * 2^e (e >= -126, and at most 121, where larger
 * values become 127 * 2^121), and
 *   codes[r][c] = x / 2^e rounded to the nearest integer, ties to even
 *   scales[r][c / 32] = e + 127; 255 for a block that holds an infinity or a NaN,
 *   which comes back as NaN
 * so that a value comes back to within 2^(e-1), and as a bf16 number.  codes:
 * [rows][width], 32-byte aligned, width = the columns rounded up to a multiple of
 * 32 (ccl_plan_act8_width), its last columns 0; scales: [rows][width / 32].
 * rows < 2^31, cols <= 2^24. */
ccl_status_t ccl_act8_pack(const void *x, size_t rows, size_t cols, size_t x_stride, ccl_dtype_t dtype, int8_t *codes,
                           uint8_t *scales, cudaStream_t stream);
ccl_status_t ccl_act8_unpack(const int8_t *codes, const uint8_t *scales, size_t rows, size_t cols, ccl_dtype_t dtype,
                             void *x, size_t x_stride, cudaStream_t stream);
ccl_status_t ccl_plan_act8_width(size_t cols, size_t *width);

/* The experts' gated feed-forward blocks (as ccl_gated_ffn) over rows in expert
 * order: rows [offsets[e], offsets[e + 1]) of x go through expert e's weights,
 * w_gate, w_up [experts][ffn][dim] and w_down [experts][dim][ffn], all contiguous
 * and bf16.  offsets is DEVICE memory, [experts + 1], as ccl_expert_order leaves
 * it (any part of it will do): the call needs no count on the host.  Offsets that
 * fall, or lie outside [0, nrows], are taken as the largest before them within
 * [0, nrows].  Rows of out before offsets[0] and from offsets[experts] on are left
 * as they were.  saved_codes, saved_scales != NULL keep g and u for the backward
 * pass in 8 bits as ccl_act8_pack keeps them, [2][nrows][width(ffn)] and
 * [2][nrows][width(ffn) / 32] (the rows of experts).  ffn >= 1.  work: ccl_plan_expert_ffn_work_bytes bytes,
 * 256-byte aligned, not shared with a concurrent call, contents irrelevant. */
ccl_status_t ccl_expert_ffn(const void *x, const int32_t *offsets, const void *w_gate, const void *w_up,
                            const void *w_down, size_t nrows, size_t experts, size_t dim, size_t ffn, ccl_dtype_t dtype,
                            ccl_act_t act, void *out, int8_t *saved_codes, uint8_t *saved_scales, void *work,
                            size_t work_bytes, cudaStream_t stream);

/* Its gradients, from grad_out, the saved g and u, and x, which is given either
 * as it was (x) or in 8 bits (x == NULL: x_codes, x_scales, as ccl_act8_pack left
 * it):
 *   dh = grad_out w_down, du = dh * act(g), dg = dh * u * act'(g), h = act(g) * u
 *   grad_x = dg w_gate + du w_up, grad_w_gate = dg^T x, grad_w_up = du^T x,
 *   grad_w_down = grad_out^T h
 * expert by expert, h, dg and du rounded to bf16 once.  A NULL gradient is not
 * computed.  An expert without rows has weight gradients 0.  accumulate != 0 adds
 * to the weight gradients: round(old + sum), one rounding.  work: planned with
 * backward = 1.  Waits that run out are counted by ccl_gated_ffn_timeouts, and
 * ccl_set_gated_ffn_wait_limit sets their limit. */
ccl_status_t ccl_expert_ffn_grad(const void *grad_out, const void *x, const int8_t *x_codes, const uint8_t *x_scales,
                                 const int32_t *offsets, const void *w_gate, const void *w_up, const void *w_down,
                                 const int8_t *saved_codes, const uint8_t *saved_scales, size_t nrows, size_t experts,
                                 size_t dim, size_t ffn, ccl_dtype_t dtype, ccl_act_t act, int accumulate, void *grad_x,
                                 void *grad_w_gate, void *grad_w_up, void *grad_w_down, void *work, size_t work_bytes,
                                 cudaStream_t stream);

/* Bytes of the work buffer; aligned and backward as for ccl_plan_gated_ffn_work_bytes.
 * A buffer planned for more rows, everything else being equal, serves fewer too,
 * although few rows may plan more bytes than many: ccl_expert_ffn then cuts its
 * sums into the parts that fit, in another order, so with other roundings, and up
 * to twice as slow (64 rows of one expert of 4096 x 4096 in the 0.5 MB of 65 rows
 * 67 us, in their own 6.8 MB 36).  The largest of the plans of the batches that
 * occur keeps every one at its speed and bits. */
ccl_status_t ccl_plan_expert_ffn_work_bytes(size_t nrows, size_t experts, size_t dim, size_t ffn, int backward,
                                            int aligned, size_t *bytes);

/* ------------------------------------------------------------------ */
/* Result checks and tracing                                           */
/* ------------------------------------------------------------------ */

/* Adds to *mismatches (a DEVICE counter the caller zeroes) the number of
 * elements, summed over ranks 1..nranks-1, whose bits differ from rank 0's.
 * After an AllReduce every rank must hold the same bits (Collective
 * Communication, Definition 1.1); the pages ask that results be checked
 * against silent corruption (section on pitfalls).  Never traps. */
ccl_status_t ccl_check_identical(const void *const *bufs, int nranks, size_t count, ccl_dtype_t dtype,
                                 unsigned long long *mismatches, cudaStream_t stream);

/* Automatic result checks, off unless CCL_CHECK is set (to anything but 0)
 * or enabled here.  While on, every AllReduce (fused or step, any order, the
 * compressed one), AllGather and Broadcast that succeeds also enqueues
 * ccl_check_identical over its outputs on the call's stream, adding to a
 * per-device counter the library owns (one cudaMalloc on the first checked
 * call on a device: make it before any stream capture).  Never traps. */
void ccl_set_check(int enabled);
/* Waits for the whole device, stores the current device's counter in
 * *mismatches (0 if nothing was checked yet) and, when reset != 0, sets the
 * counter back to 0. */
ccl_status_t ccl_check_read(unsigned long long *mismatches, int reset);

/* Debug builds (libccl_debug.so, compiled with CCL_DEBUG_BOUNDS) check every
 * global load and store of every kernel against the byte ranges of the
 * call's own buffers, library workspace included (but not the tensor-map
 * copies of the gated feed-forward block, which their maps bound); an access outside them is
 * skipped, never performed, and counted.  Waits for the device and returns
 * the count and the first offending address.  Release builds return
 * CCL_ERR_UNSUPPORTED.  Calls whose work overlaps on the GPU share the range
 * table in debug builds: run them one at a time there. */
ccl_status_t ccl_debug_faults(unsigned long long *faults, unsigned long long *first_address);

/* One traced call: the collective, its shape, the kernels it enqueued, the
 * host time it took to validate, plan and enqueue, and its device time. */
typedef struct {
    char collective[24];
    int nranks;
    int dtype;
    int op;   /* -1 where the collective takes none */
    int mode; /* or the algorithm / compressor of the _algo / _compressed calls */
    int status;
    unsigned launches;
    unsigned long long count;
    unsigned long long host_ns;
    unsigned long long seq;
    /* Device time from the start to the end of the call's work on its stream
     * (two events recorded around it; Collective Communication, libraries
     * section: time a collective against a bare baseline with a profiler
     * before tuning it).  0 until that work has completed on the device --
     * ccl_trace_read fills it in once it has -- and 0 for calls not timed:
     * made while the stream was being captured into a CUDA graph, or in a
     * process without a device. */
    unsigned long long gpu_ns;
} ccl_trace_record_t;

/* Tracing is off unless CCL_TRACE is set (to anything but 0) or enabled here.
 * The last 4096 calls are kept. */
void ccl_set_trace(int enabled);
/* Copies up to max_records of the newest records, oldest first, into out
 * (out == NULL: returns how many are held). */
size_t ccl_trace_read(ccl_trace_record_t *out, size_t max_records);
void ccl_trace_clear(void);

/* ------------------------------------------------------------------ */
/* Settings (host only; no GPU needed)                                 */
/* ------------------------------------------------------------------ */

/* Library-wide settings, read from the environment once, on first use, and
 * replaced by the setters below (Collective Communication, libraries section:
 * NCCL is steered by environment variables such as NCCL_ALGO; bucket fusion
 * section: DDP's bucket_cap_mb, 25 MB by default).
 *   CCL_MODE=fused | step (any case): every call that takes a mode argument
 *     (AllReduce, ReduceScatter, AllGather, Broadcast, Reduce, Gather,
 *     Scatter, AllToAll(v), bucket AllReduce) runs in that mode whatever it
 *     passes, so that a whole program can be re-run with the ring executed
 *     step by step (same bits, slower) without changing its calls.  Unset or
 *     empty: each call's own argument.  A mode argument that is not a valid
 *     ccl_mode_t is still rejected.  Trace records show the mode that ran.
 *   CCL_BUCKET_MB=<MiB>, a positive decimal number (e.g. 25 or 0.5): the
 *     bucket size of ccl_bucket_allreduce and ccl_bucketer_create calls that
 *     pass bucket_bytes = 0; at least 4 bytes, at most 1 TiB.
 *   CCL_HOST_PATH=staged|direct: how ccl_allreduce_host moves its buffers.
 *     staged (the default): slices go through the caller's work buffer.
 *     direct: when every buffer is page-locked host memory that the device
 *     can address (cudaHostAlloc, cudaHostRegister), one fused launch reads
 *     and writes them in place over the host link; other memory is staged.
 *     ccl_set_host_path replaces it.
 *   CCL_TRACE, CCL_CHECK: ccl_set_trace, ccl_set_check.
 * A value that cannot be read is ignored (the default stays) with one line on
 * stderr.  The settings are process-wide and may be changed at any time; a
 * call uses the values current when it is made. */
typedef struct {
    int mode_override;           /* -1: none; else CCL_MODE_FUSED or CCL_MODE_STEP */
    int trace;                   /* 1 when call tracing is on */
    int check;                   /* 1 when automatic result checks are on */
    int host_path;               /* CCL_HOST_PATH_STAGED or CCL_HOST_PATH_DIRECT */
    size_t default_bucket_bytes; /* the bucket size that bucket_bytes = 0 selects */
} ccl_config_t;

/* The current settings (CCL_ERR_INVALID_ARG for a NULL out). */
ccl_status_t ccl_get_config(ccl_config_t *out);
/* mode: CCL_MODE_FUSED or CCL_MODE_STEP forces that mode; -1 removes the
 * override (CCL_MODE is then no longer consulted).  Anything else:
 * CCL_ERR_INVALID_ARG, nothing changed. */
ccl_status_t ccl_set_mode_override(int mode);
/* bytes >= 4 sets the default bucket size; 0 restores 25 MiB
 * (CCL_DEFAULT_BUCKET_BYTES); 1 to 3: CCL_ERR_INVALID_ARG, nothing changed. */
ccl_status_t ccl_set_default_bucket_bytes(size_t bytes);
/* ccl_allreduce_host's path: CCL_HOST_PATH_STAGED (through the work buffer)
 * or CCL_HOST_PATH_DIRECT (in place over the host link when every buffer
 * allows it, else staged).  Anything else: CCL_ERR_INVALID_ARG, nothing
 * changed. */
#define CCL_HOST_PATH_STAGED 0
#define CCL_HOST_PATH_DIRECT 1
ccl_status_t ccl_set_host_path(int path);

/* ------------------------------------------------------------------ */
/* Planner (host only; no GPU needed)                                  */
/* ------------------------------------------------------------------ */

/* Chunk partition of `count` elements over nranks: off[c], len[c] (HOST arrays
 * of nranks entries, written by the call). */
ccl_status_t ccl_plan_chunks(size_t count, int nranks, size_t *off, size_t *len);

/* Ring step table, HOST array of 2*(nranks-1)*nranks*3 int32 laid out
 * [phase][s][rank] = {send chunk, recv chunk, source rank}; phase 0 is the
 * ReduceScatter phase, phase 1 the AllGather phase. */
ccl_status_t ccl_plan_ring_schedule(int nranks, int32_t *table);

/* Bucket boundaries of the reversed tensor stream: writes min(nbuckets,
 * max_buckets)+1 stream offsets into starts (bucket b covers
 * [starts[b], starts[b+1])) and the bucket count into *nbuckets. */
ccl_status_t ccl_plan_buckets(const size_t *numels, int ntensors, size_t bucket_elems, size_t *starts,
                              size_t max_buckets, size_t *nbuckets);

/* AllToAllv displacements: sdispl[i*N+j] = elements before block j in
 * send[i]; rdispl[j*N+i] = elements before block i in recv[j]. */
ccl_status_t ccl_plan_alltoallv(int nranks, const size_t *counts, size_t *sdispl, size_t *rdispl);

/* Bytes one rank would put on a link for `count` elements under a
 * compressor: INT8 block: count + 4 * ceil(count / block) (codes plus fp32
 * scales, 4b/(b+4) times fewer than fp32: 3.88 at b = 128); THRESHOLD:
 * ceil(count / 8).  TOPK depends on k: ccl_plan_topk_bytes (CCL_ERR_INVALID_ARG
 * here). */
ccl_status_t ccl_plan_compressed_bytes(size_t count, ccl_compressor_t comp, int block, size_t *bytes);

/* Slices of ccl_allreduce_host for these arguments: writes up to max_slices
 * (off, len) pairs, in elements of every rank's buffer, and the total number
 * into *nslices (off/len may be NULL to ask for the number only).  The slices
 * tile [0, count) in order; each is at most the stage length
 * floor(work_bytes / (3 * nranks * element size)) rounded down to a multiple
 * of 256 elements, starts on a multiple of 256, and they grow from 1/16 of the
 * stage length at the start and shrink the same way at the end. */
ccl_status_t ccl_plan_host_slices(size_t count, int nranks, ccl_dtype_t dtype, size_t work_bytes, size_t *off,
                                  size_t *len, size_t max_slices, size_t *nslices);

/* Arena layout: per-rank stride (bytes_per_rank rounded up to `align`, a power
 * of two >= 256) and total bytes for nranks rank buffers in one allocation. */
ccl_status_t ccl_arena_layout(int nranks, size_t bytes_per_rank, size_t align, size_t *stride, size_t *total);

/* ------------------------------------------------------------------ */
/* Misc                                                                */
/* ------------------------------------------------------------------ */

const char *ccl_status_string(ccl_status_t status);
int ccl_version(void);

/* Number of kernels this library has enqueued since it was loaded (host-side
 * counter, for accounting; thread-safe). */
unsigned long long ccl_launch_count(void);

/* Per-rank traffic of the step-by-step mode (Lesson 3, reference solution:
 * every rank counts what it sends, and an AllReduce moves 2(N-1)K/N elements
 * per rank when N divides K).  sent[j] (HOST array of nranks entries) receives
 * the elements rank j has sent in the ring steps that this host thread's
 * step-mode calls launched since the last reset: the ReduceScatter and
 * AllGather steps of AllReduce, ReduceScatter, AllGather, Reduce and bucket
 * AllReduce, and ccl_reduce_scatter_step_static.  At ReduceScatter step s
 * rank j sends chunk (j - s) mod N, at the AllReduce's AllGather step s chunk
 * (j + 1 - s) mod N, and at the AllGather entry point's step s chunk
 * (j - s) mod N (the lengths of the call's chunk partition).  Copies outside
 * the ring (placing ReduceScatter's results, Broadcast's chain, the pairwise
 * AllToAll) are not counted, nor is anything in fused mode.  reset != 0 zeroes
 * the counters after reading.  Host only; CCL_ERR_INVALID_ARG for nranks
 * outside [1, CCL_MAX_RANKS] or a NULL sent. */
ccl_status_t ccl_step_sent(int nranks, unsigned long long *sent, int reset);

/* Frees the library's cached device workspace on the current device (used by
 * step-mode ReduceScatter, Reduce and bucket AllReduce) and forgets the cached
 * address of ccl_reduce_scatter_step_static's fixed array there (the array
 * itself stays).  Safe to call at any time when no call of this library is in
 * flight; call it after a cudaDeviceReset, before the next call on that
 * device, since the reset invalidates both. */
ccl_status_t ccl_finalize(void);

#ifdef __cplusplus
}
#endif

#endif /* CCL_H */
