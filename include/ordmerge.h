/*
 * ordmerge.h -- C ABI of the GB300 (sm_103a) stable co-rank merge library
 * (libordmerge.so).
 *
 * (With it, at the end: the ordered selections of a language model, routing
 * to experts, grouping by expert and eviction from a cache.)
 *
 * Operation.  C = merge(A, B): the stable merge of two arrays that are each
 * sorted nondecreasing.  When an element of A equals an element of B, the A
 * element comes first.  The work is split by the co-rank function: for an
 * output rank k, co_rank(k) is the i (with j = k - i) such that A[0..i) and
 * B[0..j) are exactly the first k outputs, i.e. the unique i with
 *     (i == 0 || j == n || A[i-1] <= B[j])  and  (j == 0 || i == m || B[j-1] < A[i]).
 * Sources: "Co-rank Function 實作與 Basic Parallel Merge Kernel"
 * (§Co-rank Function 定義與不變式, §Binary-Search Implementation, §Important on
 * the asymmetric test); "Tiled 與 Circular Buffer Merge Kernel (Memory
 * Coalescing)" (§Block-Level Co-Rank, §Circular Buffer Merge Kernel);
 * "merge_path.cu" (coRank, mergeCpu); "排序 (Sorting) 練習題" (merge-sort
 * stages, stable sort).
 *
 * Conventions for every call below.
 *  - Array arguments are DEVICE pointers (memory the current CUDA device can
 *    address: cudaMalloc, cudaMallocAsync, managed, or a torch CUDA tensor).
 *    The caller owns them.  Element pointers must be 4-byte aligned; for
 *    key/value calls, each value array must have the same address modulo 16
 *    as its key array.  Output arrays must not overlap input arrays.
 *  - Lengths are element counts (int64).  m = 0 or n = 0 is valid (the merge
 *    is then a copy); m + n = 0 is a no-op.
 *  - Inputs must be sorted nondecreasing (signed order for int32, unsigned for
 *    uint32).  This is a precondition and is not checked; on unsorted input
 *    the output is unspecified, but every kernel still terminates.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Merge and sort calls are asynchronous with respect to the
 *    host: they validate, enqueue and return.  Errors raised while the
 *    kernels run surface at the caller's next synchronisation, and in
 *    om_device_error().
 *  - Merges allocate nothing.  The sorts' scratch (their second key and
 *    value buffers) is taken from the library's own stream-ordered memory
 *    pool (created by the first sort on each device) on `stream`
 *    (cudaMallocFromPoolAsync) and freed on the same stream (cudaFreeAsync),
 *    so it is stream-ordered; failure returns OM_ENOMEM.  The pool keeps
 *    freed scratch mapped for later calls, so a device holds up to the
 *    largest scratch any call needed until om_release_scratch().
 *  - No call exits the process or prints.  A failing call returns a status.
 */
#ifndef ORDMERGE_H
#define ORDMERGE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    OM_OK = 0,
    OM_EINVAL = 1,  /* NULL pointer with a nonzero length, negative length,
                       misaligned pointer, overlapping output */
    OM_ERANGE = 2,  /* k outside [0, m + n], or m + n overflows */
    OM_ENOMEM = 3,  /* stream-ordered scratch allocation failed */
    OM_ECUDA = 4,   /* a CUDA runtime call or kernel launch failed */
    OM_EDEVICE = 5  /* a kernel reported an error (om_device_error) */
} om_status;

/*
 * co_rank(k) of A[0..m) and B[0..n): returns i in [max(0, k-n), min(k, m)];
 * the caller derives j = k - i ("Co-rank Function 實作與 Basic Parallel Merge
 * Kernel", §Co-rank Function 定義與不變式: the function returns i only).
 * Runs one search on the device and waits for it: synchronous.  It is
 * ordered after prior work on the legacy default stream only.  Returns the
 * negated om_status (< 0) on error.
 */
int64_t om_corank_i32(int64_t k, const int32_t *A, int64_t m,
                      const int32_t *B, int64_t n);

/*
 * Batched co-rank on the device: i_out[t] = co_rank(ks[t]) for t < count.
 * ks and i_out are device arrays of int64 (each ks[t] in [0, m + n]; an
 * out-of-range k is clamped into that interval).  Asynchronous on `stream`.
 */
om_status om_corank_i32_batch(const int64_t *ks, int64_t count,
                              const int32_t *A, int64_t m,
                              const int32_t *B, int64_t n,
                              int64_t *i_out, void *stream);

/*
 * Grid-level merge-path partition: split[t] = co_rank(min(t * tile, m + n))
 * for t < count, one co-rank search per output tile boundary, run by one
 * warp each (32 probes per round) in a single launch on `stream`
 * ("Tiled 與 Circular Buffer Merge Kernel (Memory Coalescing)",
 * §Block-Level Co-Rank: one co-rank per block's output tile; "Co-rank
 * Function 實作與 Basic Parallel Merge Kernel", §Co-rank Function 定義與不變式).
 * The caller derives j_t = min(t * tile, m + n) - split[t].  split is a
 * device array of count int64 owned by the caller, 8-byte aligned, not
 * overlapping A or B.  tile >= 1 and count >= 0, else OM_EINVAL.  This is
 * the kernel om_merge_i32_noalloc runs before its tile merge; om_merge_i32
 * finds the same splitters inside its tile-merge kernel.  Allocates nothing.
 */
om_status om_partition_i32(const int32_t *A, int64_t m, const int32_t *B,
                           int64_t n, int64_t tile, int64_t count,
                           int64_t *split, void *stream);

/*
 * C[0 .. m+n) = stable merge of int32 A[0..m) and B[0..n); ties take A
 * first.  One launch on `stream`.  A merge that fits in one wave of small
 * CTAs (about 4.2 M outputs on a 152-SM GB300; the one-pass kernel: one
 * output tile per CTA, both windows loaded into shared memory at once and
 * merged by every thread) takes that kernel; a larger one takes the
 * circular-buffer tile-merge kernel, whose CTAs stream their output ranges
 * through shared-memory rings.  In either, two warps of each CTA first find
 * the co-ranks of its output range's two ends (one each).  Allocates
 * nothing.  The environment variable OM_ONE_PASS_MAX (an output count; 0:
 * never) moves the size at which the one-pass kernel stops; setting
 * OM_SUBTILES_PER_RANGE or OM_WAVES selects the tile-merge kernel.  The same
 * holds for om_merge_pairs_u32 and om_merge_keys.
 */
om_status om_merge_i32(const int32_t *A, int64_t m, const int32_t *B,
                       int64_t n, int32_t *C, void *stream);

/*
 * Stable merge of (uint32 key, uint32 value) pairs, comparing keys only
 * (unsigned order); each value travels with its key; ties take A first.
 * Outputs keysC / valsC hold m + n elements.
 */
om_status om_merge_pairs_u32(const uint32_t *keysA, const uint32_t *valsA,
                             int64_t m, const uint32_t *keysB,
                             const uint32_t *valsB, int64_t n,
                             uint32_t *keysC, uint32_t *valsC, void *stream);

/*
 * Stable sort of keys[0..n) (unsigned order), in place, carrying vals along
 * (vals may be NULL for a keys-only sort).  Built only from merges: tiles of
 * 4096 are sorted in shared memory (runs of 16 in registers, then many small
 * merges per thread block through runs of 1024 to 4096), then runs are
 * merged pairwise in co-rank-split passes ("排序 (Sorting) 練習題",
 * merge-sort stages).
 * Equal keys keep their input order.  Needs 4*n (8*n with vals) bytes of
 * stream-ordered scratch.
 */
om_status om_merge_sort_u32(uint32_t *keys, uint32_t *vals, int64_t n,
                            void *stream);

/* Human-readable name of a status (static string). */
const char *om_status_string(int status);

/*
 * Synchronises `stream`, then reads and clears the library's device error
 * word on the current device.  Returns OM_OK, OM_EDEVICE when a kernel
 * recorded an error (for example a shared-memory barrier wait that hit its
 * time limit), or OM_ECUDA.  *detail (if not NULL) receives the raw word.
 */
om_status om_device_error(void *stream, uint32_t *detail);

/* ---- tracing and counters (used by the benchmark) ---------------------- */

/*
 * With tracing on, every kernel launch is bracketed by two CUDA events on its
 * stream.  om_trace_read synchronises those events and returns, for kernel
 * kind `kind` (0 = partition, 1 = tile merge, 2 = block sort, 3 = co-rank
 * batch, 4 = the comparison merges below, 5 = one-pass merge), the number of
 * launches and their summed duration in milliseconds since the last
 * om_trace_reset.
 */
om_status om_trace_enable(int on);
om_status om_trace_reset(void);
om_status om_trace_read(int kind, int64_t *launches, double *total_ms);

/*
 * Returns the scratch the library's pool holds on the current device to the
 * system (waits for the device first).  Later calls map it again as needed.
 */
om_status om_release_scratch(void);

/* Number of kernels this library has launched since load. */
uint64_t om_launch_count(void);

/*
 * Launch planning, host only (no device call): the number of sub-tiles per
 * CTA output range the library uses for one tile-merge launch over `segs`
 * independent merges of at most `seg_len` outputs each (a merge: segs = 1;
 * a late pass of the sort: one segment per pair of runs), with sub-tiles of
 * `subtile` outputs, `bytes_per_output` bytes read plus written per output
 * and `resident_ctas` CTAs running at a time.  Ranges never cross a
 * segment.  The choice minimises  waves x (fixed cost per range + longest
 * range)  over one to eight waves, so that no launch ends on a partial wave
 * of a few CTAs.  The environment variables OM_WAVES (fixed wave count) and
 * OM_SUBTILES_PER_RANGE (fixed result) override it, here and in every call.
 * Returns a value >= 1, or 0 when an argument is not positive.
 */
int64_t om_subtiles_per_range(int64_t segs, int64_t seg_len, int64_t subtile, int64_t bytes_per_output,
                              int64_t resident_ctas);

/* ---- merge without allocating ------------------------------------------ */

/*
 * The pages have no counterpart to this call: it is a library convenience.
 *
 * Same result as om_merge_i32, in two launches that allocate nothing: the
 * partition kernel writes one co-rank splitter per output range to a fixed
 * 64 KiB array that the library keeps in device memory (a file-scope
 * __device__ object, held on every GPU that loads the library until the
 * process exits), and the tile-merge kernel reads them.  (om_merge_i32 now
 * lets each tile-merge CTA find its own splitters, so it allocates nothing
 * either; this call keeps the two-kernel form.)  For callers that cannot
 * allocate device memory on the call path: processes whose device memory is
 * reserved in full by another allocator, and code with latency bounds that
 * must not enter an allocator.
 *
 *  - m + n may be at most 2^30 = 1,073,741,824, a fixed bound of this call
 *    (the array holds 8191 output-range splitters, and ranges are lengthened
 *    as needed to fit); larger merges return OM_ERANGE and launch nothing.
 *  - The first call on each device does a one-time set-up there: it looks up
 *    the device addresses of the array and of the library's error word, sets
 *    the merge kernels' shared-memory limits and queries their occupancy.
 *    None of that allocates device memory (no memory pool is created; only
 *    the sorts make one); make that first call before any stream capture.
 *  - All calls on a device share the array.  Each call's kernels write every
 *    slot they read before reading it, so nothing needs clearing, but calls
 *    whose kernels overlap on the GPU (e.g. on different streams) race on
 *    the array and can produce wrong output: order them on one stream or
 *    with events.
 *  - With tracing off (the default) no call of this function allocates
 *    anything, on the device or the host; argument rules and errors are those
 *    of om_merge_i32.
 */
om_status om_merge_i32_noalloc(const int32_t *A, int64_t m, const int32_t *B,
                               int64_t n, int32_t *C, void *stream);

/* ---- the pages' unstaged merges, for comparison ------------------------- */

/*
 * The two merges that "merge_path.cu" measures, kept to measure what the
 * shared-memory ring design buys on this GPU.  Same result as om_merge_i32
 * (int32, ties take A first); same argument rules and errors.  Not fast paths.
 *
 * om_merge_i32_one_thread: the two-pointer merge run by one device thread
 * (one block of one thread).
 */
om_status om_merge_i32_one_thread(const int32_t *A, int64_t m,
                                  const int32_t *B, int64_t n, int32_t *C,
                                  void *stream);

/*
 * om_merge_i32_slices: one thread per slice of per_thread outputs (blocks of
 * 256 threads); each thread finds the co-ranks of both ends of its slice in
 * global memory, then merges the input intervals between them straight from
 * global memory, with no shared memory ("Co-rank Function 實作與 Basic Parallel Merge Kernel",
 * §Basic Parallel Merge Kernel; "merge_path.cu").  per_thread >= 1, else
 * OM_EINVAL.
 */
om_status om_merge_i32_slices(const int32_t *A, int64_t m, const int32_t *B,
                              int64_t n, int32_t *C, int64_t per_thread,
                              void *stream);

/* ---- other key types and descending order ------------------------------ */

/* Key types of om_merge_keys (element size 4 or 8 bytes). */
typedef enum {
    OM_KEY_I32 = 0, /* int32, signed order */
    OM_KEY_U32 = 1, /* uint32, unsigned order */
    OM_KEY_F32 = 2, /* IEEE binary32, numeric order */
    OM_KEY_I64 = 3, /* int64, signed order */
    OM_KEY_U64 = 4, /* uint64, unsigned order */
    OM_KEY_F64 = 5  /* IEEE binary64, numeric order */
} om_key_type;

typedef enum {
    OM_ASCENDING = 0,  /* inputs and output nondecreasing */
    OM_DESCENDING = 1  /* inputs and output nonincreasing */
} om_order;

/*
 * C[0 .. m+n) = stable merge of the keys A[0..m) and B[0..n) of type
 * `key_type`, both sorted in `order`; ties take A first in either order.
 * The same tile-merge kernel as om_merge_i32, for another element size and
 * comparison.  ("merge_path.cu" runs the method on float
 * keys; the co-rank test of "Co-rank Function 實作與 Basic Parallel Merge
 * Kernel", §Important, with <= and < read in the merge order.)
 *  - Floating-point keys compare by value: -0.0 and +0.0 are equal (so the
 *    A one comes first) and keep their bits.  NaN has no place in a sorted
 *    array; input holding NaN counts as unsorted (output unspecified, every
 *    kernel still terminates).
 *  - A, B and C must be aligned to the key size (4 or 8 bytes) and C must
 *    not overlap A or B.
 *  - An unknown key_type or order is OM_EINVAL.  Other rules and errors are
 *    those of om_merge_i32.
 */
om_status om_merge_keys(int key_type, int order, const void *A, int64_t m,
                        const void *B, int64_t n, void *C, void *stream);

/*
 * Stable sort of keys[0..n) of type `key_type` into `order`, in place,
 * carrying the uint32 vals along (vals may be NULL).  The pass schedule of
 * om_merge_sort_u32 with that type's compare: 4096-key tiles sorted in
 * shared memory, then co-rank-split merge passes ("排序 (Sorting) 練習題",
 * merge-sort stages).  Equal keys (including -0.0 and +0.0) keep their
 * input order in either order.
 *  - keys aligned to the key size.  Values ride only with 4-byte keys
 *    (I32, U32, F32): vals with an 8-byte key type is OM_EINVAL.  vals, if
 *    given, has the same address modulo 16 as keys and does not overlap it.
 *  - Floating-point keys must not hold NaN (unsorted output otherwise; every
 *    kernel still terminates).
 *  - Needs n * key size (plus 4 * n with vals) bytes of stream-ordered
 *    scratch.  Other rules and errors are those of om_merge_sort_u32.
 */
om_status om_merge_sort_keys(int key_type, int order, void *keys,
                             uint32_t *vals, int64_t n, void *stream);

/* ---- ordered selection: routing, grouping, eviction --------------------- */

/*
 * What a language model orders: the experts of a token by their scores, the
 * tokens by their experts, the entries of a cache by the attention they have
 * drawn.  As in the merges, ties go to the earlier (lower) index.  All calls
 * are asynchronous on `stream` and allocate nothing.
 * These calls do not need sorted input.  Their launches are in
 * om_launch_count, but om_trace_read has no kind for them.
 */

/* Value types of logits and attention weights. */
typedef enum {
    OM_VALUE_F32 = 0,
    OM_VALUE_BF16 = 1,
    OM_VALUE_F16 = 2
} om_value_type;

typedef enum {
    OM_SCORE_SOFTMAX = 0, /* s = softmax of the token's logits */
    OM_SCORE_SIGMOID = 1  /* s = 1 / (1 + exp(-logit)) */
} om_score;

/*
 * Routing to experts.  For each of `tokens` rows of `experts` logits (rows
 * row_stride values apart, each row contiguous):
 *   s_e = score of the logits;  c_e = s_e + bias_e  (bias may be NULL);
 *   the experts form `groups` groups of equal size in order, a group's score
 *   is the sum of its group_best (1 or 2) greatest c, and the group_picks
 *   groups of greatest score stay open;
 *   ids = the top_k open experts of greatest c, greatest first;
 *   weights = scale * s of those (without the bias), divided by their sum
 *   when renorm is nonzero.
 * Equal c (and equal group scores) go to the lower index.  ids and weights
 * hold tokens * top_k values.  c is computed in 32 bits; with no bias and
 * group_best = 1 (or one group) the order is taken from the logits
 * themselves, which the rounding of exp cannot tie.
 *  - An expert whose logit is -inf or NaN has no score (softmax does not
 *    count it); that one, and one whose c is -inf or NaN, is never chosen.
 *    A token with fewer than top_k experts left gets id -1 and weight 0 in
 *    the slots left over, a wholly masked one in all of them.
 *  - The renormalised weights come from shifted exponentials: they stay
 *    right when every s underflows.
 *  - The same call on the same GPU repeats bit for bit.  With another number of
 *    tokens a row's sums (softmax's, renorm's) may run in another order: its
 *    weights, and a choice by softmax scores that hangs on the last bit of one,
 *    may then differ by that bit.  Sigmoid scores are the same in every call.
 *  - 1 <= top_k <= group_picks * (experts / groups), groups divides experts.
 *    At most 1024 experts, 32 groups, top_k 32 and 2^32 tokens, else
 *    OM_ERANGE.
 */
om_status om_route_topk(int value_type, const void *logits, int64_t tokens,
                        int64_t experts, int64_t row_stride,
                        const float *bias, int score, int groups,
                        int group_picks, int group_best, int top_k, int renorm,
                        float scale, int32_t *ids, float *weights,
                        void *stream);

/*
 * Gradient of om_route_topk's weights: grad_logits (tokens * experts values
 * of value_type, dense) from grad_weights (tokens * top_k) and the ids that
 * the forward call gave.  The choice of experts is constant, the bias has no
 * gradient.  With g = scale * grad_weights and w the weights over scale:
 *   softmax            s_e * (g_e [e chosen] - sum g w)      for every e
 *   softmax, renorm    w_e * (g_e - sum g w)                 for chosen e
 *   sigmoid            g_e * s_e * (1 - s_e)                 for chosen e
 *   sigmoid, renorm    w_e * (1 - s_e) * (g_e - sum g w)     for chosen e
 * and zero elsewhere.  An id outside [0, experts), or of a logit -inf or NaN,
 * is an empty slot.  The ids of one token must differ.  Limits as above.
 */
om_status om_route_topk_backward(int value_type, const void *logits,
                                 int64_t tokens, int64_t experts,
                                 int64_t row_stride, const int32_t *ids,
                                 const float *grad_weights, int score,
                                 int top_k, int renorm, float scale,
                                 void *grad_logits, void *stream);

/*
 * Stable grouping of n slots by id: order lists the slots by rising id,
 * equal ids in slot order, and slots whose id is outside [0, groups) last;
 * offsets[g] (groups + 1 values) is where id g starts in it, offsets[groups]
 * where the ids outside do; place is the inverse, order[place[i]] = i.
 * What om_merge_sort_u32 on (id, slot) pairs gives, for few distinct ids, in
 * one launch (a cooperative one when it takes several CTAs), with the offsets.
 * n <= 2^31 - 1 and groups <= 1024, else OM_ERANGE.
 */
om_status om_group_by_id(const int32_t *ids, int64_t n, int64_t groups,
                         int32_t *offsets, int32_t *order, int32_t *place,
                         void *stream);

/*
 * Accumulated attention weight per cache entry.  weights holds the attention
 * weights of `queries` queries: value (b, hq, q, i) at b * w_batch + hq *
 * w_head + q * w_query + i.  Each of the kv_heads cache heads serves q_heads
 * / kv_heads consecutive query heads.
 *   out[b][h][i] = decay * score[b][h][i] + sum over the queries and query
 *                  heads of h of weights(b, hq, q, i)   for i < lengths[b],
 *                  0                                    up to `length`.
 * Sums run in 32 bits, by blocks of 128 rows, in an order fixed by the
 * shapes, the strides, the address of weights modulo 16 and the number of SMs:
 * the same call repeats bit for bit, and the same values at other addresses may
 * differ in the last places.  score (NULL: start from zero) and out are rows of
 * `length` floats at b * batch stride + h * head stride; out may be score
 * itself, with the same strides, or share no byte with it (nor its span with
 * that of weights).  lengths (NULL: all `length`) is a device array of batch
 * int32, clamped into [0, length]; nothing past them counts (whole aligned 16
 * bytes are read: up to 15 bytes beside the values that do).  batch * kv_heads,
 * q_heads and queries are at most 65535, strides 2^40, else OM_ERANGE.
 */
om_status om_accumulate_weights(int value_type, const void *weights,
                                int64_t batch, int64_t q_heads,
                                int64_t kv_heads, int64_t queries,
                                int64_t length, int64_t w_batch,
                                int64_t w_head, int64_t w_query,
                                const float *score, int64_t s_batch,
                                int64_t s_head, const int32_t *lengths,
                                float decay, float *out, int64_t o_batch,
                                int64_t o_head, void *stream);

/*
 * The entries of a cache that stay when each row (sequence b, head h) is cut
 * to `budget`: the first `first`, the last `last` and, of those between, the
 * ones of greatest score to fill the budget, equal scores to the lower
 * index.  A row of n = lengths[b] <= budget entries keeps all of them.
 * keep[b][h][0 .. budget) = their indices, rising, then -1; kept[b] =
 * min(n, budget).  A NaN score counts as -inf.  first + last <= budget, else
 * OM_EINVAL.  lengths as in om_accumulate_weights; batch <= 32767 and heads
 * <= 65535, else OM_ERANGE.
 */
om_status om_evict_select(const float *score, int64_t batch, int64_t heads,
                          int64_t length, int64_t s_batch, int64_t s_head,
                          const int32_t *lengths, int64_t budget,
                          int64_t first, int64_t last, int32_t *keep,
                          int32_t *kept, void *stream);

/*
 * One array of a cache for om_evict_gather: entry (b, h, i), entry_bytes
 * long, is at src + b * src_batch + h * src_head + i * src_entry, all in
 * bytes; likewise dst.
 */
typedef struct {
    const void *src;
    void *dst;
    int64_t entry_bytes;
    int64_t src_batch, src_head, src_entry;
    int64_t dst_batch, dst_head, dst_entry;
} om_cache_array;

/*
 * Moves the kept entries of `count` (at most 8) cache arrays (keys, values,
 * scores, ...) together: dst entry (b, h, j) = src entry (b, h, keep[b][h][j])
 * for j < budget, zero bytes where keep is outside [0, length).  `arrays` is
 * a host array, read before the call returns.  No dst may share a byte with a
 * src, another dst or keep, nor between its own entries.  Arrays may lie between
 * each other's rows (keys beside values in one buffer) where their strides are
 * the same; with other strides, and with keep, what counts is the span from the
 * first entry to the last.
 * In place: all arrays together may have dst = src, with the same strides;
 * keep has to rise then, as om_evict_select's does (values are lost
 * otherwise), and entries past the budget keep what they held.
 * Vectors of 16 bytes where every address allows them.  Entry strides are at
 * most 2^30 bytes, others 2^40.
 */
om_status om_evict_gather(const int32_t *keep, int64_t batch, int64_t heads,
                          int64_t budget, int64_t length,
                          const om_cache_array *arrays, int count,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ORDMERGE_H */
