/*
 * zero.h -- C ABI of libzero.so: one data-parallel rank's share of a ZeRO
 * (Zero Redundancy Optimizer, arXiv 1910.02054) mixed-precision training step,
 * on one AMD Instinct MI355X (gfx950).
 *
 * The operation, as the pages on ZeRO describe it:
 *   - every rank keeps only its own block of the training state for the long
 *     term (ZeRO mind-map page, paperbridge.wiki, section "shrink the problem:
 *     four GPUs": GPU 1 keeps block A, GPU 2 block B, and so on);
 *   - after backward, gradients are merged across ranks and split again so
 *     that each rank keeps the part it owns (same page, glossary entry
 *     "reduce-scatter", and the section on how a GPU that keeps a quarter of
 *     the state computes); the owner updates that part with mixed-precision
 *     Adam, whose state is 16-bit parameters plus fp32 master weights, first
 *     and second moments (ZeRO concept page, papers.lqhl.me, section "why it
 *     is needed");
 *   - parameters are exchanged so every rank briefly holds them in full
 *     (glossary entry "all-gather"); in Stage 3 this happens per layer, in
 *     forward/backward order, and the copy is freed afterwards (concept page,
 *     "three stages" table);
 *   - collectives run over buckets (concept page, design trade-off 1).
 *
 * On one GPU the N_d ranks are simulated: their gradient contributions are
 * resident buffers, and this library computes the arithmetic of reduce-scatter
 * for the owned partition, the Adam update, and the local layout of
 * all-gather.  No inter-GPU transfer happens here.
 *
 * Conventions for every entry point:
 *   - Device pointers are HIP device addresses owned by the caller.  The
 *     library never allocates device memory.
 *   - Host pointer arrays are read before the call returns and not kept.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Work is enqueued
 *     asynchronously; no call synchronises.  The caller keeps every buffer
 *     alive until the stream has drained.
 *   - Arguments are checked before anything is launched.  On a failed check
 *     nothing is launched and a negative zero_status is returned; the text of
 *     the last failure on the calling thread is available from
 *     zero_last_error().  The library never aborts, never prints, and lets no
 *     C++ exception cross the ABI.
 *   - Element offsets and counts are int64.  "16-bit" means ZERO_F16 or
 *     ZERO_BF16.  Buffers must be aligned to their element size.  When every
 *     base address is 16-byte aligned, the step and the reduction run the
 *     vector kernel on each piece of the shard whose offsets are multiples
 *     of 4 elements, after at most 3 leading elements; other pieces run an
 *     element kernel with the same arithmetic.
 */
#ifndef ZERO_H_
#define ZERO_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define ZERO_API __attribute__((visibility("default")))
#else
#define ZERO_API
#endif

/* Largest number of simulated ranks one fused launch reads directly. */
#define ZERO_MAX_RANKS 128

typedef struct zero_plan_s* zero_plan_t;

typedef enum zero_dtype { ZERO_F32 = 0, ZERO_F16 = 1, ZERO_BF16 = 2 } zero_dtype;

typedef enum zero_status {
  ZERO_OK = 0,
  ZERO_EINVAL = -1,          /* bad argument: null, range, alignment, overlap */
  ZERO_EUNSUPPORTED = -2,    /* valid but not supported (dtype pair, N_d) */
  ZERO_ENOMEM = -3,          /* host allocation failed */
  ZERO_EHIP = -4             /* a HIP launch failed; see zero_last_error() */
} zero_status;

/* Adam hyper-parameters, as decimal values.  The step's fp32 constants are
 * computed from them in fp64 and rounded once to fp32: beta1, 1-beta1, beta2,
 * 1-beta2, 1-beta1^t, 1-beta2^t (pow), lr, eps, grad_scale. */
typedef struct zero_adam_hyper {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double grad_scale;   /* multiplies the rank sum; 1/N_d gives the mean */
} zero_adam_hyper;

/* The N_d ranks' gradient contributions for the owner's partition.
 * ptrs[q] is rank q's buffer, either
 *   is_full[q] == 0: a compact shard-local slice of shard_total elements
 *                    (what reduce-scatter hands the owner; Stage 2 and 3), or
 *   is_full[q] == 1: rank q's whole padded flat gradient buffer of psi_pad
 *                    elements, read at the owner's ranges (Stage 1, where
 *                    gradients stay replicated).
 * is_full may be NULL (all compact).  Gradients are read only. */
typedef struct zero_grad_src {
  int32_t dtype;             /* ZERO_F16 or ZERO_BF16 */
  int32_t n;                 /* must equal the plan's n_d */
  const void* const* ptrs;   /* host array of n device pointers */
  const uint8_t* is_full;    /* host array of n flags, or NULL */
} zero_grad_src;

/* Library version: major * 10000 + minor * 100 + patch. */
ZERO_API int32_t zero_version(void);

/* Text of the last non-OK status returned on the calling thread ("" if none). */
ZERO_API const char* zero_last_error(void);

/*
 * zero_plan -- layout of the flat buckets and of every rank's shard.
 * Follows the mind-map page's four-GPU example (rank i owns the i-th
 * contiguous block) and the concept page's buckets.
 *
 *   psi          total parameters; must equal the sum of tensor_numel.
 *   n_d          simulated data-parallel ranks, >= 1.
 *   tensor_numel host array of n_tensors sizes (>= 0), in list order.
 *   bucket_cap   elements per bucket; 0 = one bucket.  Tensors are taken in
 *                list order and never split; a new bucket starts when the next
 *                tensor would push a non-empty bucket past the cap, so a tensor
 *                larger than the cap sits alone.
 *   shard_align  elements, >= 1.  Each bucket is zero-padded at its end to a
 *                multiple of n_d * shard_align, so every rank's slice
 *                S_b = padded_b / n_d is a multiple of shard_align.
 *   out          receives the plan (host memory, immutable, owned by the caller
 *                until zero_plan_destroy).  A plan may be shared by concurrent
 *                calls.
 * The padded layout must satisfy psi_pad * 4 <= INT64_MAX (fp32 buffers stay
 * byte-addressable in int64).
 * Rank r owns [flat_off_b + r*S_b, flat_off_b + (r+1)*S_b) of bucket b; its
 * shard is the concatenation of those ranges over buckets (shard_total
 * elements), bucket b's part starting at shard_off_b.
 * Errors: EINVAL for n_d < 1, shard_align < 1, bucket_cap < 0, n_tensors < 0,
 * negative sizes, sizes not summing to psi, a null pointer, or a padded
 * layout beyond that bound; ENOMEM.
 */
ZERO_API zero_status zero_plan(int64_t psi, int32_t n_d, const int64_t* tensor_numel, int32_t n_tensors,
                      int64_t bucket_cap, int32_t shard_align, zero_plan_t* out);

ZERO_API void zero_plan_destroy(zero_plan_t plan);

/* Plan queries.  Any output pointer may be NULL.  EINVAL on a null plan or an
 * index out of range. */
ZERO_API zero_status zero_plan_info(zero_plan_t plan, int64_t* psi_pad, int64_t* shard_total,
                           int32_t* n_buckets, int32_t* n_d);
ZERO_API zero_status zero_plan_bucket(zero_plan_t plan, int32_t b, int64_t* flat_off, int64_t* numel,
                             int64_t* padded, int64_t* shard_numel, int64_t* shard_off);
ZERO_API zero_status zero_plan_tensor(zero_plan_t plan, int32_t t, int32_t* bucket, int64_t* flat_off);

/*
 * zero_flatten_workspace_bytes -- device workspace zero_flatten needs for this
 * plan.  Always 0: every copy table travels in the kernel arguments (split
 * over several launches when a plan has many tensors), so flatten needs no
 * device memory of its own.  Kept so that callers can size a workspace
 * without knowing that.
 */
ZERO_API size_t zero_flatten_workspace_bytes(zero_plan_t plan);

/*
 * zero_flatten -- pack the ragged tensor list into the padded flat buckets
 * (concept page, design trade-off 1: collectives run over buckets).
 *   tensors    host array of n_tensors device pointers; tensors[t] holds
 *              tensor_numel[t] contiguous elements (may be NULL when that is 0).
 *   dt         element type of tensors and flat (ZERO_F32, ZERO_F16, ZERO_BF16).
 *   flat       device buffer of psi_pad elements.  Tensor t lands at its plan
 *              offset; every padding element is written as zero.
 *   workspace, ws_bytes  device workspace of zero_flatten_workspace_bytes()
 *              bytes; may be NULL and 0 (the size is 0).  Not touched.
 * A bit copy.  Errors: EINVAL for nulls, misaligned pointers, or flat
 * overlapping a tensor.
 */
ZERO_API zero_status zero_flatten(zero_plan_t plan, const void* const* tensors, zero_dtype dt, void* flat,
                                  void* workspace, size_t ws_bytes, void* stream);

/*
 * zero_shard_reduce -- the arithmetic of reduce-scatter for the owner's
 * partition (mind-map page, glossary entry "reduce-scatter").
 *   out[j] = ((g_0[j] + g_1[j]) + ... + g_{n_d-1}[j]) * f32(grad_scale)
 * for every j of the owner's shard (padding included), in fp32, ranks folded
 * in the fixed order 0..n_d-1 whatever `rank` is.
 *   rank   owning rank, 0 <= rank < n_d.
 *   src    the n_d contributions (see zero_grad_src).
 *   out    device fp32 buffer of shard_total elements (shard-local layout).
 * Any n_d is supported (ranks beyond ZERO_MAX_RANKS are folded by further
 * launches that continue from `out`, which keeps the same order).  Stores may
 * be held for a device-wide write window (zero_set_write_window); the result
 * never depends on it.
 * Errors: EINVAL for a bad rank, src->n != n_d, nulls, misalignment, out
 * overlapping a gradient buffer; EUNSUPPORTED for a non-16-bit dtype.
 */
ZERO_API zero_status zero_shard_reduce(zero_plan_t plan, int32_t rank, const zero_grad_src* src,
                                       double grad_scale, float* out, void* stream);

/*
 * zero_adam_step -- the owner's mixed-precision Adam update of its shard
 * (concept page, "why it is needed": fp32 master weights, first and second
 * moments, 16-bit parameters), fused with the reduction above and with the
 * local half of all-gather.  The update rule is the textbook Adam (Kingma &
 * Ba 2015, Algorithm 1), one fp32 operation per line, no FMA:
 *     g  = reduced gradient (as zero_shard_reduce computes it)
 *     m  = b1*m + c1*g            v = b2*v + c2*(g*g)
 *     mh = m / bc1                vh = v / bc2
 *     w  = w - lr * (mh / (sqrt(vh) + eps))
 *     p  = round-to-nearest-even 16-bit value of w
 *   rank        owning rank, 0 <= rank < n_d.
 *   hp          hyper-parameters (host struct).
 *   t           step number, >= 1 (bias corrections use beta^t).
 *   slices      the n_d gradient contributions (fused path, n_d <=
 *               ZERO_MAX_RANKS), or NULL to read `reduced` instead.
 *   reduced     device fp32 buffer of shard_total elements from
 *               zero_shard_reduce (grad_scale is then not applied again);
 *               ignored when slices is non-NULL.
 *   master, m, v  device fp32 buffers of shard_total elements, updated in
 *               place; they must not overlap each other, param_dst or any
 *               gradient buffer.
 *   param_dst   device 16-bit buffer receiving the updated parameters:
 *               dst_is_full != 0: the full flat parameter buffer (psi_pad
 *               elements), written only at the owner's ranges (Stage 1/2);
 *               dst_is_full == 0: the rank's resident parameter shard
 *               (shard_total elements, Stage 3).
 *   param_dt    ZERO_F16 or ZERO_BF16.
 * With slices, the kernel may hold its stores for a device-wide write window
 * (zero_set_write_window); the results never depend on it.
 * Performance: slices written just before the step with ordinary cached
 * stores slow it by 15-17% on MI355X; written with non-temporal stores (as
 * zero_shard_reduce, zero_flatten and zero_gather_pack write their outputs)
 * they cost nothing.  A producer of the slices should store them
 * non-temporally; where it cannot, zero_set_warm_read(1) recovers most of
 * the loss (3.14-3.22 -> 2.79-2.89 ms for 7.5B at N_d = 64).  Where the
 * slices sit matters too: every wave reads the same offset of all n_d slices
 * at once, and slices a power of two apart (say 256 MiB) put those reads on
 * the same HBM channels, which costs the step 4-6%; staggering them by 1-4
 * KiB, or packing them back to back, avoids it.  For about a second after a
 * large release of device memory (about 1 s per 30 GB, e.g. an emptied
 * allocator cache) the step runs 2-5% slower; keep its buffers allocated
 * from step to step.
 * Errors: EINVAL for a bad rank, t < 1, nulls, misalignment, src->n != n_d,
 * overlapping outputs; EUNSUPPORTED for non-16-bit types or for the fused
 * path with n_d > ZERO_MAX_RANKS (use zero_shard_reduce, then reduced).
 */
ZERO_API zero_status zero_adam_step(zero_plan_t plan, int32_t rank, const zero_adam_hyper* hp, int64_t t,
                           const zero_grad_src* slices, const float* reduced, float* master,
                           float* m, float* v, void* param_dst, zero_dtype param_dt,
                           int32_t dst_is_full, void* stream);

/*
 * zero_gather_pack -- the local layout of all-gather: materialise the full
 * flat buffer from all n_d shards (mind-map page, glossary entry
 * "all-gather"; Stage 3 materialises one layer at a time, concept page,
 * "three stages" table).
 *   shards  host array of n_d device pointers, each shard_total elements.
 *   dt      element type (ZERO_F32, ZERO_F16, ZERO_BF16).
 *   full    device buffer of psi_pad elements; rank q's part of bucket b goes
 *           to [flat_off_b + q*S_b, flat_off_b + (q+1)*S_b).
 * A bit copy.  Errors: EINVAL for nulls, misalignment, full overlapping a shard.
 */
ZERO_API zero_status zero_gather_pack(zero_plan_t plan, const void* const* shards, zero_dtype dt, void* full,
                             void* stream);

/*
 * zero_reshard -- re-lay out a sharded per-element state for a different
 * data-parallel degree or bucketing: the shard of rank dst_rank under dst_plan,
 * assembled from all shards under src_plan.  The sharded optimizer state must
 * survive a change of parallel degree -- a rank-local checkpoint restored at
 * another N_d (concept page, design trade-off 4 and the checklist item on
 * restoring rank-local shards after the parallel degree changes).
 *   src_plan, dst_plan  plans over the SAME tensor list (sizes, order); n_d,
 *               bucket_cap and shard_align may differ.
 *   dst_rank    0 <= dst_rank < dst n_d.
 *   src_shards  host array of src n_d device pointers, each src shard_total
 *               elements (shard-local layout).
 *   dt          element type (ZERO_F32 for master/m/v, 16-bit for params).
 *   dst_shard   device buffer of dst shard_total elements: every real element
 *               is copied from the source rank that owns the same tensor
 *               element; padding is written as zero.
 * A bit copy.  Errors: EINVAL for nulls, different tensor lists, a bad rank,
 * misalignment, or dst_shard overlapping a source shard.
 */
ZERO_API zero_status zero_reshard(zero_plan_t src_plan, zero_plan_t dst_plan, int32_t dst_rank,
                                  const void* const* src_shards, zero_dtype dt, void* dst_shard,
                                  void* stream);

/*
 * zero_set_write_window -- scheduling of the stores of zero_shard_reduce and
 * of the fused zero_adam_step (not an operation of the pages: a tuning knob of
 * this library; results are bit-identical whatever it is set to).
 * The fused step reads about ten bytes of gradient for each byte it writes.
 * With a write window, a wave whose results are ready holds its stores until
 * the GPU's constant-rate real-time counter is within the first open_ticks of
 * a period_ticks-long period, and a wave about to issue its first gradient
 * loads waits until that opening has passed, so the device's writes reach HBM
 * in bursts rather than as a thin stream between the reads.  A tick is one count of
 * that counter at the rate the device reports as hipDeviceAttributeWallClockRate
 * (100 MHz on MI355X: 10 ns).
 *   period_ticks  -1: automatic (the default): the library picks the window
 *                 per launch from the rank count, the launch size, the
 *                 kernel's occupancy and the counter's rate, and uses none for
 *                 small launches;
 *                  0: no window, stores issue as soon as results are ready;
 *                 1..100000: this period for every fused or reduce launch.
 *   open_ticks    1..period_ticks when period_ticks > 0; ignored otherwise.
 * Scope: this sets the PROCESS-WIDE DEFAULT, read by launches issued after the
 * call on every stream that has no setting of its own
 * (zero_set_stream_write_window).  The window assumes the step has HBM to
 * itself while it runs; beside other memory-heavy work (a collective or a
 * copy on another stream) it gains little or nothing, and a stream whose step
 * runs so can turn its own window off with
 * zero_set_stream_write_window(stream, 0, 0) rather than change the default
 * for everyone (measured with a concurrent copy: from 1.2% faster to no
 * difference).  Safe to call from any thread.  Adam from a `reduced`
 * buffer, the element-wise (unaligned) kernels and the copy kernels never
 * wait.
 * Errors: EINVAL for values outside these ranges (the setting is unchanged).
 */
ZERO_API zero_status zero_set_write_window(int64_t period_ticks, int64_t open_ticks);

/*
 * zero_set_warm_read -- a read of the step's own buffers just before it
 * (not an operation of the pages: a tuning knob of this library; results are
 * bit-identical whether it is on or off).  With enable = 1, every fused
 * zero_adam_step and every zero_shard_reduce that reads at least 1 GiB of
 * gradients first reads up to 256 MiB of its fp32 state (master, then m, then
 * v) or of its fp32 output with ordinary cached loads, on the same stream,
 * storing nothing.  MI355X's 256 MB memory-side
 * Infinity Cache keeps the last lines written with ordinary stores dirty;
 * when the gradient slices were just written that way (as a collective or a
 * backward kernel may write them), their write-backs otherwise fall among the
 * step's reads and cost it 15-17% (7.5B, N_d = 64).  The warm-up read moves them
 * before the step: measured, the step is then ~11% faster (7.5% for a Stage-3
 * layer, 3% for 13B at N_d = 16), and the reduction ~11%.  When the slices are
 * already clean (written non-temporally, as zero_shard_reduce and the copies
 * write) it costs the step 1-2% and the reduction 2%.  enable = 0 (the
 * default): no warm-up read.  The buffers read must be 16-byte aligned for it
 * to run.  Process-wide; read by calls issued
 * after it, from any thread.  Errors: EINVAL for any other value.
 */
ZERO_API zero_status zero_set_warm_read(int32_t enable);

/*
 * zero_set_stream_write_window -- the same setting for launches on one
 * stream only; it takes precedence over the process-wide default for every
 * zero_shard_reduce and fused zero_adam_step call issued on that stream
 * afterwards, from any thread.
 *   stream        the hipStream_t the calls are issued on (NULL = the default
 *                 stream).
 *   period_ticks  -2: remove the stream's setting (the default applies
 *                 again); -1: automatic; 0: no window; 1..100000: as above.
 *   open_ticks    as above.
 * The library keeps only the stream handle (host memory); remove the setting
 * before destroying the stream if its handle may be reused.  Safe to call
 * from any thread.  Errors: EINVAL for values outside these ranges (the
 * setting is unchanged); ENOMEM.
 */
ZERO_API zero_status zero_set_stream_write_window(void* stream, int64_t period_ticks, int64_t open_ticks);

/* ------------------------------------------------------------------------
 * Operators at the two ends of the model whose step the calls above take:
 * the vocabulary table's lookup and gradient, which read and write the flat
 * buffers a plan lays out, dropout, and the paired preference loss with the
 * gradient of its logits.  They are not operations of the pages.
 *
 * The conventions above hold for them too: nothing is allocated, nothing
 * synchronises, every table travels in the kernel arguments, and no launch
 * depends on memory that an earlier call left behind, so that every call can
 * be captured into a graph.  A workspace may be reused by the next call on
 * the same stream; two calls that can run at once (two streams, two graphs
 * replayed beside each other) need one each.  The calls are issued to the
 * current device, which has to be the one of the buffers and of the stream.
 * A call whose work exceeds one launch (2^32 work items) issues several.
 * Sums, softmax statistics and norms are held in fp32 or more and are taken
 * in an order that the sizes, the ids and the alignment of the buffers fix, so
 * that a call repeated on the same buffers gives the same bits.
 *
 * Integers in device memory (tokens, labels, offsets) cannot be checked on
 * the host.  Each kernel checks them itself: an id outside its range is
 * treated as a padding id, as each entry says, and never read or written
 * through.
 * --------------------------------------------------------------------- */

typedef enum zero_itype { ZERO_I32 = 0, ZERO_I64 = 1 } zero_itype;

/* Which elements a dropout keeps: a function of these numbers and of the
 * element's position alone, so that the backward pass asks for the same mask
 * again and no mask is stored.
 *   key = seed, then for f in (site, step): key = mix64((key ^ f) + GAMMA)
 *   element e takes the 16 bits at position (e mod 4) of
 *   mix64(key + (e div 4 + 1) * GAMMA), lowest bits first
 *   and is kept where they are >= cut = round-half-even(p * 65536)
 * mix64 and GAMMA are SplitMix64's (Steele, Lea & Flood, OOPSLA 2014).  p is
 * thereby rounded to a multiple of 2^-16; kept elements are multiplied by
 * 65536 / (65536 - cut), which keeps the mean exact. */
typedef struct zero_drop {
  double p;                /* share dropped, in [0, 1]; 1 drops everything */
  uint64_t seed;           /* e.g. one per run and rank */
  uint64_t site;           /* which dropout of the model */
  uint64_t step;           /* training step */
  const uint64_t* step_dev;/* device address read when the kernel runs, in
                              place of step (a captured graph then takes
                              another mask at each replay), or NULL */
  int64_t first;           /* e of the call's first element, >= 0 (a rank that
                              holds a piece of a tensor passes where it
                              starts) */
} zero_drop;

/*
 * zero_embed -- lookup in a table that is a tensor of the plan.
 *   out[i, c] = (16-bit or fp32 rounding of) table[tokens[i], c] * f
 *   f = fp32(scale * 65536 / (65536 - cut)); a dropped element is 0.
 *   plan, tensor  which tensor of the plan; its numel must be a multiple of
 *               hidden, and it is read as rows of `hidden` elements.
 *   params      the full flat parameter buffer (psi_pad elements), as
 *               zero_adam_step with dst_is_full or zero_gather_pack leaves it.
 *   tokens      device array of n ids; one outside [0, rows) is a padding id:
 *               its output row is zero.
 *   drop        dropout of the output, element i * hidden + c at first + that,
 *               or NULL.
 *   out         n rows of `hidden` elements, out_stride elements apart
 *               (>= hidden; what lies between rows is left as it was).
 * Errors: EINVAL for nulls, a tensor index out of range, hidden < 1 or not
 * dividing the tensor, a negative n, a short stride, misalignment, p outside
 * [0, 1], an f that is not finite, or out overlapping params or tokens; EUNSUPPORTED for more than
 * 2^31 - 2 rows or hidden above 2^24.
 */
ZERO_API zero_status zero_embed(zero_plan_t plan, int32_t tensor, int64_t hidden, const void* params,
                                zero_dtype param_dt, const void* tokens, zero_itype token_it, int64_t n,
                                double scale, const zero_drop* drop, void* out, zero_dtype out_dt,
                                int64_t out_stride, void* stream);

/*
 * zero_token_order -- the positions of n tokens in token order, equal tokens
 * in position order: what zero_embed_grad sums by.  It needs the tokens
 * alone, so that it can run beside the forward pass.
 *   rows        rows of the table; a token outside [0, rows) is a padding id
 *               and goes to the end.
 *   sorted      device int32[n]: the tokens in order, a padding id as `rows`.
 *   order       device int32[n]: the position each came from.
 *   workspace, ws_bytes  device workspace of
 *               zero_token_order_workspace_bytes(n, rows) bytes, 16-byte
 *               aligned.
 * Errors: EINVAL for nulls, misalignment, a negative n, rows < 0, a short
 * workspace or overlapping buffers; EUNSUPPORTED for n above 2^30 or rows
 * above 2^31 - 2.
 */
ZERO_API size_t zero_token_order_workspace_bytes(int64_t n, int64_t rows);
ZERO_API zero_status zero_token_order(const void* tokens, zero_itype token_it, int64_t n, int64_t rows,
                                      int32_t* sorted, int32_t* order, void* workspace, size_t ws_bytes,
                                      void* stream);

/*
 * zero_embed_grad -- the gradient of zero_embed's table: a rank's
 * contribution to zero_shard_reduce or zero_adam_step, written where those
 * read it.
 *   g[r, c] = f * sum over the positions i with tokens[i] == r, ascending,
 *             of keep(i, c) * dy[i, c]            (f as in zero_embed)
 *   The sum is fp32, in an order fixed by n, hidden and the tokens; g is
 *   rounded once.  Neither the plan, rank, accumulate, the types nor the
 *   buffers change that order: an owner's slice holds the bits that the full
 *   buffer holds there.
 *   sorted, order  what zero_token_order wrote for these n tokens.
 *   dy          n rows of `hidden` elements, dy_stride elements apart.
 *   scale, drop what the forward call had (scale may hold a loss scale too).
 *   dst         rank < 0: the full flat gradient buffer (psi_pad elements);
 *               the tensor's range is written, nothing else.
 *               rank >= 0: a compact slice of shard_total elements for that
 *               owner; the part of the tensor that the owner holds is
 *               written, nothing else.  What lies outside that part is not
 *               summed, and its rows of dy are not read.
 *   accumulate  0: every element of that range is written, a row without a
 *               token as zero.  1: g is added to what dst holds (in fp32,
 *               rounded once), for a table that is also the output matrix;
 *               rows without a token are left as they were.
 *   workspace, ws_bytes  zero_embed_grad_workspace_bytes(n, hidden) bytes,
 *               16-byte aligned; it may be the one zero_token_order used.
 * The stores are non-temporal, as zero_adam_step likes its slices.
 * Errors: as zero_embed, and EINVAL for rank >= n_d, accumulate other than 0
 * or 1, a short workspace or overlapping buffers; EUNSUPPORTED for n above
 * 2^30, or where the sums need 2^32 work items or more (n * hidden of about
 * 2^41 and beyond).
 */
ZERO_API size_t zero_embed_grad_workspace_bytes(int64_t n, int64_t hidden);
ZERO_API zero_status zero_embed_grad(zero_plan_t plan, int32_t tensor, int64_t hidden, const int32_t* sorted,
                                     const int32_t* order, int64_t n, const void* dy, zero_dtype dy_dt,
                                     int64_t dy_stride, double scale, const zero_drop* drop, void* dst,
                                     zero_dtype dst_dt, int32_t rank, int32_t accumulate, void* workspace,
                                     size_t ws_bytes, void* stream);

/*
 * zero_dropout -- dropout of n contiguous elements, with an optional residual.
 *   out[e] = residual[e] + (kept ? x[e] * fp32(65536 / (65536 - cut)) : 0)
 * in fp32, rounded once.  A dropped element contributes nothing, whatever x
 * holds there.  The backward pass is the same call on dy without a residual
 * (the residual's own gradient is dy).
 *   x, out      the same element type; out may be x or the residual itself.
 *   residual    the same type, or NULL.
 *   drop        not NULL; p = 0 keeps everything.
 * Errors: EINVAL for nulls, a negative n, misalignment, p outside [0, 1], or
 * out overlapping x or the residual without being it.
 */
ZERO_API zero_status zero_dropout(const void* x, const void* residual, void* out, int64_t n, zero_dtype dt,
                                  const zero_drop* drop, void* stream);

/*
 * zero_token_logp -- log-probability of each row's label.
 *   max[t]  = max_j logits[t, j]
 *   sum[t]  = log sum_j exp(logits[t, j] - max[t])
 *   logp[t] = (logits[t, label[t]] - max[t]) - sum[t]
 *   logits      n rows of `vocab` elements, `stride` elements apart.
 *   labels      device array of n ids; a row whose label lies outside
 *               [0, vocab) is not scored: its logits are not read, and its
 *               logp and stats are 0.
 *   logp        device fp32[n].
 *   stats       device fp32[2 * n]: max[t] and sum[t] of row t, side by side
 *               (kept apart, since their sum in fp32 loses the small one where
 *               logits are large).
 *   workspace, ws_bytes  zero_token_logp_workspace_bytes(n, vocab) bytes,
 *               16-byte aligned (few rows are split over the GPU).
 * The label's own term is added to the others' sum last and in fp64, so that
 * logp, and the label's gradient below, keep their relative accuracy where the
 * label is nearly certain.
 * -inf logits (masked ids) count as probability 0; a row of nothing else, and
 * a row with NaN or +inf, gives logp NaN, as the formula does.
 * Errors: EINVAL for nulls, n < 0, vocab < 1, a short stride, misalignment, a
 * short workspace or overlapping buffers; EUNSUPPORTED for vocab above 2^30 or
 * n above 2^31 - 1.
 */
ZERO_API size_t zero_token_logp_workspace_bytes(int64_t n, int64_t vocab);
ZERO_API zero_status zero_token_logp(const void* logits, zero_dtype dt, int64_t n, int64_t vocab, int64_t stride,
                                     const void* labels, zero_itype label_it, float* logp, float* stats,
                                     void* workspace, size_t ws_bytes, void* stream);

/*
 * zero_preference_loss -- the paired preference loss of n_pairs pairs of
 * sequences (direct preference optimisation), and its derivative by each
 * row's logp.
 *   reward[s] = beta * sum over the scored rows t of sequence s of
 *               (logp[t] - ref_logp[t])
 *   h_i       = reward[i] - reward[n_pairs + i]
 *   pair_loss[i] = -(1 - smoothing) log sigmoid(h_i) - smoothing log sigmoid(-h_i)
 *   loss      = mean of pair_loss (0 for no pairs)
 *   coef[t]   = grad_scale * d loss / d logp[t]
 * The sums over a sequence are fp64.
 *   offsets     device array of 2 * n_pairs + 1 row numbers, ascending:
 *               sequence s holds the rows [offsets[s], offsets[s + 1]), the
 *               chosen ones first, then the rejected ones in the same order.
 *               Row numbers are held to [0, n].  An empty sequence has
 *               reward 0.
 *   labels, vocab  as in zero_token_logp: a row whose label lies outside
 *               [0, vocab) counts for nothing, whatever its logp and ref_logp
 *               hold, and its coef is 0.  labels may be NULL: every row
 *               counts.
 *   logp, ref_logp  device fp32[n]; ref_logp may be NULL (zero).
 *   grad_scale  loss scale of the backward pass, 1 for none; zero_adam_step's
 *               grad_scale takes it out again.
 *   loss[1], pair_loss[n_pairs], rewards[2 * n_pairs], coef[n]  device fp32.
 *               coef of rows in no sequence is 0.
 * Errors: EINVAL for nulls, negative sizes, smoothing outside [0, 1], a
 * non-finite beta or grad_scale, beta * grad_scale / n_pairs beyond fp32,
 * misalignment or overlapping buffers;
 * EUNSUPPORTED for n_pairs above 2^29 or n above 2^31 - 1.
 */
ZERO_API zero_status zero_preference_loss(int64_t n_pairs, const void* offsets, zero_itype offset_it, int64_t n,
                                          const void* labels, zero_itype label_it, int64_t vocab,
                                          const float* logp, const float* ref_logp, double beta,
                                          double smoothing, double grad_scale, float* loss, float* pair_loss,
                                          float* rewards, float* coef, void* stream);

/*
 * zero_token_logp_grad -- gradient of the logits from the derivative by logp.
 *   dlogits[t, j] = coef[t] * ((j == label[t]) - exp((logits[t, j] - max[t]) - sum[t]))
 *   stats       what zero_token_logp wrote.
 *   coef        device fp32[n]; a row that is not scored, or whose coef is 0,
 *               gives a row of zeros and its logits are not read.
 *   dlogits     n rows, dl_stride elements apart, the logits' type; it may be
 *               the logits buffer itself (with the same stride).  What lies
 *               between rows is left as it was.
 * Errors: as zero_token_logp, and EINVAL for dlogits overlapping the logits
 * without being them.
 */
ZERO_API zero_status zero_token_logp_grad(const void* logits, zero_dtype dt, int64_t n, int64_t vocab,
                                          int64_t stride, const void* labels, zero_itype label_it,
                                          const float* stats, const float* coef, void* dlogits,
                                          int64_t dl_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_H_ */
