/*
 * reduce.h -- C ABI of libreduce: dense-array reduction on AMD Instinct
 * MI355X (gfx950).
 *
 * Four families of operations:
 *
 *   1. A 1-D fp32 vector reduced to one scalar by sum, max or min, with an
 *      accum mode that folds the old destination value into the result
 *      (TVM TIRx docs, "reduction -> sm100_packed": introduction, section
 *      "What it accepts" -- a 1-D fp32 source and a one-element
 *      destination -- and the table in "How inputs change the algorithm",
 *      row "accum").  The same reduction applied independently to each row
 *      of a row-major matrix is the segmented ("rows") form.
 *
 *   2. A row-major tile reduced column-wise by product to one row
 *      (PTO ISA "TCOLPROD": "Math Interpretation" -- dst[0,j] is the
 *      product of src[i,j] over the R valid rows, for each of the C valid
 *      columns; "Constraints" -- row-major layout, dst and src share the
 *      element type, the column counts agree, and a tile with zero valid
 *      rows or columns returns early).
 *
 *   3. Losses over rows of logits: each row of an fp32, fp16 or bf16 matrix
 *      reduced by its log-sum-exp, the rows joined into a loss, and the
 *      loss's gradient with respect to the matrix: token log-probabilities,
 *      distillation from a teacher's largest logits, a clipped policy loss
 *      and a preference loss.
 *
 *   4. The operators around the output layer whose logits those are: the
 *      root-mean-square norm of its rows with the residual's addition and an
 *      8-bit output, the balance loss of a router of experts, and the cross
 *      entropy of hidden rows against the layer, with no logits of the
 *      caller's, each with its gradient.
 *
 * Conventions shared by every entry point:
 *
 *   - Every pointer is a DEVICE pointer (HBM of the current HIP device).
 *     The caller owns all buffers and must keep them alive until the work
 *     enqueued on `stream` has completed.  The library keeps no pointer
 *     after the call returns.
 *   - Every call is asynchronous with respect to the host: it validates its
 *     arguments, enqueues kernels on `stream` and returns.  `stream` is a
 *     hipStream_t passed as an opaque pointer; NULL means the null stream.
 *     It must belong to the current HIP device, as the buffers must.
 *     Results are visible after the stream is synchronised.
 *   - The return value is a status code (enum red_status).  Errors are
 *     reported synchronously and never abort.  A status other than RED_OK
 *     means nothing was enqueued, except RED_ERR_HIP after a launch, which
 *     reports what hipGetLastError() returned.  Faults raised while a
 *     kernel runs surface at the caller's next synchronisation, as for any
 *     HIP kernel.
 *   - The destination must not overlap the source (not checked).  A
 *     gradient of logits may be written over the logits themselves:
 *     dlogits == logits with equal row strides.
 *   - Empty input (n == 0, rows == 0, R == 0 or C == 0) returns RED_OK,
 *     enqueues nothing and leaves the destination untouched, also under
 *     accum; for column products this is TCOLPROD's early return, and the
 *     empty product 1 is NOT written.  Pointers are not inspected then.
 *   - Floating point follows IEEE-754 with round to nearest even.
 *     Subnormal inputs and results are kept (no flush to zero).
 *   - max / min are IEEE-754-2008 maxNum / minNum: a quiet NaN operand is
 *     ignored; the result is NaN only if every operand is NaN.  When the
 *     extreme is a zero that occurs with both signs, either zero may be
 *     returned.
 *   - The default (non-atomic) entry points are deterministic: for a given
 *     input, device model and library build the result bits never change
 *     between runs.
 *   - Workspace.  The calls that combine per-workgroup partials in a second
 *     kernel (1-D, fused, column and column-product calls, row calls
 *     with very long rows or very few rows, the losses, the norm's gradient
 *     and the balance loss) keep those partials in a
 *     workspace (16 MiB and 128 KiB of counts, which are zero between
 *     calls) the library allocates on the first such call for a
 *     (device, stream) pair and keeps until red_release_workspace.  For
 *     hipStreamPerThread, which names a different stream in every host
 *     thread, the workspace belongs to (device, calling thread).  A call
 *     holds its workspace while it enqueues its kernels, so calls from
 *     several host threads on one stream are ordered by that stream and
 *     never interleave their kernels.  The first call on a stream allocates
 *     device memory and must not be made under HIP graph capture.
 *   - HIP graphs.  A call captured into a graph uses the workspace of its
 *     capture stream at every replay.  Replays must therefore be ordered
 *     with each other and with the calls made on that stream (replaying
 *     on the capture stream does this), and must end before that stream's
 *     workspace is released.
 *   - Thread safety: any host thread may call any entry point.
 *   - Test hooks, read from the environment and meant to be left unset
 *     outside tests: RED_TEST_FAIL_ALLOC=1 makes the creation of a workspace
 *     fail (RED_ERR_NOMEM); RED_TEST_SCRATCH_LIMIT=<bytes>
 *     lowers the static scratch limit of red_sum_max_min_f32_noalloc;
 *     RED_TEST_CUS=<1..65536> replaces the compute-unit count the launch
 *     plans start from (results then stay correct but may differ in their
 *     last bits from the device's own plan).
 */
#ifndef LIBREDUCE_REDUCE_H
#define LIBREDUCE_REDUCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RED_ABI_VERSION 3

/* A hipStream_t, passed as an opaque pointer (NULL: the null stream). */
typedef void* red_stream_t;

enum red_status {
    RED_OK = 0,
    RED_ERR_INVALID = 1, /* null pointer for non-empty input, ld too small,
                            a size whose byte extent overflows size_t, or a
                            number outside the range its argument states */
    RED_ERR_ALIGN = 2,   /* a pointer not aligned to its element size */
    RED_ERR_NOMEM = 3,   /* the per-stream workspace could not be allocated */
    RED_ERR_HIP = 4,     /* the HIP runtime reported an error */
    RED_ERR_SCRATCH = 5  /* red_sum_max_min_f32_noalloc: the grid would need
                            more than the static scratch buffer holds;
                            red_linear_ce_*: the workspace is too small */
};

/* ---------------------------------------------------------------------
 * 1-D fp32 vector -> scalar
 *
 * x      : n fp32 values, 4-byte aligned (16-byte alignment not required).
 * n      : number of elements; any n >= 0 (no minimum length).
 * out    : one fp32 value, 4-byte aligned.
 * accum  : 0 -> *out = reduce(x);  nonzero -> *out = old *out (+|max|min)
 *          reduce(x), with the old value folded in first.
 *
 * sum: the fp32 result lies within 1e-6 * (|old| + sum |x_i|) of the exact
 * sum for the sizes this library is built for (n up to 2^31); it is
 * computed with per-thread 8-wide accumulators, a fixed tree and a
 * fixed-order combine of per-workgroup partials.
 * max / min: exact (order cannot change the result).
 * ------------------------------------------------------------------- */
int red_sum_f32(const float* x, size_t n, float* out, int accum,
                red_stream_t stream);
int red_max_f32(const float* x, size_t n, float* out, int accum,
                red_stream_t stream);
int red_min_f32(const float* x, size_t n, float* out, int accum,
                red_stream_t stream);

/* Fused sum, max and min of one vector from a single read of it: out points
 * to three fp32 values, out[0] = sum, out[1] = max, out[2] = min (under
 * accum each folds its own old value first).  The TVM page's reduction
 * offers these three operators on the same 1-D source ("How inputs change
 * the algorithm", row "op"); computing them together reads x once instead
 * of three times.  Each result is bit-identical to the corresponding
 * red_sum_f32 / red_max_f32 / red_min_f32 result.  out must be 4-byte
 * aligned and must not overlap x. */
int red_sum_max_min_f32(const float* x, size_t n, float* out, int accum,
                        red_stream_t stream);

/* For callers that cannot allocate (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc): red_sum_max_min_f32
 * without any device or host allocation.  Same arguments, results (bit for
 * bit) and errors, and the same two kernels, but the per-workgroup partials
 * (12 bytes per workgroup of the first pass, at most one workgroup per
 * compute unit) live in a 16 KiB static device buffer that the library
 * declares and that each GPU it runs on holds until the process ends.
 * Calls whose grid would need more than 16 KiB of partials (devices of
 * more than 1365 compute units) return RED_ERR_SCRATCH and enqueue nothing.
 * Nothing in the buffer has to start at zero: the first kernel writes
 * every partial the second reads.  Every call on one GPU shares that GPU's
 * buffer, whatever its stream or host thread: calls that overlap in time
 * on one GPU race and give wrong results, so the caller must order them
 * (for example, issue them all on one stream).  The first call on a device
 * looks up the buffer's device address once (hipGetSymbolAddress) and
 * keeps it in a fixed table of 64 devices: on a device of index 64 or more
 * the call returns RED_ERR_HIP and enqueues nothing. */
int red_sum_max_min_f32_noalloc(const float* x, size_t n, float* out, int accum,
                                red_stream_t stream);

/* Single-pass variants: each workgroup folds its partial into *out with
 * one device-scope atomic, as the one-atomic-per-program block reduce in
 * the imxueqiu.com blog post on a Triton vector-sum kernel does (its
 * hand-written C version: warp reduce, shared-memory combine, one atomicAdd
 * by thread 0).  Same arguments and error behaviour as above.  With
 * accum == 0 the library first sets *out to the identity (-0.0 for sum, a
 * quiet NaN for max / min) on `stream`.  sum uses the hardware fp32 atomic
 * add, so its rounding order -- and its last bits -- vary from run to run
 * (same error bound); on gfx950 that atomic keeps subnormal operands and
 * results and the sign of zero, as the other entry points do (a zero sum
 * is -0 only when every term is -0); max / min fold each workgroup's result with one
 * integer atomic max / min on the fp32 bit pattern and are exact (an old
 * NaN under accum is replaced first by compare-and-swap; equal zeros of
 * both signs give +0 for max and -0 for min).  No workspace is used. */
int red_sum_f32_atomic(const float* x, size_t n, float* out, int accum,
                       red_stream_t stream);
int red_max_f32_atomic(const float* x, size_t n, float* out, int accum,
                       red_stream_t stream);
int red_min_f32_atomic(const float* x, size_t n, float* out, int accum,
                       red_stream_t stream);

/* ---------------------------------------------------------------------
 * Segmented rows: out[r] = reduce(x[r*ld .. r*ld + n)) for r < rows
 *
 * x      : row-major fp32 matrix, 4-byte aligned; row r starts at x + r*ld.
 *          Elements between n and ld in a row never affect the result.
 *          Nothing past the last row's n-th element is read; rows of 17
 *          to 64 elements with ld <= 64, or with ld <= 128 and
 *          ld - n <= n / 8, are read as one span, padding included, and
 *          the padding is dropped.
 * rows   : number of rows; n : elements reduced per row; ld : row stride
 *          in elements, ld >= n (RED_ERR_INVALID otherwise).
 * out    : rows fp32 values, 4-byte aligned.
 * accum  : nonzero folds old out[r] into row r's result.
 *
 * Rows of at most 64 elements are reduced one per thread in exactly the
 * single-precision order of the TVM page's "Algorithm" section (8 slots,
 * chunks of 8, leftovers into slot i mod 8, the 8 -> 4 -> 2 -> 1 tree,
 * accum into slot 0 first).  Longer rows are shared by 16, 32 or 64 lanes
 * (up to 1024 elements) or by a wavefront (up to 4096); rows longer still,
 * or too few rows to occupy the device, are cut into chunks reduced by
 * separate workgroups whose partials a second kernel folds in index order
 * (that case uses the stream's workspace).  Every choice depends only on
 * (rows, n, ld, alignment of x) and the device's compute-unit count, so
 * the results are deterministic.  Same tolerances as the 1-D calls.
 * ------------------------------------------------------------------- */
int red_sum_rows_f32(const float* x, size_t rows, size_t n, size_t ld,
                     float* out, int accum, red_stream_t stream);
int red_max_rows_f32(const float* x, size_t rows, size_t n, size_t ld,
                     float* out, int accum, red_stream_t stream);
int red_min_rows_f32(const float* x, size_t rows, size_t n, size_t ld,
                     float* out, int accum, red_stream_t stream);

/* ---------------------------------------------------------------------
 * Column sum / max / min: dst[j] = reduce_{i<R} src[i*ld + j], j < C
 *
 * The reduction of the TVM page ("reduction -> sm100_packed") taken along
 * the rows of a 2-D source -- the case its fast path leaves to a generic
 * fallback ("How inputs change the algorithm", last row).  Layout, ld,
 * alignment, empty-tile early return and errors as for the column product
 * below; accum folds old dst[j] into column j first.  Same identities,
 * NaN policy and tolerances as the 1-D calls: max / min exact, sum within
 * 1e-6 * (|old| + sum |x|) per column.  Deterministic.
 * ------------------------------------------------------------------- */
int red_sum_cols_f32(const float* src, size_t R, size_t C, size_t ld,
                     float* dst, int accum, red_stream_t stream);
int red_max_cols_f32(const float* src, size_t R, size_t C, size_t ld,
                     float* dst, int accum, red_stream_t stream);
int red_min_cols_f32(const float* src, size_t R, size_t C, size_t ld,
                     float* dst, int accum, red_stream_t stream);

/* ---------------------------------------------------------------------
 * Column product (TCOLPROD): dst[j] = prod_{i<R} src[i*ld + j], j < C
 *
 * src    : row-major tile of element type T, aligned to sizeof(T); row i
 *          starts at src + i*ld.  Elements between C and ld are never read.
 * R, C   : valid rows and columns; ld : row stride in elements, ld >= C
 *          (RED_ERR_INVALID otherwise -- the analogue of TCOLPROD's check
 *          that source and destination agree on the valid column count).
 * dst    : C values of the same element type T, aligned to sizeof(T).
 *
 * f32    : products accumulate in fp32; relative error <= (R-1) * 2^-24
 *          whatever the order.
 * f16/bf16 (given as uint16_t bit patterns: IEEE binary16 / bfloat16):
 *          values are widened exactly to fp32, multiplied in fp32, and the
 *          final product is rounded once to T (round to nearest even).
 * i32    : products wrap modulo 2^32 (two's complement); bit-exact.
 *
 * Deterministic: for a given shape, alignment and device, the rows are
 * split over workgroups in a fixed way and the partial products are
 * combined in a fixed order, so repeated calls give identical bits.
 * ------------------------------------------------------------------- */
int red_colprod_f32(const float* src, size_t R, size_t C, size_t ld,
                    float* dst, red_stream_t stream);
int red_colprod_f16(const uint16_t* src, size_t R, size_t C, size_t ld,
                    uint16_t* dst, red_stream_t stream);
int red_colprod_bf16(const uint16_t* src, size_t R, size_t C, size_t ld,
                     uint16_t* dst, red_stream_t stream);
int red_colprod_i32(const int32_t* src, size_t R, size_t C, size_t ld,
                    int32_t* dst, red_stream_t stream);

/* The other integer element types TCOLPROD lists ("Constraints": int16 and
 * int32 on A2A3; int16, uint16, int32, uint32 on A5).  Same arguments,
 * layout and errors as above; products wrap modulo 2^32 (u32) or 2^16 (i16,
 * u16) and are bit-exact.  The low bits of a product depend only on the low
 * bits of its factors, so i16 and u16 give the same bit patterns, and u32
 * the same bits as i32. */
int red_colprod_i16(const int16_t* src, size_t R, size_t C, size_t ld,
                    int16_t* dst, red_stream_t stream);
int red_colprod_u16(const uint16_t* src, size_t R, size_t C, size_t ld,
                    uint16_t* dst, red_stream_t stream);
int red_colprod_u32(const uint32_t* src, size_t R, size_t C, size_t ld,
                    uint32_t* dst, red_stream_t stream);

/* ---------------------------------------------------------------------
 * Losses over rows of logits
 *
 * Notation: z is a row of V logits, s the scale (1 / temperature),
 * lse = ln sum_v exp(s z_v), ln p_v = s z_v - lse, H = -sum_v p_v ln p_v.
 *
 * logits  : row-major rows x V matrix of f32, f16 or bf16 (16-bit types as
 *           uint16_t bit patterns), aligned to its element size only; row r
 *           starts at logits + r * ld, ld >= V, V < 2^31.  Elements between
 *           V and ld are never read.
 * dlogits : the gradient, same element type, row stride ldd >= V (not
 *           accumulated: every one of its rows x V elements is written, none
 *           beyond).  NULL where a call allows it: the loss alone.  It may
 *           be logits itself, with ldd == ld.
 * targets : rows column numbers.  A row whose target is not in [0, V) (-100,
 *           say) does not count: its log-probability and its gradient are 0.
 * scale   : finite and positive.
 * weight  : one fp32 factor per row (for the preference loss, per pair) in
 *           the sum that makes the loss; NULL: 1 / rows each (1 / pairs).  A
 *           row of weight 0 does not count: its outputs are 0 and its logits
 *           are not looked at.  (A pair of weight 0 adds nothing to the loss
 *           and has a gradient of 0, whatever its logits; its seq_logp is
 *           computed as any other.)  A mask and a normaliser are both weights.
 * loss    : one fp32 value, the weighted sum of row losses; accum != 0 adds
 *           it to the old value.
 *
 * Losses carry their gradient: a call given dlogits writes
 * d loss / d logits of its own sum (a factor from later in a program goes
 * into the weights), in the same pass over the logits.
 *
 * Logits are widened exactly to fp32.  A thread's statistics are fp32, what
 * is computed once per row and the sums over rows are fp64, and every result
 * is rounded once to its type.  A term below 2^-126 of its row's largest
 * counts as 0 (in the sum of a distilled row's columns that are not listed: of
 * the largest among these).  Logits of -inf have probability 0.  A row with a
 * NaN or +inf, or with nothing but -inf, has NaN results unless it does not
 * count (the lse of nothing but -inf is -inf); its neighbours are not touched
 * by it.  A row filled with one finite value is
 * uniform, the type's lowest value included.
 * All results are deterministic.
 * ------------------------------------------------------------------- */

/* logp[r] = ln p_target, lse[r], and, where entropy is not NULL,
 * entropy[r] = H.  A row whose target is no column still has its lse and
 * entropy. */
int red_token_logprob_f32(const float* logits, size_t rows, size_t V, size_t ld,
                          const int64_t* targets, float scale, float* logp, float* lse,
                          float* entropy, red_stream_t stream);
int red_token_logprob_f16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                          const int64_t* targets, float scale, float* logp, float* lse,
                          float* entropy, red_stream_t stream);
int red_token_logprob_bf16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                           const int64_t* targets, float scale, float* logp, float* lse,
                           float* entropy, red_stream_t stream);

/* The gradient of red_token_logprob: with g = glogp[r] and h = gentropy[r]
 * the gradients of the row's two outputs,
 *   dlogits[r, v] = s (g (delta_{v, target} - p_v) - h p_v (ln p_v + H)).
 * lse and entropy are what the forward call wrote, and p_v = exp(s z_v - lse)
 * with lse as it is: its fp32 rounding, |lse| 2^-24, is a relative error of
 * every p_v.  gentropy and entropy
 * are both NULL where the entropy has no gradient.  Where g (or the target's
 * column) and h are 0 the row's logits are not looked at. */
int red_token_logprob_grad_f32(const float* logits, size_t rows, size_t V, size_t ld,
                               const int64_t* targets, float scale, const float* lse,
                               const float* entropy, const float* glogp, const float* gentropy,
                               float* dlogits, size_t ldd, red_stream_t stream);
int red_token_logprob_grad_f16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                               const int64_t* targets, float scale, const float* lse,
                               const float* entropy, const float* glogp, const float* gentropy,
                               uint16_t* dlogits, size_t ldd, red_stream_t stream);
int red_token_logprob_grad_bf16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                                const int64_t* targets, float scale, const float* lse,
                                const float* entropy, const float* glogp, const float* gentropy,
                                uint16_t* dlogits, size_t ldd, red_stream_t stream);

/* Distillation from a teacher of which each row keeps K entries: columns
 * idx[r * ldk + k] and their logits val[r * ldk + k] (fp32; log-probabilities
 * are logits too).  An entry whose column is not in [0, V) is padding.
 * 1 <= K <= 1024, ldk >= K, V <= 393216.
 *
 * teacher_lse NULL: the teacher is the softmax of the row's entries,
 *   q_k = exp(s val_k) / sum_j exp(s val_j),
 *   row loss = sum_k q_k (ln q_k - ln p_{idx_k}).
 * A row of padding alone (or of -inf alone) does not count; a NaN among the
 * entries makes NaN of the row.
 *
 * teacher_lse given (ln sum exp(s .) over the teacher's whole row): q_k =
 * exp(s val_k - teacher_lse), and the columns not listed, with the teacher's
 * rest q_r = 1 - sum q and the student's p_r = their sum of p, count as one:
 *   row loss = sum_k q_k (ln q_k - ln p_{idx_k}) + q_r (ln q_r - ln p_r).
 * The rest is 0 where sum q >= 1 or every column is listed, and where the
 * columns outside are masked (s z more than 745.2 below the row's largest:
 * nothing even in double precision) and 1 - sum q is no more than the rounding
 * of teacher_lse, (1 + |teacher_lse|) 2^-20.
 *
 * An entry of probability 0 adds nothing.  Each entry of a column listed
 * more than once counts.  row_loss, where not NULL, takes the rows' losses
 * without their weights.  (The factor 1 / s^2 that some recipes put on this
 * loss goes into the weights.) */
int red_distill_topk_f32(const float* logits, size_t rows, size_t V, size_t ld,
                         const int64_t* idx, const float* val, size_t K, size_t ldk,
                         const float* teacher_lse, const float* weight, float scale,
                         float* loss, int accum, float* row_loss, float* dlogits, size_t ldd,
                         red_stream_t stream);
int red_distill_topk_f16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                         const int64_t* idx, const float* val, size_t K, size_t ldk,
                         const float* teacher_lse, const float* weight, float scale,
                         float* loss, int accum, float* row_loss, uint16_t* dlogits, size_t ldd,
                         red_stream_t stream);
int red_distill_topk_bf16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                          const int64_t* idx, const float* val, size_t K, size_t ldk,
                          const float* teacher_lse, const float* weight, float scale,
                          float* loss, int accum, float* row_loss, uint16_t* dlogits, size_t ldd,
                          red_stream_t stream);

/* Clipped policy loss.  With A = advantage[r], ratio = exp(ln p_target -
 * old_logp[r]) and d = ref_logp[r] - ln p_target,
 *   row loss = -min(ratio A, clip(ratio, 1 - clip_low, 1 + clip_high) A)
 *              + kl_coef (exp(d) - d - 1) - entropy_coef H.
 * Where the two products are equal the first one's gradient is taken.
 * clip_low, clip_high >= 0 (infinity: no bound); kl_coef and entropy_coef
 * finite; ref_logp may be NULL where kl_coef is 0 and is not read then.
 * logp takes ln p_target, entropy (NULL: not wanted) H. */
int red_policy_loss_f32(const float* logits, size_t rows, size_t V, size_t ld,
                        const int64_t* targets, const float* old_logp, const float* ref_logp,
                        const float* advantage, const float* weight, float scale,
                        float clip_low, float clip_high, float kl_coef, float entropy_coef,
                        float* loss, int accum, float* logp, float* entropy, float* dlogits,
                        size_t ldd, red_stream_t stream);
int red_policy_loss_f16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                        const int64_t* targets, const float* old_logp, const float* ref_logp,
                        const float* advantage, const float* weight, float scale,
                        float clip_low, float clip_high, float kl_coef, float entropy_coef,
                        float* loss, int accum, float* logp, float* entropy, uint16_t* dlogits,
                        size_t ldd, red_stream_t stream);
int red_policy_loss_bf16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                         const int64_t* targets, const float* old_logp, const float* ref_logp,
                         const float* advantage, const float* weight, float scale,
                         float clip_low, float clip_high, float kl_coef, float entropy_coef,
                         float* loss, int accum, float* logp, float* entropy, uint16_t* dlogits,
                         size_t ldd, red_stream_t stream);

/* Preference loss of `pairs` pairs of packed sequences.  Sequence i has the
 * rows [starts[i], starts[i + 1]); sequences 0 .. pairs - 1 are the chosen
 * ones and pairs .. 2 pairs - 1 the rejected ones of the same pairs (2 pairs
 * + 1 starts, nondecreasing; bounds outside [0, rows] are moved into it).
 * Rows of no sequence have a gradient of 0.  pairs == 0 is empty input: nothing
 * is written, dlogits neither.  With S_i the sum of ln p_target over
 * the sequence's rows that count (average != 0: their mean; an empty
 * sequence has 0), ref_logp[i] the same from a reference model (NULL: 0),
 *   D = (S_c - ref_c) - (S_r - ref_r),   h = beta D - margin,
 *   RED_PREF_SIGMOID: loss = -(1 - smoothing) ln sigmoid(h)
 *                            - smoothing ln sigmoid(-h)
 *   RED_PREF_HINGE  : loss = max(0, 1 - h)
 *   RED_PREF_SQUARED: loss = ((h - 1/2) / beta)^2
 * beta > 0, margin finite, 0 <= smoothing <= 1, rows <= 524288, pairs <=
 * 131072.  seq_logp takes the 2 pairs values S_i.  The logits are read twice
 * when there is a gradient: it needs the whole pair's sum. */
enum red_preference { RED_PREF_SIGMOID = 0, RED_PREF_HINGE = 1, RED_PREF_SQUARED = 2 };
int red_preference_loss_f32(const float* logits, size_t rows, size_t V, size_t ld,
                            const int64_t* targets, const int64_t* starts, size_t pairs,
                            const float* ref_logp, const float* weight, int kind, float beta,
                            float margin, float smoothing, int average, float* loss, int accum,
                            float* seq_logp, float* dlogits, size_t ldd, red_stream_t stream);
int red_preference_loss_f16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                            const int64_t* targets, const int64_t* starts, size_t pairs,
                            const float* ref_logp, const float* weight, int kind, float beta,
                            float margin, float smoothing, int average, float* loss, int accum,
                            float* seq_logp, uint16_t* dlogits, size_t ldd, red_stream_t stream);
int red_preference_loss_bf16(const uint16_t* logits, size_t rows, size_t V, size_t ld,
                             const int64_t* targets, const int64_t* starts, size_t pairs,
                             const float* ref_logp, const float* weight, int kind, float beta,
                             float margin, float smoothing, int average, float* loss, int accum,
                             float* seq_logp, uint16_t* dlogits, size_t ldd,
                             red_stream_t stream);

/* ---------------------------------------------------------------------
 * Around the output layer
 *
 * Matrices are row-major f32, f16 or bf16 (16-bit types as uint16_t bit
 * patterns), aligned to their element size, with a row stride of at least
 * their columns (where there is one row the stride is not looked at).
 * Elements between the columns and the stride are neither read nor written.
 * Values are widened exactly to fp32; every result is rounded once to its
 * type.  A row with a NaN or an infinity has NaN results (but see the norm for
 * an infinity) and touches no other row's (it does touch what is summed over
 * rows).  All results are deterministic.
 * ------------------------------------------------------------------- */

/* Root-mean-square norm of rows of D values, D <= 16384, with the residual's
 * addition before it:
 *   h = x + residual (NULL: x),   rstd = (mean h^2 + eps)^(-1/2),
 *   y = h rstd weight.
 * sum (NULL: not wanted) takes h, y the norm, both rounded once from the exact
 * sum's fp32 value: y does not start from the rounded h.  y8 with scale8 (both
 * or neither; y or y8 or both must be given) takes the row in 8 bits, OCP
 * e4m3: scale8[r] = max |y| / 448 and y8 = round(y / scale8[r]), to nearest even; a row
 * whose largest |y| is below 1e-35 has scale 0 and zeros, and a NaN in y is a
 * NaN in y8 and does not count for the scale.  rstd (NULL: not wanted) is what
 * the gradient needs.  The sum of squares is fp64: no finite row overflows.
 * A row in whose h there is an infinity and no NaN has rstd 0: its y and y8 are
 * NaN at the infinities and 0 elsewhere, with a scale of 0; a test of rstd for 0
 * finds it, its gradient is NaN.
 * weight has D values.  eps >= 0 and finite; with eps 0 a row of zeros has NaN.
 * sum and y may each be x or residual themselves, with the same stride (two
 * outputs never the same). */
int red_add_rmsnorm_f32(const float* x, size_t rows, size_t D, size_t ldx,
                        const float* residual, size_t ldr, const float* weight, float eps,
                        float* sum, size_t lds, float* y, size_t ldy, uint8_t* y8, size_t ldy8,
                        float* scale8, float* rstd, red_stream_t stream);
int red_add_rmsnorm_f16(const uint16_t* x, size_t rows, size_t D, size_t ldx,
                        const uint16_t* residual, size_t ldr, const uint16_t* weight, float eps,
                        uint16_t* sum, size_t lds, uint16_t* y, size_t ldy, uint8_t* y8, size_t ldy8,
                        float* scale8, float* rstd, red_stream_t stream);
int red_add_rmsnorm_bf16(const uint16_t* x, size_t rows, size_t D, size_t ldx,
                        const uint16_t* residual, size_t ldr, const uint16_t* weight, float eps,
                        uint16_t* sum, size_t lds, uint16_t* y, size_t ldy, uint8_t* y8, size_t ldy8,
                        float* scale8, float* rstd, red_stream_t stream);

/* The gradient of red_add_rmsnorm: with n = h rstd and g = dy weight,
 *   dx = (g - n mean(g n)) rstd + dsum,   dweight = sum over rows of dy n,
 * dx being the gradient of x and of the residual alike, dsum (NULL: none) the
 * gradient that arrives at h past the norm.  h and rstd are the forward call's.
 * dweight (NULL: not wanted) is fp32; accum != 0 adds to its old values.  dx
 * may be h, dy or dsum itself, with the same stride.  Uses the stream's
 * workspace. */
int red_rmsnorm_grad_f32(const float* h, size_t rows, size_t D, size_t ldh,
                         const float* weight, const float* rstd, const float* dy, size_t lddy,
                         const float* dsum, size_t ldds, float* dx, size_t lddx, float* dweight,
                         int accum, red_stream_t stream);
int red_rmsnorm_grad_f16(const uint16_t* h, size_t rows, size_t D, size_t ldh,
                         const uint16_t* weight, const float* rstd, const uint16_t* dy, size_t lddy,
                         const uint16_t* dsum, size_t ldds, uint16_t* dx, size_t lddx, float* dweight,
                         int accum, red_stream_t stream);
int red_rmsnorm_grad_bf16(const uint16_t* h, size_t rows, size_t D, size_t ldh,
                         const uint16_t* weight, const float* rstd, const uint16_t* dy, size_t lddy,
                         const uint16_t* dsum, size_t ldds, uint16_t* dx, size_t lddx, float* dweight,
                         int accum, red_stream_t stream);

/* Balance loss of a router of E experts, E <= 2048, over rows of logits, of
 * which each row has chosen the K experts experts[r * ldk + k] (one that is
 * not in [0, E) is padding; one listed twice counts twice; 1 <= K <= 1024,
 * ldk >= K, not looked at for one row).  With p_r the softmax of row r and n_e the number of choices of
 * expert e among the rows that count,
 *   P_e = sum_r weight[r] p_re,   f_e = n_e / sum n,
 *   loss = balance_coef E sum_e f_e P_e + z_coef sum_r weight[r] lse_r^2.
 * weight: one factor per row (NULL: 1 / rows each); a row of weight 0 does not
 * count: its logits and choices are not looked at and its gradient is 0.
 * counts takes the n_e, prob (NULL: not wanted) the P_e.  dlogits (NULL: the
 * loss alone) takes the gradient, for which the counts are constants; it may be
 * logits itself, with the same stride.  Where nothing was chosen the first term
 * is 0.  A row with a NaN makes the loss a NaN, and not the other rows'
 * gradients.  balance_coef and z_coef finite, rows < 2^31.  accum != 0 adds to
 * the old loss.  Uses the stream's workspace. */
int red_router_balance_f32(const float* logits, size_t rows, size_t E, size_t ld,
                           const int64_t* experts, size_t K, size_t ldk, const float* weight,
                           float balance_coef, float z_coef, float* loss, int accum,
                           int64_t* counts, float* prob, float* dlogits, size_t ldd,
                           red_stream_t stream);
int red_router_balance_f16(const uint16_t* logits, size_t rows, size_t E, size_t ld,
                           const int64_t* experts, size_t K, size_t ldk, const float* weight,
                           float balance_coef, float z_coef, float* loss, int accum,
                           int64_t* counts, float* prob, uint16_t* dlogits, size_t ldd,
                           red_stream_t stream);
int red_router_balance_bf16(const uint16_t* logits, size_t rows, size_t E, size_t ld,
                           const int64_t* experts, size_t K, size_t ldk, const float* weight,
                           float balance_coef, float z_coef, float* loss, int accum,
                           int64_t* counts, float* prob, uint16_t* dlogits, size_t ldd,
                           red_stream_t stream);

/* Cross entropy of hidden rows (rows x D) against an output layer weight
 * (V x D) and targets, in pieces of the vocabulary:
 *   z_v = scale hidden[r] . weight[v],  lse = ln sum_v exp z_v,
 *   loss = sum_r row_weight[r] (lse - z_target + z_coef lse^2).
 * row_weight: one factor per row (NULL: 1 / rows each).  A row of weight 0, or
 * whose target is not in [0, V) (-100, say), does not count: its outputs are 0
 * and its hidden values are not looked at.  logp takes z_target - lse, lse the
 * log-sum-exp (NULL: not wanted).  dhidden and dweight (NULL: not wanted) take
 * the gradients, of the inputs' type; every element of their rows is written.
 * accum != 0 adds to the old loss.  No output may lie over an input.
 *
 * Products are of the 16-bit values, summed in fp32; subnormal values count.
 * A logit's gradient over its row's weight (up to a power of two) is rounded
 * to the inputs' type before it is multiplied by weight or hidden rows: half a
 * step of each term, 2^-8 (bf16) or 2^-11 (f16) of it at most, and in f16 at
 * least 2^-29 of the row's weight.  For dweight in f16 the hidden values are
 * taken to within 2^-22 where the rows' weights differ in magnitude; a row's part
 * of dweight keeps that accuracy however small its weight is beside others', down
 * to 2^-100 of the largest.  In f16 1 + 2 z_coef lse must stay below 2000 in
 * magnitude (gradients overflow otherwise).  A row with a NaN or an
 * infinity has a NaN loss, and NaN in dhidden's row; dweight sums over rows.
 * A weight that is NaN or infinite leaves logp and lse as they are and makes the
 * loss no finite number and dhidden's row NaN.
 *
 * D a multiple of 8 and at most 65536; the rows of weight aligned to 16 bytes
 * (RED_ERR_ALIGN, or RED_ERR_INVALID where ldw is no multiple of 8);
 * rows <= 2^20, V <= 2^24, ldw <= 2^21; scale positive, z_coef finite.
 *
 * workspace: device memory of the caller's, aligned to 256 bytes, whose needed
 * size red_linear_ce_workspace_* gives (on the device of the call; dhidden,
 * dweight: whether they are wanted).  It holds nothing between calls; calls
 * that share one must be ordered.  RED_ERR_SCRATCH where it is too small.  It
 * takes the hidden rows once or, for dweight, twice, 8 bytes a row for each 128
 * or 256 columns, for gradients a piece of their logits' gradients (256 MiB or
 * 2048 columns), the logits themselves in fp32 where they are one piece, at most
 * 512 MiB and, for D below 640, at most 384 KiB times D (others are computed a
 * second time), and for dhidden its fp32 sums. */
int red_linear_ce_f16(const uint16_t* hidden, size_t rows, size_t D, size_t ldh,
                      const uint16_t* weight, size_t V, size_t ldw, const int64_t* targets,
                      const float* row_weight, float scale, float z_coef, float* loss, int accum,
                      float* logp, float* lse, uint16_t* dhidden, size_t lddh, uint16_t* dweight,
                      size_t lddw, void* workspace, size_t workspace_bytes, red_stream_t stream);
int red_linear_ce_workspace_f16(size_t rows, size_t D, size_t V, int dhidden, int dweight,
                                size_t* bytes);
int red_linear_ce_bf16(const uint16_t* hidden, size_t rows, size_t D, size_t ldh,
                      const uint16_t* weight, size_t V, size_t ldw, const int64_t* targets,
                      const float* row_weight, float scale, float z_coef, float* loss, int accum,
                      float* logp, float* lse, uint16_t* dhidden, size_t lddh, uint16_t* dweight,
                      size_t lddw, void* workspace, size_t workspace_bytes, red_stream_t stream);
int red_linear_ce_workspace_bf16(size_t rows, size_t D, size_t V, int dhidden, int dweight,
                                size_t* bytes);

/* ---------------------------------------------------------------------
 * Utilities
 * ------------------------------------------------------------------- */

/* Waits for the work enqueued on `stream` to finish, then frees the
 * workspace the library holds for (current device, stream) -- for
 * hipStreamPerThread, the calling thread's.  Call it before destroying a
 * stream that library calls used, or before a thread that used
 * hipStreamPerThread exits; a later call on the stream allocates a new
 * workspace.  RED_OK when there is nothing to free; RED_ERR_HIP when the
 * synchronisation or the free fails.  The stream must still exist. */
int red_release_workspace(red_stream_t stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* red_status_str(int status);

/* RED_ABI_VERSION of the built library. */
int red_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBREDUCE_REDUCE_H */
