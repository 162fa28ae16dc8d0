/*
 * btq.h -- C ABI of libbtq, the hybrid int4/BF16 codec for tensor-parallel
 * partial sums on AMD Instinct MI355X (gfx950).
 *
 * Source of the method: the page "Revolutionizing LLM Inference: The Power of
 * Efficient Low-Bit Communication" (aiexpert.world), a summary of the paper
 * "Towards Efficient Low-Bit Communication for Tensor Parallel LLM Inference".
 * Its section "The Hybrid Quantization Algorithm" gives three steps:
 *   Calibration  -- per-feature parameters from moving averages of the
 *                   minimum and maximum observed on each device;
 *   Selection    -- rank features by quantization range and keep a number
 *                   of them in BF16;
 *   Inference    -- the selected features stay BF16 and the others are sent
 *                   as 4-bit integers; after communication everything is
 *                   converted back and summed across devices.
 * Section "Combating Quantization Errors with Tensor Parallelism" places the
 * quantization on each device's partial sum, before the sum.
 *
 * Four calls follow those steps: btq_calib_update, btq_select_outliers,
 * btq_compress_pack (the sender) and btq_decompress_reduce (the receiver).
 * Here all P shards' partial sums sit in one GPU's HBM, so the exchange
 * between devices is the identity: the buffers written by btq_compress_pack
 * are the ones read by btq_decompress_reduce. The other calls widen the path:
 * a bf16-output receiver, other readings of the selection step and a packed
 * row pitch. Two more groups cover what stands next to the path in a
 * transformer: the 8-bit linear layer whose partial sums the sender takes
 * (btq_quantize_rows, btq_int8_matmul, btq_int8_linear) with the norms that
 * read the receiver's sum (btq_block_norm), and what lies between two linear
 * layers of an attention block: btq_head_norm_rope, a paged 4-bit cache
 * (btq_kv_append, btq_kv_gather) and btq_kv_attention over it.
 *
 * Conventions shared by every call
 *  - Tensor pointers are DEVICE pointers (hipMalloc'd or from PyTorch) to
 *    caller-owned, contiguous, row-major memory with the last index fastest.
 *    The library never allocates, frees or keeps them.
 *  - bf16 values are raw 16-bit patterns (uint16_t).
 *  - A pointer must be aligned to its element type (BTQ_ERR_ALIGN
 *    otherwise). Fast kernels run when x, packed, outliers and y are 16-byte
 *    aligned, the per-feature arrays 16-byte aligned, and H and H-k are
 *    multiples of 8 (the receivers: up to 8 shards per launch, see
 *    btq_decompress_reduce); every other layout runs on a general kernel
 *    that is correct but much slower.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *    Every call checks its arguments on the host, enqueues its kernels on
 *    `stream` and returns. It does not synchronize, print, throw or abort.
 *    The library holds no mutable global state, so calls on different
 *    streams may run concurrently as long as their buffers do not overlap.
 *  - Return value: BTQ_OK (0) or a negative btq_status. On an argument or
 *    shape error nothing is enqueued and no HIP call is made. A fault while
 *    the kernels run surfaces at the caller's next synchronization.
 *  - Sizes: 1 <= P <= 65535, 1 <= H <= 2^30, 0 <= k <= H, T >= 0, and
 *    P*T*H < 2^62. T == 0 is an empty batch: compress and decompress do
 *    nothing, and calibration rejects it (its min/max would be undefined).
 *  - Floating point: every fp32 step is one IEEE round-to-nearest-even
 *    operation. Divisions are correctly rounded. Nothing is flushed to zero.
 *    Inputs must be finite; NaN and Inf give unspecified (but in-bounds)
 *    results.
 *
 * Layouts
 *  x            bf16 [P,T,H]     partial sums, one [T,H] block per shard
 *  run_min/max  fp32 [P,H]
 *  scale        fp32 [P,H]       4-bit step of feature h on shard p
 *  rscale       fp32 [P,H]       1/scale
 *  zero_point   u8   [P,H]       0..15
 *  outlier_idx  i32  [k]         BF16 features, ascending h
 *  fmap         i32  [H]         fmap[h] = j (int4 slot j of h), or -1-i when
 *                                h = outlier_idx[i]
 *  cmap         i32  [H-k]       cmap[j] = h of int4 slot j, ascending
 *  packed       u8   [P,T,Bq]    Bq = btq_packed_row_bytes(H,k) = ceil((H-k)/2);
 *                                slot 2b in the low nibble of byte b, slot
 *                                2b+1 in the high nibble; an odd H-k leaves
 *                                the last high nibble 0
 *  outliers     bf16 [P,T,k]     outliers[p,t,i] = x[p,t,outlier_idx[i]]
 *  y            fp32 [T,H]       (bf16 [T,H] for the bf16-output receiver)
 */
#ifndef BTQ_H
#define BTQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BTQ_OK = 0,
  BTQ_ERR_ARG = -1,        /* null pointer, unknown option, factor out of range */
  BTQ_ERR_SHAPE = -2,      /* a size, a stride or the pitch out of range        */
  BTQ_ERR_ALIGN = -3,      /* pointer not aligned to its element type           */
  BTQ_ERR_WORKSPACE = -4,  /* workspace smaller than the *_workspace_bytes size */
  BTQ_ERR_HIP = -5,        /* a HIP call failed (hipGetLastError, cleared)      */
  BTQ_ERR_SCRATCH = -6     /* sizes beyond btq_calib_update_noalloc's scratch    */
} btq_status;

/*
 * Calibration -- "The Hybrid Quantization Algorithm", Calibration bullet.
 *
 * For every shard p and feature h, takes the batch minimum and maximum over
 * the T tokens of x[p,:,h]. Then it updates the running extremes:
 *   first_batch != 0 : run = batch value
 *   otherwise        : run = fl(fl(a*run) + fl(c*batch)),  a = momentum,
 *                      c = fl(1 - a), all fp32 (moving average; the page
 *                      gives no formula -- the momentum weights the old value)
 *   x        bf16 [P,T,H]   in, T >= 1
 *   momentum in [0,1): the weight of the running value (BTQ_ERR_ARG
 *            otherwise, NaN included)
 *   run_min  fp32 [P,H]     in/out (ignored on input when first_batch != 0)
 *   run_max  fp32 [P,H]     in/out
 *   workspace  device scratch of at least btq_calib_workspace_bytes(P,T,H)
 *              bytes (may be NULL if that size is 0); its contents are
 *              overwritten and need no initial value.
 * Batch extremes are exact, and -0 and +0 count as equal. The result does
 * not depend on how the kernels split the token axis.
 */
int btq_calib_update(const uint16_t *x, int64_t P, int64_t T, int64_t H,
                     float momentum, int first_batch,
                     float *run_min, float *run_max,
                     void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes for btq_calib_update (0 for invalid sizes). */
size_t btq_calib_workspace_bytes(int64_t P, int64_t T, int64_t H);

/*
 * btq_calib_update without a workspace and without any allocation, for
 * callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc.
 *
 * Arguments, checks and results are those of btq_calib_update, bit for bit
 * (the result does not depend on how the token axis is split). The partial
 * extremes live in a static device array of BTQ_NOALLOC_SCRATCH_BYTES on
 * each GPU, held until the process ends; the call uses as many token chunks
 * as that array holds, so 2*P*H*4 bytes must fit it (P*H <= 2^20), else it
 * returns BTQ_ERR_SCRATCH and enqueues nothing. It calls no hipMalloc or
 * hipFree; its first call on a device looks up the array's address there.
 * Every call on one GPU uses that GPU's one array: calls that may overlap
 * on one GPU (different streams, or host threads) race and must be ordered
 * by the caller. Nothing in the array needs an initial value.
 */
#define BTQ_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
int btq_calib_update_noalloc(const uint16_t *x, int64_t P, int64_t T, int64_t H,
                             float momentum, int first_batch,
                             float *run_min, float *run_max, void *stream);

/*
 * Selection -- "The Hybrid Quantization Algorithm", Calibration bullet
 * (per-feature parameters) and Selection bullet (rank by range, keep k).
 *
 * Per (p,h):  lo = min(run_min,0), hi = max(run_max,0), width = hi - lo,
 *             scale = width/15 (1 if below 2^-126), rscale = 1/scale,
 *             zero_point = clamp(rint_half_even(-lo/scale), 0, 15).
 * Per h:      score = width[0,h] + width[1,h] + ... (fp32, p ascending).
 * The k features with the highest score are kept in BF16 (ties: lower h
 * first). They are shared by all shards, because the receiver must know
 * every sender's layout.
 *   run_min, run_max  fp32 [P,H]  in
 *   scale, rscale     fp32 [P,H]  out
 *   zero_point        u8   [P,H]  out, values 0..15
 *   outlier_idx       i32  [k]    out, the BF16 features in ascending h
 *   fmap              i32  [H]    out
 *   cmap              i32  [H-k]  out
 *   workspace  at least btq_select_workspace_bytes(P,H,k) bytes of scratch.
 * Pointers for zero-length outputs (k == 0, or k == H for cmap) may be NULL.
 */
int btq_select_outliers(const float *run_min, const float *run_max,
                        int64_t P, int64_t H, int64_t k,
                        float *scale, float *rscale, uint8_t *zero_point,
                        int32_t *outlier_idx, int32_t *fmap, int32_t *cmap,
                        void *workspace, size_t workspace_bytes, void *stream);

/* Scratch bytes for the ranked selections: P*H floats (0 for invalid sizes). */
size_t btq_select_workspace_bytes(int64_t P, int64_t H, int64_t k);

/*
 * Sender side of inference -- "The Hybrid Quantization Algorithm", Inference
 * bullet; quantization before the sum per "Combating Quantization Errors
 * with Tensor Parallelism".
 *
 * For each token row (p,t), the int4 slots j = 0..H-k-1 take feature
 * h = cmap[j]:  q = clamp(rint_half_even(fl(x*rscale[p,h])) + zero_point[p,h],
 * 0, 15), packed two per byte into a row of Bq = btq_packed_row_bytes(H,k)
 * bytes (rows follow each other with no gap). The BF16 features are copied
 * bit for bit: outliers[p,t,i] = x[p,t,outlier_idx[i]].
 *   x            bf16 [P,T,H]    in
 *   rscale       fp32 [P,H], zero_point u8 [P,H]   in (from a selection call)
 *   outlier_idx  i32 [k], cmap i32 [H-k]           in (from a selection call)
 *   packed       u8   [P,T,Bq]   out
 *   outliers     bf16 [P,T,k]    out
 * The maps are trusted: outlier_idx and cmap must partition 0..H-1, each in
 * ascending order, as the selection calls write them.
 */
int btq_compress_pack(const uint16_t *x, int64_t P, int64_t T, int64_t H, int64_t k,
                      const float *rscale, const uint8_t *zero_point,
                      const int32_t *outlier_idx, const int32_t *cmap,
                      uint8_t *packed, uint16_t *outliers, void *stream);

/*
 * Receiver side of inference -- "The Hybrid Quantization Algorithm",
 * Inference bullet (convert back, sum across devices).
 *
 * y[t,h] = sum over p = 0..P-1 of term_p, in fp32, where
 *   fmap[h] = j >= 0:  term_p = (q_p - zero_point[p,h]) * scale[p,h], q_p
 *                      the code of slot j in packed row (p,t)
 *   fmap[h] = -1-i:    term_p = the bf16 value outliers[p,t,i]
 * Features kept in BF16 are summed in p order from +0, so they equal a
 * sequential fp32 sum bit for bit. int4 features are evaluated as
 * fma(q_p, scale, acc) from the constant -sum_p zero_point*scale, which
 * stays within 1e-3*|y| + 1e-2*max_p scale[p,h] of the sequential sum.
 * (The 512 features of a block that holds a scale of 2^104 or more are
 * computed as the sequential sum itself.)
 *   packed [P,T,Bq], outliers [P,T,k]   in, as written by btq_compress_pack
 *   scale fp32 [P,H], zero_point u8 [P,H], fmap i32 [H]   in
 *   y      fp32 [T,H]   out
 * Fast kernel: H a multiple of 8, Bq a multiple of 4 and at least 8,
 * 16-byte aligned scale, fmap and y, and the message and outlier block of
 * every 8 shards under 2^31 bytes. More than 8 shards, or a message past
 * 2^31 bytes, run it once per group of shards (8, or fewer so that each
 * group's message fits), in shard order; each later group starts from the y
 * the earlier ones wrote (y is read as well as written), so BF16 features
 * keep their sequential sum. Anything else takes a general kernel (correct,
 * much slower, and exactly the sequential sum).
 */
int btq_decompress_reduce(const uint8_t *packed, const uint16_t *outliers,
                          int64_t P, int64_t T, int64_t H, int64_t k,
                          const float *scale, const uint8_t *zero_point, const int32_t *fmap,
                          float *y, void *stream);

/* Code bytes per packed row: ceil((H-k)/2); -1 if H < 1 or k is outside [0,H]. */
int64_t btq_packed_row_bytes(int64_t H, int64_t k);

/* ------------------------------------------------------------------------
 * Widened path.
 * ------------------------------------------------------------------------ */

/*
 * Receiver with bf16 output -- "The Hybrid Quantization Algorithm",
 * Inference bullet (after communication the tensors convert back to BF16).
 *
 * The same sum as btq_decompress_reduce, rounded once from fp32 to bf16
 * (round to nearest even): y[t,h] = bf16(fp32 sum), bit for bit the rounding
 * of what btq_decompress_reduce writes. y is bf16 [T,H] (uint16 bits), 2-byte
 * aligned (16-byte aligned for the fast kernel). More than 8 shards take the
 * general kernel here (there is no fp32 buffer to carry a group's sum): the
 * result is then the rounding of the sequential sum, bit for bit.
 */
int btq_decompress_reduce_bf16(const uint8_t *packed, const uint16_t *outliers,
                               int64_t P, int64_t T, int64_t H, int64_t k,
                               const float *scale, const uint8_t *zero_point,
                               const int32_t *fmap, uint16_t *y, void *stream);

/* How a feature's P per-shard ranges become its rank score. */
typedef enum {
  BTQ_SCORE_SUM = 0,   /* width[0,h] + width[1,h] + ... (fp32, p ascending)    */
  BTQ_SCORE_MAX = 1    /* max over p of width[p,h] (exact)                     */
} btq_score_rule;

/*
 * btq_select_outliers with a choice of rank score -- "The Hybrid
 * Quantization Algorithm", Selection bullet: features are ranked by their
 * quantization ranges, which are per device, and the page does not say how
 * one feature's ranges on the P devices combine. BTQ_SCORE_SUM is the
 * reading btq_select_outliers uses; BTQ_SCORE_MAX ranks a feature by its
 * widest shard. Only the score (and so the set and maps) changes; every
 * other output and argument is as in btq_select_outliers. Any other
 * score_rule returns BTQ_ERR_ARG.
 */
int btq_select_outliers_rule(const float *run_min, const float *run_max,
                             int64_t P, int64_t H, int64_t k, int score_rule,
                             float *scale, float *rscale, uint8_t *zero_point,
                             int32_t *outlier_idx, int32_t *fmap, int32_t *cmap,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Selection with the BF16 set given by the caller -- the comparison in
 * "Key Observations and Future Directions" (features picked at random
 * instead of by range), and any other selection rule computed elsewhere.
 *
 * Same parameters and maps as btq_select_outliers, with the ranking
 * replaced by the given set:
 *   features      i32 [k]  in, HOST memory: k distinct features in
 *                          ascending order, each in [0, H). Anything else
 *                          returns BTQ_ERR_ARG and enqueues nothing.
 *   outlier_idx   i32 [k]  out (device): a copy of features, made by a
 *                          host-to-device copy on `stream`. Keep `features`
 *                          unchanged until the stream has passed this call.
 * Every other argument is as in btq_select_outliers. No workspace is needed.
 */
int btq_select_features(const float *run_min, const float *run_max,
                        int64_t P, int64_t H, int64_t k, const int32_t *features,
                        float *scale, float *rscale, uint8_t *zero_point,
                        int32_t *outlier_idx, int32_t *fmap, int32_t *cmap, void *stream);

/*
 * Per-shard BF16 sets -- a second reading of "The Hybrid Quantization
 * Algorithm", Selection bullet: the ranges that rank features are per
 * device, so every shard keeps its own k widest features (ranked by its own
 * range, ties to the lower h) in BF16. The message keeps its size (k BF16
 * values and H-k codes per row), but each shard lays it out by its own map,
 * so the receiver reads every shard's map.
 *
 * btq_select_outliers_per_shard: parameters as in btq_select_outliers, plus
 *   outlier_idx  i32 [P,k]      out, shard p's BF16 features, ascending h
 *   fmap         i32 [P,H]      out, shard p's map (slot j, or -1-i)
 *   cmap         i32 [P,H-k]    out, shard p's int4 features, ascending h
 *   workspace    at least btq_select_workspace_bytes(P,H,k) bytes.
 * btq_compress_pack_per_shard: btq_compress_pack with outlier_idx [P,k] and
 *   cmap [P,H-k]; row (p,t) is coded with shard p's maps. Same layouts.
 * btq_decompress_reduce_per_shard: btq_decompress_reduce with fmap [P,H]:
 *   term_p follows shard p's map. Features BF16 on every shard are summed in
 *   shard order from +0, exactly; the others are within the receiver's
 *   tolerance of the sequential sum. Past 8 shards (or a message past 2^31
 *   bytes) the fast kernel runs once per group of up to 6 shards, each
 *   later group adding to y as in btq_decompress_reduce.
 */
int btq_select_outliers_per_shard(const float *run_min, const float *run_max,
                                  int64_t P, int64_t H, int64_t k,
                                  float *scale, float *rscale, uint8_t *zero_point,
                                  int32_t *outlier_idx, int32_t *fmap, int32_t *cmap,
                                  void *workspace, size_t workspace_bytes, void *stream);
int btq_compress_pack_per_shard(const uint16_t *x, int64_t P, int64_t T, int64_t H, int64_t k,
                                const float *rscale, const uint8_t *zero_point,
                                const int32_t *outlier_idx, const int32_t *cmap,
                                uint8_t *packed, uint16_t *outliers, void *stream);
int btq_decompress_reduce_per_shard(const uint8_t *packed, const uint16_t *outliers,
                                    int64_t P, int64_t T, int64_t H, int64_t k,
                                    const float *scale, const uint8_t *zero_point,
                                    const int32_t *fmap, float *y, void *stream);

/* Set layout of the *_ex calls: one set for all shards, or one per shard. */
typedef enum { BTQ_SETS_SHARED = 0, BTQ_SETS_PER_SHARD = 1 } btq_sets;
/* Output type of btq_decompress_reduce_ex. */
typedef enum { BTQ_Y_F32 = 0, BTQ_Y_BF16 = 1 } btq_ytype;

/*
 * The sender and receiver with every option: the set layout, the output
 * type, and a packed row pitch. Row (p,t) of the message starts at byte
 * (p*T+t)*packed_pitch; its first Bq bytes hold the codes and the sender
 * writes the rest of the row as zeros, which the receiver never reads.
 * packed_pitch = Bq is the layout of btq_compress_pack; btq_packed_pitch(H,k)
 * (Bq rounded up to 128) starts every row on a cache line, so the kernels
 * write and read whole lines (the message grows by less than 128 bytes a
 * row). packed_pitch < Bq returns BTQ_ERR_SHAPE. The fast kernels need a
 * pitch that is a multiple of 4.
 * For sets == BTQ_SETS_PER_SHARD outlier_idx, cmap and fmap carry one set
 * per shard as in the *_per_shard calls. y_type BTQ_Y_BF16 makes y bf16
 * [T,H] (uint16 bits). Any other sets or y_type returns BTQ_ERR_ARG.
 */
int btq_compress_pack_ex(const uint16_t *x, int64_t P, int64_t T, int64_t H, int64_t k,
                         const float *rscale, const uint8_t *zero_point,
                         const int32_t *outlier_idx, const int32_t *cmap, int sets,
                         uint8_t *packed, int64_t packed_pitch, uint16_t *outliers,
                         void *stream);
int btq_decompress_reduce_ex(const uint8_t *packed, int64_t packed_pitch,
                             const uint16_t *outliers, int64_t P, int64_t T, int64_t H, int64_t k,
                             const float *scale, const uint8_t *zero_point, const int32_t *fmap,
                             int sets, void *y, int y_type, void *stream);

/* Recommended packed row pitch for the *_ex calls: the code bytes rounded up
 * to a multiple of 128; -1 for invalid sizes. */
int64_t btq_packed_pitch(int64_t H, int64_t k);

/* ------------------------------------------------------------------------
 * Around the codec: the 8-bit linear layer that makes the partial sums, and
 * the block norm that reads the reduced sum.
 *
 * Extra conventions of these calls
 *  - Value types are BTQ_T_F32, BTQ_T_BF16 (raw 16-bit patterns) and, for
 *    norm outputs, BTQ_T_INT8. Any other value returns BTQ_ERR_ARG.
 *  - Sums, statistics and norms are fp32 (integer sums int32, exact; sums of
 *    norm rows past 32768 fp64, rounded once). Each
 *    output is rounded once, to nearest even (codes: see the calls).
 *  - NaN and Inf are carried, not excluded: see each call.
 *  - T == 0 does nothing. Sizes: P <= 65535, H, N, K in [1, 2^30], and every
 *    tensor under 2^62 elements.
 * ------------------------------------------------------------------------ */

typedef enum { BTQ_T_F32 = 0, BTQ_T_BF16 = 1, BTQ_T_INT8 = 2 } btq_type;

/*
 * Per-row 8-bit codes: activations (one scale a token) or, once, weights
 * (one scale an output channel).
 *
 * For every row of K values, m = max|x| and
 *   scale = m/127, code = x*(127/m) rounded to the nearest integer, ties away
 *   from zero; codes lie in -127..127.
 * For bf16 input the codes are those of exact arithmetic, ties included. A
 * row with m/127 below 2^-126 (a row of zeros among them) gets scale 1 and
 * codes 0. A row that holds NaN or Inf gets scale NaN and codes 0, so that
 * everything computed from it is NaN.
 *   x      fp32 or bf16 [P,T,K]  in; row (p,t) starts at element
 *                                p*x_shard + t*x_pitch, its K values are
 *                                contiguous (a row-parallel layer's shards can
 *                                be column slices of one [T,P*K] matrix). Rows
 *                                may overlap or coincide; strides are >= 0.
 *   q      i8   [P,T,K]          out, contiguous
 *   scale  fp32 [P,T]            out
 */
int btq_quantize_rows(const void *x, int x_type, int64_t x_shard, int64_t x_pitch,
                      int64_t P, int64_t T, int64_t K, int8_t *q, float *scale, void *stream);

/*
 * Matrix product of 8-bit codes with a scale for each token and each output
 * channel, for all P shards:
 *   y[p,t,n] = (sum over k of a[p,t,k]*w[p,n,k]) * a_scale[p,t] * w_scale[p,n]
 *              (+ bias[p,n])
 * The sum is exact in int32 (K <= 131071, BTQ_ERR_SHAPE beyond it); it is
 * then rounded to fp32, multiplied by a_scale, by w_scale, added to bias, each
 * one fp32 operation, and rounded to the output type. y has the sender's
 * layout: bf16 y is an x of btq_compress_pack.
 *   a        i8 [P,T,K]  in; row (p,t) starts at p*a_shard + t*a_pitch
 *            (a_shard 0: one set of rows for all shards, as in a
 *            column-parallel layer). Strides are >= 0.
 *   a_scale  fp32        in; of row (p,t) at p*as_shard + t, as_shard >= 0
 *   w        i8 [P,N,K], w_scale fp32 [P,N]  in, contiguous
 *   bias     fp32 [P,N]  in, or NULL
 *   y        fp32 or bf16 [P,T,N]  out, contiguous
 * The fastest kernels run when a, w and their strides are multiples of 16 (so K
 * is, and weights are best stored so); rows on any other byte are as exact and
 * take 1.1 to 2.2 times as long. K < 16, N >= 2^20 and a_pitch >= 2^22 run on
 * a general kernel that is several times slower.
 */
int btq_int8_matmul(const int8_t *a, int64_t a_shard, int64_t a_pitch,
                    const float *a_scale, int64_t as_shard,
                    const int8_t *w, const float *w_scale, const float *bias,
                    int64_t P, int64_t T, int64_t N, int64_t K,
                    void *y, int y_type, void *stream);

/*
 * btq_quantize_rows on x, then btq_int8_matmul of its codes: a linear layer
 * with 8-bit weights on fp32 or bf16 activations. Bit for bit the result of
 * the two calls; small ones run in one launch. workspace: device scratch of at least
 * btq_int8_linear_workspace_bytes(P,T,K) bytes, 16-byte aligned, with no
 * initial value. x_shard == 0 quantizes one set of T rows for all shards.
 */
int btq_int8_linear(const void *x, int x_type, int64_t x_shard, int64_t x_pitch,
                    const int8_t *w, const float *w_scale, const float *bias,
                    int64_t P, int64_t T, int64_t N, int64_t K,
                    void *y, int y_type, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes for btq_int8_linear: P*T*((K rounded up to 16) + 4). 0 for
 * T == 0 and for sizes that the call refuses, P*T rows of that many bytes past
 * 2^62 among them. */
size_t btq_int8_linear_workspace_bytes(int64_t P, int64_t T, int64_t K);

typedef enum { BTQ_NORM_NONE = 0, BTQ_NORM_RMS = 1, BTQ_NORM_LAYER = 2 } btq_norm;

/*
 * The norms after one block and before the next, with the block's gate, its
 * residual scale and the residual sum, in one pass:
 *   u  = post(y)
 *   r' = residual + alpha * (gate * u)
 *   n  = pre(r')
 * where, over the H features of a row,
 *   BTQ_NORM_NONE   norm(v) = v
 *   BTQ_NORM_RMS    norm(v) = v * (1/sqrt(mean(v^2) + eps)) * weight
 *   BTQ_NORM_LAYER  the same of v - mean(v), plus bias
 * All of it is fp32; n is computed from r' before r' is rounded to its type.
 *   y             fp32 or bf16 [T,H]  in (the receiver's output), or NULL:
 *                 then r' = residual, and post and gate must be NONE and NULL
 *   residual      fp32 or bf16 [T,H]  in
 *   post_weight, post_bias, pre_weight, pre_bias  fp32 [H] in, or NULL (1, 0);
 *                 bias only for BTQ_NORM_LAYER (BTQ_ERR_ARG otherwise)
 *   gate          fp32 or bf16 [gate_rows,H]  in, or NULL (1). gate_rows
 *                 divides T; token t takes gate row t / (T/gate_rows): 1 is a
 *                 gate per feature, T one per token and feature, between them
 *                 one per sequence of equal length.
 *   residual_out  [T,H] of the residual's type, out, or NULL. It may be
 *                 residual itself; no other overlap is allowed.
 *   n             [T,H] out: fp32, bf16, or int8 codes of each row as
 *                 btq_quantize_rows defines them (of the fp32 n), or NULL
 *   n_scale       fp32 [T] out, with int8 n only (else NULL)
 * eps >= 0 and finite, alpha finite. NaN and Inf spread to their row's
 * norms as the formulas give them. A row whose sum of squares passes the
 * largest fp32 (values near 2^64/sqrt(H)) is normed as if it were Inf: to 0
 * where its values are finite.
 * The same call gives the same bits every time. A row's do not depend on the
 * rows around it, except that for 4096 < H <= 8192 its sums are added in one
 * order for T <= 256 and in another for more.
 */
int btq_block_norm(const void *y, int y_type, const void *residual, int r_type,
                   int64_t T, int64_t H,
                   int post, const float *post_weight, const float *post_bias, float post_eps,
                   const void *gate, int gate_type, int64_t gate_rows, float alpha,
                   int pre, const float *pre_weight, const float *pre_bias, float pre_eps,
                   void *residual_out, void *n, int n_type, float *n_scale, void *stream);

/* ------------------------------------------------------------------------
 * Attention between two linear layers: the norm and the rotation of heads, a
 * paged cache of keys and values in 4-bit codes, and attention over it, for all
 * P shards.
 *
 * Extra conventions of these calls
 *  - Heads: x[p,t,h,:] starts at element p*x_shard + t*x_pitch + h*x_head and its
 *    D features are contiguous, so the heads of a fused projection's rows are
 *    taken where they lie. Strides are >= 0. Those of an output leave no element to
 *    two heads: each (of a size above 1) is at least what the smaller ones span.
 *  - A batch is B sequences one after another: the rows of sequence b are
 *    seq_starts[b] <= t < seq_starts[b+1] (i32 [B+1], ascending), lengths[b] (i32
 *    [B]) is the number of its tokens in the cache WITH those rows, so row t has
 *    the place lengths[b] - seq_starts[b+1] + t. Rows before seq_starts[0] and
 *    from seq_starts[B] on belong to no sequence and are left as they are.
 *    A sequence may have no rows, or no tokens.
 *  - page_table i32 [B,max_pages]: the page that holds places i*page_size .. of a
 *    sequence. An entry outside [0,pages) is no page: it is not read, and its
 *    places are not in the cache. The table's places, max_pages*page_size, may be
 *    2^30 at most.
 *  - These arrays are read on the device. Whatever they hold, no call touches
 *    memory outside its tensors. Starts are cut to [0,T] and lengths to the table's
 *    places, and rows and places follow from the cut ones; where starts do not
 *    ascend, the results are unspecified.
 *  - cache u8 [P,pages,Hk,page_size/32,btq_kv_block_bytes(D)], 16-byte aligned;
 *    page_size a power of 2 from 32 to 65536, D a multiple of 32 up to 256.
 *    A block holds 32 tokens of a key head:
 *      keys    [32][D/2]  feature 2i in the low nibble of byte i, 2i+1 in the high
 *      values  [D][16]    token 2i in the low nibble of byte i, 2i+1 in the high
 *      words   u32 [32] of the keys, then u32 [32] of the values: the bf16 bits
 *              of the scale in the high half, those of 128 + z in the low half
 *    A code c stands for scale*(c - z).
 *  - rope: cos_table and sin_table fp32 [rope_rows,rope_dim/2], row = position.
 *    The first rope_dim features (even, <= D) turn in pairs (a, b) ->
 *    (a*cos - b*sin, b*cos + a*sin), each product and sum one fp32 operation:
 *    BTQ_ROPE_HALF pairs feature i with i + rope_dim/2, BTQ_ROPE_PAIRS 2i with
 *    2i+1, both by column i. Both tables NULL: no rotation. A position outside
 *    the table turns its features to NaN.
 *  - NaN and Inf are carried: see each call.
 * ------------------------------------------------------------------------ */

typedef enum { BTQ_ROPE_HALF = 0, BTQ_ROPE_PAIRS = 1 } btq_rope;

/* Bytes of a block of 32 tokens of a key head, 32*D + 256; 0 for a D that the
 * cache does not take. */
int64_t btq_kv_block_bytes(int64_t D);

/*
 * The norm of each query and key head over its D features, with the rotation by
 * its token's position, in one pass:
 *   y = rope(norm(x) * weight)
 * in fp32, rounded once. norm is a btq_norm over the head (no bias).
 *   x         fp32 or bf16 [P,T,q_heads+k_heads,D] in: query heads first
 *   q_weight, k_weight  fp32 or NULL (1): the weights of head h of shard p start
 *             at p*qw_shard + h*qw_head (k: kw_*, h from 0); strides 0 for one
 *             set of D weights
 *   positions i32 [T] in, or NULL without tables
 *   y         fp32 or bf16 [P,T,q_heads+k_heads,D] out, strides of its own. It
 *             may be x itself (same address, type and strides); no other overlap.
 * 1 <= D <= 65536, q_heads and k_heads >= 0, one of them at least. NaN and Inf
 * spread to their head as the formulas give them. The vector kernel takes
 * D <= 1024, D and rope_dim multiples of 16, heads, weights and tables on 16
 * bytes, and fewer than 2^25 heads a shard; others take a general one.
 */
int btq_head_norm_rope(const void *x, int x_type, int64_t x_shard, int64_t x_pitch, int64_t x_head,
                       int64_t P, int64_t T, int64_t q_heads, int64_t k_heads, int64_t D,
                       int norm, const float *q_weight, int64_t qw_shard, int64_t qw_head,
                       const float *k_weight, int64_t kw_shard, int64_t kw_head, float eps,
                       const int32_t *positions, const float *cos_table, const float *sin_table,
                       int64_t rope_rows, int64_t rope_dim, int rope,
                       void *y, int y_type, int64_t y_shard, int64_t y_pitch, int64_t y_head,
                       void *stream);

/*
 * Appends the batch's keys, rotated by their places, and values to the cache.
 * For each row of D fp32 values (a key after its rotation), with 0 in the range,
 * lo = min(0, x), hi = max(0, x):
 *   scale = (hi - lo)/15 rounded up to bf16; below 2^-126: 1
 *   z     = rint(-lo/scale),  code = clamp(rint(x/scale) + z, 0, 15)
 * rint is to nearest even; the quotients are rounded once, so for bf16 rows
 * without rotation the codes are those of exact arithmetic, ties included. No
 * value moves by more than scale/2. A row that holds NaN or Inf, or whose range
 * passes the largest fp32, gets scale NaN and codes 0: queries that see it get NaN.
 *   k, v      fp32 or bf16 (both x_type) [P,T,Hk,D] in
 * A row whose place is negative (more rows than lengths[b]) or has no page is
 * dropped. Other places of the pages keep what they hold. A block of 32 places that a call
 * writes must belong to one sequence of it: sequences may share the pages of a prefix that
 * is there already, not one that both write, not even at places of their own (a byte holds
 * two of them). Calls that write one page must not run at once, and one that reads it
 * must wait for them.
 */
int btq_kv_append(const void *k, const void *v, int x_type, int64_t k_shard, int64_t k_pitch,
                  int64_t k_head, int64_t v_shard, int64_t v_pitch, int64_t v_head,
                  int64_t P, int64_t T, int64_t Hk, int64_t D,
                  const int32_t *seq_starts, const int32_t *lengths, int64_t B,
                  const int32_t *page_table, int64_t max_pages,
                  const float *cos_table, const float *sin_table, int64_t rope_rows,
                  int64_t rope_dim, int rope,
                  uint8_t *cache, int64_t pages, int64_t page_size, void *stream);

/*
 * What the cache holds for the batch's rows: k[p,t,h,:] = scale*(code - z) of the
 * key at row t's place, v the same of the value, in fp32, rounded once. Rows
 * without a place in the cache get zeros.
 *   k, v      fp32 or bf16 (both y_type) [P,T,Hk,D] out; one may be NULL
 * With lengths as btq_kv_append had them it reads back what that call wrote; with
 * others any stretch of the cached sequences.
 */
int btq_kv_gather(const int32_t *seq_starts, const int32_t *lengths, int64_t B,
                  const int32_t *page_table, int64_t max_pages,
                  const uint8_t *cache, int64_t pages, int64_t page_size,
                  int64_t P, int64_t T, int64_t Hk, int64_t D,
                  void *k, void *v, int y_type, int64_t k_shard, int64_t k_pitch, int64_t k_head,
                  int64_t v_shard, int64_t v_pitch, int64_t v_head, void *stream);

/*
 * Attention of the batch's queries over the cache. Query head h reads key head
 * h/(Hq/Hk). For a row at place i, over the keys j in the cache that it sees,
 *   t[j] = scale * sum_d q[d]*k[j,d],  out = sum_j exp(t[j])*v[j] / sum_j exp(t[j])
 *   lse  = log(sum_j exp(t[j]))
 * It sees j < lengths[b], and j <= i if causal, and j > i - window if window > 0.
 * A row that sees no key gets out 0 and lse -Inf.
 * Scores and sums are fp32; the weight exp(t - max)*(scale of v[j]) is rounded to
 * bf16 for the second product. NaN or Inf in a query gives NaN; a NaN key or value
 * gives NaN to the queries that see it and to no others.
 * With many queries a sequence, those of up to 128 (query, head) pairs are held as fp16
 * relative to the largest of them: exact down to 2^-27 of it. With queries of up to 2^100,
 * scale up to 2^30 and values of up to 2^80 nothing overflows where q.k and the scores do
 * not, whatever the number of keys. Larger values may give NaN: the sums on the way hold up to
 * 2^8*(143*1024 + 15*keys) steps of a value's scale.
 *   q         bf16 [P,T,Hq,D] in; fastest with heads on 16 bytes
 *   scale     > 0, at most 2^127
 *   max_length  an upper bound of lengths (0: the table's places) by which the
 *             keys are split over the chip. Longer sequences are as correct,
 *             and may be slower.
 *   out       fp32 (8-byte aligned) or bf16 (4-byte aligned) [P,T,Hq*D] out,
 *             contiguous: an x of btq_int8_linear
 *   lse       fp32 [P,T,Hq] out, or NULL
 *   workspace at least btq_kv_attention_workspace_bytes bytes of the same sizes,
 *             16-byte aligned, with no initial value (NULL if that is 0). Calls at
 *             the same time need one each.
 * One launch, or two where keys are split. The same call gives the same bits. By
 * which kernel and in which pieces keys are summed is chosen by the sizes, and where
 * equal shares of a batch's keys are taken also by all its lengths, so the last bits
 * of a sequence's result may differ between batches; the contents of other sequences
 * do not matter.
 */
int btq_kv_attention(const void *q, int64_t q_shard, int64_t q_pitch, int64_t q_head,
                     int64_t P, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                     const int32_t *seq_starts, const int32_t *lengths, int64_t B,
                     const int32_t *page_table, int64_t max_pages,
                     const uint8_t *cache, int64_t pages, int64_t page_size,
                     float scale, int causal, int64_t window, int64_t max_length,
                     void *out, int out_type, float *lse,
                     void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes for btq_kv_attention (0 for sizes that it refuses). max_length
 * 0 stands for the table's places, max_pages*page_size. */
size_t btq_kv_attention_workspace_bytes(int64_t P, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                        int64_t B, int64_t max_pages, int64_t page_size,
                                        int64_t max_length);

/* Static text for a btq_status value (never NULL). */
const char *btq_status_str(int status);

/* Library version, "major.minor.patch". */
const char *btq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BTQ_H */
