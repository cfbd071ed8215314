/*
 * kld_eval.h -- C ABI of the MI355X (gfx950) quantized-vs-base logit comparison.
 *
 * The operation. For every token position the caller holds two rows of
 * next-token logits over the full vocabulary: one from the base (BF16) model
 * and one from the quantized model. For each row pair the library computes
 *   - the KL divergence KL(P_base || Q_quant) of the quantized model's softmax
 *     from the base model's softmax, in nats, at temperature 1, over all
 *     `vocab` entries ("Mistral-Small-4-119B-2603 GSQ-RCO IQ3_S GGUF" model card,
 *     "How it was made" step 5 and the "Quality" section; "Qwen3.6 27B
 *     Quantization Benchmark", section "Understand KLD and Same Top P");
 *   - the argmax of each row, ties broken toward the lowest index, and whether
 *     the two argmaxes agree -- the "Same Top P" / same-top-1 test (same
 *     section of the Qwen3.6 benchmark page; "Unsloth Dynamic 3.0 GGUFs",
 *     "The Divergence-300 @32 Metric", which calls top-1 an argmax on one
 *     prediction);
 * and reduces the per-token values to the mean KLD, the max KLD (with its row)
 * and the fraction of rows whose top tokens agree, over every row evaluated
 * (the "Raw benchmark data" table of the Qwen3.6 page reports exactly such
 * means). The base logits are produced once and compared against each quant
 * in turn ("Measurement method" on the same page), so rows can be fed in any
 * order and in pieces, and reduced once.
 *
 * Layout. `base` and `quant` are device pointers to row-major, contiguous
 * [n_rows, vocab] arrays; row r starts at element r * vocab. Element types are
 * IEEE float32 or bfloat16 (1 sign, 8 exponent, 7 mantissa bits), chosen per
 * tensor at create time; bfloat16 is widened exactly to float32. All logits
 * must be finite: non-finite inputs give unspecified (but memory-safe)
 * results. The fastest path needs vocab % 8 == 0 and 16-byte-aligned row
 * pointers; any other shape is still handled, more slowly.
 *
 * Ownership. The caller owns `base`, `quant` and every `*_out` array (device
 * memory). The handle owns its per-token buffers (max_rows rows), the
 * reduction partials and a pinned host summary. Nothing is retained from the
 * caller's pointers after the work enqueued by a call has run.
 *
 * Streams. `stream` is a hipStream_t passed as void*; NULL means the default
 * stream. kld_eval_rows only enqueues work. kld_eval_reduce orders itself
 * after every earlier kld_eval_rows call on this handle, whatever stream it
 * used, and blocks until the summary is on the host.
 *
 * Errors. Every call returns a kld_status. Arguments are validated on the host
 * before any work is enqueued; an invalid call enqueues and writes nothing.
 * Errors reported by HIP while enqueueing or running work are latched in the
 * handle and returned by the next kld_eval_reduce / kld_eval_destroy.
 * kld_eval_last_error() returns a message for the calling thread's last
 * non-OK status. No C++ exception crosses this interface.
 *
 * Threading. Calls on one handle may come from several threads as long as
 * concurrent kld_eval_rows calls cover disjoint row ranges (the reductions
 * share one workspace per handle and run one at a time); results are
 * deterministic: for one handle they are bit-identical whatever the chunking,
 * call order or streams (the launch shape, and so the summation order, is a
 * function of the element types and the handle's max_rows only).
 */
#ifndef KLD_EVAL_H
#define KLD_EVAL_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kld_eval kld_eval; /* opaque handle */

typedef enum kld_dtype {
    KLD_DTYPE_F32 = 0,  /* IEEE binary32 */
    KLD_DTYPE_BF16 = 1  /* bfloat16, raw 16-bit patterns */
} kld_dtype;

typedef enum kld_status {
    KLD_OK = 0,
    KLD_ERR_INVALID_ARG = -1,      /* NULL pointer, vocab < 1, bad dtype, negative count ... */
    KLD_ERR_NO_DEVICE = -2,        /* no HIP device visible */
    KLD_ERR_UNSUPPORTED_ARCH = -3, /* current device is not gfx950 */
    KLD_ERR_OUT_OF_MEMORY = -4,    /* a device or pinned allocation failed */
    KLD_ERR_RANGE = -5,            /* row_offset + n_rows exceeds max_rows */
    KLD_ERR_HIP = -6,              /* HIP reported an error (latched) */
    KLD_ERR_BAD_HANDLE = -7,       /* NULL, destroyed or foreign handle */
    KLD_ERR_EMPTY = -8             /* reduce over zero rows */
} kld_status;

typedef struct kld_eval_summary {
    int64_t n_rows;      /* rows reduced */
    double kld_sum;      /* sum of per-token KLD (float64 accumulation, fixed order) */
    double kld_mean;     /* kld_sum / n_rows */
    double kld_max;      /* largest per-token KLD */
    int64_t kld_max_row; /* lowest row index attaining kld_max */
    int64_t n_match;     /* rows whose base and quant argmax agree */
    double same_top1;    /* n_match / n_rows */
} kld_eval_summary;

/*
 * Token-conditioned metrics over the rows whose next-token id t is in
 * [0, vocab). With log p(t) = z[t] - lse, per model:
 *   ppl_base = exp(-logp_base_sum / n_scored), ppl_quant likewise -- the
 *   "Mean PPL(Q)" column of the Qwen3.6 benchmark's "Raw benchmark data"
 *   table; ppl_ratio = ppl_quant / ppl_base, the perplexity ratio of the
 *   GSQ-RCO model card's "Quality" section; dp = q(t) - p(t), the change of
 *   the actual token's probability ("points" in that section), with its mean
 *   and its root mean square (the table's "RMS Δp (%)", as a fraction here).
 * A perplexity past the largest double is +inf; ppl_ratio is computed as
 * exp((logp_base_sum - logp_quant_sum) / n_scored), the same quantity, and
 * stays finite there. With n_scored == 0 every mean is NaN.
 */
typedef struct kld_eval_token_summary {
    int64_t n_scored;      /* rows with 0 <= t < vocab */
    int64_t n_invalid;     /* rows with t >= vocab: not scored, counted here */
    double logp_base_sum;  /* sum of log p_base(t) over scored rows (float64, fixed order) */
    double logp_quant_sum; /* sum of log p_quant(t) */
    double ppl_base;       /* exp(-logp_base_sum / n_scored) */
    double ppl_quant;      /* exp(-logp_quant_sum / n_scored) */
    double ppl_ratio;      /* ppl_quant / ppl_base = exp((logp_base_sum - logp_quant_sum) / n_scored) */
    double dp_mean;        /* mean of q(t) - p(t) */
    double dp_rms;         /* sqrt(mean of (q(t) - p(t))^2) */
} kld_eval_token_summary;

/*
 * Create a handle on the current HIP device for rows of `vocab` logits.
 *   vocab      1 .. 2^31-1 entries per row
 *   max_rows   >= 1: capacity of the per-token buffers (rows addressable by
 *              row_offset + r in kld_eval_rows)
 *   base_dtype, quant_dtype: a kld_dtype each
 * Returns KLD_ERR_INVALID_ARG, KLD_ERR_NO_DEVICE, KLD_ERR_UNSUPPORTED_ARCH or
 * KLD_ERR_OUT_OF_MEMORY on failure, with *out set to NULL.
 */
kld_status kld_eval_create(kld_eval** out, int64_t vocab, int64_t max_rows,
                           int32_t base_dtype, int32_t quant_dtype);

/*
 * Compare n_rows row pairs and store their per-token results at handle rows
 * [row_offset, row_offset + n_rows). Row r of `base`/`quant` is handle row
 * row_offset + r. Asynchronous on `stream`.
 *   kld_out          float32[n_rows]  KL(P_base || Q_quant) per row, nats
 *   match_out        uint8[n_rows]    1 when the argmaxes agree, else 0
 *   argmax_base_out  int32[n_rows]    lowest index of the base row's maximum
 *   argmax_quant_out int32[n_rows]    lowest index of the quant row's maximum
 * Each *_out is an optional device array (NULL skips it); the handle's own
 * buffers are always written. n_rows == 0 is a no-op. Rows whose single
 * pass's fp32 sums would lose the 1e-5 relative accuracy (one row far
 * flatter than the other, or far-apart dominant tokens) are evaluated a
 * second time in float64 by the same kernel (kld_eval_copy_row_flags reports
 * which, and why). Returns
 * KLD_ERR_RANGE when row_offset + n_rows > max_rows, KLD_ERR_INVALID_ARG for
 * NULL inputs or negative counts, KLD_ERR_HIP if the launch fails.
 */
kld_status kld_eval_rows(kld_eval* h, const void* base, const void* quant,
                         int64_t n_rows, int64_t row_offset,
                         float* kld_out, uint8_t* match_out,
                         int32_t* argmax_base_out, int32_t* argmax_quant_out,
                         void* stream);

/*
 * kld_eval_rows plus the token-conditioned metrics, in the same pass.
 *   tokens           int32[n_rows] device array: the id of the token that
 *                    follows each position. 0 <= t < vocab is scored; t < 0
 *                    marks a position with no next token (not scored); t >=
 *                    vocab is not scored and counted as invalid. NULL makes
 *                    this call identical to kld_eval_rows.
 *   logp_base_out    float32[n_rows]  log p_base(t), NaN where not scored
 *   logp_quant_out   float32[n_rows]  log p_quant(t), NaN where not scored
 *   dp_out           float32[n_rows]  p_quant(t) - p_base(t), NaN where not scored
 * Other arguments, outputs and errors as for kld_eval_rows; every *_out may be
 * NULL. Rows written by kld_eval_rows are "not scored".
 */
kld_status kld_eval_rows_tokens(kld_eval* h, const void* base, const void* quant,
                                const int32_t* tokens, int64_t n_rows, int64_t row_offset,
                                float* kld_out, uint8_t* match_out,
                                int32_t* argmax_base_out, int32_t* argmax_quant_out,
                                float* logp_base_out, float* logp_quant_out, float* dp_out,
                                void* stream);

/*
 * kld_eval_rows with its kernel timed by the launch itself, for callers that
 * measure the row pass without adding packets to the stream.
 *   start_event, stop_event  hipEvent_t (as void*), each may be NULL; created
 *                    by the caller (with timing, on the handle's device) and
 *                    still owned by it. The row kernel's dispatch records
 *                    start when the call's first launch begins and stop when
 *                    its last launch ends (hipExtLaunchKernel); the
 *                    elapsed time between them is the row pass alone. Neither
 *                    is recorded when n_rows == 0 or the call fails before
 *                    launching.
 * Results, outputs, ordering and errors as for kld_eval_rows (bit-identical
 * per-token results).
 */
kld_status kld_eval_rows_timed(kld_eval* h, const void* base, const void* quant,
                               int64_t n_rows, int64_t row_offset,
                               float* kld_out, uint8_t* match_out,
                               int32_t* argmax_base_out, int32_t* argmax_quant_out,
                               void* stream, void* start_event, void* stop_event);

/*
 * Reduce handle rows [0, n_rows) -- which must all have been written by
 * kld_eval_rows -- to a summary: float64 sum and mean of the per-token KLD,
 * the max and its lowest row, the match count and fraction. Deterministic:
 * the result depends only on the per-token values, not on how the rows were
 * chunked or which streams computed them. Blocks until *out is filled.
 * The handle keeps the results of its last reduction: a reduction (this call,
 * kld_eval_reduce_tokens or kld_eval_reduce_segments) over the same rows or
 * segments, with no kld_eval_rows* or kld_eval_rows_topk call in between,
 * returns them without launching anything.
 * Returns KLD_ERR_EMPTY for n_rows == 0, KLD_ERR_RANGE for n_rows > max_rows,
 * or a latched KLD_ERR_HIP.
 */
kld_status kld_eval_reduce(kld_eval* h, int64_t n_rows, kld_eval_summary* out, void* stream);

/*
 * kld_eval_reduce without the wait: enqueues the same reduction of handle rows
 * [0, n_rows) on `stream` and returns. The summary (the same bits
 * kld_eval_reduce returns) is written to *out, which must be memory the
 * device can write: device memory, or pinned host memory (hipHostMalloc);
 * read it once the stream has reached this point. Ordered after earlier
 * kld_eval_rows calls on any stream, and later reductions of this handle on
 * other streams order after it; rows overwritten by a later kld_eval_rows
 * call before this work runs give an undefined summary. Returns
 * KLD_ERR_INVALID_ARG for a NULL out, KLD_ERR_EMPTY for n_rows == 0,
 * KLD_ERR_RANGE for n_rows > max_rows, KLD_ERR_HIP for a latched error or a
 * failed launch.
 */
kld_status kld_eval_reduce_async(kld_eval* h, int64_t n_rows, kld_eval_summary* out, void* stream);

/*
 * Token-conditioned summary of handle rows [0, n_rows), computed by the same
 * deterministic reduction as kld_eval_reduce (float64 sums in a fixed order).
 * Blocks until *out is filled. Errors as for kld_eval_reduce.
 */
kld_status kld_eval_reduce_tokens(kld_eval* h, int64_t n_rows, kld_eval_token_summary* out, void* stream);

/*
 * Per-segment summaries: segment s covers handle rows
 * [offsets[s], offsets[s + 1]), for s in [0, n_segments) -- one summary per
 * context, per fixed-length chunk or per domain, as the pages report them
 * (GSQ-RCO model card, "Quality": per domain, over chunks of 512 tokens).
 *   offsets     host int64[n_segments + 1], non-decreasing, offsets[0] >= 0,
 *               offsets[n_segments] <= max_rows; every row in a segment must
 *               have been written. Segments may be empty and need not cover
 *               every row.
 *   kld_out     host kld_eval_summary[n_segments] (NULL skips). An empty
 *               segment has n_rows 0, NaN mean and fraction, kld_max -inf and
 *               kld_max_row -1.
 *   tok_out     host kld_eval_token_summary[n_segments] (NULL skips).
 * A segment [0, n) gives bit-for-bit what kld_eval_reduce and
 * kld_eval_reduce_tokens give for n rows. The handle grows a workspace for
 * more than one segment on first use (KLD_ERR_OUT_OF_MEMORY if that fails).
 * Blocks until the outputs are filled. Returns KLD_ERR_INVALID_ARG for NULL
 * offsets, n_segments outside [1, 2^30] or decreasing offsets, KLD_ERR_RANGE
 * for offsets outside [0, max_rows], or a latched KLD_ERR_HIP.
 */
kld_status kld_eval_reduce_segments(kld_eval* h, const int64_t* offsets, int64_t n_segments,
                                    kld_eval_summary* kld_out, kld_eval_token_summary* tok_out,
                                    void* stream);

/*
 * Copy the log-normalisers log(sum_i exp z_i) of handle rows
 * [row_offset, row_offset + n_rows), as computed by kld_eval_rows, to device
 * arrays (float32[n_rows] each, NULL skips). Asynchronous on `stream`, ordered
 * after earlier kld_eval_rows calls on any stream.
 */
kld_status kld_eval_copy_lse(kld_eval* h, int64_t row_offset, int64_t n_rows,
                             float* lse_base_out, float* lse_quant_out, void* stream);

/*
 * Conditioning flags of handle rows [row_offset, row_offset + n_rows): one
 * byte per row, written by the kld_eval_rows / kld_eval_rows_tokens call that
 * last wrote the row (0 for rows no such call has written; kld_eval_rows_topk
 * does not touch them). A nonzero byte means the row's single-pass fp32 sums
 * could not be trusted to the stated accuracy, and the same call evaluated
 * the row a second time in float64 (the KL definition of the GSQ-RCO model
 * card, "How it was made" step 5, summed term by term) and stored that
 * result. Bits:
 *   KLD_ROW_FLAG_AMPLIFIED   the sums' rounding is amplified past the KL
 *                            tolerance: one distribution far flatter than
 *                            the other
 *   KLD_ROW_FLAG_QUANT_MASS  the quant row's mass relative to its maximum is
 *                            under 1/4 of the base row's: its normaliser lost
 *                            bits to cancellation
 *   KLD_ROW_FLAG_CARRIED     rescales moved more mass between the two sums
 *                            than the quant normaliser's bound allows: one
 *                            row's running maximum jumped by tens of nats
 *                            while the other's did not
 *   flags_out   device uint8[n_rows], owned by the caller
 * Asynchronous on `stream`, ordered after earlier kld_eval_rows calls on any
 * stream. Returns KLD_ERR_INVALID_ARG for a NULL flags_out (with n_rows > 0)
 * or negative counts, KLD_ERR_RANGE when row_offset + n_rows > max_rows,
 * KLD_ERR_HIP if the copy fails.
 */
enum {
    KLD_ROW_FLAG_AMPLIFIED = 1,
    KLD_ROW_FLAG_QUANT_MASS = 2,
    KLD_ROW_FLAG_CARRIED = 4
};
kld_status kld_eval_copy_row_flags(kld_eval* h, int64_t row_offset, int64_t n_rows, uint8_t* flags_out,
                                   void* stream);

/*
 * Gradient of the per-token KL(P_base || Q_quant) with respect to the
 * quantized logits: grad[r][i] = scale * (q_i - p_i), where p and q are the
 * softmaxes of base row r and quant row r (the derivative of the log-sum-exp
 * is the softmax). This is the first step of the backward pass of the loss the
 * GSQ-RCO model card's end-to-end tuning minimises, KL(BF16 || quantized) of
 * the next-token distributions ("How it was made" step 7); `scale` is the
 * row's weight in that loss (1/N for the mean over N rows).
 *   base, quant  the same rows that kld_eval_rows evaluated into handle rows
 *                [row_offset, row_offset + n_rows): the float64
 *                log-normalisers saved there are reused, so this call reads
 *                the rows once more and needs no reduction
 *   grad_out     device [n_rows, vocab] row-major array of grad_dtype
 *                (KLD_DTYPE_F32, or KLD_DTYPE_BF16 rounded to nearest even),
 *                owned by the caller
 * Asynchronous on `stream`, ordered after earlier kld_eval_rows calls on any
 * stream. Rows overwritten by a later kld_eval_rows before this call's work
 * runs give undefined gradients. Returns KLD_ERR_INVALID_ARG for NULL
 * pointers, a bad grad_dtype or a non-finite scale, KLD_ERR_RANGE when
 * row_offset + n_rows > max_rows, KLD_ERR_HIP if the launch fails.
 */
kld_status kld_eval_grad(kld_eval* h, const void* base, const void* quant, int64_t n_rows,
                         int64_t row_offset, double scale, void* grad_out, int32_t grad_dtype,
                         void* stream);

/*
 * Base rows stored as their top-K tokens plus the rest of the mass -- the form
 * the GSQ-RCO model card tunes against ("How it was made" step 7: the BF16
 * model's top-128 distributions and the rest of the mass).
 *
 * kld_eval_topk_compress: for each of n_rows base rows ([n_rows, vocab] device
 * array of the handle's base dtype) store
 *   idx_out   int32[n_rows][k]  the k largest logits' indices, most probable
 *                               first, equal logits by lowest index (+0 and -0
 *                               are equal), so idx_out[r][0] is the argmax
 *   logp_out  float32[n_rows][k] their log-probabilities z - lse
 *   rest_out  float32[n_rows]   the probability of every other token, summed
 *                               over those tokens (0 when k == vocab)
 * k in [1, min(vocab, 1024)]. Device arrays, owned by the caller; handle rows
 * are not touched. Asynchronous on `stream`. Deterministic.
 *
 * kld_eval_rows_topk: like kld_eval_rows, with the base given in that stored
 * form (the same k) and the quantized rows in full ([n_rows, vocab] of the
 * handle's quant dtype). Per row it computes the KL divergence of both
 * distributions coarsened to the k stored tokens plus one outcome "any other
 * token":
 *   KL_k = sum_j p_j (log p_j - log q_j) + R (log R - log Q_rest)
 * (p_j = exp(logp[j]), R = rest; q_j, Q_rest from the quantized row; a term
 * with R == 0 is 0) -- the full KL when k == vocab, never more than it
 * otherwise -- and the top-1 match of the quantized argmax (lowest index)
 * with idx[0]. Results go to handle rows [row_offset, row_offset + n_rows)
 * exactly as kld_eval_rows writes them (kld, match, argmax_base = idx[0],
 * argmax_quant, log-normaliser of the quant row; the base log-normaliser is
 * NaN and no token is scored), so kld_eval_reduce and the segmented reduction
 * summarize them. Stored indices must be distinct and in [0, vocab): a row
 * that breaks this gets a NaN divergence and match 0. Needs vocab / 8 bytes of
 * on-chip memory per workgroup: KLD_ERR_INVALID_ARG when the device has too
 * little (vocab beyond about one million on gfx950).
 * Both return KLD_ERR_INVALID_ARG for NULL pointers, negative counts or a bad
 * k, KLD_ERR_RANGE when row_offset + n_rows > max_rows, KLD_ERR_HIP if a
 * launch fails.
 */
kld_status kld_eval_topk_compress(kld_eval* h, const void* base, int64_t n_rows, int32_t k,
                                  int32_t* idx_out, float* logp_out, float* rest_out, void* stream);

kld_status kld_eval_rows_topk(kld_eval* h, const int32_t* topk_idx, const float* topk_logp,
                              const float* topk_rest, int32_t k, const void* quant,
                              int64_t n_rows, int64_t row_offset,
                              float* kld_out, uint8_t* match_out,
                              int32_t* argmax_base_out, int32_t* argmax_quant_out,
                              void* stream);

/*
 * Gradient of the coarsened divergence KL_k of kld_eval_rows_topk with respect
 * to the quantized logits, the stored form held fixed -- the first step of the
 * backward pass of the GSQ-RCO model card's tuning phase against the top-128
 * distributions and the rest of the mass ("How it was made" step 7). With q the
 * quantized softmax, S the stored tokens, P = sum_j p_j, R = rest and Q_rest
 * the quantized mass outside S:
 *   grad[r][i] = scale * (q_i (P + R) - p_i)                 for i in S
 *   grad[r][i] = scale * q_i (P + R - R / Q_rest)            otherwise
 * (q - p when k == vocab). `scale` is the row's weight in the loss.
 *   topk_idx, topk_logp, k, quant
 *                the stored indices and log-probabilities and the quantized
 *                rows that kld_eval_rows_topk evaluated into handle rows
 *                [row_offset, row_offset + n_rows): the quant log-normaliser
 *                and the factors P + R and P + R - R / Q_rest that call saved
 *                there are reused (R enters only through them), so this call
 *                reads each quant row once more; rows last written by
 *                kld_eval_rows hold no such factors and give undefined
 *                gradients
 *   grad_out     device [n_rows, vocab] row-major array of grad_dtype
 *                (KLD_DTYPE_F32, or KLD_DTYPE_BF16 rounded to nearest even),
 *                owned by the caller; every entry is written
 * A row whose stored indices are not distinct and in [0, vocab) is written as
 * NaN. Asynchronous on `stream`, ordered after earlier calls on any stream.
 * Returns KLD_ERR_INVALID_ARG for NULL pointers, a bad k or grad_dtype or a
 * non-finite scale, KLD_ERR_RANGE when row_offset + n_rows > max_rows,
 * KLD_ERR_HIP if the launch fails.
 */
kld_status kld_eval_grad_topk(kld_eval* h, const int32_t* topk_idx, const float* topk_logp, int32_t k,
                              const void* quant, int64_t n_rows, int64_t row_offset, double scale,
                              void* grad_out, int32_t grad_dtype, void* stream);

/*
 * Measurement aid, not a step of the method: the attainable HBM read rate for
 * the row kernels' access pattern, to set their timing against. Reads n_rows
 * rows of row_bytes bytes from `a` (and, when `b` is not NULL, the same rows
 * of `b`) once, one workgroup of waves_per_row waves (1 or 4) per row,
 * 16-byte non-temporal loads from 1 KiB tiles, four tiles per row in flight
 * per wave -- the row kernel's load shapes with no arithmetic -- and writes
 * sink[r] = the XOR of every 32-bit word of row r of a (and b), so that the
 * reads are not removed and can be checked. Device pointers on the current
 * device; a, b 16-byte aligned, row_bytes a positive multiple of 16; sink is
 * uint32[n_rows], owned by the caller. Asynchronous on `stream`; no handle is
 * involved. start_event / stop_event (hipEvent_t as void*, each may be NULL,
 * created by the caller with timing): recorded by the probe's first launch
 * when it begins and by its last when it ends, as kld_eval_rows_timed does,
 * so the probe and the row pass are timed the same way. Returns
 * KLD_ERR_INVALID_ARG for NULL a or sink, negative n_rows, a bad row_bytes or
 * waves_per_row or misaligned pointers, KLD_ERR_HIP if the launch fails.
 */
kld_status kld_eval_read_probe(const void* a, const void* b, int64_t n_rows, int64_t row_bytes,
                               int32_t waves_per_row, uint32_t* sink, void* stream,
                               void* start_event, void* stop_event);

/*
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation. The same
 * comparison as kld_eval_rows over rows [0, n_rows) followed by
 * kld_eval_reduce, with no handle: it calls no allocator, enqueues everything
 * on `stream` and never blocks.
 *   base, quant   device [n_rows, vocab] arrays of base_dtype / quant_dtype
 *   kld_out       float32[n_rows], required (the reduction reads it)
 *   match_out     uint8[n_rows], required (the reduction reads it)
 *   argmax_base_out, argmax_quant_out   int32[n_rows], optional (NULL skips)
 *   summary_out   device memory for one kld_eval_summary, written by the
 *                 last kernel of the call; read it after the stream reaches
 *                 that point
 * The results are bit-identical to kld_eval_rows + kld_eval_reduce on a
 * handle created with max_rows = n_rows. The reduction's partials live in a
 * fixed workspace inside the library, one per GPU, sized for at most
 * 4,194,304 rows (320 KiB); calls on one GPU share it, so calls that overlap
 * on one GPU (two streams, or two threads) race and must be serialised by the
 * caller. Needs a gfx950 as the current device.
 * Returns KLD_ERR_INVALID_ARG for NULL required pointers, a bad vocab or
 * dtype, or negative n_rows; KLD_ERR_EMPTY for n_rows == 0; KLD_ERR_RANGE for
 * n_rows > 4194304; KLD_ERR_UNSUPPORTED_ARCH / KLD_ERR_NO_DEVICE for the
 * device; KLD_ERR_HIP if a launch fails.
 */
kld_status kld_eval_compare_noalloc(const void* base, const void* quant, int64_t vocab, int64_t n_rows,
                                    int32_t base_dtype, int32_t quant_dtype,
                                    float* kld_out, uint8_t* match_out,
                                    int32_t* argmax_base_out, int32_t* argmax_quant_out,
                                    kld_eval_summary* summary_out, void* stream);

/*
 * Operators around the model's vocabulary, for callers that let the compared
 * models answer (beam search over the same logit rows) or that carry the KL
 * gradient back to the embedding table. They take no handle and allocate
 * nothing: everything is enqueued on `stream` of the current device (a
 * gfx950), scratch memory is the caller's workspace, and every call may be
 * captured into a HIP graph. A workspace is 16-byte aligned device memory of
 * at least the size its query gives; nothing in it outlives the call's work, so
 * one may be used again by later calls on the same stream. Calls whose work may
 * overlap (two streams, two graphs) need one each. Device pointers must not
 * overlap one another unless stated. Errors of every call: KLD_ERR_INVALID_ARG,
 * KLD_ERR_RANGE past a stated limit, KLD_ERR_NO_DEVICE,
 * KLD_ERR_UNSUPPORTED_ARCH, KLD_ERR_HIP if a launch fails; arguments are
 * checked before anything is enqueued. Results do not depend on timing: the
 * same inputs give the same bits.
 *
 * kld_eval_beam_select: one step of beam search. Item i holds n_beams beams of
 * scores s_w = scores[i][w]; beam w's next-token logits are row
 * i * n_beams + w of `logits`. Logits that are not finite (NaN, either
 * infinity) are excluded tokens: they add nothing to the normaliser and are
 * never chosen. A live beam offers every other token v at
 * s_w + z_v - log(sum exp z); a finished beam offers only itself, as token
 * eos_token at s_w, whatever its logits are; a beam whose score is not finite
 * is empty and offers nothing. The n_select best of all beams together
 * are chosen, best first, equal scores by lowest beam, then lowest id. Scores
 * are compared as in float64 (one beam's candidates by their logits).
 *   logits       device rows of `vocab` elements of `dtype`, row_stride
 *                elements apart (>= vocab), n_items * n_beams of them (at most
 *                4,194,304); any alignment of the type
 *   n_beams      1 .. 64, n_select 1 .. 64
 *   finished     uint8[n_items][n_beams], nonzero for a finished beam, or NULL
 *                for none; needs an eos_token
 *   eos_token    id that ends a beam, in [0, vocab), or -1 for none
 *   scores_out   float32[n_items][n_select]  (a score past float32's range
 *                becomes an infinity and keeps its parent and token)
 *   parents_out  int32[n_items][n_select]  the chosen candidate's beam
 *   tokens_out   int32[n_items][n_select]  its token
 *   finished_out uint8[n_items][n_select]  1 if the beam was finished or the
 *                token is eos_token
 * Where fewer candidates exist the remaining outputs are score -inf, parent -1,
 * token -1, finished 0, which the next step, kld_eval_beam_reorder and
 * kld_eval_embed take as an empty beam. scores_out and finished_out may be
 * scores and finished themselves when n_select == n_beams. n_items == 0 is a
 * no-op.
 */
kld_status kld_eval_beam_select_workspace(int64_t vocab, int32_t dtype, int64_t n_items, int32_t n_beams,
                                          int32_t n_select, int64_t* bytes_out);

kld_status kld_eval_beam_select(const void* logits, int32_t dtype, int64_t vocab, int64_t row_stride,
                                int64_t n_items, int32_t n_beams, int32_t n_select, const float* scores,
                                const uint8_t* finished, int32_t eos_token, float* scores_out,
                                int32_t* parents_out, int32_t* tokens_out, uint8_t* finished_out,
                                void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Beam states (key and value caches, token histories, recurrent states) follow
 * the chosen beams, in place: beam w of item i becomes what beam parents[i][w]
 * was, over the item's first lengths[i] positions. A parent outside
 * [0, n_beams) leaves its beam as it is, positions from lengths[i] on are left
 * as they are.
 *   states       host array of n_states device pointers, read before the call
 *                returns; all of one geometry, none overlapping another
 *   parents      int32[n_items][n_beams] (n_items * n_beams at most 4,194,304)
 *   geometry     byte q of position t of outer index o of beam
 *                r = i * n_beams + w lies at r * beam_stride + o * outer_stride
 *                + t * position_bytes + q: [beams, heads, positions, dim] has
 *                n_outer = heads, [beams, positions, heads, dim] has n_outer = 1;
 *                strides in bytes, without overlap (a stride whose count is 1
 *                is not looked at)
 *   lengths      int32[n_items], taken into [0, n_positions], or NULL for
 *                n_positions everywhere
 * A count of zero is a no-op.
 *
 * kld_eval_beam_reorder_check makes the call's checks of the states and their
 * geometry alone, on the host, and enqueues nothing: states of several
 * geometries take a call each, and a caller who has had all of them checked
 * first is not left with some of them moved when a later one is refused.
 */
kld_status kld_eval_beam_reorder_check(void* const* states, int32_t n_states, int64_t n_items, int32_t n_beams,
                                       int64_t beam_stride, int64_t n_outer, int64_t outer_stride,
                                       int64_t n_positions, int64_t position_bytes);

kld_status kld_eval_beam_reorder(void* const* states, int32_t n_states, int64_t n_items, int32_t n_beams,
                                 const int32_t* parents, int64_t beam_stride, int64_t n_outer, int64_t outer_stride,
                                 int64_t n_positions, int64_t position_bytes, const int32_t* lengths, void* stream);

/*
 * Embedding lookup with scaling: out[n] = scale * table[tokens[n]], formed in
 * float64 and rounded once to out_dtype (nearest even). A negative id gives a zero row, an id >=
 * vocab a NaN row (it is never used as an address).
 *   table        device [vocab, dim] rows of table_dtype, table_stride elements
 *                apart (>= dim); dim 1 .. 2^24
 *   tokens       int32[n_tokens]
 *   out          [n_tokens, dim] rows of out_dtype, out_stride elements apart
 * Elements between the rows are left as they are. n_tokens == 0 is a no-op.
 */
kld_status kld_eval_embed(const void* table, int32_t table_dtype, int64_t vocab, int64_t dim, int64_t table_stride,
                          const int32_t* tokens, int64_t n_tokens, double scale, void* out, int32_t out_dtype,
                          int64_t out_stride, void* stream);

/*
 * Gradient of the lookup with respect to the table:
 *   out[v] = scale * sum over { n : tokens[n] == v } of grad[n]
 * summed in float32 in an order fixed by the sizes and the tokens, scaled and
 * added in float64, and rounded once to out_dtype. Ids outside [0, vocab) add nothing.
 *   grad         device [n_tokens, dim] rows of grad_dtype, grad_stride
 *                elements apart (>= dim); n_tokens at most 4,194,304
 *   out          [vocab, dim] rows of out_dtype, out_stride elements apart;
 *                vocab at most 2^24
 *   accumulate   0: every row is written, zero where no token names it;
 *                otherwise the sums are added to what `out` holds (rows that
 *                no token names are left as they are)
 * With n_tokens == 0 the rows are zeroed, or nothing is done when accumulating.
 */
kld_status kld_eval_embed_grad_workspace(int64_t vocab, int64_t dim, int64_t n_tokens, int64_t* bytes_out);

kld_status kld_eval_embed_grad(const void* grad, int32_t grad_dtype, int64_t grad_stride, const int32_t* tokens,
                               int64_t n_tokens, int64_t vocab, int64_t dim, double scale, void* out,
                               int32_t out_dtype, int64_t out_stride, int32_t accumulate, void* workspace,
                               int64_t workspace_bytes, void* stream);

/*
 * Operators with which an 8-bit model answers: rows rounded to 8-bit integers
 * with a scale each, the product of such rows with 8-bit weights (its logit
 * rows, or any of its linear layers), and drawing tokens from logit rows. As
 * the operators around the vocabulary: no handle, nothing allocated, everything
 * enqueued on `stream` of the current device, each call may be captured into a
 * HIP graph, arguments are checked before anything is enqueued, and the same
 * inputs give the same bits.
 *
 * kld_eval_quantize_int8: for each of n_rows rows of `dim` elements,
 *   scales[r] = a / 127 rounded to float32, a the row's largest magnitude
 *   q[r][i]   = 127 x[r][i] / a to the nearest whole number, ties to even, of
 *               the exact quotient: -127 .. 127
 * A row of zeros (dim 0 apart, which is refused) has scale 0 and q 0, a row with
 * a NaN or an infinity has scale NaN and q 0, so that what is computed from it
 * is NaN. Weights [n_cols, dim] have a scale per output channel in the same way.
 *   x            device rows of dtype, x_stride elements apart (>= dim); dim 1 .. 2^24
 *   q            int8 rows, q_stride elements apart (>= dim); any alignment
 *   scales       float32[n_rows]
 * Elements between the rows are left as they are. n_rows == 0 is a no-op.
 */
kld_status kld_eval_quantize_int8(const void* x, int32_t dtype, int64_t dim, int64_t x_stride, int64_t n_rows,
                                  int8_t* q, int64_t q_stride, float* scales, void* stream);

/*
 * Product of 8-bit rows with 8-bit weights:
 *   out[m][n] = x_scales[m] * w_scales[n] * sum_k x[m][k] * w[n][k]
 * The sum is exact (32-bit integers; dim at most 131071, KLD_ERR_RANGE beyond;
 * all 256 values of a byte are allowed). It is rounded to float32 and scaled,
 * within 3 * 2^-24 of the value and 2^-149, then rounded to out_dtype (nearest even).
 *   x            int8[n_rows][dim], x_stride bytes apart (>= dim)
 *   w            int8[n_cols][dim], w_stride bytes apart (>= dim)
 *   x_scales, w_scales   float32[n_rows], float32[n_cols], any values
 *   out          [n_rows, n_cols] rows of out_dtype, out_stride elements apart (>= n_cols)
 * n_rows at most 4,194,304, n_cols at most 2^31 - 1. Rows may start anywhere;
 * fastest where x, w and their strides are multiples of 16 bytes. Elements
 * between the rows of `out` are left as they are, bytes between the rows of x and
 * w do not matter. n_rows == 0 is a no-op.
 */
kld_status kld_eval_matmul_int8(const int8_t* x, int64_t x_stride, const float* x_scales, int64_t n_rows,
                                const int8_t* w, int64_t w_stride, const float* w_scales, int64_t n_cols,
                                int64_t dim, void* out, int32_t out_dtype, int64_t out_stride, void* stream);

/*
 * Draw one token from each of n_rows logit rows, from given random numbers.
 * Logits that are not finite are excluded tokens. With M the largest of the
 * others and w_v = exp((z_v - M) / temperature), tokens are ordered by logit,
 * equal logits by lowest id, and kept are
 *   - the first top_k of that order;
 *   - of those the shortest run from its beginning whose sum of w is at least
 *     top_p times the sum over all of those (always one token);
 *   - of those the ones with w >= min_p, min_p taken into [2^-64, 1].
 * The token is the first kept one, in order of ids, at which the running sum of
 * the kept w exceeds uniforms[r] times their whole sum; logp is the logarithm of
 * w over that sum, the log-probability with which it was drawn. Weights are formed
 * in float64 and rounded to 2^-45 of themselves, sums of them are exact or in float64,
 * and a sum that equals a border but for 2^-44 of itself counts as reaching it. Where no
 * limit is set the whole sum may hold tokens below 2^-64 that are not drawn, 2^-42 of it
 * at most.
 *   logits       device rows of `vocab` elements of dtype, row_stride elements
 *                apart (>= vocab); any alignment of the type; vocab and n_rows at most 4,194,304
 *   uniforms     float32[n_rows] in [0, 1): values outside are taken to its ends,
 *                NaN to 0
 *   temperatures, top_ks, top_ps, min_ps   device arrays [n_rows] (int32 for top_ks,
 *                else float32), or NULL: then temperature, top_k, top_p, min_p hold
 *                for every row (not NaN: KLD_ERR_INVALID_ARG). A temperature of 0 or
 *                less, or NaN, takes the largest logit (lowest id, logp 0); a top_k
 *                of 0 or less, a top_p of 1 or more or NaN, a min_p of 0 or less or
 *                NaN is no limit
 *   tokens_out   int32[n_rows], logp_out  float32[n_rows]
 * A row with no finite logit gets token -1 and logp -inf, which kld_eval_embed
 * takes as no token. n_rows == 0 is a no-op. The workspace is as described above
 * for the operators around the vocabulary.
 */
kld_status kld_eval_sample_workspace(int64_t vocab, int32_t dtype, int64_t n_rows, int64_t* bytes_out);

kld_status kld_eval_sample(const void* logits, int32_t dtype, int64_t vocab, int64_t row_stride, int64_t n_rows,
                           const float* uniforms, const float* temperatures, double temperature,
                           const int32_t* top_ks, int32_t top_k, const float* top_ps, double top_p,
                           const float* min_ps, double min_p, int32_t* tokens_out, float* logp_out,
                           void* workspace, int64_t workspace_bytes, void* stream);

/* Synchronize the handle's work and free it. NULL is a no-op returning KLD_OK. */
kld_status kld_eval_destroy(kld_eval* h);

/* Message for the calling thread's last non-OK status ("" if none). */
const char* kld_eval_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* KLD_EVAL_H */
