/*
 * er_requests.h -- C ABI of liber.so, continued: what many requests bring to a step.  Products of a block-quantized matrix
 * with any number of tokens, low-rank adapters of the requests beside them, and tokens sampled from logits by each request's
 * parameters.  The conventions of er.h hold for every call here.
 */
#ifndef ER_REQUESTS_H
#define ER_REQUESTS_H

#include "er.h"
#include "er_pages.h" /* ER_BF16 */

#ifdef __cplusplus
extern "C" {
#endif

/* Low-rank adapters of one matrix shape [rows x cols], for the requests that share the matrix: adapter i adds
 * scale_i * B_i (A_i x) to the product, A_i [rank_i x cols], B_i [rows x rank_i].  The handle owns them in the layout that
 * er_matrix_mul reads (A as fp16 rows, each times a power of two, B as it is); it belongs to the device it was created on.
 *   type      ER_F16 or ER_BF16: the type of every A and B
 *   slots     adapters that it holds (1..4096);  max_rank  1..256
 * A's values enter the products exactly but for those below 2^-31 (ER_F16: 2^-28) of their row's largest. */
typedef struct er_adapters er_adapters;
typedef struct {
    int32_t rows, cols, slots, max_rank, type;
} er_adapters_config;
/* Every slot starts empty.  Synchronises the device.  cols: a positive multiple of 32. */
ER_API er_status er_adapters_create(const er_adapters_config *cfg, er_adapters **out);
ER_API void er_adapters_destroy(er_adapters *ad);
/* Bytes of device memory that the handle owns (0 for NULL). */
ER_API size_t er_adapters_device_bytes(const er_adapters *ad);
/* Puts an adapter into `slot` (over what is there): a_dev [rank][cols], b_dev [rows][rank], dense.  Queued on `stream`: calls
 * queued before it that use the slot still see the old one, calls after it the new one, captured ones too when they are
 * replayed; calls on other streams are the caller's to order.  rank 1..max_rank; scale finite. */
ER_API er_status er_adapters_set(er_adapters *ad, int32_t slot, int32_t rank, float scale, const void *a_dev,
                                 const void *b_dev, void *stream);
/* Empties `slot`, in the same order: tokens with its number get no adapter. */
ER_API er_status er_adapters_clear(er_adapters *ad, int32_t slot, void *stream);

/* y[t] = W x[t] + scale_a B_a (A_a x[t]), a = ids_dev[t], for the tokens t < n_tokens: the product of er_matrix_gemv for any
 * number of rows of three types, with the adapters of the requests.
 *   x_dev   rows of mat's cols values of `type` (ER_F32, ER_F16, ER_BF16), x_stride values apart
 *   y_dev   rows of mat's rows values of `type`, y_stride values apart; must not overlap x_dev
 *   adapters, ids_dev  both or neither: int32 [n_tokens], the slot of each token; a negative number or an empty slot: none.
 *           A number past the slots gets none too and sets flag bit 1 (er_matrix_mul_error).  A shape of the matrix.
 *   work_dev  er_matrix_mul_work_bytes of scratch, 256-byte aligned.  Its contents need no preparation and mean nothing after
 *           the call; calls that may run at the same time take scratch of their own each.  Those that one host thread queues on
 *           one stream share it; other threads' calls, on that stream too, do not: a call is up to four launches.
 * Sums are fp32; beyond 16 tokens the tensor cores add, which cut a sum off at 2^-23 of it 8 times for 64 columns: in calls of up to
 * 128 tokens sums of 16 such steps (fp32 rows: of 2, in calls of any size) go on to nearest, in larger ones all columns add up there.
 * 16-bit rows enter the products exactly, as fp16 numbers times a power of two of their row, but for values below 2^-31 (fp16 rows:
 * 2^-28) of their row's largest; fp32 rows as fp16 pairs (2^-22).  W's values (at most 19 bits) enter exactly; beyond 16 tokens, where
 * a row's largest scale is 256 and more (Q4_0: 4096), within 2^-32 (2^-36) of that scale times 128 (8).
 * A row of x with an infinity or a NaN gives a row of NaN of y, a row of W with such a scale a column of NaN; infinities and NaN
 * of an adapter stay with the tokens of its slot.  Results do not depend on timing.
 * ER_EINVAL: sizes, strides, alignment, a handle of another device than the current one or of another shape; n_tokens *
 * rows, n_tokens * cols must be below 2^40, n_tokens below 2^24. */
typedef struct {
    int32_t n_tokens, type;
    const void *x_dev;
    void *y_dev;
    int64_t x_stride, y_stride;
    const er_adapters *adapters;
    const int32_t *ids_dev;
    void *work_dev;
    size_t work_bytes;
} er_matrix_mul_args;
/* Scratch of a call with n_tokens rows of `type`, with adapters or without (NULL); 0 for what er_matrix_mul refuses. */
ER_API size_t er_matrix_mul_work_bytes(const er_matrix *mat, const er_adapters *adapters, int32_t n_tokens, int32_t type);
ER_API er_status er_matrix_mul(const er_matrix *mat, const er_matrix_mul_args *a, void *stream);
/* Synchronises the device, then reports and clears the matrix's flags: bit 1: an adapter number was past the slots, bit 2: a
 * wait inside a kernel gave up (internal error; that call's y is unspecified).  Returns ER_EDEVICE if *code != 0. */
ER_API er_status er_matrix_mul_error(er_matrix *mat, int32_t *code);
/* Failure injection for tests of the bounded waits, as er_kv_inject_wait_shortfall: with extra > 0 the first CTA of
 * er_matrix_mul's product waits, in calls made (or captured) from then on, for `extra` more arrivals than there are (calls of up
 * to 16 tokens have no such waits).  extra = 0 restores normal calls.  ER_EINVAL outside 0..1024. */
ER_API er_status er_matrix_mul_inject_wait_shortfall(er_matrix *mat, int32_t extra);

/* A token of each row of logits, by its request's parameters and a given random number, beside er_decode_step's greedy argmax.
 * Of row i ([vocab] values of `type`, rows `stride` values apart), with T = temperature, in this order:
 *   1. w_j = exp((x_j - max x) / T).  NaN and -infinity have no mass; of +infinities every one has mass 1 and nothing else any.
 *   2. in the order of falling logit, ties by index (-0 and 0 tie), the first top_k are kept (top_k <= 0 or >= vocab: all);
 *   3. of these the ones before which the sum of w is below top_p times their sum, the first always (top_p >= 1 or NaN: all);
 *   4. of these the ones with w_j >= min_p, the first always (min_p <= 0 or NaN: all).
 * tokens_dev[i]: the lowest index at which the running sum of the kept w, in the order of the vocabulary, is above uniform_dev[i]
 * times their sum; uniform in [0, 1) (below or NaN: 0; 1 and above: the last kept with a mass).
 * logprobs_dev[i] (may be NULL): log of the token's share of the kept sum.
 * T <= 0 or NaN, top_k 1, top_p <= 0: the largest logit, lowest index on ties, and 0; T in (0, 2^-120) counts as 2^-120.  A row without any mass (all NaN or
 * -infinity): token -1 and -infinity.  Arrays of parameters are [n_rows] or NULL (temperature 1, nothing left out); top_k64_dev is
 * top_k in 64 bits, for callers who have it so: with both ER_EINVAL.
 * The choice is that of the definition in 64 bits, but where a border lies within some 2^-40 of the sum; masses below 2^-45 of
 * the largest count as none, and at temperatures above 1e30 logits below 2^-86 are multiples of 2^-109.  vocab: at most
 * ER_SAMPLE_MAX_VOCAB (else ER_EUNSUPPORTED).  One launch, no scratch. */
#define ER_SAMPLE_MAX_VOCAB 262144
typedef struct {
    int32_t n_rows, vocab, type;
    const void *logits_dev;
    int64_t stride;
    const float *temperature_dev;
    const int32_t *top_k_dev;
    const float *top_p_dev, *min_p_dev, *uniform_dev;
    int32_t *tokens_dev;
    float *logprobs_dev;
    const int64_t *top_k64_dev;
} er_sample_args;
ER_API er_status er_sample(const er_sample_args *a, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* ER_REQUESTS_H */
