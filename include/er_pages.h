/*
 * er_pages.h -- C ABI of liber.so, continued: a paged 4-bit K/V cache shared by
 * many sequences.  The conventions of er.h hold for every call here.
 */
#ifndef ER_PAGES_H
#define ER_PAGES_H

#include "er.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bfloat16 (GGUF's type code), a type of the rows of the calls below only. */
enum { ER_BF16 = 30 };

/* Paged 4-bit K/V cache: the cache of many sequences of any length in one pool
 * of fixed-size pages, with the calls that give pages to sequences, write rows
 * and attend over them.  It stands beside er_kv (at most 16 sequences, each
 * with its own fixed capacity, fp16 or Q8_0 rows) for callers that run the
 * projections themselves, for instance with er_matrix_gemv.
 *
 * Rows.  Each head's row of head_dim values is kept as head_dim / 32 Q4_0 blocks
 * of one fp16 scale d and 32 codes c in 0..15; a value reads back as d (c - 8).
 * Quantiser, for every row written, in float32: m = the value of largest size
 * of the block (the first of them), d = fp16(bf16(-m / 8)) limited to +-2720,
 * c = clamp(round(x / d) + 8, 0, 15) with halves away from zero, c = 8 where d
 * is 0.  The scale has 8 significant bits, so d (c - 8) has at most 11: every
 * value is an fp16 number exactly (against an fp16 scale's 11 bits this moves
 * a block's values by at most 1 in 512, where a code's step is 1 in 8).  Values
 * past 21760 saturate; a block with a NaN reads back as NaN.
 *
 * Pool.  pool_dev is the caller's memory, er_pages_pool_bytes long, 16-byte
 * aligned: [n_layers][n_pages][n_kv_heads][page_rows / 16] tiles of 16 rows,
 * 18 * head_dim bytes each, hd = head_dim:
 *   K codes  8 hd bytes  row by row, hd / 8 words of 32 bits a row.  Word
 *            t * (hd / 32) + b (t < 4, b < hd / 32) holds the dims 32 b + 8 t + j,
 *            j < 8: dim 2 i + e of those 8 at bits 4 i + 16 e (i < 4, e < 2).
 *   K scales hd bytes    fp16 [16 rows][hd / 32]
 *   V codes  8 hd bytes  words [hd / 64][8 g][4 t][4 u]: word (q, g, t, u) holds
 *            the dims 64 q + 16 u + g (low nibble of each byte) and that + 8 (high
 *            nibble), of row 2 t + e + 8 i in byte i + 2 e (i < 2, e < 2)
 *   V scales hd bytes    fp16 [4 t][hd / 32][2 i][2 e] of row 2 t + e + 8 i
 * A slot is page * page_rows + row of the page.  Nothing initialises the pool:
 * rows are read only after they are written.
 *
 * Configuration.  page_rows: a multiple of 16 up to 1024; head_dim 64 or 128
 * (else ER_EUNSUPPORTED); kv_type ER_Q4_0 (another er_dtype: ER_EUNSUPPORTED);
 * n_pages * page_rows < 2^31 and that times n_kv_heads < 2^35.  The handle owns scratch only; it belongs to the
 * device it was created on, and so do the pool and every array of a call (a pool of another device, or a call with another
 * device current, is ER_EINVAL).
 * The calls of one handle share its scratch: order them (one stream, or
 * events), captured graphs of them included.  Work that overlaps takes a handle
 * each: any number of handles may be made over one pool. */
typedef struct er_pages er_pages;
typedef struct {
    int32_t n_layers, n_pages, page_rows, n_kv_heads, head_dim, kv_type;
} er_pages_config;
/* Bytes of the pool, or 0 for a configuration that er_pages_create refuses. */
ER_API size_t er_pages_pool_bytes(const er_pages_config *cfg);
/* Allocates the handle's scratch and synchronises the device. */
ER_API er_status er_pages_create(const er_pages_config *cfg, void *pool_dev, er_pages **out);
ER_API void er_pages_destroy(er_pages *p);

/* One step's block tables and slot maps, built on the device from the requests'
 * lengths.  Request b < n_seqs (<= 1024) holds lens_dev[b] rows in the pages of
 * tables_dev[b][0 .. ceil(lens / page_rows) - 1] and brings new_dev[b] tokens.  In
 * order of b, a request is admitted while the pages that it and those before it
 * need are at most *free_count_dev and their new tokens at most max_tokens; the
 * first that does not fit and every one after it get nothing (flag bit 0).  A
 * request with a negative length or count, or whose rows pass its table
 * (table_stride pages) or 2^31 - 1025, gets nothing either, by itself (flag bit 1).  Written:
 *   tables_dev           [n_seqs][table_stride]: the new pages' entries only; the
 *                        i-th page given out is free_dev[*free_count_dev - 1 - i]
 *   lens_out_dev         [n_seqs] lens + admitted tokens (may be lens_dev)
 *   free_count_out_dev   [1] (may be free_count_dev)
 *   q_start_dev          [n_seqs + 1]: request b's tokens are rows q_start[b] ..
 *                        q_start[b + 1] - 1 of the step
 *   positions_dev, slots_dev, seqs_dev  [max_tokens]: a token's position, slot and
 *                        request; 0, -1, -1 behind the last token
 * Other outputs must not overlap the inputs. */
typedef struct {
    int32_t n_seqs, max_tokens, table_stride;
    const int32_t *lens_dev, *new_dev, *free_dev, *free_count_dev;
    int32_t *tables_dev, *lens_out_dev, *free_count_out_dev, *q_start_dev, *positions_dev, *slots_dev, *seqs_dev;
} er_pages_plan_args;
ER_API er_status er_pages_plan(er_pages *p, const er_pages_plan_args *a, void *stream);
/* Gives back the pages of every request with done_dev[b] != 0: they go on top of
 * free_dev in order of request and block, *free_count_dev grows, lens_dev[b]
 * becomes 0 and the table's entries of the pages become -1.  An entry outside the
 * pool, or one for which free_dev (n_pages long) has no room, is dropped (flag
 * bit 1).  n_seqs * table_stride: at most 2^31 - 1024. */
ER_API er_status er_pages_release(er_pages *p, int32_t n_seqs, const int32_t *done_dev, int32_t *lens_dev,
                                  int32_t *tables_dev, int32_t table_stride, int32_t *free_dev,
                                  int32_t *free_count_dev, void *stream);

/* (cos, sin) of p * base^(-2 i / head_dim), computed in float64, as fp32
 * out_dev[n_positions][head_dim / 2][2], the table er_pages_append reads.  Memory of
 * another device than the current one is ER_EINVAL. */
ER_API er_status er_rope_table(int32_t head_dim, double base, int32_t n_positions, float *out_dev, void *stream);

/* Norms of queries and keys for each head, their rotation and the K/V append, in
 * one pass.  Row t < n_tokens of q_dev ([n_heads][head_dim] of `type`, rows
 * q_stride values apart), k_dev and v_dev ([n_kv_heads][head_dim]):
 *   y = x * gain / sqrt(mean(x^2) + eps) over the head (no gain: y = x), then, with
 *   a rope table, pair i rotated by row positions_dev[t] of the table:
 *   (a, b) -> (a cos - b sin, b cos + a sin); rope_style ER_ROPE_PAIRS pairs the
 *   dims (2 i, 2 i + 1), ER_ROPE_HALVES (i, i + head_dim / 2).
 * Queries go to q_out_dev (`type`, rows q_out_stride apart, may be q_dev itself),
 * keys (normed and rotated) and values (as they are) into slot slots_dev[t] of
 * `layer`.  Queries are worked in float32: with eps above 2^-90, a query row whose
 * squares' sum passes float32's largest number becomes zeros.  A key's codes are those of the formula in float64 rounded to float32:
 * rows near a border are computed again in float64.
 *   - A row with a negative slot is skipped whole: nothing of it is read or
 *     written.  A slot past the pool, or with a rope table a position outside
 *     it, skips the row too and sets flag bit 1.
 *   - Rows may come in any order; two rows with one slot leave it unspecified.
 *   - n_heads = 0 (q_dev NULL) appends only.  `type`: ER_F32, ER_F16, ER_BF16.
 *     Strides: at least a row's values; any alignment of the type's own size. */
typedef enum { ER_ROPE_PAIRS = 0, ER_ROPE_HALVES = 1 } er_rope_style;
typedef struct {
    int32_t n_tokens, n_heads, type, rope_style, rope_positions;
    const void *q_dev, *k_dev, *v_dev;
    void *q_out_dev;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const float *q_gain_dev, *k_gain_dev;  /* [head_dim] or NULL */
    const float *rope_dev;                 /* [rope_positions][head_dim / 2][2] or NULL */
    const int32_t *positions_dev;          /* [n_tokens] (NULL without a rope table) */
    const int32_t *slots_dev;              /* [n_tokens] */
    float eps;
} er_pages_append_args;
ER_API er_status er_pages_append(er_pages *p, int32_t layer, const er_pages_append_args *a, void *stream);

/* Rows slots_dev[0 .. n - 1] of `layer` as values of `type` (ER_F32, ER_F16 exactly,
 * ER_BF16 rounded), k_out_dev and v_out_dev [n][n_kv_heads][head_dim] (either may
 * be NULL).  A negative slot's row is left as it was; one past the pool too, with
 * flag bit 1. */
ER_API er_status er_pages_read(er_pages *p, int32_t layer, int32_t n, const int32_t *slots_dev, int32_t type,
                               void *k_out_dev, void *v_out_dev, void *stream);

/* Attention of new tokens over the paged cache.  Sequence b < n_seqs has the rows
 * q_start_dev[b] .. q_start_dev[b + 1] - 1 of q_dev ([n_tokens][n_heads][head_dim] of
 * `type`, rows q_stride values apart) and lens_dev[b] cached rows, its new tokens'
 * own among them, in the pages of tables_dev[b] ([n_seqs][table_stride]).  Token i of
 * its n_b tokens is at position p = lens_dev[b] - n_b + i and attends rows
 * max(0, p - window + 1) .. p (window 0: rows 0 .. p); query head h reads KV head
 * h / (n_heads / n_kv_heads):
 *   out = sum_r softmax_r(scale * q . k_r) v_r     (scale 0: 1 / sqrt(head_dim))
 * out_dev: `type`, rows out_stride apart; may be q_dev itself.  lse_dev (fp32 [n_tokens][n_heads], may
 * be NULL): log of sum_r exp(scale q . k_r).  A token that attends no row (p < 0) gets zeros and
 * -infinity.  Any mix of single tokens and prompts; rows of q_dev that belong to
 * no sequence are left alone.  Scores, softmax and sums are fp32; fp32 queries
 * and the probabilities of every type enter the tensor cores as two fp16 halves
 * each (2^-22), 16-bit queries exactly (but for values below 2^-31 of their row's
 * largest).  Results do not depend on timing.
 *   - A q_start_dev that falls or passes n_tokens, a length below 0, past the
 *     table or past 2^31 - 1025, and a table entry outside the pool set flag bit 1 and leave that
 *     sequence's outputs unspecified (a q_start_dev that falls: all outputs); nothing outside the pool is read.
 *   - A NaN in a cached row makes NaN of at least its 32 dims (of a value) or of
 *     the whole head (of a key) in every token that attends the row, and of
 *     nothing in those that do not.
 *   - n_heads must be a multiple of n_kv_heads, at most 64 times it, and n_tokens
 *     times that ratio below 2^31 - 1024. */
typedef struct {
    int32_t n_seqs, n_tokens, n_heads, type, table_stride, window;
    const void *q_dev;
    void *out_dev;
    float *lse_dev;
    int64_t q_stride, out_stride;
    const int32_t *q_start_dev, *lens_dev, *tables_dev;
    float scale;
} er_pages_attention_args;
ER_API er_status er_pages_attention(er_pages *p, int32_t layer, const er_pages_attention_args *a, void *stream);

/* Failure injection for tests of the bounded waits, as er_kv_inject_wait_shortfall
 * for the paged attention: with extra > 0 the first CTA of each of its kernels waits,
 * in calls made (or captured) from then on, for `extra` more arrivals than there are.
 * The wait runs out (er_set_wait_limit_ns) and the kernel returns.  extra = 0 (the
 * default) restores normal calls.  ER_EINVAL outside 0..1024. */
ER_API er_status er_pages_inject_wait_shortfall(er_pages *p, int32_t extra);

/* Synchronises the device, then reports and clears the handle's flags: bit 0: a
 * request was not admitted (pages or rows ran out), bit 1: a length, position,
 * slot or table entry was out of range, bit 2: a wait inside a kernel gave up
 * (internal error): what that attention and any later one of the handle wrote before
 * this call is unspecified.  Returns ER_EDEVICE if *code != 0, else ER_OK. */
ER_API er_status er_pages_error(er_pages *p, int32_t *code);

#ifdef __cplusplus
}
#endif
#endif /* ER_PAGES_H */
