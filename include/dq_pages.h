/*
 * dq_pages.h -- paged KV cache in microscaled 4-bit floats: the part of libdq's
 * C ABI for serving many sequences of different lengths from one pool.
 *
 * What it computes
 * ----------------
 * A pool holds pages of page_size tokens; a row (sequence) is a list of pages
 * and a length, so rows share pages, grow, shrink and end without moving their
 * tokens.  A token's key and value of one KV head are held in 4-bit floats
 * (e2m1: 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign) with an e4m3 scale for every 16
 * channels:
 *   s = e4m3(min(448, max|x| / 6 / 2^exp)),  code = e2m1(x / (2^exp s)),
 *   held value = 2^exp s code,
 * both roundings to nearest, ties to even; exp is k_exp or v_exp, one for the
 * pool (a layer whose values are small needs a negative one: s below 2^-6 loses
 * precision and below 2^-10 becomes 0).  A page also carries a summary of its
 * keys, from which dq_pages_select tells cheaply which pages a query may need.
 *
 * A decode step of a model, with every argument in device memory and nothing
 * read back, so that it can be captured into a CUDA graph once:
 *   dq_pages_resize   each row gets room for its new token(s)
 *   per layer: dq_pages_append, then dq_pages_attention (or dq_pages_select and
 *   dq_pages_attention over what it chose)
 *
 * Conventions (beside those of dq.h: device pointers, 16-byte alignment, status
 * codes, work enqueued on `stream`, argument errors found on the host before
 * anything is enqueued)
 * ------------------------------------------------------------------------
 * - rows: device int32 [n_rows], the table rows of this call's sequences; NULL
 *   = rows 0 .. n_rows - 1.  A negative entry is a padding row: it holds
 *   nothing, and its queries' outputs are those of an empty sequence.  A call that
 *   writes (resize, fork, append) names a row once.
 * - cu: device int32 [n_rows + 1], where each row's new tokens begin among the
 *   call's n_tok tokens; NULL = one token for each row.  A row's n new tokens are
 *   its LAST n: they stand at positions [seq_len - n, seq_len), so a call that
 *   brings tokens follows a dq_pages_resize that counted them.  max_new is a
 *   bound on n over the call's rows (the host plans the launch with it).
 * - What only the device can see (row numbers, counts and page numbers out of
 *   range, a pool without free pages, non-finite input) is skipped there,
 *   latched in the status word and returned by dq_pages_check().  Nothing is
 *   read or written out of range for it; outputs that depend on it are
 *   unspecified (a table's entry that names no page: those of the row's queries).
 * - Nothing is allocated: the caller owns all buffers.  Calls that share a
 *   workspace must be ordered (one stream, or events between streams; two
 *   captured graphs that may run at the same time need a workspace each).
 *   Calls that change the same rows, pages or counts must be ordered as well.
 */
#ifndef DQ_PAGES_H
#define DQ_PAGES_H

#include "dq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DQ_PAGES_MAX_ROWS 1024          /* rows of a table and of a call */
#define DQ_PAGES_MAX_PAGES (1 << 20)    /* pages of a pool */
#define DQ_PAGES_MAX_SELECT 512         /* pages chosen for a row and KV head */

typedef struct {
    int n_layers;           /* >= 1: one table of rows serves every layer */
    int n_pages;            /* [1, DQ_PAGES_MAX_PAGES] */
    int page_size;          /* tokens: 16, 32, 64 or 128 */
    int n_kv_heads;         /* [1, 128] */
    int n_q_heads;          /* a multiple G n_kv_heads with G <= 16; query head h reads KV head h / G */
    int head_dim;           /* 64 or 128 */
    int max_seqs;           /* rows of the table, [1, DQ_PAGES_MAX_ROWS] */
    int max_pages_per_seq;  /* [1, 65536], and max_pages_per_seq * page_size <= 2^22 */
    int dtype;              /* DQ_F16 or DQ_BF16: keys, values, queries, outputs */
    int k_exp, v_exp;       /* [-16, 16] */
} dq_pages_config;

/*
 * Buffers (device).  dq_pages_sizes() gives the bytes of each, in field order.
 *
 * pages   [n_layers][n_pages][n_kv_heads][P d 9/8 bytes], P = page_size: the
 *         page's tokens in blocks of b = min(P, 64), each
 *           key codes    [b][d / 2]               channel 2j low, 2j + 1 high half of byte j
 *           key scales   [b][d / 16]
 *           value codes  [b / 8][d / 16][4][16]   8 tokens, 16 channels, pair of
 *                        tokens, channel: even token low, odd token high half
 *           value scales [b / 8][d / 16][4][2]    the same order
 * summary [n_layers][n_pages][n_kv_heads][2 d + 16 bytes]: int8 [d] largest and
 *         int8 [d] smallest held key of each channel over the page's tokens,
 *         int32 e, 12 unused bytes.  In units of 2^k_exp the largest is at most
 *         2^e times its byte and the smallest at least 2^e times its: bytes are
 *         rounded up and down, e = E - 7 for the largest magnitude m 2^E,
 *         m in [1/2, 1) (0 where every key is 0).  dq_pages_append works it out
 *         anew from all tokens that the page holds then; a copy or a move takes
 *         it along.  A row that is shortened leaves it: until the next append to
 *         the page it bounds the tokens that are left, and those that are gone.
 * table   int32 [max_seqs][max_pages_per_seq]: the pages of each row in order; -1
 *         behind the last.  All -1 at the start.
 * seq_len int32 [max_seqs], 0 at the start.
 * refs    int32 [n_pages]: rows that hold the page; 0 = free.  0 at the start.
 * status  16 bytes, 0 at the start.
 * workspace: 0 at the start, used by every call but dq_pages_append, _read, _fork
 *         and _select: 12 bytes a page and some 43 MB for the parts that attention's
 *         CTAs join.  Every call leaves it fit for the next one, a call whose wait
 *         ran out too.
 */
typedef struct {
    void *pages, *summary;
    int *table, *seq_len, *refs;
    void *status, *workspace;
} dq_pages_buffers;

#define DQ_PAGES_NUM_BUFFERS 7

/* Byte size of every dq_pages_buffers field into bytes[].  Host only.
 * Errors: DQ_EINVAL, DQ_EUNSUPPORTED (head_dim, page_size, dtype, G). */
dq_status dq_pages_sizes(const dq_pages_config *cfg, size_t bytes[DQ_PAGES_NUM_BUFFERS]);

/*
 * Set the lengths of n rows: row rows[i] to lens[i] tokens (device int32 [n]).
 * lens[i] = 0 frees a row.  In this order:
 *   1. pages wholly behind a row's new length lose a reference;
 *   2. a row that grows past a partly filled last page which other rows hold too
 *      takes a copy of it in every layer (copy on write).  Of several growing
 *      rows that alone share the page, the last in the list keeps it;
 *   3. each row in list order takes the lowest free pages: the copy's first.
 * All or nothing: a pool with too few free pages (DQ_ENOMEM from
 * dq_pages_check), a length outside [0, max_pages_per_seq * page_size], a row
 * >= max_seqs or a row named twice (DQ_EINVAL) changes nothing.  Negative rows
 * are skipped.  New pages hold whatever they held; dq_pages_append fills them.
 * Errors: DQ_EINVAL, DQ_EALIGN, DQ_ECUDA.
 */
dq_status dq_pages_resize(const dq_pages_config *cfg, const dq_pages_buffers *bufs, const int *rows,
                          const int *lens, int n, void *stream);

/*
 * Fork: row dst[i] becomes a second holder of row src[i]'s pages and takes its
 * length (device int32 [n]).  No token is copied: dq_pages_resize copies a partly
 * filled last page when one of its holders grows.  Several dst may name one src.
 * Every dst must be empty (length 0), named once, and no src of the call;
 * otherwise, or where a row is >= max_seqs, nothing changes (DQ_EINVAL from
 * dq_pages_check).  Pairs with a negative row are skipped.
 * Errors: DQ_EINVAL, DQ_ECUDA.
 */
dq_status dq_pages_fork(const dq_pages_config *cfg, const dq_pages_buffers *bufs, const int *src,
                        const int *dst, int n, void *stream);

/*
 * Compact: with n live pages, the i-th live page numbered n or more (ascending)
 * moves to the i-th free number below n, in every layer, and the tables follow:
 * afterwards the live pages are [0, n).
 * Errors: DQ_EINVAL, DQ_EALIGN, DQ_ECUDA.
 */
dq_status dq_pages_compact(const dq_pages_config *cfg, const dq_pages_buffers *bufs, void *stream);

/*
 * Quantise the new tokens of n_rows rows into their pages of one layer and bring
 * the summaries of the pages they touch up to date.
 *   k, v : device, dtype, [n_tok][n_kv_heads][head_dim] with the given strides in
 *          elements (multiples of 8; channels are contiguous)
 * A page that more than one row holds is not written (DQ_EINVAL from
 * dq_pages_check: the row was forked after it was resized), nor is a row that
 * `rows` names twice with new tokens (DQ_EINVAL).  A non-finite value
 * latches DQ_ENONFINITE; its block's held values are then finite but unspecified.
 * Errors: DQ_EINVAL, DQ_EALIGN, DQ_ECUDA.
 */
dq_status dq_pages_append(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *k,
                          const void *v, long long k_tok_stride, long long k_head_stride, long long v_tok_stride,
                          long long v_head_stride, const int *rows, const int *cu, int n_rows, int n_tok, int max_new,
                          void *stream);

/*
 * The held values of the last n tokens of each row, rounded once to dtype (exact
 * in bf16): k_out, v_out [n_tok][n_kv_heads][head_dim] contiguous.  Positions
 * below 0 (n > seq_len) give zeros.
 * Errors: DQ_EINVAL, DQ_EALIGN, DQ_ECUDA.
 */
dq_status dq_pages_read(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, void *k_out, void *v_out,
                        const int *rows, const int *cu, int n_rows, int n_tok, int max_new, void *stream);

/*
 * Attention of each row's newest tokens over its pages of one layer:
 *   out_h = sum_j softmax_j(sm_scale q_h . k_j) v_j,  j <= the query's position
 *   q   : device, dtype, [n_tok][n_q_heads][head_dim], strides in elements
 *         (multiples of 8; channels are contiguous)
 *   out : device, dtype, [n_tok][n_q_heads][head_dim] contiguous
 *   lse : device fp32 [n_tok][n_q_heads] or NULL: log sum_j exp(sm_scale q_h . k_j)
 *   sel : device int32 [n_rows][n_kv_heads][n_sel] or NULL: attend to these pages
 *         of the row alone (ordinals, distinct, -1 ignored; cu must be NULL).
 *         Ordinals behind the row's last page are ignored.
 * A query that no key is visible to gives out = 0 and lse = -inf.
 * Precision: logits, sums and accumulators are fp32.  Queries are held in binary16 after a
 * scaling by a power of two (a bf16 channel below 2^-38 of its query's largest loses bits);
 * exponentials are off by up to 2^-22; a weight is rounded to binary16 (11 bits) for its
 * product with the value, once more at each raise of the running maximum within its 128 keys
 * (rows of many new tokens), while the sum that divides takes it unrounded.  An output is so within about
 * 2^-11 of sum_j weight_j |v_j| beside its own rounding.  The result is the same every time.
 * A call over more than 2^35 (row, KV head, token) triples may be refused (DQ_EINVAL from
 * dq_pages_check).
 * Errors: DQ_EINVAL, DQ_EALIGN, DQ_ECUDA.
 */
dq_status dq_pages_attention(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                             long long q_tok_stride, long long q_head_stride, void *out, float *lse, const int *rows,
                             const int *cu, int n_rows, int n_tok, int max_new, const int *sel, int n_sel,
                             float sm_scale, void *stream);

/*
 * Test support for the timeout path: an attention call over rows 0 .. n_rows - 1 (sm_scale 1, no chosen pages) whose barriers
 * wait for an arrival that nobody makes, for limit_ns at most (clamped to [1000, 10^9]) instead of the 2 s of
 * every other call.  The kernel returns, `out` holds nothing of use, and dq_pages_check reports DQ_ETIMEOUT.
 * Errors: as dq_pages_attention.
 */
dq_status dq_pages_test_expire_wait(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                                    long long q_tok_stride, long long q_head_stride, void *out, const int *cu, int n_rows,
                                    int n_tok, int max_new, unsigned long long limit_ns, void *stream);

/*
 * Choose pages for each row's one query token and KV head.  With the group's
 * query heads q_h, Q+ = sum_h max(q_h, 0) and Q- = sum_h min(q_h, 0) a page's score
 *   sum_c Q+_c largest_c + Q-_c smallest_c
 * bounds sum_h q_h . k from above for every key k of the page.  It is computed in
 * whole numbers, so that it is the same in every order: Q+- (summed in 64 bits,
 * rounded to fp32) go to the nearest whole number, ties to even, of Q+- r with
 * r = 127 / max|Q+-|, quotient and product rounded to fp32; the page's bytes
 * are used as they are, and the sum is scaled by 2^e.  With the rounded Q+- the score
 * is a bound up to half a unit of Q+- for each channel's byte.
 *   sel : device int32 [n_rows][n_kv_heads][n_sel]: the ordinals of the first
 *         keep_first and the last keep_last pages and of those with the highest
 *         scores (the lower ordinal where scores are equal), n_sel in all,
 *         ascending, then -1 where the row has fewer pages
 * Requires keep_first + keep_last <= n_sel <= DQ_PAGES_MAX_SELECT and
 * max_pages_per_seq <= 16384 (else DQ_EUNSUPPORTED).  A non-finite query makes its
 * group's scores 0.
 * Errors: DQ_EINVAL, DQ_EALIGN, DQ_EUNSUPPORTED, DQ_ECUDA.
 */
dq_status dq_pages_select(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                          long long q_tok_stride, long long q_head_stride, const int *rows, int n_rows, int *sel,
                          int n_sel, int keep_first, int keep_last, void *stream);

/*
 * Synchronize `stream`, then return the gravest of what earlier calls on these buffers
 * latched and clear that alone: what else they latched, and what calls on other
 * streams latch meanwhile, is there for the next dq_pages_check.  In this order:
 * DQ_ETIMEOUT (a bounded device wait ran out: that call's output is not valid),
 * DQ_ENOMEM (a resize found too few free pages), DQ_EINVAL (a row, length, count or
 * page number out of range, a row named twice, a write to a shared page: three
 * reports), DQ_ENONFINITE, or DQ_OK; DQ_ECUDA if the stream reports an error.
 */
dq_status dq_pages_check(const dq_pages_buffers *bufs, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DQ_PAGES_H */
