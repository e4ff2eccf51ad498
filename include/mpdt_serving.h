/*
 * mpdt_serving.h -- C ABI of the serving operators in libmpdt.so: a paged
 * key/value cache, attention over it, the bookkeeping of its pages, and the
 * log probabilities of given tokens with their gradient.
 *
 * The conventions of mpdt.h hold (device pointers, arguments checked on the
 * host before anything is launched, no allocation, no synchronisation, no
 * state between calls, stream order, mpdt_last_error()), with two additions:
 *   - Strides are in ELEMENTS and named in the structures below.  Rows that are
 *     written (of out, of a cache that is appended to) share no bytes.
 *   - An operator that needs device scratch takes a workspace of the size that
 *     its *_workspace function names; it may be shared by calls on one stream.
 *
 * Numbers that only the device knows (page numbers, lengths, offsets) cannot
 * be refused by the host.  They are cut to the buffers instead, and nothing is
 * read or written out of range: a page number outside [0, pages) holds no
 * keys, a length past width * page_size counts as that, an offset outside the
 * tokens is moved to their border.
 *
 * One call takes fewer than 2^24 rows of logits or of a page table (the gradient:
 * of pieces of rows, 8192 values of 16 bits or 4096 of 32), and fewer than 2^27 new
 * tokens to append.
 */
#ifndef MPDT_SERVING_H
#define MPDT_SERVING_H

#include <stdint.h>

#include "mpdt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MPDT_BF16 = 0,
    MPDT_F16 = 1,
    MPDT_F32 = 2,
    MPDT_E4M3 = 3   /* OCP FP8, only as a cache's type */
} mpdt_dtype;

/* One layer's cache: element (page, slot, head, d) of K lies at
 * page * page_stride + slot * slot_stride + head * head_stride + d, and the
 * same of V.  Any order of slots and heads will do. */
typedef struct {
    void* k;
    void* v;
    int64_t page_stride, slot_stride, head_stride;
    int64_t pages;          /* at least 1 */
    int64_t page_size;      /* tokens of a page, any positive number */
    int64_t kv_heads;
    int64_t dim;            /* a multiple of 16, at most 128 */
    int dtype;              /* MPDT_BF16, MPDT_F16 or MPDT_E4M3 */
    const float* k_scale;   /* [kv_heads], for MPDT_E4M3: a key is its code's value times k_scale[head] */
    const float* v_scale;
} mpdt_paged_kv;

/* The sequences of a batch.  Sequence b has lens[b] tokens in all, of which
 * the last cu_q[b + 1] - cu_q[b] are new; its token t lies in page
 * table[b * ld_table + t / page_size], slot t % page_size. */
typedef struct {
    const int32_t* table;
    int64_t ld_table;       /* >= width */
    const int32_t* cu_q;    /* [seqs + 1], ascending */
    const int32_t* lens;    /* [seqs] */
    int64_t seqs, width;
    int64_t tokens;         /* new tokens of all sequences */
} mpdt_sequences;

/* Write new keys and values to their places in the cache: row i of k_new /
 * v_new [tokens, kv_heads, dim] is the i-th new token of the batch.  dtype is
 * the cache's, or MPDT_BF16 / MPDT_F16 for an MPDT_E4M3 cache, where a value x
 * becomes e4m3_rne(clamp(x / scale[head], -448, 448)).  Tokens whose place
 * does not exist (position below 0, no such page) are dropped. */
mpdt_status paged_kv_append(const mpdt_paged_kv* kv, const mpdt_sequences* seq, int dtype,
                            const void* k_new, int64_t k_token, int64_t k_head,
                            const void* v_new, int64_t v_token, int64_t v_head, void* stream);

/* Attention of the new tokens over the cache (which holds their own keys and
 * values already).  New token t of a sequence with n tokens, nq of them new,
 * stands at position p = n - nq + t and sees the keys j <= p; with window > 0
 * only those with j > p - window.  Query head h reads KV head
 * h / (heads / kv_heads).  s = scale * (q . k), then softcap * tanh(s /
 * softcap) where softcap > 0 (any finite one: a large cap lets the score through;
 * the cap adds a few roundings of the capped score, in chunks up to 2^-22 of a
 * softcap of at most 64); out = sum softmax(s) v, lse = log sum exp(s).
 * A token that sees no key gets out = 0 and lse = -inf.  Keys and values past a
 * sequence's end or on pages that do not exist are never looked at; a value that
 * is no number or infinite, hidden from one token but seen by another of the same
 * sequence, may reach both.  Rows of q that belong
 * to no sequence are not written.  q and out [tokens, heads, dim] in q_dtype
 * (the cache's type, or either 16-bit type for an MPDT_E4M3 cache); lse
 * [tokens, heads] FP32 or NULL. */
int64_t paged_attention_workspace(const mpdt_paged_kv* kv, const mpdt_sequences* seq, int64_t heads);
mpdt_status paged_attention(const mpdt_paged_kv* kv, const mpdt_sequences* seq, int64_t heads, int q_dtype,
                            const void* q, int64_t q_token, int64_t q_head,
                            void* out, int64_t out_token, int64_t out_head,
                            float* lse, int64_t lse_token, float scale, float softcap, int64_t window,
                            void* workspace, int64_t workspace_bytes, void* stream);

/* A cache as its pages: planes (layers, K and V) x pages blocks of page_bytes,
 * with a counter of holders for each page and the sequences' rows of pages. */
typedef struct {
    void* kv;               /* may be NULL where nothing is moved */
    int64_t plane_stride, page_stride;  /* BYTES */
    int64_t page_bytes;
    int64_t planes, pages;
    int64_t page_size;
    int32_t* refs;          /* [pages]: holders of a page; 0: free */
    int32_t* table;         /* [rows, width] */
    int64_t ld_table;
    int32_t* lens;          /* [rows] */
    int64_t rows, width;    /* no rows: the four calls below do nothing */
} mpdt_pages;

/* Bytes of workspace for each of the four below (cache_free needs none). */
int64_t cache_pages_workspace(int64_t pages, int64_t rows);

/* Row r becomes a copy of row parent[r] (itself or no row: it stays): whole pages
 * are shared and their counters raised, a part-filled last page is copied in every
 * plane to a free page of its own, the lowest free pages going to the rows in
 * ascending order.  What row r held before is forgotten.  A row that names
 * another one in the same call is no parent.  Where pages are missing,
 * nothing changes and *shortfall says how many (0 otherwise). */
mpdt_status cache_fork(const mpdt_pages* c, const int32_t* parent, int32_t* shortfall, void* workspace,
                       int64_t workspace_bytes, void* stream);

/* Room for add[r] (>= 0) more tokens in row r: the pages that its new length
 * needs, the lowest free ones in ascending order of rows.  Where pages are
 * missing, nothing changes and *shortfall says how many; where a row of the table
 * is full, nothing changes and it says how many pages were asked for. */
mpdt_status cache_extend(const mpdt_pages* c, const int32_t* add, int32_t* shortfall, void* workspace,
                         int64_t workspace_bytes, void* stream);

/* Rows with drop[r] != 0 give up their pages (counters lowered) and become
 * empty: length 0, table entries -1. */
mpdt_status cache_free(const mpdt_pages* c, const int32_t* drop, void* stream);

/* All pages with holders into the lowest numbers: with n of them, the i-th
 * free page below n takes the i-th used page from n on, in every plane, and
 * counters and tables follow. */
mpdt_status cache_compact(const mpdt_pages* c, void* workspace, int64_t workspace_bytes, void* stream);

/* For each row x of logits [rows, vocab] (leading dimension ld; BF16, FP16 or
 * FP32) and its target t: lse = log sum exp(x), logprob = x[t] - lse,
 * entropy = -sum p log p with p = exp(x - lse), and the `top` (0 to 64, at
 * most vocab) largest log probabilities in descending order with their indices
 * (ties to the lower index).  A target outside [0, vocab) has logprob 0.
 * Logits of -inf have p = 0; a row of nothing else has lse = -inf, entropy 0 and
 * log probabilities -inf.  NaN or +inf in a row make its results NaN. */
int64_t token_logprobs_workspace(int dtype, int64_t rows, int64_t vocab, int64_t top);
mpdt_status token_logprobs(int dtype, int64_t rows, int64_t vocab, const void* logits, int64_t ld,
                           const int64_t* targets, int64_t top, float* logprob, float* lse, float* entropy,
                           float* top_logprobs, int64_t* top_indices, void* workspace, int64_t workspace_bytes,
                           void* stream);

/* The gradient of sum(g_logprob * logprob + g_entropy * entropy) in the
 * logits, from what token_logprobs gave:
 *   grad[j] = g_logprob * ([j = t] - p_j) - g_entropy * p_j * (log p_j + entropy).
 * Either gradient may be NULL (0).  A target outside [0, vocab) drops the
 * first term; a row with lse = -inf has gradient 0.  grad: logits' type. */
mpdt_status token_logprobs_backward(int dtype, int64_t rows, int64_t vocab, const void* logits, int64_t ld,
                                    const int64_t* targets, const float* lse, const float* entropy,
                                    const float* g_logprob, const float* g_entropy, void* grad, int64_t ld_grad,
                                    void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MPDT_SERVING_H */
