/*
 * sgemv_kv.h -- C ABI of the decode-path operators of libsgemv.so that stand between the GEMVs of sgemv.h
 * and its beam step: a paged KV cache held in 4 bits (block tables and slot maps, writing, reading,
 * attention) and the log-probabilities of the head's logits.
 *
 * The conventions of sgemv.h hold: status codes, no allocation, no synchronisation, argument errors found
 * on the host before anything is launched, `stream` and `status_dev` as described there. Device pointers
 * are 16-byte aligned unless a function says otherwise. What a call writes overlaps neither its inputs nor what else it
 * writes, but where a function says so: SGEMV_ERR_ARG. (Rows may lie between other rows, as in a fused projection's
 * output; whether such rows share bytes is not looked into.)
 *
 * Cache bytes. The cache is n_pages pages; a page holds `page` tokens of every KV head; head h of page p
 * starts at p * page_bytes + h * head_bytes and is page / 16 subtiles of 16 tokens, sub_bytes each. Token
 * tau (0..15) of a subtile, with D = dim, g = group:
 *   K  [0, 8D)        panels of P = min(D, 128) dims: dim d at (d / P) * 8P + tau * P / 2 + (d % P) / 2, the
 *                     low nibble for even d
 *   V  [8D, 16D)      dim d = c + 8n + 32i (c < 8, n < 4): with w = (tau / 2 % 2) * (D / 32) + i, nibble n of the
 *                     16-bit word at 8D + (w / 4) * 512 + (4c + tau / 4) * 16 + (w % 4) * 4 + (tau % 2) * 2
 *   scales [16D, ..)  {fp16 scale, fp16 zero point}: K group j at 16D + 64j + 4 tau, V group j 64 D/g bytes later
 * The interleaving of V puts the same dim of two neighbouring tokens into the two halves of a 32-bit word,
 * the pair that a matrix instruction contracts over; K does so with dims n and n + 4 of one token.
 * A group of g values v of one token and head is quantised as a weight group of the packed weight format:
 * s = fp16((mx - mn) / 15) with mn = min(0, min v) and mx = max(0, max v), 1 where that is 0; z = clamp(rint(
 * -mn / s), 0, 15); q = clamp(rint(v / s) + z, 0, 15); all in binary32. The value is (q - z) * s.
 */
#ifndef SGEMV_KV_H
#define SGEMV_KV_H

#include "sgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { SGEMV_F16 = 0, SGEMV_BF16 = 1, SGEMV_F32 = 2 };

/* A paged 4-bit cache. total_bytes are allocated by the caller; unwritten bytes may hold anything. */
typedef struct {
    int32_t heads, dim, group, page, n_pages, reserved;
    uint64_t sub_bytes, head_bytes, page_bytes, total_bytes;
} sgemv_kv_layout;

/*
 * sgemv_kv_layout_query -- host only, pure. heads 1..1024 KV heads, dim 64, 128 or 256, group 64 or 128 (at
 * most dim), page 16, 32, 64, 128 or 256 tokens, n_pages >= 1. Errors: SGEMV_ERR_ARG (out is NULL),
 * SGEMV_ERR_SHAPE.
 */
int sgemv_kv_layout_query(int heads, int dim, int group, int page, int n_pages, sgemv_kv_layout* out);

/*
 * sgemv_kv_plan -- block tables and slot maps of one step, from the requests' lengths. Request r holds
 * len[r] tokens in ceil(len / page) pages, listed in row r of the block table; it keeps its first keep[r]
 * (<= len: fewer to take draft tokens back, 0 to release it) and add[r] new tokens follow them.
 *   len_dev, add_dev : int32 [n_req]; keep_dev the same, or NULL to keep everything.
 *   table_dev        : int32, row r at table_dev + r * table_stride, table_cols columns. Entries of new pages are
 *                      written; entries past a request's last page are left as they are.
 *   free_dev         : int32 [n_pages], a stack of free page ids whose top is entry *free_count_dev - 1.
 *   len_out_dev      : int32 [n_req], keep + add.       free_count_out_dev : int32, the stack's new height.
 *   q_start_dev      : int32 [n_req + 1], prefix sums of add: request r's new tokens are q_start[r] .. q_start[r+1].
 *   slots_dev        : int64 [n_slots]: new token t lives at page id slots[t] / page, place slots[t] % page; -1
 *   pos_dev          : int32 [n_slots]: its position in its request; -1 for t >= q_start[n_req].
 * Pages that requests give up are handed out first, in request order and ascending blocks, to the requests
 * that grow, in the same order; then pages are popped from the stack. What is left of the given-up pages is
 * pushed, in order. The inputs len and free_count are not written: a caller swaps two buffers from step to step.
 * A page has one owner here: if two rows list one (a shared prefix), it goes back when the first of them gives it up,
 * while the other still reads it. Attention does not mind shared pages; who shares them keeps count of the users and
 * hands this call only what is to go.
 * Device-reported, and then nothing is taken or released (len_out = len, free_count_out = free_count, q_start all
 * 0, every slot and position -1): SGEMV_ERR_ARG (negative counts, keep > len, more new tokens than n_slots, a
 * stack height outside 0..n_pages), SGEMV_ERR_SHAPE (a row needs more than table_cols pages, the free pages run out, or
 * more pages than there are are given up or needed). A page id outside 0..n_pages-1 in a block that is given up (it
 * goes where the page would) or that a new token falls into: SGEMV_ERR_ARG, and -1 in that token's slot.
 * Pointers are 4-byte aligned (slots: 8-byte). n_req 0 and n_slots 0 are allowed.
 * Errors returned: SGEMV_ERR_ARG, SGEMV_ERR_SHAPE (page; n_req above 16384, n_slots or n_pages above 2^30),
 * SGEMV_ERR_ALIGN, SGEMV_ERR_CUDA.
 */
int sgemv_kv_plan(int n_req, int page, int n_pages, const int32_t* len_dev, const int32_t* keep_dev,
                  const int32_t* add_dev, int32_t* table_dev, int table_cols, int64_t table_stride, int32_t* free_dev,
                  const int32_t* free_count_dev, int32_t* len_out_dev, int32_t* free_count_out_dev,
                  int32_t* q_start_dev, int64_t* slots_dev, int32_t* pos_dev, int n_slots, int32_t* status_dev,
                  void* stream);

/*
 * sgemv_kv_append -- quantise K and V rows into the cache.
 *   k_dev, v_dev : dtype (fp16 or bf16) [n_tokens][heads][dim]; dims are contiguous, a token's and a head's rows
 *                  start *_token_stride and *_head_stride elements apart (multiples of 8; that of an axis of length 1 is not used).
 *   slots_dev    : int64 [n_tokens], 8-byte aligned, as sgemv_kv_plan writes them. A negative slot is skipped;
 *                  one past the cache is skipped and reported (SGEMV_ERR_ARG). Slots are distinct.
 *   status_dev   : nullable; SGEMV_ERR_NONFINITE if a row holds inf or NaN, or a range too wide for an fp16 scale;
 *                  such a group is stored as zeros.
 * Every byte of a written token's nibbles and scales is set, none of its neighbours'.
 * Errors returned: SGEMV_ERR_ARG, SGEMV_ERR_FORMAT (layout fields), SGEMV_ERR_ALIGN, SGEMV_ERR_SHAPE (n_tokens * heads
 * past 2^31 - 1 rows of 128), SGEMV_ERR_CUDA.
 */
int sgemv_kv_append(const sgemv_kv_layout* layout, void* cache_dev, int dtype, const void* k_dev,
                    int64_t k_token_stride, int64_t k_head_stride, const void* v_dev, int64_t v_token_stride,
                    int64_t v_head_stride, const int64_t* slots_dev, int n_tokens, int32_t* status_dev, void* stream);

/*
 * sgemv_kv_read -- the values the cache holds for the tokens at slots_dev, rounded once to dtype (fp16, bf16 or
 * fp32), into contiguous k_dev, v_dev [n_tokens][heads][dim]. A negative slot reads as zeros; one past the
 * cache does too, and is reported (SGEMV_ERR_ARG). Errors returned: as sgemv_kv_append.
 */
int sgemv_kv_read(const sgemv_kv_layout* layout, const void* cache_dev, const int64_t* slots_dev, int n_tokens,
                  int dtype, void* k_dev, void* v_dev, int32_t* status_dev, void* stream);

/* What sgemv_kv_attention reads and writes beside the cache. */
typedef struct {
    int32_t dtype;      /* of q and out: SGEMV_F16 or SGEMV_BF16 */
    int32_t heads_q;    /* query heads, a multiple of the cache's heads; query head a reads KV head a / (heads_q / heads) */
    int32_t n_req, n_tokens;
    int32_t max_q;      /* at least every request's number of new tokens */
    int32_t window;     /* 0, or each token sees only the last `window` positions, its own among them */
    int32_t table_cols;
    float scale;        /* factor of q . k */
    int64_t table_stride;
    int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride; /* elements, multiples of 8 as in append */
    const void* q_dev;             /* [n_tokens][heads_q][dim] */
    const int32_t* q_start_dev;    /* [n_req + 1], as sgemv_kv_plan writes it */
    const int32_t* len_dev;        /* [n_req] tokens in the cache, the new ones included */
    const int32_t* table_dev;      /* block table: page ids */
    const uint64_t* tree_dev;      /* nullable [n_tokens]: see below */
    void* out_dev;                 /* [n_tokens][heads_q][dim] */
    float* lse_dev;                /* nullable [n_tokens][heads_q] */
    void* workspace_dev;           /* SGEMV_KV_WORKSPACE bytes */
    uint64_t workspace_bytes;
} sgemv_kv_query;

/* Bytes of workspace of any sgemv_kv_attention call. The caller zeroes them once, before the first call; every
 * call leaves zero what it needs zero. Calls that may run at the same time need workspaces of their own. */
#define SGEMV_KV_WORKSPACE (32u << 20)

/*
 * sgemv_kv_attention -- out = softmax(scale * q K^T) V over the cache, with the values (q - z) * s the cache
 * stands for; scores, the softmax's maximum and sum, and out's sums are held in 32 bits. What is rounded to fp16 on the
 * way: a query row in units of a power of two of its own (exact above 2^-25 of its largest element); the softmax's
 * weights before they meet V (11 bits); and, for requests with many rows, V's values (11 bits). So out is off by 2^-11
 * (2^-10 there) of the weighted sum of V's magnitudes s (q + z) and its own rounding, lse by 2^-19 beside what 32-bit
 * scores are.
 * New token i of request r (n = q_start[r+1] - q_start[r] of them, already in the cache) is at position
 * p = len[r] - n + i and sees positions j <= p, and j > p - window where window > 0. With tree_dev (window
 * must be 0, max_q <= 64) it sees every position before len - n, and new token m of its request where bit m of
 * tree_dev[q_start[r] + i] is set: the draft tokens of a token tree, each seeing its ancestors.
 * Pages before the one that holds the first position that a request's new tokens see (len - n - window + 1) are
 * not looked at: with a window they may be free, their table entries anything.
 * A token that sees nothing gets out = 0 and lse = -inf. lse is the natural logarithm of the softmax's sum.
 * out may be q itself (the same address and strides). Rows of out past q_start[n_req] are not written. What the cache holds past len is never used.
 * Results do not depend on the order in which the GPU runs the call's parts: the same inputs give the same bits.
 * Device-reported: SGEMV_ERR_ARG (a request with q_start out of order or out of range, n > max_q, a negative
 * length; a page id outside the cache), SGEMV_ERR_SHAPE (len needs more than table_cols pages, or passes 2^30): such a request's
 * rows are not written, keys of a page outside the cache are left out; SGEMV_ERR_TIMEOUT (a bounded wait for a
 * copy gave up: out is invalid).
 * Errors returned: SGEMV_ERR_ARG, SGEMV_ERR_FORMAT (layout fields), SGEMV_ERR_SHAPE (heads_q; n_tokens times query
 * heads a KV head, or n_req, above 2^30), SGEMV_ERR_ALIGN, SGEMV_ERR_CUDA.
 */
int sgemv_kv_attention(const sgemv_kv_layout* layout, const void* cache_dev, const sgemv_kv_query* query,
                       int32_t* status_dev, void* stream);

/*
 * sgemv_logprobs -- log-probabilities of rows of logits: lp = x - lse, lse = ln sum exp(x), sums in 32 bits.
 *   logits_dev : dtype (any of the three) [rows][vocab], rows `stride` elements apart; aligned to its element.
 *   tokens_dev : int32 [rows][n_tok] (n_tok 0..64; NULL if 0): tok_logp_dev fp32 [rows][n_tok] gets the tokens' lp;
 *                token -1 gets 0, any other outside the vocabulary NaN and SGEMV_ERR_ARG in status_dev.
 *   lse_dev, entropy_dev : fp32 [rows], nullable. Entropy in nats.
 *   top        : 0..64 alternatives: top_tok_dev int32, top_logp_dev fp32 [rows][top], highest first, equal logits by
 *                the lower token; past the vocabulary -1 and -inf.
 *   logp_dev   : nullable fp32 [rows][vocab], contiguous: every lp, the rows that sgemv_beam_step reads.
 * -inf logits (banned tokens) have probability 0 and lp -inf. A row of nothing else has lse -inf, every lp -inf
 * and entropy 0. A row with NaN or +inf has NaN in every output and -1 in top_tok, and status_dev gets
 * SGEMV_ERR_NONFINITE. Pointers are aligned to their element. logp_dev may be logits_dev (fp32, stride vocab). rows 0 is
 * allowed.
 * Errors returned: SGEMV_ERR_ARG, SGEMV_ERR_SHAPE (vocab outside 1..2^24), SGEMV_ERR_ALIGN, SGEMV_ERR_CUDA.
 */
int sgemv_logprobs(const void* logits_dev, int dtype, int rows, int vocab, int64_t stride, const int32_t* tokens_dev,
                   int n_tok, int top, float* tok_logp_dev, float* lse_dev, float* entropy_dev, int32_t* top_tok_dev,
                   float* top_logp_dev, float* logp_dev, int32_t* status_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMV_KV_H */
