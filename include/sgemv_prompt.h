/*
 * sgemv_prompt.h -- C ABI of the prompt-path operators of libsgemv.so: matrices in block-scaled 4-bit floating point (quantisation,
 * reading back, the product of two of them, for 1 to many rows, where the GEMVs of sgemv.h end at 8) and causal attention over packed
 * prompts' own keys and values (sgemv_kv_attention of sgemv_kv.h reads a 4-bit cache).
 *
 * The conventions of sgemv.h hold: status codes, no allocation, no synchronisation, argument errors found on the host before anything
 * is launched, `stream` and `status_dev` as described there. No call needs a workspace. Device pointers are 16-byte aligned unless a
 * function says otherwise. What a call writes overlaps neither its inputs nor what else it writes: SGEMV_ERR_ARG. (Rows may lie between
 * other rows, as in a fused projection's output; whether such rows share bytes is not looked into.)
 *
 * 4-bit matrices. A matrix of `rows` rows of `k` values holds for every value a code of one sign, two exponent and one mantissa bits
 * (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; the sign is bit 3), for every `block` consecutive values of a row a scale byte, and for every
 * row an fp32 power of two; a value is code * scale * row scale.
 *   block 32  The scale is 2^(b - 127), b its byte, with b - 127 = floor(log2 m) - 2 for the block's largest magnitude m (at least
 *             -127; b = 0 where m = 0). The row scale is 1.
 *   block 16  The row scale is 2^e, e the least integer of at least -100 with M <= 2688 * 2^e for the row's largest magnitude M (e = 0
 *             where M = 0). The scale is the e4m3 number nearest to m / 2^e / 6 (ties to even).
 * A code is the nearest to x / (scale * row scale), ties to the even code, magnitudes past 6 to 6; of magnitude 0 where the scale is 0.
 * Codes of magnitude 0 may have either sign. A row with an infinite or NaN element has row scale NaN (0x7FC00000), codes and scales 0:
 * every value that it stands for, and every product with it, is NaN.
 * (The row's power of two stands where other formats of this kind have one scale a tensor: no pass over the tensor comes first, a token
 * does not depend on the others of its call, and as a power of two it rounds nothing.)
 * Bytes, with kp = k up to a multiple of 64, T = 128 rows a tile (a matrix of up to 64 rows: the next power of two, 8 at least):
 *   codes   [ceil(rows / T)][kp / 32][T][16]: byte j of a row's 32 values holds value 2j in its low and 2j + 1 in its high nibble
 *   scales  at scale_off, [ceil(rows / 128)][ceil(kp / (4 block))][512]: scale s of the 4 of row 32 j + i of 128 at 16 i + 4 j + s
 *   rows    at row_off, fp32 [rows up to a multiple of 128]
 * so that the operands of the tensor cores' instruction are contiguous copies: 128-byte groups of 8 rows of 16 bytes for the codes, and
 * the scales as they go into tensor memory. Codes and scales of the columns k .. are 0; bytes of rows past the last are never used.
 */
#ifndef SGEMV_PROMPT_H
#define SGEMV_PROMPT_H

#include "sgemv_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A 4-bit matrix: total_bytes are allocated by the caller. */
typedef struct {
    int32_t rows, k, block, tile, kp, reserved;
    uint64_t scale_off, row_off, total_bytes;
} sgemv_fp4_layout;

/*
 * sgemv_fp4_layout_query -- host only, pure. rows 0..2^24 (calls with a matrix of no rows do nothing), k 1..2^20, block 16 or 32.
 * Errors: SGEMV_ERR_ARG (out is NULL), SGEMV_ERR_SHAPE.
 */
int sgemv_fp4_layout_query(int rows, int k, int block, sgemv_fp4_layout* out);

/*
 * sgemv_fp4_quantize -- the 4-bit matrix of x.
 *   x_dev      : dtype (fp16 or bf16) [rows][k], rows `stride` (at least k) elements apart, aligned to its element. (Rows of aligned
 *                16-byte pieces, stride and k multiples of 8, are read faster.)
 *   packed_dev : layout->total_bytes.
 *   status_dev : nullable; SGEMV_ERR_NONFINITE if x holds inf or NaN.
 * Errors returned: SGEMV_ERR_ARG, SGEMV_ERR_FORMAT (layout fields), SGEMV_ERR_ALIGN, SGEMV_ERR_CUDA.
 */
int sgemv_fp4_quantize(const sgemv_fp4_layout* layout, const void* x_dev, int dtype, int64_t stride, void* packed_dev,
                       int32_t* status_dev, void* stream);

/*
 * sgemv_fp4_read -- the values that a 4-bit matrix stands for, into out_dev, dtype (fp16, bf16 or fp32) [rows][k], rows `stride` (at
 * least k) elements apart, aligned to its element. bf16 and fp32 hold them exactly within their range (six significant bits).
 * Errors returned: as sgemv_fp4_quantize.
 */
int sgemv_fp4_read(const sgemv_fp4_layout* layout, const void* packed_dev, void* out_dev, int dtype, int64_t stride, void* stream);

/*
 * sgemv_fp4_product -- y[t][n] = sum over k of x[t][k] * w[n][k], of the values that the two 4-bit matrices stand for (equal k and
 * block). Products are exact and summed in 32 bits by the tensor cores; y is rounded once.
 *   y_dev      : dtype (fp16 or bf16) [x rows][w rows], rows `stride` (at least w rows) elements apart, aligned to its element.
 *   status_dev : nullable; SGEMV_ERR_TIMEOUT if a bounded wait for a copy gave up (y is then invalid).
 * The same inputs give the same bits: sums are split by sizes alone and joined in a fixed order.
 * Errors returned: SGEMV_ERR_ARG, SGEMV_ERR_FORMAT (layout fields; different k or block), SGEMV_ERR_ALIGN, SGEMV_ERR_SHAPE (more than
 * 2^28 - 1 tiles of 128 x 128), SGEMV_ERR_CUDA.
 */
int sgemv_fp4_product(const sgemv_fp4_layout* w_layout, const void* w_dev, const sgemv_fp4_layout* x_layout, const void* x_dev,
                      void* y_dev, int dtype, int64_t stride, int32_t* status_dev, void* stream);

/* What sgemv_prompt_attention reads and writes. */
typedef struct {
    int32_t dtype;              /* of q, k, v and out: SGEMV_F16 or SGEMV_BF16 */
    int32_t heads_q, heads;     /* query heads, a multiple of the KV heads; query head a reads KV head a / (heads_q / heads) */
    int32_t dim;                /* 64 or 128 */
    int32_t n_req, n_tokens;
    int32_t causal;             /* 1: a token sees those up to itself; 0: all of its request */
    int32_t window;             /* 0, or (causal only) each token sees only the last `window` tokens, itself among them */
    float scale;                /* factor of q . k; |scale| up to 2^127 */
    int32_t reserved;
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride; /* elements, positive multiples of 8 (below 2^38); that of */
    int64_t v_token_stride, v_head_stride, out_token_stride, out_head_stride; /* an axis of length 1 is not used */
    const void* q_dev;          /* [n_tokens][heads_q][dim] */
    const void* k_dev;          /* [n_tokens][heads][dim] */
    const void* v_dev;
    const int32_t* start_dev;   /* [n_req + 1]: request r's tokens are start[r] .. start[r + 1] */
    const int32_t* length_dev;  /* nullable [n_req]: only the first length[r] of them (a padded batch) */
    void* out_dev;              /* [n_tokens][heads_q][dim] */
    float* lse_dev;             /* nullable [n_tokens][heads_q] */
} sgemv_prompt_query;

/*
 * sgemv_prompt_attention -- out = softmax(scale * q K^T) V of each request's tokens over its own keys and values: scores, the
 * softmax's sum and out's sums are held in 32 bits; the softmax's weights are rounded to dtype (11 or 8 bits) before they meet V, as the
 * matrix instruction takes both in one type. In fp16 a weight is also held to no less than 2^-27 of its row's largest (below that it is
 * 0), which n keys down there add up to n * 2^-27 * max |v| in out; in bf16, elements of v below 2^-87 lose bits. lse is the natural
 * logarithm of the softmax's sum, of unrounded weights.
 * Keys and values that a token does not see do not enter its outputs, whatever they hold. A NaN or infinite element of v that it sees
 * makes that dim of its output NaN or infinite. Scores follow the softmax: with one that is NaN or infinity (NaN elements of q or k,
 * infinite ones, products that leave binary32) a row's output and lse are NaN; one of minus infinity beside finite ones has weight 0;
 * where a token sees no other than such, output and lse are NaN.
 * Rows that belong to no request (past start[n_req], or past a request's length) are neither used nor written. Requests of no tokens are
 * allowed. out may be q itself (the same address and strides); out's rows do not overlap one another.
 * The same inputs give the same bits.
 * Device-reported: SGEMV_ERR_ARG (a request with start out of order or out of range, or a length outside 0..start[r + 1] - start[r]: its
 * rows are not written, and nobody's where starts out of order make the others overlap to more than n_tokens); SGEMV_ERR_TIMEOUT (a bounded wait for a copy gave up: out is invalid).
 * Errors returned: SGEMV_ERR_ARG, SGEMV_ERR_SHAPE (dim; heads_q; strides; n_tokens times heads_q above 2^30; n_req above 2^26),
 * SGEMV_ERR_ALIGN, SGEMV_ERR_CUDA.
 */
int sgemv_prompt_attention(const sgemv_prompt_query* query, int32_t* status_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMV_PROMPT_H */
