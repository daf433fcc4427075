/*
 * e2ttt_tokens.h -- C ABI of the two ends of a hybrid model: the lookup of
 * tokens' vectors with its gradient, and the choice of the next token from a
 * row of logits.  In the same library (libe2ttt.so) as the chunk update
 * (e2ttt.h) and the other operators of a layer (e2ttt_layer.h), whose
 * conventions hold here too: device pointers owned by the caller, nothing
 * allocated, freed or synchronised, work queued on `stream`, arguments checked
 * on the host before any device call, every result the same bit for bit from
 * call to call.  What a device tensor holds (tokens, settings of a row) cannot
 * be checked on the host; what the kernels make of values out of range is said
 * below.
 */
#ifndef E2TTT_TOKENS_H
#define E2TTT_TOKENS_H

#include "e2ttt.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Token lookup: out[n] = scale table[tokens[n]], a product in 32 bits rounded to
 * io_dtype; and its gradient, a dense tensor: dtable[v] = scale times the sum, in
 * 32 bits, of dout[n] over the n with tokens[n] = v, 0 for a v that no token
 * names.  Up to 16 of them are added up in the order of n; more are cut into
 * pieces, at the multiples of 16 of all places in the order of their tokens,
 * whose sums are then added up, in an order that the tokens alone determine.
 *   tokens  [tokens] int32 or int64; one outside [0, vocab) reads a row of
 *           zeros and has no part in the gradient
 *   table, dtable  [vocab][width] table_dtype contiguous
 *   out, dout      [tokens][width] io_dtype contiguous
 * Tensors are aligned to their elements; where every row starts on 16 bytes
 * they are read and written in wider pieces.  Outputs must not overlap any
 * other buffer.  vocab up to 2^24, width up to 2^20, tokens below 2^31.
 */
typedef struct {
    int32_t table_dtype, io_dtype; /* e2ttt_dtype, in any combination */
    int32_t token_bytes;           /* 4 or 8 */
    float scale;                   /* finite */
    int64_t tokens, vocab, width;
} e2ttt_embedding_desc;

E2TTT_API int e2ttt_embedding_forward(const e2ttt_embedding_desc* desc, const void* tokens, const void* table, void* out,
                        void* stream);

/*   workspace  >= e2ttt_embedding_backward_workspace_size(desc) bytes, 256-byte
 *              aligned; clobbered (NULL when that is 0) */
E2TTT_API size_t e2ttt_embedding_backward_workspace_size(const e2ttt_embedding_desc* desc);
E2TTT_API int e2ttt_embedding_backward(const e2ttt_embedding_desc* desc, const void* dout, const void* tokens, void* dtable,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token for each row of logits, from a given random number of the row.
 *
 * With temperature T > 0 and x the row's largest logit, token i has the weight
 *   w_i = 2^-44 round(2^44 exp((logit_i - x) / T)),
 * a whole number of 2^-44, so that sums of weights are exact (a token of less
 * than 2^-45 of the largest one's probability is never chosen).  There are two
 * exceptions: without any filter, and with top_p but no top_k on rows of more than
 * 8192, the row's sum is one of weights before they are rounded, in 64-bit floats.
 * It is off by 2^-45 of the largest weight per logit at most, so that the token may
 * be a neighbour, or top_p keep one more or less, where u or top_p is within 2^-27
 * of a border.  (Rows of equal logits are exact all the same.)  The tokens are
 * put in order of falling logit, equal ones by index, and kept are
 *   1. the first top_k of them (0 or less: all);
 *   2. of those, as many as it takes for their weight to reach top_p of that of
 *      all those (1 or more: all; at least the first one);
 *   3. of those, the ones with exp((logit_i - x) / T) >= min_p, and the first.
 * Of what is kept, in order of index, the token is the first at which the
 * running sum of weights exceeds u times their sum, and logprob the natural
 * log of its share of that sum.  T <= 0 takes the largest logit, the first of
 * equal ones, with logprob 0.
 *   logits  [rows] of vocab values io_dtype, row_stride elements apart
 *   u       [rows] fp32 in [0, 1); others are taken as the nearest in it
 *   temperature, top_p, min_p  [rows] fp32 or NULL; top_k [rows] int32 or NULL:
 *           settings of each row, in place of the descriptor's (a NaN switches
 *           the filter off; as a temperature it is taken as 0)
 *   token   [rows] int64;  logprob  [rows] fp32 or NULL
 * A logit of NaN or -infinity is never chosen; a row that holds nothing else
 * gives token -1 and logprob NaN.  Where logits are +infinity, those tokens
 * alone have weight, equal ones.
 * A min_p above 1 is taken as 1.  Outputs must not overlap any other buffer.
 * vocab up to E2TTT_SAMPLE_VOCAB, rows below 2^22.
 */
#define E2TTT_SAMPLE_VOCAB 262136 /* 2^18 - 8 */
typedef struct {
    int32_t io_dtype;
    int32_t top_k;
    float temperature; /* >= 0, finite */
    float top_p;       /* >= 0 */
    float min_p;       /* in [0, 1] */
    int32_t reserved;  /* 0 */
    int64_t rows, vocab, row_stride;
} e2ttt_sample_desc;

E2TTT_API size_t e2ttt_sample_workspace_size(const e2ttt_sample_desc* desc);
E2TTT_API int e2ttt_sample(const e2ttt_sample_desc* desc, const void* logits, const float* u, const float* temperature,
                        const int32_t* top_k, const float* top_p, const float* min_p, int64_t* token, float* logprob,
                        void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* E2TTT_TOKENS_H */
