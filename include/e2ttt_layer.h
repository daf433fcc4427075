/*
 * e2ttt_layer.h -- C ABI of the operators a hybrid layer has beside the chunk
 * update of e2ttt.h, in the same library (libe2ttt.so).
 *
 * The paper's models are hybrids: sliding window attention and the E2-TTT
 * branch side by side in a layer ("Rethinking Expressivity and Efficiency in
 * Test-Time Training", atlas summary "Approach").  Here are the attention for
 * prompts and training (forward and backward over packed sequences), the
 * attention of new tokens over a paged cache for serving (in the queries' type or
 * in 8 bits), the gated linear recurrence, whose state is a vector where the
 * chunk update's is a matrix, and the norm with the residual's addition that
 * stands before the branches.
 *
 * Conventions, as in e2ttt.h: every tensor pointer is a DEVICE pointer owned
 * by the caller; the library never allocates, frees or synchronises; work is
 * queued on `stream`; arguments are validated on the host before any device
 * call and the status is returned; no exception crosses the ABI; NaN and Inf
 * reach the results that depend on them and, masked, no other.  Statuses and types are those of e2ttt.h.  Every result is the
 * same bit for bit from call to call (no floating-point atomics).
 * Attention calls whose launch would take 2^24 workgroups or more are
 * E2TTT_ERR_UNSUPPORTED: each is a tile of one key head, of 128 (token, head)
 * rows or 64 keys in bf16 and 16 in fp32, at least one for every sequence, or
 * 4 KiB of new keys where a cache is extended.
 * What a device tensor holds (offsets, lengths, page indices) cannot be
 * checked on the host: the kernels clamp it, so that bad values give wrong
 * results but no access outside the tensors.
 */
#ifndef E2TTT_LAYER_H
#define E2TTT_LAYER_H

#include "e2ttt.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Causal attention with grouped heads over packed sequences.
 *
 * Sequence s holds tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1 of the packed
 * tensors.  Query head h reads key head h / (heads / kv_heads).  The query at
 * position i of its sequence sees the keys at positions j <= i, and with
 * window > 0 only j > i - window:
 *   s_ij = scale <q_i, k_j>,  lse_i = log sum_j exp(s_ij),
 *   out_i = sum_j exp(s_ij - lse_i) v_j.
 */
typedef struct {
    int32_t io_dtype;           /* e2ttt_dtype of q, k, v, out and their gradients */
    int32_t window;             /* 0: no window */
    int64_t tokens, seqs;       /* packed tokens N, sequences S */
    int64_t heads, kv_heads, D; /* heads a multiple of kv_heads; D a multiple of 8 up to 128 */
    float scale;                /* > 0, finite */
    int32_t reserved;           /* 0 */
    /* strides in elements, multiples of 16 bytes, of q [N][heads][D],
     * k and v [N][kv_heads][D] over tokens and heads (the last dimension is
     * contiguous), of tokens up to 2^23; so views of one projection's output,
     * or of tensors that hold head after head, need no copy */
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
} e2ttt_attention_desc;

/*
 *   q, k, v     as above, 16-byte aligned
 *   cu_seqlens  [S + 1] int32, non-decreasing, from 0 to N; tokens before
 *               the first or from the last on (room to spare in a packed
 *               buffer) belong to no sequence and see nothing.  (A call of
 *               no sequences, S = 0, returns without writing anything.)
 *   out         [N][heads][D] contiguous; 0 for tokens of no sequence
 *   lse         [N][heads] fp32 (natural log), or NULL; -infinity there
 *   workspace   >= e2ttt_attention_workspace_size(desc) bytes, 256-byte
 *               aligned; clobbered (NULL when that is 0)
 * bf16: bf16 MFMA with fp32 accumulation; scores, softmax and output sums are
 * fp32, the probabilities are rounded to bf16 once as an operand.  fp32: fp32
 * MFMA throughout.  out and lse must not overlap any other buffer.
 */
E2TTT_API size_t e2ttt_attention_workspace_size(const e2ttt_attention_desc* desc);
E2TTT_API int e2ttt_attention_forward(const e2ttt_attention_desc* desc, const void* q, const void* k, const void* v,
                        const int32_t* cu_seqlens, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of <dout, out> with respect to q, k, v, from the forward's
 * inputs, out and lse.  dout, dq [N][heads][D] and dk, dv [N][kv_heads][D]
 * contiguous, 16-byte aligned; a key head's gradient is the sum over the
 * query heads that share it.  Those of tokens of no sequence are 0.  Outputs must not overlap any other buffer.
 */
E2TTT_API size_t e2ttt_attention_backward_workspace_size(const e2ttt_attention_desc* desc);
E2TTT_API int e2ttt_attention_backward(const e2ttt_attention_desc* desc, const void* q, const void* k, const void* v,
                        const void* out, const float* lse, const void* dout, const int32_t* cu_seqlens,
                        void* dq, void* dk, void* dv,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention of new tokens over a paged cache (serving: a chunk of a prompt, or
 * one token per sequence).  Sequence s has cached[s] tokens in the cache and
 * cu_seqlens[s + 1] - cu_seqlens[s] new ones, at positions cached[s],
 * cached[s] + 1, ...; position p of it is slot p % page_size of page
 * table[s][p / page_size].  With k and v given, the call writes the new
 * tokens' keys and values into their slots and attends over cached and new
 * ones; with k = v = NULL the slots hold them already.  Scores, mask and
 * window as above, over positions.  A new token always sees itself; rows that
 * see nothing (of tokens outside every sequence; k = v = NULL and a negative
 * length) give 0.
 * Slots that no query sees may hold anything.  A page index outside the pool
 * is read as zeros and not written.
 */
typedef struct {
    e2ttt_attention_desc a; /* tokens, seqs: the new tokens, packed */
    int64_t pages;          /* pages in the pool */
    int64_t page_size;      /* tokens per page, a power of two */
    int64_t table_width;    /* page indices per sequence in table */
    /* strides in elements, multiples of 16 bytes, of k_cache and v_cache over
     * pages, key heads and slots (head dimension contiguous) */
    int64_t kc_page, kc_head, kc_slot, vc_page, vc_head, vc_slot;
} e2ttt_paged_desc;

E2TTT_API size_t e2ttt_paged_workspace_size(const e2ttt_paged_desc* desc);
E2TTT_API int e2ttt_paged_attention(const e2ttt_paged_desc* desc, const void* q, const void* k, const void* v,
                        void* k_cache, void* v_cache, const int32_t* table, const int32_t* cu_seqlens,
                        const int32_t* cached, void* out,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same over a cache in 8 bits: k_cache and v_cache hold OCP e4m3 values,
 * and k_scale and v_scale [pages][kv_heads][page_size] contiguous a scale for
 * every slot and key head, a power of two 2^(b - 127) as its biased exponent b
 * (OCP e8m0; 255 is NaN).  A key or value that the call writes gets the smallest
 * such scale with max|x| <= 448 scale (1 for zeros), and x / scale rounded to
 * nearest even; one that holds a NaN or an Inf becomes NaN as a whole.  Queries
 * see keys and values as the cache holds them, the new ones among them.
 * Probabilities are rounded to bf16 as operands, as over a cache of bf16; a
 * value's scale goes into its probability, which loses bits, as the smallest
 * numbers of bf16 do, where the values are all below some 2^-110.
 * io_dtype is bf16, in which an 8-bit value times its scale is exact, and D a
 * multiple of 16 (else E2TTT_ERR_UNSUPPORTED).  The cache's strides count
 * elements of one byte, in multiples of 16.  Everything else as above.
 */
E2TTT_API size_t e2ttt_paged8_workspace_size(const e2ttt_paged_desc* desc);
E2TTT_API int e2ttt_paged8_attention(const e2ttt_paged_desc* desc, const void* q, const void* k, const void* v,
                        void* k_cache, void* v_cache, void* k_scale, void* v_scale, const int32_t* table,
                        const int32_t* cu_seqlens, const int32_t* cached, void* out,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gated linear recurrence of every channel over packed sequences:
 *   h_t = a_t h_{t-1} + x_t,  out_t = h_t,
 * from h0 of each sequence (0 where h0 is NULL) to its state after its last
 * token (h0 where it has none).  Held in 32 bits; out is rounded once.
 *   x           [tokens][width] io_dtype, x_tok elements from token to token
 *   a           [tokens][width] gate_dtype, a_tok elements from token to token;
 *               gates, of magnitude up to 1: products of them over stretches of
 *               a sequence are formed, which larger ones could take past the range
 *   h0, state   [seqs][width] fp32, or NULL; state may be h0 (in place)
 *   cu_seqlens  [seqs + 1] int32, as for the attention; out is 0 for tokens of
 *               no sequence
 *   out         [tokens][width] io_dtype contiguous
 *   starts      NULL, or, for the backward, [tokens / E2TTT_SCAN_TILE + seqs][width]
 *               fp32: the state before token E2TTT_SCAN_TILE j of sequence s, in
 *               row cu_seqlens[s] / E2TTT_SCAN_TILE + s + j; other rows are left alone
 *   workspace   >= e2ttt_scan_workspace_size(desc) bytes, 256-byte aligned;
 *               clobbered (NULL when that is 0); calls that overlap in time need
 *               one each: with a workspace that another call overwrites meanwhile the
 *               results are not defined, and are NaN, without an error, where a part of
 *               the call has waited in vain for what the workspace should have told it
 * Tensors are aligned to their elements.  Outputs must not overlap any other
 * buffer.  tokens up to 2^31 - 4097, seqs below 2^28, width up to 2^24, and
 * (tokens / E2TTT_SCAN_TILE + seqs) ceil(width / 64) up to 2^22 (else
 * E2TTT_ERR_UNSUPPORTED; the forward takes more tokens of short sequences).
 */
#define E2TTT_SCAN_TILE 128
typedef struct {
    int32_t io_dtype;
    int32_t gate_dtype; /* of a: fp32, or io_dtype */
    int64_t tokens, seqs, width;
    int64_t x_tok, a_tok; /* at least width, up to 2^31 */
} e2ttt_scan_desc;

E2TTT_API size_t e2ttt_scan_workspace_size(const e2ttt_scan_desc* desc);
E2TTT_API int e2ttt_scan_forward(const e2ttt_scan_desc* desc, const void* x, const void* a, const float* h0,
                        const int32_t* cu_seqlens, void* out, float* state, float* starts,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of <dout, out> + <dstate, state>, from the forward's inputs and
 * starts:
 *   g_t = dout_t + a_{t+1} g_{t+1}  (+ dstate after the last token),
 *   dx_t = g_t,  da_t = g_t h_{t-1},  dh0 = a_1 g_1  (dstate for no token).
 * dout, dx [tokens][width] io_dtype and da [tokens][width] gate_dtype
 * contiguous; dstate (or NULL: 0) and dh0 (or NULL) [seqs][width] fp32.  dx and
 * da are 0 for tokens of no sequence.  Outputs must not overlap any other buffer.
 */
E2TTT_API size_t e2ttt_scan_backward_workspace_size(const e2ttt_scan_desc* desc);
E2TTT_API int e2ttt_scan_backward(const e2ttt_scan_desc* desc, const void* dout, const void* x, const void* a,
                        const float* starts, const float* dstate, const int32_t* cu_seqlens, void* dx, void* da,
                        float* dh0, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Root-mean-square norm with the residual's addition:
 *   h = x + residual, rounded to the stream's type (h = x without residual),
 *   rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd weight,
 * y in the stream's type, or with bits8 in OCP e4m3 with an fp32 scale per
 * row: scale = max|y| / 448 (1 for a row of zeros, NaN for one that holds a
 * NaN, and at least 2^-149), y8 = round(y / scale).
 *   x, residual, h  [rows][width] io_dtype contiguous; weight [width] fp32
 *   y               [rows][width] io_dtype, or uint8 with bits8
 *   scale           [rows] fp32, with bits8 only; rstd [rows] fp32 or NULL
 * Tensors are aligned to their elements; rows that all start on 16 bytes (the
 * tensors, and width times the element's size) are read in wider loads.
 * residual = h = NULL for the norm alone.  h may be residual or x (in place);
 * any other overlap of an output is E2TTT_ERR_ALIAS.
 */
typedef struct {
    int32_t io_dtype;
    int32_t bits8;
    int64_t rows, width; /* width up to 65536 */
    float eps;
    int32_t reserved; /* 0 */
} e2ttt_norm_desc;

E2TTT_API int e2ttt_norm_forward(const e2ttt_norm_desc* desc, const void* x, const void* residual,
                        const float* weight, void* y, float* scale, void* h, float* rstd, void* stream);

/*
 * With xhat = h rstd and g = dy weight:
 *   dx = dh + rstd (g - xhat mean(g xhat))   (also the residual's gradient),
 *   dweight = sum over rows of dy xhat.
 * dy, h, dh (or NULL), dx [rows][width] io_dtype; dweight [width] fp32.
 * dx may be dh (in place); any other overlap of an output is an error.
 */
E2TTT_API size_t e2ttt_norm_backward_workspace_size(const e2ttt_norm_desc* desc);
E2TTT_API int e2ttt_norm_backward(const e2ttt_norm_desc* desc, const void* dy, const void* h, const float* weight,
                        const float* rstd, const void* dh, void* dx, float* dweight,
                        void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* E2TTT_LAYER_H */
