/*
 * ss_attn.h -- the operators of libssscan.so (MI355X, gfx950) of a layer that mixes tokens by
 * linear attention, and of the choice of the next token: linear attention with a decay for each
 * head, the norms of its queries and keys with their position rotation, and sampling from logits.
 *
 * Conventions, status codes and error reporting are those of ss_scan.h and ss_lm.h, with these
 * additions:
 *  - Heads lie side by side in a token's row: head h of a (batch, seqlen, heads, width) operand
 *    starts h * width elements into the row.  A row stride counts elements between two tokens'
 *    first elements and is at least heads * width, so that a projection's output that holds
 *    several operands side by side is read in place.
 *  - Operands are aligned to their elements; rows of 16-byte chunks (base, row stride and head
 *    width multiples of 16 bytes) are read fastest.
 *  - Outputs are contiguous.
 */
#ifndef SS_ATTN_H
#define SS_ATTN_H

#include "ss_lm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention with a decay for each head.  With a = exp(log_decay[h]), per batch row and
 * head, from the state S_{-1} = h0:
 *   S_t = a S_{t-1} + k_t v_t^T              (k_t v_t^T alone where reset[b,t] != 0)
 *   o_t = scale * S_t^T q_t
 * A reset starts a new sequence at its row: nothing of the state before it remains, whatever it
 * held.  Row t takes nothing from the rows behind it, whatever they hold.
 *
 *   q, k      : (batch, seqlen, qk_heads, k_dim) dtype, each with its own row stride
 *   v         : (batch, seqlen, heads, v_dim) dtype, with a row stride; heads is a multiple of
 *               qk_heads, and head h uses the queries and keys of head h / (heads / qk_heads)
 *   log_decay : (heads,) fp32, at most 0 (a head that forgets everything has -infinity)
 *   h0        : (batch, heads, k_dim, v_dim) fp32, or NULL (zero)
 *   reset     : (batch, seqlen) bytes, or NULL (no resets)
 *   o         : (batch, seqlen, heads, v_dim) dtype output
 *   h_last    : (batch, heads, k_dim, v_dim) fp32 output, the state after the last row, or NULL;
 *               may be exactly h0
 * scale must be finite.  k_dim and v_dim above 256, heads * k_dim, heads * v_dim and, where seqlen is
 * above 1, row strides above 2^20 elements, and seqlen from 2^30 on are SS_ERR_UNSUPPORTED.
 * The state is fp32 throughout.  bf16: it and the products q k^T are rounded to bf16 where they
 * enter a product with q or v.  fp32: products are formed from three bf16 parts of each operand,
 * which hold its 24 bits.  An infinity in q, k, v or the state gives infinities or NaN in the rows
 * and states that see it, and none in the others.
 */
size_t ss_lattn_workspace_bytes(int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim,
                                int64_t v_dim, ss_dtype dtype); /* 0: none needed */

ss_status ss_lattn_fwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                       int64_t v_row_stride, const float* log_decay, float scale, const float* h0,
                       const uint8_t* reset, void* o, float* h_last, void* workspace, size_t workspace_bytes,
                       int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim, int64_t v_dim,
                       ss_dtype dtype, hipStream_t stream);

/*
 * ss_lattn_bwd -- gradients of sum(d_o * o) + sum(dh_last * h_last) with respect to q, k, v and
 * h0 (log_decay is a constant of the layer and has none).  With G_t the gradient of S_t,
 *   G_t = scale q_t d_o_t^T + a G_{t+1}   (the last row: + dh_last; nothing of G_{t+1} where
 *                                          reset[b,t+1] != 0)
 *   dq_t = scale S_t d_o_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dh0 = a G_0  (0 where reset[b,0] != 0)
 * and dq and dk are summed over the heads that share them.  Nothing of the forward is kept: S is
 * formed again.
 *   d_o     : (batch, seqlen, heads, v_dim) dtype, with a row stride
 *   dh_last : (batch, heads, k_dim, v_dim) fp32, or NULL (zero)
 *   dq, dk  : (batch, seqlen, qk_heads, k_dim) dtype outputs
 *   dv      : (batch, seqlen, heads, v_dim) dtype output
 *   dh0     : (batch, heads, k_dim, v_dim) fp32 output, or NULL
 */
size_t ss_lattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim,
                                    int64_t v_dim, ss_dtype dtype);

ss_status ss_lattn_bwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                       int64_t v_row_stride, const float* log_decay, float scale, const float* h0,
                       const uint8_t* reset, const void* d_o, int64_t do_row_stride, const float* dh_last, void* dq,
                       void* dk, void* dv, float* dh0, void* workspace, size_t workspace_bytes, int64_t batch,
                       int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim, int64_t v_dim, ss_dtype dtype,
                       hipStream_t stream);

/*
 * ss_lattn_step -- one token of the recurrence, in place on the state:
 *   h    : (batch, heads, k_dim, v_dim) fp32, read and overwritten
 *   q, k : (batch, qk_heads, k_dim) dtype, each with its own row stride
 *   v    : (batch, heads, v_dim) dtype, with a row stride
 *   o    : (batch, heads, v_dim) dtype output
 */
ss_status ss_lattn_step(float* h, const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                        const void* v, int64_t v_row_stride, const float* log_decay, float scale, void* o,
                        int64_t batch, int64_t qk_heads, int64_t heads, int64_t k_dim, int64_t v_dim, ss_dtype dtype,
                        hipStream_t stream);

/*
 * Norms of queries and keys for each head, and their position rotation, in one pass.  For each
 * token and head, x of q or k:
 *   y = x / sqrt(mean(x^2) + eps) * w
 * and of y's first 2 n elements, n = half_rotary, pair i is turned by the angle
 * pos[token] * inv_freq[i], formed and reduced to one turn in 64 bits:
 *   (y1, y2) -> (y1 cos - y2 sin, y2 cos + y1 sin)
 * Pair i is elements (i, i + n), or (2 i, 2 i + 1) with interleaved != 0.  The rest stays.
 *
 *   q        : (tokens, q_heads, width) dtype, with a row stride
 *   k        : (tokens, k_heads, width) dtype, with a row stride
 *   w_q, w_k : (width,) fp32
 *   pos      : (tokens,) int64
 *   inv_freq : (half_rotary,) fp32; NULL if half_rotary is 0
 *   qo, ko   : (tokens, q_heads, width), (tokens, k_heads, width) dtype outputs
 * width is at most 512, q_heads and k_heads at most 2^24 (SS_ERR_UNSUPPORTED above); width is at least
 * 2 half_rotary; eps is finite and not negative.  The mean of the squares is fp32: a head whose squares
 * sum past its range is normed to 0, with gradient 0; squares below its range (of elements below 2^-63)
 * lose bits or count as 0, so that a head of such elements is normed by eps, and with eps 0 to infinities
 * or NaN, as a head of zeros then is to NaN.
 */
ss_status ss_qknorm_fwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const float* w_q,
                        const float* w_k, const int64_t* pos, const float* inv_freq, float eps, int interleaved,
                        void* qo, void* ko, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t width,
                        int64_t half_rotary, ss_dtype dtype, hipStream_t stream);

/*
 * ss_qknorm_bwd -- gradients of sum(dqo * qo) + sum(dko * ko) with respect to q, k, w_q and w_k.
 *   dqo, dko   : (tokens, q_heads, width), (tokens, k_heads, width) dtype, contiguous
 *   dq, dk     : the same shapes, dtype outputs
 *   dw_q, dw_k : (width,) fp32 outputs, sums over the tokens and heads in a fixed order
 */
size_t ss_qknorm_bwd_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t width);

ss_status ss_qknorm_bwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const float* w_q,
                        const float* w_k, const int64_t* pos, const float* inv_freq, float eps, int interleaved,
                        const void* dqo, const void* dko, void* dq, void* dk, float* dw_q, float* dw_k,
                        void* workspace, size_t workspace_bytes, int64_t tokens, int64_t q_heads, int64_t k_heads,
                        int64_t width, int64_t half_rotary, ss_dtype dtype, hipStream_t stream);

/*
 * Sampling: one token for each row of logits from one given random number.  The row's tokens are
 * ordered by logit, the largest first, equal ones by index, l_0 >= l_1 >= ...; token j has weight
 * w_j = exp((l_j - l_0) / temperature), and of them remain
 *   1. the first top_k                                          (all with top_k <= 0)
 *   2. those before which the weights sum to less than top_p of the sum over 1.   (all with top_p >= 1)
 *   3. those with w_j >= min_p                                  (all with min_p <= 0)
 * and always the first.  The token is the first of these at which the running sum of their
 * weights exceeds u times their whole sum (the last that has a weight if none does).
 * Weights and sums have 64 bits: each weight is rounded to a multiple of 2^-min(50, 62 - b), b the
 * number of bits of vocab, so that a whole row's sum fits and does not depend on its order.
 *
 * A temperature that is not above 0 takes the largest logit, the first of its equals.  Logits
 * that are NaN or -infinity are never taken: a row without another has token -1.  If the largest
 * is +infinity, the tokens that hold it share the weight.  NaN top_p and min_p are off; a NaN u is 0.
 *
 *   logits : (rows, vocab) dtype, row_stride elements apart
 *   u      : (rows,) fp32, in [0, 1)
 *   temperature, top_k, top_p, min_p : (rows,) fp32, int32, fp32, fp32, or NULL: every row then has
 *            the value beside it
 *   token  : (rows,) int64 output
 * vocab is at most 2^24 (SS_ERR_UNSUPPORTED above).
 */
size_t ss_sample_workspace_bytes(int64_t rows, int64_t vocab, ss_dtype dtype); /* 0: none needed */

ss_status ss_sample(const void* logits, int64_t row_stride, const float* u, const float* temperature,
                    float temperature_all, const int32_t* top_k, int32_t top_k_all, const float* top_p,
                    float top_p_all, const float* min_p, float min_p_all, int64_t* token, void* workspace,
                    size_t workspace_bytes, int64_t rows, int64_t vocab, ss_dtype dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_ATTN_H */
