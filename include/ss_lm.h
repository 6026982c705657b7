/*
 * ss_lm.h -- the operators of libssscan.so that stand beside the scan in a
 * recurrent language model (MI355X, gfx950): the gated linear recurrence, the
 * gated feed-forward projection, and the softmax cross entropy of a vocabulary
 * projection, each with its backward pass.
 *
 * Conventions, status codes and error reporting are those of ss_scan.h, with
 * these additions:
 *  - `dtype` is the element type of the activations, the weights of the two
 *    matrix operators and all their gradients.  Products of bf16 operands are
 *    accumulated in fp32; softmax statistics, losses and recurrent states are
 *    fp32; every other result is rounded once from fp32, to nearest even.
 *  - A row stride counts elements between two rows' first elements and is at
 *    least the row's length; rows are (batch, seqlen) or tokens in order, so a
 *    column slice of a wider contiguous tensor is read in place.
 *  - Workspace contents on entry are unused; sizes depend on the shape alone.
 *    Workspaces are 256-byte aligned and overlap nothing.
 *  - Outputs overlap neither the inputs nor each other.
 *  - Sizes whose launch would take 2^32 threads or more along a grid's axis are
 *    SS_ERR_UNSUPPORTED.
 *  - Every sum is taken in a fixed order: results are the same from run to run.
 */
#ifndef SS_LM_H
#define SS_LM_H

#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated linear recurrence, per batch row b and channel d:
 *   k[d] = c * log(1 + exp(decay[d]))                   (the decay rate, c > 0)
 *   a_t  = exp(-k[d] * sigmoid(r[b,t,d]))               (0 where reset[b,t] != 0)
 *   h_t  = a_t * h_{t-1} + sqrt(1 - a_t^2) * sigmoid(i[b,t,d]) * x[b,t,d]
 *   y[b,t,d] = h_t
 * r and i are the gates before their sigmoids.  A reset starts a new sequence
 * at its row: nothing of the state before it remains.
 *
 *   x, r, i : (batch, seqlen, dim) dtype, each with its own row stride (the
 *             three may be column slices of one projection's output)
 *   decay   : (dim,) fp32
 *   h0      : (batch, dim) fp32, or NULL (zero)
 *   reset   : (batch, seqlen) bytes, or NULL (no resets)
 *   y       : (batch, seqlen, dim) dtype output
 *   h_last  : (batch, dim) fp32 output, the state after the last row, or NULL
 *   ckpt    : (ceil(seqlen/32), batch, dim) fp32 output, the state entering
 *             every 32nd row, for ss_glr_bwd; or NULL
 * h_last may be exactly h0.  c must be finite and positive.  Row strides (and
 * dim) above 2^20 elements are SS_ERR_UNSUPPORTED.
 */
size_t ss_glr_ckpt_bytes(int64_t batch, int64_t seqlen, int64_t dim);
size_t ss_glr_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim); /* 0: none needed */

ss_status ss_glr_fwd(const void* x, int64_t x_row_stride, const void* r, int64_t r_row_stride, const void* i,
                     int64_t i_row_stride, const float* decay, float c, const float* h0, const uint8_t* reset,
                     void* y, float* h_last, float* ckpt, void* workspace, size_t workspace_bytes, int64_t batch,
                     int64_t seqlen, int64_t dim, ss_dtype dtype, hipStream_t stream);

/*
 * ss_glr_bwd -- gradients of sum(dy * y) + sum(dh_last * h_last) with respect
 * to every input of ss_glr_fwd.  The states are rebuilt from ckpt as written
 * by ss_glr_fwd for the same inputs, or, with ckpt NULL, from a pass of its
 * own over the inputs.
 *   dy         : (batch, seqlen, dim) dtype
 *   dh_last    : (batch, dim) fp32, or NULL (zero)
 *   dx, dr, di : (batch, seqlen, dim) dtype outputs, rows grad_row_stride
 *                elements apart (the three may be column slices of one tensor)
 *   ddecay     : (dim,) fp32 output
 *   dh0        : (batch, dim) fp32 output, or NULL
 * with_ckpt of the workspace query: whether the call is given ckpt.
 */
size_t ss_glr_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int with_ckpt);

ss_status ss_glr_bwd(const void* x, int64_t x_row_stride, const void* r, int64_t r_row_stride, const void* i,
                     int64_t i_row_stride, const float* decay, float c, const float* h0, const uint8_t* reset,
                     const void* dy, const float* dh_last, const float* ckpt, void* dx, void* dr, void* di,
                     int64_t grad_row_stride, float* ddecay, float* dh0, void* workspace, size_t workspace_bytes,
                     int64_t batch, int64_t seqlen, int64_t dim, ss_dtype dtype, hipStream_t stream);

/*
 * ss_glr_step -- one token of the recurrence, in place on the state:
 *   h       : (batch, dim) fp32, read and overwritten
 *   x, r, i : (batch, dim) dtype, each with its own row stride
 *   y       : (batch, dim) dtype output
 */
ss_status ss_glr_step(float* h, const void* x, int64_t x_row_stride, const void* r, int64_t r_row_stride,
                      const void* i, int64_t i_row_stride, const float* decay, float c, void* y, int64_t batch,
                      int64_t dim, ss_dtype dtype, hipStream_t stream);

/*
 * Gated feed-forward projection:
 *   h = act(x Wg^T) * (x Wu^T)
 * elementwise product; act is silu(g) = g sigmoid(g), or gelu in its tanh form,
 * 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))).  Both products, the
 * activation and the product are one kernel; x Wg^T and x Wu^T are not stored.
 *
 *   x        : (tokens, dim) dtype, rows x_row_stride elements apart
 *   w_gate, w_up : (features, dim) dtype
 *   h        : (tokens, features) dtype output
 * bf16 with dim a multiple of 8: x, w_gate and w_up must be 16-byte aligned and
 * x_row_stride a multiple of 8 (SS_ERR_INVALID_ARG otherwise).  Other dims, and
 * fp32, take any element-aligned operands; bf16 ones may first be copied to
 * padded rows in the workspace.
 * fp32 products of more than a few rows are formed from three bf16 parts of each
 * operand, six products of parts accumulated in fp32: each product is within
 * 2^-23 of itself (fp32 rounds one by up to 2^-24), and operands below 2^-110
 * keep no bits below 2^-134.  Infinities, NaN and numbers up to the largest
 * give what fp32 arithmetic gives.
 */
typedef enum { SS_ACT_SILU = 0, SS_ACT_GELU = 1 } ss_activation;

size_t ss_glu_workspace_bytes(int64_t tokens, int64_t dim, int64_t features, ss_dtype dtype); /* 0: none needed */

ss_status ss_glu_fwd(const void* x, int64_t x_row_stride, const void* w_gate, const void* w_up, void* h,
                     ss_activation act, void* workspace, size_t workspace_bytes, int64_t tokens, int64_t dim,
                     int64_t features, ss_dtype dtype, hipStream_t stream);

/*
 * ss_glu_bwd -- gradients of sum(dh * h), both products formed again from x:
 *   dh      : (tokens, features) dtype
 *   dx      : (tokens, dim) dtype output, or NULL (not wanted)
 *   dw_gate, dw_up : (features, dim) dtype outputs, or both NULL
 * The gradients of x Wg^T and x Wu^T are rounded to dtype between the
 * products (of up to 32 bf16 tokens dw_gate and dw_up take what the rounding
 * leaves too).  Alignment as for ss_glu_fwd.
 */
size_t ss_glu_bwd_workspace_bytes(int64_t tokens, int64_t dim, int64_t features, ss_dtype dtype);

ss_status ss_glu_bwd(const void* x, int64_t x_row_stride, const void* w_gate, const void* w_up, const void* dh,
                     void* dx, void* dw_gate, void* dw_up, ss_activation act, void* workspace,
                     size_t workspace_bytes, int64_t tokens, int64_t dim, int64_t features, ss_dtype dtype,
                     hipStream_t stream);

/*
 * Softmax cross entropy of a vocabulary projection: with logits l = x w^T,
 *   lse[i]  = log(sum_j exp(l[i,j]))
 *   loss[i] = lse[i] - l[i, target[i]]
 * without storing the logits.  A row whose target equals ignore_index, or lies
 * outside [0, vocab), has loss 0 and no gradient: dx is 0 there and nothing of
 * its x or dloss, whatever they hold, enters dw.
 *
 *   x      : (tokens, dim) dtype, rows x_row_stride elements apart
 *   w      : (vocab, dim) dtype
 *   target : (tokens,) int64
 *   loss, lse : (tokens,) fp32 outputs
 * Alignment of x, x_row_stride and w as for ss_glu_fwd.
 */
size_t ss_xent_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab, ss_dtype dtype);

ss_status ss_xent_fwd(const void* x, int64_t x_row_stride, const void* w, const int64_t* target,
                      int64_t ignore_index, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                      int64_t tokens, int64_t dim, int64_t vocab, ss_dtype dtype, hipStream_t stream);

/*
 * ss_xent_bwd -- gradients of sum(dloss * loss), lse as ss_xent_fwd gave it.
 * The vocabulary is taken in pieces: a piece's logits are formed again, their
 * gradient is rounded to dtype in the workspace, and its parts of dx and dw
 * follow before the next piece reuses the space.
 *   dloss : (tokens,) fp32
 *   dx    : (tokens, dim) dtype output, or NULL (not wanted)
 *   dw    : (vocab, dim) dtype output, or NULL
 */
size_t ss_xent_bwd_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab, ss_dtype dtype);

ss_status ss_xent_bwd(const void* x, int64_t x_row_stride, const void* w, const int64_t* target,
                      int64_t ignore_index, const float* lse, const float* dloss, void* dx, void* dw,
                      void* workspace, size_t workspace_bytes, int64_t tokens, int64_t dim, int64_t vocab,
                      ss_dtype dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_LM_H */
