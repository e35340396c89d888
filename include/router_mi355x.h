/*
 * router_mi355x.h - C ABI of the router's side of the grouped products on MI355X (gfx950): per-expert counts
 * with their offsets, the balance loss of a batch of tokens, and its gradient. Same library, status codes, error
 * messages (gemm_last_error) and conventions as gemm_mi355x.h: every tensor pointer is a caller-owned DEVICE
 * pointer, launches are asynchronous on `stream`, no entry point allocates device memory or synchronises,
 * errors are returned and never thrown.
 *
 * `batch` sequences of `tokens` tokens each choose among `experts` experts. Of the logits x of a token:
 *   ROUTER_SOFTMAX   p_e = exp(x_e) / sum_j exp(x_j)
 *   ROUTER_SIGMOID   p_e = s(x_e) / sum_j s(x_j),   s(x) = 1 / (1 + exp(-x))
 * A token whose mask is 0 (padding) counts nowhere, whatever its logits hold; one whose logits are all -inf has
 * p = 0, and scores below 2^-126 may be 0. With n_b the unmasked tokens of sequence b, c_be how often they chose
 * expert e, and k choices a token:
 *   P_be = sum over its tokens of p_e / n_b     f_be = experts * c_be / (k * n_b)
 *   loss = coef / batch * sum over b, e of f_be * P_be         (a sequence without tokens adds 0)
 * so that an even choice gives coef. batch = 1: one loss over all tokens; more: one for each sequence. Sums are held in
 * fp32 and run in a fixed order: results repeat bit for bit.
 */
#ifndef ROUTER_MI355X_H
#define ROUTER_MI355X_H

#include "gemm_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ROUTER_SOFTMAX = 0, ROUTER_SIGMOID = 1 } router_scores;

/* logits: (batch, tokens, experts) of type F16 / BF16 / F32, element e of token t of sequence b at
 * b * logits_batch + t * logits_ld + e. chosen: (batch, tokens, k) indices of index_bytes 4 (int32) or 8
 * (int64) each, contiguous; an index outside [0, experts) is no choice, one that a token names twice counts
 * twice. mask: (batch, tokens) bytes, or NULL: all count.
 * Outputs: counts int32 (batch, experts), valid int32 (batch) = n_b, probs fp32 (batch, experts) = P, loss fp32 (1),
 * and, unless NULL, cu_seqlens int32 (experts + 1): the running sum of the counts over all sequences, 0 first, as the
 * grouped products take it for rows in the order of their experts (wrong past 2^31 choices).
 * workspace: router_balance_workspace bytes, 16-byte aligned; its contents need no preparation, and calls that
 * follow each other on a stream may share it. 1 <= experts <= 2048, 1 <= k <= experts, batch <= 65535, batch * tokens
 * * k below 2^31. Rows do not overlap; sequences follow each other or alternate row by row (tokens
 * outermost). batch = 0 or tokens = 0 gives zeros. */
typedef struct {
  int32_t batch, tokens, experts, k;
  int32_t type;   /* gemm_dtype of the logits */
  int32_t scores; /* router_scores */
  int32_t index_bytes;
  float coef;
  const void* logits;
  const void* chosen;
  const uint8_t* mask; /* or NULL */
  int32_t* counts;
  int32_t* valid;
  int32_t* cu_seqlens; /* or NULL */
  float* probs;
  float* loss;
  void* workspace;
  int64_t workspace_bytes;
  int64_t logits_ld, logits_batch;
} router_balance_args;
gemm_status router_balance(const router_balance_args* args, void* stream);
/* Bytes of workspace (-1 for a negative size, or one that router_balance refuses as too large). */
int64_t router_balance_workspace(int32_t batch, int32_t tokens, int32_t experts);

/* The gradient of grad * loss with respect to the logits (the counts are constants):
 *   w_be = grad * coef * experts * c_be / (batch * k * n_b^2)
 *   softmax: dx_e = p_e (w_e - sum_j p_j w_j)       sigmoid: the same times (1 - s(x_e))
 * of the counts and valid that router_balance gave. (Computed with the counts less the sequence's smallest one, which
 * changes nothing as p sums to 1: even counts have a gradient of exactly 0.) Masked tokens get 0. grad: device
 * fp32 (1), or NULL for 1. dlogits has the logits' type and its own strides, and may be the logits
 * themselves. */
typedef struct {
  int32_t batch, tokens, experts, k;
  int32_t type;
  int32_t scores;
  float coef;
  const void* logits;
  const uint8_t* mask; /* or NULL */
  const int32_t* counts;
  const int32_t* valid;
  const float* grad; /* or NULL */
  void* dlogits;
  int64_t logits_ld, logits_batch, dlogits_ld, dlogits_batch;
} router_balance_backward_args;
gemm_status router_balance_backward(const router_balance_backward_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ROUTER_MI355X_H */
