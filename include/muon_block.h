/*
 * muon_block.h -- C ABI of the operators around a block's products (same
 * library, status codes and dtypes as muon.h; memory, streams, workspaces and
 * errors as in muon_ops.h).
 *
 *  - norm: layer norm and root-mean-square norm of rows, with the residual
 *    added ahead of them, and their gradient.
 *  - gate: the largest logits of each token and their softmax weights, which
 *    muon_route and muon_combine take; and the gradient.
 *  - balance: the loss that keeps the experts' loads even, the count of every
 *    expert, and the gradient.
 *  - mx: weights held in four bits (e2m1 in blocks of 32 with an e8m0 scale, the
 *    Open Compute Project's microscaling formats 1.0) and the linear and
 *    expert layers over them, without gradients.
 */
#ifndef MUON_BLOCK_H
#define MUON_BLOCK_H

#include "muon_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_NORM_LAYER = 0, /* xhat = (s - mean) / sqrt(var + eps), var the mean of (s - mean)^2 */
  MUON_NORM_RMS = 1    /* xhat = s / sqrt(mean(s^2) + eps)                                  */
} muon_norm_t;

/* Rows of cols elements; strides in elements, a row's elements contiguous.
 * rows up to 2^31 - 1024, cols up to 2^24. */
typedef struct {
  int32_t dtype;   /* of x, residual, w, b, y, s and their gradients */
  int32_t kind;    /* muon_norm_t                                     */
  int64_t rows, cols;
  int64_t ldx;     /* row stride of x                                 */
  int64_t ldr;     /* row stride of the residual                      */
  int64_t ldg;     /* row stride of dy                                */
  int64_t ldd;     /* row stride of ds                                */
  double eps;      /* at least 0                                      */
} muon_norm_desc_t;

/* s = x + residual (s is x where residual is NULL; the argument s is then NULL
 * too), y = xhat w + b.  w and b [cols] may be NULL; y and s are contiguous.  y comes from the
 * float32 sum.  stats: NULL, or 2 rows float32 that the gradient needs. */
int muon_norm_forward(const muon_norm_desc_t* desc, const void* x, const void* residual, const void* w, const void* b,
                      void* y, void* s, float* stats, void* stream);

/* Workspace of muon_norm_backward (host only). */
int muon_norm_workspace(const muon_norm_desc_t* desc, uint64_t* bytes);

/* With g = dy w: dx = (g - mean(g) - xhat mean(g xhat)) / sqrt(var + eps) + ds
 * (no mean(g) for MUON_NORM_RMS; ds NULL: none), contiguous, the gradient of
 * x and of the residual alike; dw = sum over rows of dy xhat; db = sum of dy.
 * Each of dx, dw and db is NULL where not wanted.  x and residual as in the forward pass, or s for x and NULL:
 * that reads and keeps one tensor less, and takes s as it was rounded. */
int muon_norm_backward(const muon_norm_desc_t* desc, const void* dy, const void* x, const void* residual, const void* w,
                       const float* stats, const void* ds, void* dx, void* dw, void* db, void* workspace,
                       uint64_t workspace_bytes, void* stream);

/* A router's logits [tokens, experts], rows ldz apart; experts up to 1024,
 * top <= experts.  mask: NULL, or one byte a token, 0 for a token that takes no part. */
typedef struct {
  int32_t dtype;      /* of the logits and their gradient                       */
  int32_t experts, top;
  int32_t normalize;  /* gate: weights sum to one over the chosen (1), or are
                         the softmax over all experts (0)                       */
  int64_t tokens, ldz;
} muon_gate_desc_t;

/* ids [tokens, top]: the experts of the `top` largest logits in falling order, ties to
 * the lower index, NaN ahead of all; -1 for a masked token, and where only logits of -inf are left.
 * weights [tokens, top] float32, 0 where the id is -1. */
int muon_gate_forward(const muon_gate_desc_t* desc, const void* logits, const uint8_t* mask, float* weights,
                      int32_t* ids, void* stream);
/* dlogits [tokens, experts], contiguous, from dweights and what the forward pass gave.  logits
 * are not read where normalize is 1. */
int muon_gate_backward(const muon_gate_desc_t* desc, const void* logits, const uint8_t* mask, const float* weights,
                       const int32_t* ids, const float* dweights, void* dlogits, void* stream);

/* Workspace of muon_balance_forward (host only). */
int muon_balance_workspace(const muon_gate_desc_t* desc, uint64_t* bytes);

/* loss = experts sum_e f_e P_e: f_e = c_e / (T top), c_e the entries of ids
 * [tokens, top] (int64, ids_bytes 8, or int32, 4) that name e, P_e the mean over
 * tokens of softmax(logits)_e, T the number of tokens that the mask leaves.  Ids
 * outside [0, experts) are not counted; a row of -inf alone has no probabilities.  T = 0 gives 0.
 * counts [experts]: c_e.  shares [experts + 1] float32: what the gradient needs.
 * tokens top up to 2^31 - 1024. */
int muon_balance_forward(const muon_gate_desc_t* desc, const void* logits, const void* ids, int32_t ids_bytes,
                         const uint8_t* mask, float* loss, int32_t* counts, float* shares, void* workspace,
                         uint64_t workspace_bytes, void* stream);
/* dlogits[t][e] = dloss experts / T p_te (f_e - sum_i p_ti f_i), contiguous; 0 for
 * masked tokens.  dloss: one float32 on the device.  (The counts have no gradient.) */
int muon_balance_backward(const muon_gate_desc_t* desc, const void* logits, const uint8_t* mask, const float* shares,
                          const float* dloss, void* dlogits, void* stream);

/* A weight [k, n], or `groups` of them w_stride elements apart, held in four
 * bits along k.  k and n up to 2^23; groups n k and rows k, with k in steps of 512, n at least 4 and rows in steps of 4,
 * below 2^35. */
typedef struct {
  int32_t dtype;     /* of the weight; of x, bias, residual and y */
  int32_t act;       /* muon_act_t                                */
  int32_t groups;    /* 0: one weight                             */
  int32_t w_layout;  /* quantize: 0: element (i, j) at i ldw + j; 1: at j ldw + i */
  int64_t rows, k, n;
  int64_t ldx, ldw, w_stride, ldr;
} muon_mx_desc_t;

/* Sizes of one weight's (times max(groups, 1)) four-bit form:
 *  values [ceil(k / 128)][n][64]: the e2m1 values of each column by slices of 128, two a byte, lower half first;
 *  scales [ceil(k / 512)][n][16]: byte 4 g + s is the e8m0 scale of the 32 values g (0..3) of slice s (0..3) of 512.
 * Both 16-byte aligned; what pads k is zero. */
int muon_mx_sizes(const muon_mx_desc_t* desc, uint64_t* values_bytes, uint64_t* scales_bytes);

/* A block's scale is 2^(floor(log2 max |w|) - 2), at least 2^-127; values are
 * rounded to nearest (ties to even), and saturate at 6 scales.  A block that holds an infinity or NaN is NaN. */
int muon_mx_quantize(const muon_mx_desc_t* desc, const void* w, uint8_t* values, uint8_t* scales, void* stream);
/* w [groups][n][k] contiguous (the transpose of [k, n]) in desc's dtype: exact in both. */
int muon_mx_dequantize(const muon_mx_desc_t* desc, const uint8_t* values, const uint8_t* scales, void* w,
                       void* stream);

/* Workspace of muon_mx_linear (host only): x in four bits, and partial sums. */
int muon_mx_linear_workspace(const muon_mx_desc_t* desc, uint64_t* bytes);

/* y = act(Q(x) W + bias) + residual, contiguous [rows, n]; Q takes each row of x
 * [rows, k] to four bits along k, the sums are float32.  offsets as in muon_ops.h where groups > 0 (no
 * residual then); bias [max(groups, 1), n] and residual may be NULL. */
int muon_mx_linear(const muon_mx_desc_t* desc, const int32_t* offsets, const void* x, const uint8_t* values,
                   const uint8_t* scales, const void* bias, const void* residual, void* y, void* workspace,
                   uint64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MUON_BLOCK_H */
