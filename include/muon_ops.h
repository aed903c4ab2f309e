/*
 * muon_ops.h -- C ABI of the layer operators that make the gradients a Muon
 * step consumes (same library, status codes and dtypes as muon.h).
 *
 *  - linear: y = act(x W + b) + r over one weight, or over the experts of a
 *    3-D weight [E, K, N] whose rows are grouped by expert; and its gradient.
 *  - route, dispatch, combine: entries sorted by expert, rows moved to that
 *    order and back with weights, and the gradients of both moves.
 *  - dropout from a counter-based generator, with an optional residual.
 *
 * Memory: every pointer is a DEVICE pointer on the current device, aligned to
 * its element; 16-byte aligned rows take the faster loads.  Workspaces belong
 * to the caller, must be 16-byte aligned and may be reused once the calls that
 * were given them have run.  Nothing is allocated, nothing is kept between
 * calls and no call synchronises, so calls may be captured into a HIP graph
 * and may run on several streams at once with workspaces of their own.
 *
 * Errors: as in muon.h; arguments are checked before anything is enqueued.
 * Sums, activations and weights' products are float32; what is stored in
 * bf16 (z and dz among it) is rounded to nearest even once.  No result depends on the order in
 * which workgroups run.
 */
#ifndef MUON_OPS_H
#define MUON_OPS_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_ACT_NONE = 0,
  MUON_ACT_RELU = 1,
  MUON_ACT_SILU = 2,      /* z / (1 + e^-z)                                                 */
  MUON_ACT_GELU = 3,      /* z Phi(z), Phi the normal distribution function                  */
  MUON_ACT_GELU_TANH = 4  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2                 */
} muon_act_t;

/* A linear layer.  x [rows, k], y [rows, n]; weight [k, n] (w_layout 0: element
 * (i, j) at i ldw + j) or its transpose in memory (1: at j ldw + i).
 * groups = 0: one weight.  groups > 0: that many weights w_stride elements
 * apart, and calls take `offsets`, groups + 1 int32 on the device, non
 * decreasing from 0 to <= rows: rows offsets[e] .. offsets[e + 1] meet weight e;
 * rows past offsets[groups] give zero.  (Offsets that break this give
 * unspecified values, never an access outside the tensors.)  Sizes go up to 2^31 - 1024.  Strides are in
 * elements; a row's elements are contiguous. */
typedef struct {
  int32_t dtype;     /* muon_dtype_t of x, W, b, r, y, z and their gradients */
  int32_t act;       /* muon_act_t                                            */
  int32_t groups;
  int32_t w_layout;
  int64_t rows, k, n;
  int64_t ldx;       /* row stride of x                                       */
  int64_t ldw;       /* row stride of W as stored                             */
  int64_t w_stride;  /* from one expert's weight to the next                  */
  int64_t ldr;       /* row stride of the residual (forward)                  */
  int64_t ldg;       /* row stride of the gradient read (dy, or dz where act'
                        was applied)                                          */
} muon_linear_desc_t;

typedef enum {
  MUON_LINEAR_FORWARD = 0,
  MUON_LINEAR_GRAD_ACT = 1,
  MUON_LINEAR_GRAD_INPUT = 2,
  MUON_LINEAR_GRAD_WEIGHT = 3,
  MUON_LINEAR_BACKWARD = 4
} muon_linear_op_t;

/* Workspace of one of the calls below, for pointers that are 16-byte
 * aligned or not (host only; 0 for many shapes).  A large bf16 product of odd
 * sizes copies its operands there. */
int muon_linear_workspace(const muon_linear_desc_t* desc, int32_t op, uint64_t* bytes);

/* z = x W + b, y = act(z) + r.  bias [max(groups, 1), n], residual (groups = 0
 * only) and z may be NULL; y and z are contiguous [rows, n].  z is the value
 * the gradient of the activation is taken at. */
int muon_linear_forward(const muon_linear_desc_t* desc, const int32_t* offsets, const void* x, const void* w,
                        const void* bias, const void* residual, void* y, void* z, void* workspace,
                        uint64_t workspace_bytes, void* stream);

/* dz = dy act'(z) (contiguous; NULL: not stored) and db[e] = sum of dz over the
 * rows of e (NULL: not computed).  z is NULL when act is MUON_ACT_NONE.
 * Rows past offsets[groups] give dz = 0. */
int muon_linear_grad_act(const muon_linear_desc_t* desc, const int32_t* offsets, const void* dy, const void* z,
                         void* dz, void* db, void* workspace, uint64_t workspace_bytes, void* stream);

/* dx = dz W^T, contiguous [rows, k]; rows past offsets[groups] are zero. */
int muon_linear_grad_input(const muon_linear_desc_t* desc, const int32_t* offsets, const void* dz, const void* w,
                           void* dx, void* workspace, uint64_t workspace_bytes, void* stream);

/* dW[e] = x[rows of e]^T dz[rows of e], contiguous in the layout of w_layout
 * ([k, n], or [n, k] for 1); zero for an expert without rows. */
int muon_linear_grad_weight(const muon_linear_desc_t* desc, const int32_t* offsets, const void* x, const void* dz,
                            void* dw, void* workspace, uint64_t workspace_bytes, void* stream);

/* The three steps above in one call: dx, dw and db, each NULL where not wanted,
 * from x, W, z and dy; dz stays in the workspace.  In bf16 dz is rounded for the
 * products, so that dx and dW carry one rounding more than their own; up to 64 rows,
 * or 16 for each group on average, what that loses is kept and added, which the three
 * steps alone do not do. */
int muon_linear_backward(const muon_linear_desc_t* desc, const int32_t* offsets, const void* x, const void* w,
                         const void* z, const void* dy, void* dx, void* dw, void* db, void* workspace,
                         uint64_t workspace_bytes, void* stream);

#define MUON_ROUTE_MAX_EXPERTS 1024

/* Workspace of muon_route for so many entries. */
int muon_route_workspace(int64_t entries, int32_t experts, uint64_t* bytes);

/* Stable counting sort of tokens x top expert choices.  ids: [tokens, top],
 * int64 (ids_bytes 8) or int32 (4); an id outside [0, experts) is not routed.
 *  offsets [experts + 1]: first sorted row of each expert, and their total;
 *  order [tokens top]: the flat entry (token top + choice) of each sorted row,
 *    in flat order within an expert; -1 past the total;
 *  position [tokens, top]: the sorted row of each entry, or -1. */
int muon_route(const void* ids, int32_t ids_bytes, int64_t tokens, int32_t top, int32_t experts, int32_t* offsets,
               int32_t* order, int32_t* position, void* workspace, uint64_t workspace_bytes, void* stream);

/* Rows of h elements moved by `position` and `offsets` of muon_route.  Row
 * strides (ldx, ldg, ldr) in elements; outputs are contiguous. */
typedef struct {
  int32_t dtype;
  int32_t experts;
  int32_t top;
  int32_t reserved;
  int64_t tokens, h;
  int64_t ldx, ldg, ldr;
} muon_move_desc_t;

/* xs[position[t][j]] = x[t]; rows past the routed ones are zero. */
int muon_dispatch(const muon_move_desc_t* desc, const int32_t* offsets, const int32_t* position, const void* x,
                  void* xs, void* stream);
/* dx[t] = sum_j dxs[position[t][j]]  (row stride of dxs: ldx). */
int muon_dispatch_grad(const muon_move_desc_t* desc, const int32_t* position, const void* dxs, void* dx,
                       void* stream);
/* y[t] = sum_j weights[t][j] ys[position[t][j]] + residual[t]  (ys: ldx,
 * residual: ldr, NULL for none; weights: contiguous float32). */
int muon_combine(const muon_move_desc_t* desc, const int32_t* position, const float* weights, const void* ys,
                 const void* residual, void* y, void* stream);
/* dys[position[t][j]] = weights[t][j] dy[t], zero past the routed rows;
 * dweights[t][j] = <dy[t], ys[position[t][j]]>, zero where not routed.  Either
 * output may be NULL (dy: ldg, ys: ldx). */
int muon_combine_grad(const muon_move_desc_t* desc, const int32_t* offsets, const int32_t* position,
                      const float* weights, const void* ys, const void* dy, void* dys, float* dweights, void* stream);

/* y = keep x 65536 / (65536 - D) + residual with D = 65536 p rounded to the nearest (ties to even), over n
 * contiguous elements.  Element i is kept when lane i mod 8 (16 bits, low half
 * of word 0 first) of Philox4x32-10 with counter (i div 8, offset) and key
 * `seed` is at least D.  D = 65536 is refused.  state: NULL, or two uint64 on the device {seed, offset}
 * that take their place (so that a captured call can be given new ones).
 * The gradient of x is the same call on dy without a residual. */
int muon_dropout(int32_t dtype, int64_t n, const void* x, const void* residual, void* y, double p, uint64_t seed,
                 uint64_t offset, const uint64_t* state, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MUON_OPS_H */
