/*
 * moe_ops.h -- C ABI of the operators around the Stable LatentMoE layer, in the
 * same library as moe.h: what a Transformer block that serves or trains with
 * the layer needs beside it.
 *
 *   moe_route, moe_route_backward     routing from given logits: softmax or
 *                                     sigmoid scores, selection bias, groups of
 *                                     experts, masked experts
 *   moe_norm, moe_norm_backward       layer norm and RMS norm of rows
 *   moe_linear, moe_linear_backward   matrix product with bias, activation and
 *                                     residual in its epilogue
 *   moe_clip_grads                    global norm of many gradient tensors, and
 *                                     clipping
 *
 * The conventions of moe.h hold: device pointers on the current device,
 * row-major and contiguous in the stated shape, 16-byte aligned unless stated;
 * the caller owns every buffer; the library never allocates or synchronises;
 * arguments are checked on the host before anything is launched; work is
 * enqueued on `stream` in order and can be captured into a CUDA graph;
 * identical inputs give bitwise-identical outputs.  Outputs must not overlap
 * inputs or each other unless stated.  A workspace is 256-byte aligned, need
 * not be initialised, and belongs to one call at a time: two calls that may
 * run at the same time (on two streams, or in two graphs) need one each.
 */
#ifndef MOE_B200_OPS_H
#define MOE_B200_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- routing */

typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

typedef struct {
  int64_t T;           /* tokens, 0 <= T <= 2^31 - 1 */
  int32_t E;           /* experts, 1 <= E <= 1024 */
  int32_t k;           /* experts per token, 1 <= k <= min(32, keep_groups * E / groups) */
  int32_t groups;      /* groups of E / groups consecutive experts, 1 <= groups <= 32, dividing E; 1: none */
  int32_t keep_groups; /* groups kept per token, 1 <= keep_groups <= groups */
  int32_t group_top;   /* a group's score is the sum of its 1 or 2 largest keys (at most E / groups) */
  moe_score score;
  int32_t renorm;      /* != 0: weights divided by their sum over the chosen experts */
  float scale;         /* factor of the weights, finite */
  moe_dtype dtype;     /* of the logits (and of dlogits): MOE_F32, MOE_BF16 or MOE_F16 */
} moe_route_desc;

/* Routing of logits[T, E]:
 *   s = softmax(l) or sigmoid(l) over the experts of a token;
 *   key_e = s_e + bias[e]                  (bias[E] fp32, or NULL for none)
 *   groups > 1: the keep_groups groups with the largest group score remain;
 *   idx[t, 0..k-1] = the experts with the k largest keys among the remaining
 *     groups, in descending order of the key;
 *   w[t, j] = scale * s_{idx_j}, with renorm scale * s_{idx_j} / sum_j' s_{idx_j'}.
 * Equal keys (and equal group scores) go to the lower index.  The order is that
 * of the keys as real numbers: keys that fp32 cannot tell apart are compared in
 * fp64 (without a bias, the logits themselves are compared).
 * A masked expert (logit -inf or NaN) has s = 0 and comes after every unmasked
 * one; a group with no unmasked expert comes after every other.  Where fewer
 * than k unmasked experts remain, masked ones of the kept groups follow in
 * ascending order with weight 0; where all the chosen ones are masked, the
 * weights are 0.  An expert whose bias is -inf or NaN is ordered as a masked one,
 * but keeps the weight of its score.  (A sigmoid score below 2^-126 counts as 0
 * beside chosen ones whose sum is above 1e-18: a share of less than 1e-20.)
 * A row's k indices are always distinct and in [0, E), as moe_permute needs them.
 * A +inf logit is the limit of large ones.
 * idx [T, k] int32, w [T, k] fp32. */
MOE_API moe_status moe_route(const moe_route_desc* d, const void* logits, const float* bias, int32_t* idx, float* w,
                             moe_stream_t stream);

/* Gradient of moe_route's weights with the selection held fixed:
 *   ds_j = scale * dw_j, with renorm scale * (dw_j - sum_j' p_j' dw_j') / sum_j' s_j',
 *          p_j = s_j / sum_j' s_j' (0 where all the chosen ones are masked);
 *   sigmoid: dl_e = ds_j s_e (1 - s_e) at the chosen experts, 0 elsewhere;
 *   softmax: dl_e = s_e (ds_e - sum_j s_j ds_j), ds 0 where e is not chosen.
 * idx[T, k] holds distinct experts in [0, E): an index out of range is recorded
 * as a device fault (moe_device_error, site 11) and adds nothing, a repeated one
 * (site 12) counts once.  dw [T, k] fp32; dlogits [T, E] in the logits' type,
 * every element written.  Masked experts get 0, and their dw is not used.  groups, keep_groups and
 * group_top only have to be valid. */
MOE_API moe_status moe_route_backward(const moe_route_desc* d, const void* logits, const int32_t* idx,
                                      const float* dw, void* dlogits, moe_stream_t stream);

/* ---------------------------------------------------------------- norms */

typedef enum { MOE_NORM_LAYER = 0, MOE_NORM_RMS = 1 } moe_norm_kind;

typedef struct {
  int64_t T;          /* rows, 0 <= T <= 2^31 - 1 */
  int32_t H;          /* row length, 1 <= H <= 16384 (MOE_ERR_UNSUPPORTED above) */
  moe_norm_kind kind;
  float eps;          /* finite, >= 0 */
  moe_dtype dtype;    /* x, y, dy, dx: MOE_F32, MOE_BF16 or MOE_F16 */
} moe_norm_desc;

/* y = (x - mean) * rstd * gamma + beta per row of x[T, H], with
 *   mean = sum x / H (layer norm; 0 for RMS norm),
 *   rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),
 * computed in fp32 and rounded once to the type of y.  gamma, beta [H] fp32, each
 * NULL for none (1 and 0).  mean, rstd [T] fp32 receive the statistics for the
 * backward pass, or are NULL (mean has to be NULL for RMS norm).  y may be x. */
MOE_API moe_status moe_norm(const moe_norm_desc* d, const void* x, const float* gamma, const float* beta, void* y,
                            float* mean, float* rstd, moe_stream_t stream);

/* With xh = (x - mean) rstd and g = dy gamma:
 *   dx = rstd * (g - [layer norm: sum g / H] - xh * sum(g xh) / H)   per row
 *   dgamma = sum_t dy xh,  dbeta = sum_t dy                          fp32 [H]
 * x, dy, dx [T, H]; mean (NULL for RMS norm) and rstd from moe_norm.  dgamma and
 * dbeta may be NULL.  The sums over the rows run in a fixed order.  T = 0 writes
 * zeros to dgamma and dbeta.  dx may be dy or x.
 * Workspace: moe_norm_backward_workspace_size(d) bytes (0 for a bad descriptor). */
MOE_API size_t moe_norm_backward_workspace_size(const moe_norm_desc* d);
MOE_API moe_status moe_norm_backward(const moe_norm_desc* d, const void* dy, const void* x, const float* gamma,
                                     const float* mean, const float* rstd, void* dx, float* dgamma, float* dbeta,
                                     void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- linear */

typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_SILU = 2,      /* a * sigmoid(a) */
  MOE_ACT_GELU = 3,      /* a * (1 + erf(a / sqrt 2)) / 2 */
  MOE_ACT_GELU_TANH = 4  /* a * (1 + tanh(sqrt(2 / pi) (a + 0.044715 a^3))) / 2 */
} moe_act;

typedef struct {
  int64_t M;       /* rows of x, 0 <= M <= 2^31 - 1 */
  int32_t N;       /* rows of the weight: columns of y; a multiple of 8 */
  int32_t K;       /* columns of x and of the weight; a multiple of 8 */
  moe_act act;
  moe_dtype dtype; /* x, weight and, in the backward pass, all matrices: MOE_BF16 or MOE_F16 */
  moe_dtype y_out; /* y and the residual: equal to dtype, or MOE_F32 */
} moe_linear_desc;

/* y = act(x[M, K] . W[N, K]^T + bias) + residual, on the tensor cores with fp32
 * accumulation; bias, activation and residual are applied to the fp32
 * accumulator and y is rounded once.  (Activations by fast exponentials and
 * reciprocals: a relative error of at most 2^-19 + 2^-21 z, z the exponent's size: |a|,
 * a^2 / 2 or 2 sqrt(2 / pi) (|a| + 0.044715 |a|^3); sigmoids and exponentials below
 * 2^-126 count as 0.)
 * bias [N] fp32, residual [M, N] in the type
 * of y, each NULL for none; pre [M, N] in `dtype` receives x W^T + bias for the
 * backward pass, or is NULL.  y may be the residual.  N or K not a multiple of 8
 * is MOE_ERR_UNSUPPORTED, as is MOE_F32 for `dtype`.
 * Workspace: moe_linear_workspace_size(d) bytes (may be 0: ws may be NULL then). */
MOE_API size_t moe_linear_workspace_size(const moe_linear_desc* d);
MOE_API moe_status moe_linear(const moe_linear_desc* d, const void* x, const void* weight, const float* bias,
                              const void* residual, void* pre, void* y, void* ws, size_t ws_bytes,
                              moe_stream_t stream);

/* With dp = dy act'(pre) (pre from moe_linear; NULL for MOE_ACT_NONE):
 *   dx = dp . W [M, K],  dweight = dp^T . x [N, K],  dbias = sum_m dp [N] fp32
 * dp is rounded once to `dtype` as the products' operand, where there is an
 * activation (with it the gradients carry two roundings: about 1.4 times the error
 * that the rounding of dx and dweight alone leaves; and MOE_F16 loses dp below 2^-25, so
 * the loss has to be scaled, as it has for dy itself); dbias is summed from the
 * unrounded fp32 dp in a fixed order.  dx, dweight and dbias may each be NULL; dx
 * and dweight are in `dtype`, dy [M, N] in `dtype`.  relu'(0) = 0.  The residual's
 * gradient is dy itself.  M = 0 writes zeros to dweight and dbias.
 * Workspace: moe_linear_backward_workspace_size(d) bytes (0 for a bad descriptor). */
MOE_API size_t moe_linear_backward_workspace_size(const moe_linear_desc* d);
MOE_API moe_status moe_linear_backward(const moe_linear_desc* d, const void* dy, const void* pre, const void* x,
                                       const void* weight, void* dx, void* dweight, float* dbias, void* ws,
                                       size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- clipping */

typedef enum { MOE_CLIP_L2 = 0, MOE_CLIP_MAX = 1 } moe_clip_norm;

/* One gradient tensor: n elements of `dtype` at `in` (read) and `out` (written),
 * each aligned to its element size only; out may be in (clipping in place), and
 * must not overlap it otherwise, nor any other tensor's. */
typedef struct {
  const void* in;
  void* out;
  int64_t n;       /* >= 0; the pointers of an empty tensor are not looked at */
  moe_dtype dtype; /* MOE_F32, MOE_BF16 or MOE_F16, each tensor its own */
} moe_grad_tensor;

/* norm = sqrt(sum of g^2) or max |g| over all elements of all tensors (the host
 * array `list`, 0 <= count <= 65536), norm_out[0] = norm (fp32, device), and
 *   out = g * min(1, max_norm / (norm + 1e-6)),
 * the factor in fp32 and the product rounded once to each tensor's type.  max_norm:
 * finite, >= 0.  Squares are added up in a fixed order and so that neither large nor
 * small fp32 values overflow or vanish: the 4 or 8 of 16 bytes in fp32 where it holds
 * them, else in fp64, and these sums in fp64.  Where norm_out is not finite (a gradient
 * is inf or NaN, or the norm is beyond the largest fp32 number) nothing is scaled:
 * out = g.  `list` is read during the call only.
 * Workspace: moe_clip_grads_workspace_size(list, count) bytes (0 for a bad list). */
MOE_API size_t moe_clip_grads_workspace_size(const moe_grad_tensor* list, int32_t count);
MOE_API moe_status moe_clip_grads(const moe_grad_tensor* list, int32_t count, moe_clip_norm kind, float max_norm,
                                  float* norm_out, void* ws, size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_B200_OPS_H */
