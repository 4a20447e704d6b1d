/*
 * zc_ops.h -- C ABI of libzc_ops: the operators of a training step around the
 * codec of zc.h, which make the buffers it compresses and use the buffers it
 * decodes.
 *   MoE all-to-all (pith.science, Figure 2): zc_route picks each token's
 *   experts, zc_expert_slots lays the (token, choice) pairs out as
 *   per-expert chunks and gives their counts on the device (the d_counts of
 *   zc_compress_dev), zc_dispatch moves the token rows there, zc_combine
 *   joins the experts' rows again; zc_route_grad and zc_combine_grad are
 *   their gradients (the gradient of zc_dispatch is zc_combine without
 *   weights).
 *   Reduce-scatter and all-gather (Figure 3): zc_grad_norm and zc_adamw take
 *   the summed gradients (zc_decompress_reduce) to the new parameters (the
 *   d_in of zc_compress).
 * Every sum, softmax statistic, norm and optimizer value is held in fp32 or
 * fp64; a result of fewer bits is rounded from that once, to nearest with ties
 * to even.  Every result has one order of additions: the same inputs give the
 * same bits.
 *
 * Status codes are zc.h's.  All calls are thread-safe and keep no state between
 * calls; the library allocates no memory.  Calls are asynchronous on the given
 * stream (a hipStream_t; NULL is the null stream) of the current device, only
 * launch kernels, and can be captured into a HIP graph: what is passed by value
 * (a step's number and rates among it) is replayed as captured.
 */
#ifndef ZC_OPS_H
#define ZC_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "zc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define ZC_BF16 0
#define ZC_F16 1
#define ZC_F32 2
#define ZC_E4M3 3            /* 8-bit float, 4 exponent and 3 mantissa bits,
                                no infinities (AdamW states only)           */

#define ZC_MAX_EXPERTS 1024
#define ZC_MAX_TOPK 32
#define ZC_MAX_ROW_VALUES (1 << 28)

#define ZC_SCORE_SOFTMAX 0
#define ZC_SCORE_SIGMOID 1
#define ZC_GROUP_MAX 0
#define ZC_GROUP_TOP2 1

typedef struct {
    int32_t experts;     /* E, 1 .. ZC_MAX_EXPERTS                          */
    int32_t k;           /* choices per token, 1 .. ZC_MAX_TOPK, <= E       */
    int32_t score;       /* ZC_SCORE_*                                      */
    int32_t groups;      /* G, divides E; 1 .. 64                           */
    int32_t top_groups;  /* 1 .. G, with k <= top_groups E / G              */
    int32_t group_score; /* ZC_GROUP_*                                      */
    int32_t renorm;      /* 1: the k weights are divided by their sum       */
    float scale;         /* factor on the weights                           */
} zc_router;

/*
 * Expert choice of every token.  With s_e = exp(x_e - max x) / sum exp(x -
 * max x) or 1 / (1 + exp(-x_e)) over a token's E logits x, and key_e = s_e +
 * bias_e:
 *   - with G > 1 groups of E / G neighbouring experts, a group's score is its
 *     largest key (ZC_GROUP_MAX) or the fp32 sum of its two largest
 *     (ZC_GROUP_TOP2), and only the top_groups best groups take part;
 *   - the k experts of the largest keys are chosen, in that order; equal keys
 *     (and groups of equal score) go to the lowest index;
 *   - their weights are scale s_e, or scale s_e / (sum of the k chosen s) with
 *     renorm.  With softmax that is the softmax over the chosen logits alone,
 *     and is computed so: it does not vanish where a bias chooses experts
 *     whose s does.  With sigmoid the weights are 0 where the fp32 sum is 0
 *     (all chosen logits below -88).  The bias is for balance: it takes part
 *     in the choice alone.
 * An expert with logit -inf or bias -inf is never chosen and counts for no
 * group; a choice for which no expert is left has expert -1 and weight 0.  A
 * NaN key ranks below every number.  A NaN or +inf logit makes a softmax
 * token's weights NaN.  The exponentials are summed in fp64 and the sum is
 * rounded to fp32: two orders of additions give the same sum, and with it the
 * same choice, but for the rare one that lies within fp64's rounding of the
 * middle of two fp32 numbers.
 *   d_logits     device, dtype ZC_BF16 / ZC_F16 / ZC_F32, aligned to it;
 *                token t's logits start at element t row_stride, row_stride
 *                >= 0
 *   tokens       >= 0
 *   d_bias       device fp32[E], or NULL
 *   d_valid      device uint8[tokens], or NULL: a token with 0 gets experts
 *                -1 and weights 0
 *   d_experts    device int32[tokens][k], written
 *   d_weights    device fp32[tokens][k], written
 * No workspace.  Returns ZC_OK once queued, ZC_EINVAL or ZC_EHIP.
 */
int zc_route(const void* d_logits, int32_t dtype, int64_t tokens,
             int64_t row_stride, const zc_router* router, const float* d_bias,
             const uint8_t* d_valid, int32_t* d_experts, float* d_weights,
             void* stream);

/*
 * Gradient of zc_route's weights with respect to the logits, the choice
 * itself held fixed (it has no gradient, nor has the bias).  With g =
 * d_weights_grad and S the sum of the chosen scores,
 *   ds_j = scale g_j, or with renorm scale (g_j - sum_i g_i s_i / S) / S (0
 *   where zc_route's weights are 0 because S is);
 *   sigmoid: dx_e = s_e (1 - s_e) ds_e;  softmax: dx_e = s_e (ds_e - sum_i
 *   ds_i s_i), over all E.
 *   router          as for zc_route; the group fields and k <= top_groups E /
 *                   G are not used (the choice is given)
 *   d_experts       device int32[tokens][k], a token's entries distinct;
 *                   entries outside 0 .. E - 1 take no part; a token without
 *                   any other has a gradient of zeros, whatever its logits
 *   d_weights_grad  device fp32[tokens][k]
 *   d_logits_grad   device, dtype, [tokens][E] without gaps, every entry
 *                   written
 */
int zc_route_grad(const void* d_logits, int32_t dtype, int64_t tokens,
                  int64_t row_stride, const zc_router* router,
                  const int32_t* d_experts, const float* d_weights_grad,
                  void* d_logits_grad, void* stream);

/*
 * Slots of the (token, choice) pairs in a buffer of per-expert chunks.  The
 * pairs are ordered by expert, and by index within one (a stable counting
 * sort); pair i's row is its place in that order.  Pairs whose expert is
 * outside 0 .. E - 1 come last.
 *   d_experts  device int32[pairs]; pair i is choice i % k of token i / k
 *   experts    E, 1 .. ZC_MAX_EXPERTS
 *   row_values values per row, the unit of d_counts, 0 ..
 *              ZC_MAX_CHUNK_VALUES
 *   d_slots    device int32[pairs], written: the row, or ~row (a negative
 *              number) for a pair without an expert
 *   d_counts   device int64[E + 1], 8-byte aligned, written: row_values times
 *              the rows of each expert, then of the pairs without one; sums
 *              to pairs row_values
 *   d_ws       device workspace, 4-byte aligned, ws_bytes >=
 *              zc_slots_workspace_bytes(pairs, experts); need not be cleared
 * Returns ZC_OK once queued, ZC_EINVAL (pairs outside 0 .. 2^31 - 1),
 * ZC_ENOSPC or ZC_EHIP.
 */
size_t zc_slots_workspace_bytes(int64_t pairs, int32_t experts);
int zc_expert_slots(const int32_t* d_experts, int64_t pairs, int32_t experts,
                    int64_t row_values, int32_t* d_slots, int64_t* d_counts,
                    void* d_ws, size_t ws_bytes, void* stream);

/*
 * Token rows to their slots: row d_slots[t k + j] of d_rows is token t's
 * row; the rows of pairs without an expert (slot ~row) are zeros.  Slots
 * outside the tokens k rows are ignored, and a row that no slot names is left
 * as it was; no row may be named twice (zc_expert_slots names each once).
 *   d_x      device, dtype, aligned to it; token t's row starts at element
 *            t row_stride, row_stride >= 0 (0 repeats one row)
 *   row_values  0 .. ZC_MAX_ROW_VALUES
 *   d_slots  device int32[tokens][k], k in 1 .. ZC_MAX_TOPK, tokens k < 2^31
 *   d_rows   device, dtype, [tokens k][row_values], written
 */
int zc_dispatch(const void* d_x, int32_t dtype, int64_t tokens,
                int64_t row_values, int64_t row_stride, const int32_t* d_slots,
                int32_t k, void* d_rows, void* stream);

/*
 * Weighted sum of each token's rows, in fp32 in the order of the choices:
 *   d_out[t] = base[t] + sum_j w[t][j] d_rows[slot[t][j]]
 * Pairs without an expert (negative slots), and slots outside the tokens k
 * rows, add nothing.
 *   d_weights  device fp32[tokens][k], or NULL for weights of one
 *   d_base     device, dtype, row t at element t base_stride, or NULL for 0
 *   d_out      device, dtype, [tokens][row_values], written; may be d_base
 *              itself where base_stride is row_values
 *   other arguments as for zc_dispatch
 */
int zc_combine(const void* d_rows, int32_t dtype, int64_t tokens,
               int64_t row_values, const int32_t* d_slots, int32_t k,
               const float* d_weights, const void* d_base, int64_t base_stride,
               void* d_out, void* stream);

/*
 * Gradients of zc_combine with weights (its base's gradient is d_out_grad
 * itself):
 *   d_rows_grad[slot[t][j]] = w[t][j] d_out_grad[t]
 *   d_weights_grad[t][j]    = <d_out_grad[t], d_rows[slot[t][j]]> in fp32
 * The rows of pairs without an expert (slot ~row) get zeros, their weights'
 * gradients 0.  Slots outside the tokens k rows are ignored (gradient 0), and
 * a row of d_rows_grad that no slot names is left as it was.
 *   d_out_grad  device, dtype, row t at element t row_stride
 */
int zc_combine_grad(const void* d_out_grad, int32_t dtype, int64_t tokens,
                    int64_t row_values, int64_t row_stride, const void* d_rows,
                    const int32_t* d_slots, int32_t k, const float* d_weights,
                    void* d_rows_grad, float* d_weights_grad, void* stream);

/* One tensor of a list: n values at data (device, aligned to their type). */
typedef struct {
    const void* data;
    int64_t n;
} zc_tensor;

/*
 * Norm of all values of a list of gradients, and the factor that clips it:
 *   d_norm[0] = sqrt(sum of squares), summed in fp64
 *   d_norm[1] = min(1, max_norm / (d_norm[0] + 1e-6)), or 1 where max_norm is
 *               not positive; NaN where d_norm[0] is not finite, which makes
 *               zc_adamw skip the step
 *   tensors  host array; dtype ZC_BF16 or ZC_F32 for all of them, together
 *            below 2^24 pieces of 32 KB (a tensor's last may be shorter)
 *   d_norm   device fp32[2], written
 *   d_ws     device workspace, 8-byte aligned, ws_bytes >=
 *            zc_grad_norm_workspace_bytes(...) (0 for a short list, then it
 *            may be NULL); need not be cleared
 * Returns ZC_OK once queued, ZC_EINVAL, ZC_ENOSPC or ZC_EHIP.
 */
size_t zc_grad_norm_workspace_bytes(const zc_tensor* tensors, int32_t count,
                                    int32_t dtype);
int zc_grad_norm(const zc_tensor* tensors, int32_t count, int32_t dtype,
                 float max_norm, float* d_norm, void* d_ws, size_t ws_bytes,
                 void* stream);

/* Values per scale of the 8-bit AdamW states. */
#define ZC_STATE_BLOCK 256

/* One tensor of an AdamW step; all pointers are device pointers. */
typedef struct {
    void* param;         /* n parameters, param_dtype; updated              */
    float* master;       /* fp32 parameters that param is rounded from, or
                            NULL (all tensors of a call alike)              */
    const void* grad;    /* n gradients, grad_dtype                         */
    void* avg;           /* first state, n values of state_dtype; updated   */
    void* sq;            /* second state                                    */
    float* avg_scale;    /* fp32[ceil(n / 256)] scales of 8-bit states,     */
    float* sq_scale;     /* else unused                                     */
    int64_t n;
} zc_adamw_tensor;

typedef struct {
    int32_t param_dtype; /* ZC_BF16 or ZC_F32 (master only with ZC_BF16)    */
    int32_t grad_dtype;  /* ZC_BF16 or ZC_F32                               */
    int32_t state_dtype; /* ZC_F32 or ZC_E4M3                               */
    int32_t pad;         /* 0                                               */
    int64_t step;        /* number of this step, from 1                     */
    double lr, beta1, beta2, eps, weight_decay;
} zc_adamw_config;

/*
 * One AdamW step with decoupled weight decay over a list of tensors.  With
 * g = grad times *d_grad_scale, in fp32:
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * p is master where there is one (param is then its rounding), else param.
 * With ZC_F32 states, avg holds m and sq holds v.  With ZC_E4M3, avg holds m
 * and sq holds sqrt(v), each as e4m3 values times the scale of their block of
 * 256 (the last of a tensor may be shorter): scale = largest |x| / 448, and
 * a positive sqrt(v) is stored as at least 2^-9 of its scale, so that no
 * denominator vanishes below its step; a block whose largest is below 1e-30
 * is stored as zeros.  The step itself uses m and v before they are rounded.
 * A NaN stays in its own value; an infinity leaves no finite value in its
 * block.
 * Every operation is rounded to fp32 in the order of the formulas, with the
 * factors 1 - beta, 1 - lr weight_decay, lr / (1 - beta1^step) and
 * 1 / sqrt(1 - beta2^step) made in fp64.  One step is rounded otherwise, that
 * of a parameter kept in ZC_BF16 alone beside ZC_E4M3 states: m times the
 * denominator's reciprocal to 1 unit in the last place, in fused
 * multiplications and additions, within 4 units in fp32's last place before
 * the parameter is rounded to bf16.  (No state follows from it.)
 *   tensors       host array of count entries, n >= 0, together below 2^24
 *                 pieces of 2048 values (a tensor's last may be shorter)
 *   d_grad_scale  device fp32, or NULL for 1: a factor on every gradient, for
 *                 example d_norm + 1 of zc_grad_norm.  If it is not finite,
 *                 the step changes nothing.
 * Returns ZC_OK once queued, ZC_EINVAL or ZC_EHIP.
 */
int zc_adamw(const zc_adamw_tensor* tensors, int32_t count,
             const zc_adamw_config* config, const float* d_grad_scale,
             void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ZC_OPS_H */
