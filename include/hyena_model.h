/*
 * hyena_model.h -- C ABI of the operators between the layers of a sequence
 * model and its weights on MI355X (gfx950), in libhyena_model.so:
 *
 *   hyena_norm_*   layer norm and root-mean-square norm over the channels of a
 *                  row (forward, from one row up, and backward),
 *   hyena_xent_*   the softmax cross entropy of a readout over a vocabulary,
 *                  without keeping the logits (forward and backward),
 *   hyena_grad_norm, hyena_adamw_step
 *                  the norm of all gradients and an AdamW step, each over a
 *                  list of tensors in a few launches.
 *
 * Status codes and element types are hyena_conv.h's; data, pointers, streams,
 * workspaces and errors are treated as hyena_layer.h says: DEVICE pointers
 * owned by the caller, no allocation, nothing kept between calls, argument
 * checks on the host before any HIP call, outputs and workspaces apart from
 * inputs and from each other (HYENA_ERR_ALIAS) except where updated in place,
 * pointers to no elements may be NULL, a workspace for each call that may run at
 * the same time, the same bits run to run, kernels only (every call can be
 * captured into a HIP graph).  Data pointers need the alignment of their
 * elements; multiples of 16 bytes in pointers and rows are fastest.
 */
#ifndef HYENA_MODEL_H
#define HYENA_MODEL_H

#include <stdint.h>

#include "hyena_conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- norm over a row's channels ----------------------------------------------
 *
 *     HYENA_NORM_LAYER:  mean = sum_d x_d / D,  var = sum_d (x_d - mean)^2 / D
 *     HYENA_NORM_RMS:    mean = 0,              var = sum_d x_d^2 / D
 *     rstd = 1 / sqrt(var + eps),   y_d = (x_d - mean) rstd w_d + b_d
 *
 * x [M, D] has row stride ldx >= D, y [M, D] row stride ldy; w and b [D] or NULL
 * (1 and 0); all in `dtype`.  mean and rstd [M] float32 are written where not
 * NULL (what the backward wants; mean is not used for the rms kind and may not
 * be given).  eps >= 0 and finite.  A row of equal values with eps = 0 has
 * rstd = inf.  Precision: fp32 throughout, deviations from the mean are summed
 * after the mean is known, y is rounded once. */
enum hyena_norm_kind { HYENA_NORM_LAYER = 0, HYENA_NORM_RMS = 1 };

int hyena_norm_fwd(const void *x, const void *w, const void *b, int64_t M,
                   int64_t D, int64_t ldx, int64_t ldy, int kind, float eps,
                   void *y, float *mean, float *rstd, int dtype, void *stream);

/* Backward for dy ([M, D], row stride lddy), with u = (x - mean) rstd, g = w dy:
 *     dx = rstd (g - [mean of g] - u mean(g u)),  dw = sum_m dy u,  db = sum_m dy
 * ([mean of g] only for the layer kind).  dx [M, D] has row stride lddx; dw and
 * db [D]; all in `dtype`.  Any output may be NULL, not all.  w NULL is 1; mean is
 * NULL for the rms kind.  `workspace`: at least hyena_norm_workspace bytes,
 * 16-byte aligned, overwritten.  Sums are fp32, outputs rounded once. */
int hyena_norm_bwd(const void *x, const void *w, const void *dy,
                   const float *mean, const float *rstd, int64_t M, int64_t D,
                   int64_t ldx, int64_t lddy, int64_t lddx, int kind, void *dx,
                   void *dw, void *db, void *workspace,
                   int64_t workspace_bytes, int dtype, void *stream);

/* Bytes of workspace the backward needs.  Host only. */
int hyena_norm_workspace(int64_t M, int64_t D, int dtype, int64_t *bytes_out);

/* ---- softmax cross entropy of a readout ----------------------------------------
 *
 *     z = x w^T + bias,   lse_i = log sum_v exp(z_iv),   loss_i = lse_i - z_i,target_i
 *
 * x [M, K] (row stride ldx >= K), w [V, K] contiguous, bias [V] or NULL, all in
 * `dtype`; target int64 [M]; loss and lse float32 [M].  A row whose target lies
 * outside [0, V) has none: its loss and lse are 0, its gradient is 0, it adds
 * nothing to dw and db whatever its x holds (NaN included), and costs nothing but
 * the reading of its target (in a forward of no more than 16 rows, what any row does:
 * the weights stream through whatever the targets are).  The logits are kept nowhere: the forward keeps a
 * maximum and a sum for every tile of columns, the backward forms dz in pieces of
 * the vocabulary in its workspace.  A logit of -inf (by bias) is an entry that
 * cannot occur.  Sizes: M and V up to 2^31 - 1024, K below 2^20, and M V and
 * M K + V K up to 2^42 in fp32 and 2^44 in bf16.  Precision: bf16 products are
 * summed in fp32, fp32 products and sums are fp32; logits, maxima, sums, lse and loss
 * stay fp32; an exp(y) is off by (|y| + 2) 2^-23 of itself.  loss is formed as
 * (max z - z_target) + log sum exp(z - max z), so that small ones keep their digits. */
int hyena_xent_fwd(const void *x, const void *w, const void *bias,
                   const int64_t *target, int64_t M, int64_t K, int64_t V,
                   int64_t ldx, float *loss, float *lse, void *workspace,
                   int64_t workspace_bytes, int dtype, void *stream);

/* Backward for dloss (float32 [M]) from the forward's lse:
 *     dz_iv = dloss_i (exp(z_iv - lse_i) - [v = target_i]),
 *     dx = dz w,  dw = dz^T x,  db = sum_i dz_i
 * dx [M, K] has row stride lddx; dw [V, K], db [V] contiguous; all in `dtype`.
 * Any output may be NULL, not all.  bf16: softmax - [target] (with dloss, or else x
 * with dloss, for dw) is rounded to bf16 as operand of the products, dloss being over
 * the largest |dloss|; db sums unrounded values; sums are fp32, outputs rounded once.
 * (In dw, a dloss below 2^-126 of the largest counts as 0.)  A row whose lse is not
 * finite has gradients of NaN.  Where the dloss of a row with a target is not finite, neither
 * is any element of dw and db (NaN for a NaN), nor that row of dx. */
int hyena_xent_bwd(const void *x, const void *w, const void *bias,
                   const int64_t *target, const float *lse, const float *dloss,
                   int64_t M, int64_t K, int64_t V, int64_t ldx, int64_t lddx,
                   void *dx, void *dw, void *db, void *workspace,
                   int64_t workspace_bytes, int dtype, void *stream);

/* Bytes of workspace (16-byte aligned, overwritten) the forward (backward = 0)
 * or the backward with all its outputs (backward = 1) needs.  Host only. */
int hyena_xent_workspace(int64_t M, int64_t K, int64_t V, int dtype,
                         int backward, int64_t *bytes_out);

/* ---- AdamW over many tensors -----------------------------------------------------
 *
 * `tensors` is an array of n descriptors in HOST memory, read before the call
 * returns.  Tensors are contiguous, of any sizes (0 among them) below 2^40
 * elements; param and grad are `dtype`.  Nothing that a step writes may overlap
 * anything else of it (HYENA_ERR_ALIAS), in one tensor or between two. */
typedef struct hyena_tensor {
    void *param;           /* [numel] */
    const void *grad;      /* [numel] */
    void *exp_avg;         /* [numel]: m, float32 or e4m3 codes */
    void *exp_avg_sq;      /* [numel]: v in float32, or sqrt(v) in e4m3 codes */
    float *exp_avg_scale;  /* 8 bits: [ceil(numel / 256)], else not used */
    float *exp_avg_sq_scale;
    float *master;         /* [numel] or NULL: the fp32 value of which param is the rounding */
    int64_t numel;
} hyena_tensor;

/* With g = grad_scale grad (grad_scale: float32, one element on the device, or
 * NULL: 1), t = step >= 1:
 *     m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * p is master where there is one (param gets its rounding), else param itself;
 * in bf16 without a master a move below half a unit in param's last place is
 * lost.  Where lr_dev (float32), step_dev or seed_dev (int64) is given, one element
 * on the device, it takes lr's, step's or seed's place, so that a captured step can
 * be replayed with others (a *step_dev below 1 counts as 1).  If *grad_scale is
 * not finite, nothing is written: the step is skipped.  All in fp32, param rounded
 * once.
 *
 * state_bits 32: m and v are float32.  state_bits 8: m and r = sqrt(v) are held
 * as codes c of 8 bits (OCP e4m3: 3 bits of mantissa, up to 448) with a scale s
 * for every 256 elements, m = c s and v = (c s)^2; p takes the new m and v before
 * they are rounded.  s becomes the largest magnitude / 448 (a block whose largest
 * is below 2^-117 counts as zeros), and x / s is rounded to one of the two codes around
 * it at random, up with the probability of its place between them, so that
 * moments keep changing where a step moves them by less than half a code: with the same
 * seed in every step an element would be rounded by the same bits each time, and those with low
 * ones never up, so that the seed has to differ from step to step.  (r and
 * not v, since e4m3 spans 2^18 from its least to its largest.)  The random bits
 * are a function of seed (its low 32 bits), of the tensor's place k in the list
 * and of the element's index i: with mix the last steps of murmur3,
 *     h = mix(low(i) ^ mix(seed + 0x9E3779B9 k + high(i))),   in 32 bits,
 * the low 16 bits of h / 65536 for m, the high ones for r; up where the place
 * plus that reaches 1. */
int hyena_adamw_step(const hyena_tensor *tensors, int64_t n, double lr,
                     double beta1, double beta2, double eps,
                     double weight_decay, int64_t step, int64_t seed,
                     const float *lr_dev, const int64_t *step_dev,
                     const int64_t *seed_dev, const float *grad_scale,
                     int state_bits, int dtype, void *stream);

/* norm[0] = sqrt(sum of grad^2 over all tensors) (only grad and numel are
 * read), and, where scale is not NULL, scale[0] = min(1, max_norm / norm) (1
 * where norm is 0; NaN where norm is infinite or NaN, which skips the step); max_norm
 * is at least 0 and may be infinite.
 * Squares are summed in 64 bits.  `workspace`: at least
 * hyena_grad_norm_workspace bytes for tensors of `numel` elements together. */
int hyena_grad_norm(const hyena_tensor *tensors, int64_t n, double max_norm,
                    float *norm, float *scale, void *workspace,
                    int64_t workspace_bytes, int dtype, void *stream);

int hyena_grad_norm_workspace(int64_t n, int64_t numel, int64_t *bytes_out);

/* Static English text for a status code of this header's calls. */
const char *hyena_model_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* HYENA_MODEL_H */
