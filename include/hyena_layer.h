/*
 * hyena_layer.h -- C ABI of the operators around the gated convolution of
 * hyena_conv.h in a sequence layer on MI355X (gfx950), in libhyena_layer.so:
 *
 *   hyena_scan_*    a gated linear recurrence along time (forward, backward,
 *                   one token),
 *   hyena_linear_*  a matrix product with bias, activation and residual in
 *                   its epilogue (forward, from one row up, and backward),
 *   hyena_conv_step, hyena_conv_cache_fill
 *                   the gated convolution for one token at a time.
 *
 * Status codes and element types are hyena_conv.h's.  As there: every pointer
 * is a DEVICE pointer owned by the caller; nothing is allocated or kept
 * between calls; work is enqueued on `stream` (a hipStream_t, NULL the
 * default stream) and the call returns without waiting; argument checks run
 * on the host before any HIP call; outputs and workspaces must not overlap
 * inputs or each other (HYENA_ERR_ALIAS) except where a buffer is said to be
 * updated in place.  A pointer to no elements may be NULL.  Calls that may run
 * at the same time need workspaces of their own.  Results are the same run to
 * run.  The launches are kernels only, so every call can be captured into a HIP
 * graph.
 *
 * Alignment: data pointers need the alignment of their elements (else
 * HYENA_ERR_ALIGN), and sizes and row strides are free.  Multiples of 16 bytes
 * are fastest.
 */
#ifndef HYENA_LAYER_H
#define HYENA_LAYER_H

#include <stdint.h>

#include "hyena_conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- gated linear recurrence ---------------------------------------------
 *
 *     a[b,t,d] = sigmoid(g[b,t,d])  or  exp(g[b,t,d])
 *     s[b,t,d] = a[b,t,d] s[b,t-1,d] + k[b,t,d] v[b,t,d],   s[b,-1,d] = s0[b,d] or 0
 *     y[b,t,d] = q[b,t,d] s[b,t,d]
 *
 * Where a is 0 (g = -inf: the first row of a packed document) the earlier
 * state is dropped whatever it holds, infinities and NaN included; a is also 0
 * for finite g below about -87, where it is below fp32's least normal number.
 *
 * q, k, v, g are [B, L, D] with D contiguous and one row stride `ld` >= D for
 * all four: row (b, t) of each starts (b L + t) ld elements after its pointer
 * (ld = D for separate tensors; 4 D for the column slices of one projection's
 * output).  y is [B, L, D] contiguous.  States are float32: s0, s_last [B, D],
 * `states` [B, ceil(L / 64), D] with s[b, 64 c - 1, :] in row c (row 0: s0 or
 * zero), what the backward wants of the forward.
 * Precision: gates, products, states and their sums are fp32 for both types;
 * y is rounded once. */
enum hyena_gate {
    HYENA_GATE_SIGMOID = 0, /* a = 1 / (1 + exp(-g)) */
    HYENA_GATE_LOG = 1      /* a = exp(g): a decay for g <= 0, growth above; exp(g), the
                               states and their gradients have to fit fp32 */
};

/* Forward.  s0 may be NULL (zero).  Any of y, s_last, states may be NULL (not
 * computed), not all three; q may be NULL where y is.  L = 0 writes s_last
 * only.  `workspace`: at least hyena_scan_workspace bytes, 16-byte aligned,
 * contents need not be initialised; overwritten. */
int hyena_scan_fwd(const void *q, const void *k, const void *v, const void *g,
                   int64_t B, int64_t L, int64_t D, int64_t ld, int gate,
                   const float *s0, void *y, float *s_last, float *states,
                   void *workspace, int64_t workspace_bytes, int dtype,
                   void *stream);

/* Backward for the upstream gradients dy ([B, L, D] contiguous) and ds_last
 * ([B, D] float32, of s_last; NULL is zero), from the forward's inputs and
 * `states`:
 *     ds_t = q_t dy_t + c_{t+1},   c_t = a_t ds_t  (c_L = ds_last),
 *     dq = dy s,  dk = ds v,  dv = ds k,  dg = ds s_{t-1} da/dg,  ds0 = c_0.
 * Where a is 0, c and dg are 0.  dq, dk, dv, dg share the row stride `ldd`
 * >= D (element type `dtype`); ds0 is float32 [B, D].  Any output may be NULL,
 * not all five.  workspace as for the forward. */
int hyena_scan_bwd(const void *q, const void *k, const void *v, const void *g,
                   const void *dy, const float *states, const float *ds_last,
                   int64_t B, int64_t L, int64_t D, int64_t ld, int64_t ldd,
                   int gate, void *dq, void *dk, void *dv, void *dg,
                   float *ds0, void *workspace, int64_t workspace_bytes,
                   int dtype, void *stream);

/* Bytes of workspace either direction needs (written to *bytes_out; may be
 * 0).  Host only. */
int hyena_scan_workspace(int64_t B, int64_t L, int64_t D, int dtype,
                         int64_t *bytes_out);

/* One token of B sequences: q, k, v, g are [B, D] with row stride `ld`, y is
 * [B, D] contiguous, `state` is float32 [S, D].  Sequence b's state is row
 * slots[b] (int32; NULL: row b, S >= B) and is replaced by the new one in
 * `state_out` (same layout; NULL or == state: in place; rows of no sequence
 * are not written).  A slot outside [0, S) marks an inactive entry: its y row
 * is zero and no state is read or written.  Active slots must differ. */
int hyena_scan_step(const void *q, const void *k, const void *v, const void *g,
                    int64_t B, int64_t D, int64_t ld, int gate, float *state,
                    float *state_out, int64_t S, const int32_t *slots, void *y,
                    int dtype, void *stream);

/* ---- the gated convolution, one token at a time ----------------------------
 *
 * `cache` is a pool of S rings of R >= l_h rows, [S, R, D] in `dtype`: row
 * t % R of ring slots[b] holds x_t = k_t v_t of sequence b's row t, rounded
 * once (as the convolution's forward rounds its matrix-core operand).
 * pos[b] (int64, device) is the number of rows sequence b has had before.
 *     y = q (h_0 x_pos + sum_{s=1}^{min(pos, l_h - 1)} h_s x_{pos-s})
 * and x_pos is written to its ring row; the caller advances pos.  q, k, v are
 * [B, D] with row stride ld; h is [D / group_size, l_h], l_h <= 128; y [B, D]
 * contiguous.  A slot outside [0, S) or pos < 0 marks an inactive entry: its
 * y row is zero and its ring is left alone.  slots NULL: ring b, S >= B.
 * Active slots must differ.  x_pos itself enters the sum in fp32.  A ring must
 * be below 2 GiB (else HYENA_ERR_UNSUPPORTED). */
int hyena_conv_step(const void *q, const void *k, const void *v, const void *h,
                    int64_t B, int64_t D, int64_t ld, int64_t group_size,
                    int64_t l_h, void *cache, int64_t S, int64_t R,
                    const int64_t *pos, const int32_t *slots, void *y,
                    int dtype, void *stream);

/* After a prompt of lens[b] rows (int64, device; NULL: L for all; clamped to
 * [0, L]) in k, v ([B, L, D], row stride ld): its last min(lens[b], R) rows of
 * x = k v into the rings.  pos[b] = lens[b] then continues with
 * hyena_conv_step.  Inactive slots as there. */
int hyena_conv_cache_fill(const void *k, const void *v, int64_t B, int64_t L,
                          int64_t D, int64_t ld, void *cache, int64_t S,
                          int64_t R, const int64_t *lens,
                          const int32_t *slots, int dtype, void *stream);

/* ---- matrix product with an epilogue ---------------------------------------
 *
 *     z = x w^T + bias,   y = act(z) + residual
 *
 * x [M, K] (row stride ldx >= K), w [N, K] contiguous, bias [N] or NULL,
 * residual [M, N] (row stride ldr) or NULL, y [M, N] (row stride ldy).
 * `preact`, if given, receives z ([M, N] contiguous, `dtype`), which the
 * backward of an activation wants.  Precision: bf16 products are summed in
 * fp32 on the matrix cores and z, the activation and the residual sum stay
 * fp32 until y (and preact) are rounded once; fp32 products and sums are fp32.
 * y may be the residual itself (same pointer and stride): it is then updated
 * in place. */
enum hyena_act {
    HYENA_ACT_NONE = 0,
    HYENA_ACT_RELU = 1,
    HYENA_ACT_GELU = 2,    /* z Phi(z), Phi the normal distribution function */
    HYENA_ACT_SILU = 3,    /* z / (1 + exp(-z)) */
    HYENA_ACT_SIGMOID = 4  /* 1 / (1 + exp(-z)) */
};

/* `workspace`: at least hyena_linear_workspace(..., backward = 0) bytes,
 * 16-byte aligned (NULL where that is 0). */
int hyena_linear_fwd(const void *x, const void *w, const void *bias,
                     const void *residual, int64_t M, int64_t N, int64_t K,
                     int64_t ldx, int64_t ldr, int64_t ldy, int act, void *y,
                     void *preact, void *workspace, int64_t workspace_bytes,
                     int dtype, void *stream);

/* Backward for dy ([M, N], row stride lddy; the residual's gradient is dy):
 *     dz = dy act'(z),  dx = dz w,  dw = dz^T x,  db = sum over rows of dz
 * with z = `preact` (NULL where act is HYENA_ACT_NONE).  dx [M, K] has row
 * stride lddx; dw [N, K] and db [N] are contiguous; all in `dtype`.  Any
 * output may be NULL, not all.  bf16: dz is rounded once to bf16 as matrix-core
 * operand (exact without an activation); db sums the unrounded dz; sums are
 * fp32, outputs rounded once.  x is only read for dw, w only for dx (NULL
 * allowed otherwise). */
int hyena_linear_bwd(const void *x, const void *w, const void *preact,
                     const void *dy, int64_t M, int64_t N, int64_t K,
                     int64_t ldx, int64_t lddy, int64_t lddx, int act,
                     void *dx, void *dw, void *db, void *workspace,
                     int64_t workspace_bytes, int dtype, void *stream);

/* Bytes of workspace the forward (backward = 0) or the backward with all its
 * outputs (backward = 1) needs.  Host only. */
int hyena_linear_workspace(int64_t M, int64_t N, int64_t K, int act, int dtype,
                           int backward, int64_t *bytes_out);

/* Static English text for a status code of this header's calls. */
const char *hyena_layer_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* HYENA_LAYER_H */
