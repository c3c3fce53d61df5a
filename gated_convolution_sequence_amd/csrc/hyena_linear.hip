// Matrix product with bias, activation and residual in its epilogue, and its
// backward, for MI355X (gfx950) (hyena_layer.h has the formulas and layouts).
//
// Every product is C[m, n] = sum_c A[m, c] B[n, c] with free strides, in
// 16 x 16 tiles: one thread per output element, operands staged through LDS.

#include "layer_common.h"

namespace layer {
namespace {

__device__ inline float act_value(int act, float z) {
    switch (act) {
    case HYENA_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case HYENA_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case HYENA_ACT_SILU: return z / (1.0f + __expf(-z));
    case HYENA_ACT_SIGMOID: return decay<false>(z);
    default: return z;
    }
}

__device__ inline float act_slope(int act, float z) {
    switch (act) {
    case HYENA_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case HYENA_ACT_GELU:
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * __expf(-0.5f * z * z) * 0.39894228040143268f;
    case HYENA_ACT_SILU: {
        float slope;
        const float p = decay<false>(z, slope);
        return p + z * slope;
    }
    case HYENA_ACT_SIGMOID: {
        float slope;
        decay<false>(z, slope);
        return slope;
    }
    default: return 1.0f;
    }
}

struct GemmParams {
    const void *a, *b;                // C[m, n] = sum_c a[m sam + c sac] b[n sbn + c sbc]
    int64_t M, N, C, sam, sac, sbn, sbc;
    const void *az;                   // a is multiplied by act'(az) (same strides as a over [M, N] of z), or null
    int64_t szm, szc;
    const void *bias, *residual;
    int64_t ldr, ldy;
    void *y, *preact;
    int act;                          // epilogue activation
    int act_a;                        // activation whose slope multiplies a
};

template <bool F32>
__global__ __launch_bounds__(256) void gemm_kernel(GemmParams p) {
    __shared__ float ta[16][17], tb[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t tiles_n = ceil_div(p.N, 16);
    const int64_t m0 = (blockIdx.x / tiles_n) * 16, n0 = (blockIdx.x % tiles_n) * 16;
    float acc = 0.0f;
    for (int64_t c0 = 0; c0 < p.C; c0 += 16) {
        const int64_t m = m0 + ty, n = n0 + ty, c = c0 + tx;
        float a = 0.0f, b = 0.0f;
        if (m < p.M && c < p.C) {
            a = load1<F32>(p.a, m * p.sam + c * p.sac);
            if (p.az) {
                a *= act_slope(p.act_a, load1<F32>(p.az, m * p.szm + c * p.szc));
                if constexpr (!F32) a = (float)(bf16_t)a;
            }
        }
        if (n < p.N && c < p.C) b = load1<F32>(p.b, n * p.sbn + c * p.sbc);
        ta[ty][tx] = a, tb[ty][tx] = b;
        __syncthreads();
        for (int i = 0; i < 16; ++i) acc += ta[ty][i] * tb[tx][i];
        __syncthreads();
    }
    const int64_t m = m0 + ty, n = n0 + tx;
    if (m >= p.M || n >= p.N) return;
    if (p.bias) acc += load1<F32>(p.bias, n);
    if (p.preact) store1<F32>(p.preact, m * p.N + n, acc);
    acc = act_value(p.act, acc);
    if (p.residual) acc += load1<F32>(p.residual, m * p.ldr + n);
    store1<F32>(p.y, m * p.ldy + n, acc);
}

// db[n] = sum over rows of dy act'(z): one wave per column.
template <bool F32>
__global__ __launch_bounds__(64) void bias_grad_kernel(const void *dy, const void *z, int64_t M, int64_t N,
                                                       int64_t lddy, int act, void *db) {
    const int64_t n = blockIdx.x;
    float sum = 0.0f;
    for (int64_t m = threadIdx.x; m < M; m += 64) {
        const float d = load1<F32>(dy, m * lddy + n);
        sum += z ? d * act_slope(act, load1<F32>(z, m * N + n)) : d;
    }
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (threadIdx.x == 0) store1<F32>(db, n, sum);
}

int gemm(const GemmParams &p, bool f32, hipStream_t stream) {
    if (p.M == 0 || p.N == 0) return HYENA_OK;
    const int64_t blocks = ceil_div(p.M, 16) * ceil_div(p.N, 16);
    if (blocks > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(f32 ? gemm_kernel<true> : gemm_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return launch_status();
}

int check_linear(int64_t M, int64_t N, int64_t K, int act, int dtype) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    if (act < HYENA_ACT_NONE || act > HYENA_ACT_SIGMOID) return HYENA_ERR_UNSUPPORTED;
    int64_t n;
    if (!mul_fits(M, N, 4, &n) || !mul_fits(M, K, 4, &n) || !mul_fits(N, K, 4, &n)) return HYENA_ERR_SHAPE;
    const int64_t most = (int64_t)1 << 31;
    if (M >= most || N >= most || K >= most) return HYENA_ERR_SHAPE;
    return HYENA_OK;
}

}  // namespace
}  // namespace layer

using namespace layer;

extern "C" {

int hyena_linear_workspace(int64_t M, int64_t N, int64_t K, int act, int dtype, int backward, int64_t *bytes_out) {
    const int st = check_linear(M, N, K, act, dtype);
    if (st != HYENA_OK) return st;
    if (!bytes_out) return HYENA_ERR_NULL;
    (void)backward;
    *bytes_out = 0;
    return HYENA_OK;
}

int hyena_linear_fwd(const void *x, const void *w, const void *bias, const void *residual, int64_t M, int64_t N,
                     int64_t K, int64_t ldx, int64_t ldr, int64_t ldy, int act, void *y, void *preact,
                     void *workspace, int64_t workspace_bytes, int dtype, void *stream) {
    const int st = check_linear(M, N, K, act, dtype);
    if (st != HYENA_OK) return st;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (ldx < K || ldy < N || (residual && ldr < N) || !mul_fits(M, ldx, eb, &n) || !mul_fits(M, ldy, eb, &n) ||
        (residual && !mul_fits(M, ldr, eb, &n)))
        return HYENA_ERR_SHAPE;
    if (M == 0 || N == 0) return HYENA_OK;
    if (!y || (K > 0 && (!x || !w))) return HYENA_ERR_NULL;
    if (!aligned(x, eb) || !aligned(w, eb) || !aligned(bias, eb) || !aligned(residual, eb) || !aligned(y, eb) ||
        !aligned(preact, eb) || !aligned(workspace, 16))
        return HYENA_ERR_ALIGN;
    int64_t need = 0;
    hyena_linear_workspace(M, N, K, act, dtype, 0, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const Rows rr = {residual, M, N * eb, ldr * eb}, ry = {y, M, N * eb, ldy * eb}, rp = {preact, M, N * eb, N * eb};
    const Rows rw = {need > 0 ? workspace : nullptr, 1, need, need};
    const Rows in[3] = {{x, M, K * eb, ldx * eb}, {w, N, K * eb, K * eb}, {bias, 1, N * eb, N * eb}};
    for (const Rows &r : in)
        if (overlap(ry, r) || overlap(rp, r) || overlap(rw, r)) return HYENA_ERR_ALIAS;
    if ((overlap(ry, rr) && !same_range(ry, rr)) || overlap(rp, rr) || overlap(rw, rr) || overlap(ry, rp) ||
        overlap(rw, ry) || overlap(rw, rp))
        return HYENA_ERR_ALIAS;
    GemmParams p = {};
    p.a = x, p.b = w, p.M = M, p.N = N, p.C = K;
    p.sam = ldx, p.sac = 1, p.sbn = K, p.sbc = 1;
    p.bias = bias, p.residual = residual, p.ldr = ldr, p.ldy = ldy, p.y = y, p.preact = preact, p.act = act;
    return gemm(p, dtype == HYENA_DTYPE_F32, (hipStream_t)stream);
}

int hyena_linear_bwd(const void *x, const void *w, const void *preact, const void *dy, int64_t M, int64_t N,
                     int64_t K, int64_t ldx, int64_t lddy, int64_t lddx, int act, void *dx, void *dw, void *db,
                     void *workspace, int64_t workspace_bytes, int dtype, void *stream) {
    int st = check_linear(M, N, K, act, dtype);
    if (st != HYENA_OK) return st;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (lddy < N || (dw && ldx < K) || (dx && lddx < K) || !mul_fits(M, lddy, eb, &n) ||
        (dw && !mul_fits(M, ldx, eb, &n)) || (dx && !mul_fits(M, lddx, eb, &n)))
        return HYENA_ERR_SHAPE;
    if (!dx && !dw && !db) return HYENA_ERR_NULL;
    const bool rows = M > 0 && N > 0;
    if (rows && (!dy || (act != HYENA_ACT_NONE && !preact) || (dx && K > 0 && !w) || (dw && K > 0 && !x)))
        return HYENA_ERR_NULL;
    if (!aligned(x, eb) || !aligned(w, eb) || !aligned(preact, eb) || !aligned(dy, eb) || !aligned(dx, eb) ||
        !aligned(dw, eb) || !aligned(db, eb) || !aligned(workspace, 16))
        return HYENA_ERR_ALIGN;
    int64_t need = 0;
    hyena_linear_workspace(M, N, K, act, dtype, 1, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const Rows in[4] = {{dw ? x : nullptr, M, K * eb, ldx * eb}, {dx ? w : nullptr, N, K * eb, K * eb},
                        {act != HYENA_ACT_NONE ? preact : nullptr, M, N * eb, N * eb}, {dy, M, N * eb, lddy * eb}};
    const Rows out[4] = {{dx, M, K * eb, lddx * eb}, {dw, N, K * eb, K * eb}, {db, 1, N * eb, N * eb},
                         {need > 0 ? workspace : nullptr, 1, need, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Rows &r : in)
            if (overlap(out[i], r)) return HYENA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HYENA_ERR_ALIAS;
    }
    const bool f32 = dtype == HYENA_DTYPE_F32;
    hipStream_t s = (hipStream_t)stream;
    const void *z = act != HYENA_ACT_NONE ? preact : nullptr;
    if (dx) {
        GemmParams p = {};
        p.a = dy, p.b = w, p.M = M, p.N = K, p.C = N;
        p.sam = lddy, p.sac = 1, p.sbn = 1, p.sbc = K;
        p.az = z, p.szm = N, p.szc = 1, p.act_a = act, p.y = dx, p.ldy = lddx;
        if ((st = gemm(p, f32, s)) != HYENA_OK) return st;
    }
    if (dw) {
        GemmParams p = {};
        p.a = dy, p.b = x, p.M = N, p.N = K, p.C = M;
        p.sam = 1, p.sac = lddy, p.sbn = 1, p.sbc = ldx;
        p.az = z, p.szm = 1, p.szc = N, p.act_a = act, p.y = dw, p.ldy = K;
        if ((st = gemm(p, f32, s)) != HYENA_OK) return st;
    }
    if (db && N > 0) {
        hipLaunchKernelGGL(f32 ? bias_grad_kernel<true> : bias_grad_kernel<false>, dim3((unsigned)N), dim3(64), 0, s,
                           dy, z, M, N, lddy, act, db);
        st = launch_status();
    }
    return st;
}

}  // extern "C"
