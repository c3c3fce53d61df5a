// Gated linear recurrence along time for MI355X (gfx950):
//     s_t = a_t s_{t-1} + k_t v_t,   y_t = q_t s_t,   a = sigmoid(g) or exp(g),
// and its backward (hyena_layer.h has the formulas and layouts).
//
// One lane walks one channel of one batch row through time.

#include "layer_common.h"

namespace layer {
namespace {

struct ScanParams {
    const void *q, *k, *v, *g, *dy;
    const float *s0, *ds_last, *states_in;
    void *y, *dq, *dk, *dv, *dg;
    float *s_last, *states, *ds0;
    int64_t B, L, D, ld, ldd;
};

template <bool F32, bool LOG>
__global__ __launch_bounds__(64) void scan_fwd_kernel(ScanParams p) {
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i % p.D;
    const int64_t chunks = ceil_div(p.L, kStateRows);
    float s = p.s0 ? p.s0[i] : 0.0f;
    for (int64_t t = 0; t < p.L; ++t) {
        const int64_t e = (b * p.L + t) * p.ld + d;
        if (p.states && t % kStateRows == 0) p.states[(b * chunks + t / kStateRows) * p.D + d] = s;
        const float a = decay<LOG>(load1<F32>(p.g, e));
        s = (a == 0.0f ? 0.0f : a * s) + load1<F32>(p.k, e) * load1<F32>(p.v, e);
        if (p.y) store1<F32>(p.y, (b * p.L + t) * p.D + d, load1<F32>(p.q, e) * s);
    }
    if (p.s_last) p.s_last[i] = s;
}

template <bool F32, bool LOG>
__global__ __launch_bounds__(64) void scan_bwd_kernel(ScanParams p) {
    __shared__ float sm[kStateRows][64];
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i % p.D;
    const int64_t chunks = ceil_div(p.L, kStateRows);
    float c = p.ds_last ? p.ds_last[i] : 0.0f;
    for (int64_t n = chunks - 1; n >= 0; --n) {
        float s = p.states_in[(b * chunks + n) * p.D + d];
        const int rows = (int)min((int64_t)kStateRows, p.L - n * kStateRows);
        for (int r = 0; r < rows; ++r) {
            sm[r][threadIdx.x] = s;  // the state before row r
            const int64_t e = (b * p.L + n * kStateRows + r) * p.ld + d;
            const float a = decay<LOG>(load1<F32>(p.g, e));
            s = (a == 0.0f ? 0.0f : a * s) + load1<F32>(p.k, e) * load1<F32>(p.v, e);
        }
        for (int r = rows - 1; r >= 0; --r) {
            const int64_t row = b * p.L + n * kStateRows + r, e = row * p.ld + d, o = row * p.ldd + d;
            const float dy = load1<F32>(p.dy, row * p.D + d);
            float slope;
            const float a = decay<LOG>(load1<F32>(p.g, e), slope);
            const float prev = sm[r][threadIdx.x];
            const float ds = load1<F32>(p.q, e) * dy + c;
            if (p.dq) store1<F32>(p.dq, o, dy * s);
            if (p.dk) store1<F32>(p.dk, o, ds * load1<F32>(p.v, e));
            if (p.dv) store1<F32>(p.dv, o, ds * load1<F32>(p.k, e));
            if (p.dg) store1<F32>(p.dg, o, a == 0.0f ? 0.0f : ds * prev * slope);
            c = a == 0.0f ? 0.0f : a * ds;
            s = prev;
        }
    }
    if (p.ds0) p.ds0[i] = c;
}

int check_sizes(int64_t B, int64_t L, int64_t D, int gate, int dtype) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    if (gate != HYENA_GATE_SIGMOID && gate != HYENA_GATE_LOG) return HYENA_ERR_UNSUPPORTED;
    int64_t n;
    if (B < 0 || L < 0 || D < 0) return HYENA_ERR_SHAPE;
    if (!mul_fits(B, L, 1, &n) || !mul_fits(n, D, 4, &n) || !mul_fits(B, D, 4, &n)) return HYENA_ERR_SHAPE;
    if (L > (int64_t)1 << 40 || D > (int64_t)1 << 30 || B > (int64_t)1 << 30) return HYENA_ERR_SHAPE;
    return HYENA_OK;
}

template <typename K> int launch(K kernel, const ScanParams &p, void *stream) {
    const int64_t blocks = ceil_div(p.B * p.D, 64);
    if (blocks > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64), 0, (hipStream_t)stream, p);
    return launch_status();
}

}  // namespace
}  // namespace layer

using namespace layer;

extern "C" {

int hyena_scan_workspace(int64_t B, int64_t L, int64_t D, int dtype, int64_t *bytes_out) {
    const int st = check_sizes(B, L, D, HYENA_GATE_SIGMOID, dtype);
    if (st != HYENA_OK) return st;
    if (!bytes_out) return HYENA_ERR_NULL;
    *bytes_out = 0;
    return HYENA_OK;
}

int hyena_scan_fwd(const void *q, const void *k, const void *v, const void *g, int64_t B, int64_t L, int64_t D,
                   int64_t ld, int gate, const float *s0, void *y, float *s_last, float *states, void *workspace,
                   int64_t workspace_bytes, int dtype, void *stream) {
    int st = check_sizes(B, L, D, gate, dtype);
    if (st != HYENA_OK) return st;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (ld < D || !mul_fits(B * L, ld, eb, &n)) return HYENA_ERR_SHAPE;
    if (B == 0 || D == 0) return HYENA_OK;
    if (!y && !s_last && !states) return HYENA_ERR_NULL;
    if (L > 0 && (!k || !v || !g || (y && !q))) return HYENA_ERR_NULL;
    if (!aligned(q, eb) || !aligned(k, eb) || !aligned(v, eb) || !aligned(g, eb) || !aligned(y, eb) ||
        !aligned(s0, 4) || !aligned(s_last, 4) || !aligned(states, 4) || !aligned(workspace, 16))
        return HYENA_ERR_ALIGN;
    int64_t need = 0;
    hyena_scan_workspace(B, L, D, dtype, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const Rows in[5] = {{y ? q : nullptr, B * L, D * eb, ld * eb}, {k, B * L, D * eb, ld * eb},
                        {v, B * L, D * eb, ld * eb}, {g, B * L, D * eb, ld * eb}, {s0, B, D * 4, D * 4}};
    const Rows out[4] = {{y, B * L, D * eb, D * eb}, {s_last, B, D * 4, D * 4},
                         {states, B * ceil_div(L, kStateRows), D * 4, D * 4},
                         {need > 0 ? workspace : nullptr, 1, need, need}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (overlap(out[i], in[j])) return HYENA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HYENA_ERR_ALIAS;
    }
    ScanParams p = {};
    p.q = q, p.k = k, p.v = v, p.g = g, p.s0 = s0;
    p.y = y, p.s_last = s_last, p.states = states;
    p.B = B, p.L = L, p.D = D, p.ld = ld;
    const bool f32 = dtype == HYENA_DTYPE_F32, lg = gate == HYENA_GATE_LOG;
    return launch(f32 ? (lg ? scan_fwd_kernel<true, true> : scan_fwd_kernel<true, false>)
                      : (lg ? scan_fwd_kernel<false, true> : scan_fwd_kernel<false, false>), p, stream);
}

int hyena_scan_bwd(const void *q, const void *k, const void *v, const void *g, const void *dy, const float *states,
                   const float *ds_last, int64_t B, int64_t L, int64_t D, int64_t ld, int64_t ldd, int gate, void *dq,
                   void *dk, void *dv, void *dg, float *ds0, void *workspace, int64_t workspace_bytes, int dtype,
                   void *stream) {
    int st = check_sizes(B, L, D, gate, dtype);
    if (st != HYENA_OK) return st;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (ld < D || ldd < D || !mul_fits(B * L, ld, eb, &n) || !mul_fits(B * L, ldd, eb, &n)) return HYENA_ERR_SHAPE;
    if (B == 0 || D == 0) return HYENA_OK;
    if (!dq && !dk && !dv && !dg && !ds0) return HYENA_ERR_NULL;
    if (L > 0 && (!q || !k || !v || !g || !dy || !states)) return HYENA_ERR_NULL;
    if (!aligned(q, eb) || !aligned(k, eb) || !aligned(v, eb) || !aligned(g, eb) || !aligned(dy, eb) ||
        !aligned(dq, eb) || !aligned(dk, eb) || !aligned(dv, eb) || !aligned(dg, eb) || !aligned(states, 4) ||
        !aligned(ds_last, 4) || !aligned(ds0, 4) || !aligned(workspace, 16))
        return HYENA_ERR_ALIGN;
    int64_t need = 0;
    hyena_scan_workspace(B, L, D, dtype, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const Rows in[7] = {{q, B * L, D * eb, ld * eb}, {k, B * L, D * eb, ld * eb}, {v, B * L, D * eb, ld * eb},
                        {g, B * L, D * eb, ld * eb}, {dy, B * L, D * eb, D * eb},
                        {states, B * ceil_div(L, kStateRows), D * 4, D * 4}, {ds_last, B, D * 4, D * 4}};
    const Rows out[6] = {{dq, B * L, D * eb, ldd * eb}, {dk, B * L, D * eb, ldd * eb}, {dv, B * L, D * eb, ldd * eb},
                         {dg, B * L, D * eb, ldd * eb}, {ds0, B, D * 4, D * 4},
                         {need > 0 ? workspace : nullptr, 1, need, need}};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 7; ++j)
            if (overlap(out[i], in[j])) return HYENA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HYENA_ERR_ALIAS;
    }
    ScanParams p = {};
    p.q = q, p.k = k, p.v = v, p.g = g, p.dy = dy, p.states_in = states, p.ds_last = ds_last;
    p.dq = dq, p.dk = dk, p.dv = dv, p.dg = dg, p.ds0 = ds0;
    p.B = B, p.L = L, p.D = D, p.ld = ld, p.ldd = ldd;
    const bool f32 = dtype == HYENA_DTYPE_F32, lg = gate == HYENA_GATE_LOG;
    return launch(f32 ? (lg ? scan_bwd_kernel<true, true> : scan_bwd_kernel<true, false>)
                      : (lg ? scan_bwd_kernel<false, true> : scan_bwd_kernel<false, false>), p, stream);
}

}  // extern "C"
