// One token at a time for MI355X (gfx950): the recurrence of hyena_scan.hip
// and the gated convolution with a ring cache of past rows of x = k v
// (hyena_layer.h has the formulas and layouts).

#include "layer_common.h"

namespace layer {
namespace {

struct StepParams {
    const void *q, *k, *v, *g, *h;
    const float *state;
    float *state_out;
    void *cache, *y;
    const int64_t *pos;
    const int32_t *slots;
    int64_t B, L, D, ld, S, R, group_size, l_h;
};

__device__ inline int64_t slot_of(const StepParams &p, int64_t b) { return p.slots ? p.slots[b] : b; }

template <bool F32, bool LOG>
__global__ __launch_bounds__(256) void scan_step_kernel(StepParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i % p.D, e = b * p.ld + d;
    const int64_t slot = slot_of(p, b);
    float y = 0.0f;
    if (slot >= 0 && slot < p.S) {
        const float a = decay<LOG>(load1<F32>(p.g, e));
        const float s = (a == 0.0f ? 0.0f : a * p.state[slot * p.D + d]) + load1<F32>(p.k, e) * load1<F32>(p.v, e);
        p.state_out[slot * p.D + d] = s;
        y = load1<F32>(p.q, e) * s;
    }
    store1<F32>(p.y, i, y);
}

template <bool F32>
__global__ __launch_bounds__(256) void conv_step_kernel(StepParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i % p.D, e = b * p.ld + d;
    const int64_t slot = slot_of(p, b), pos = p.pos[b];
    float y = 0.0f;
    if (slot >= 0 && slot < p.S && pos >= 0) {
        const int64_t f = d / p.group_size * p.l_h;
        const float x = load1<F32>(p.k, e) * load1<F32>(p.v, e);
        float acc = load1<F32>(p.h, f) * x;
        for (int64_t s = 1; s < p.l_h && s <= pos; ++s)
            acc += load1<F32>(p.h, f + s) * load1<F32>(p.cache, (slot * p.R + (pos - s) % p.R) * p.D + d);
        store1<F32>(p.cache, (slot * p.R + pos % p.R) * p.D + d, x);
        y = load1<F32>(p.q, e) * acc;
    }
    store1<F32>(p.y, i, y);
}

// One thread per channel of each of the R last rows.
template <bool F32>
__global__ __launch_bounds__(256) void cache_fill_kernel(StepParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t rows = min(p.R, p.L);
    if (i >= p.B * rows * p.D) return;
    const int64_t d = i % p.D, r = i / p.D % rows, b = i / p.D / rows;
    const int64_t slot = slot_of(p, b);
    int64_t len = p.pos ? p.pos[b] : p.L;
    len = len < 0 ? 0 : len > p.L ? p.L : len;
    const int64_t t = len - 1 - r;
    if (slot < 0 || slot >= p.S || t < 0) return;
    const int64_t e = (b * p.L + t) * p.ld + d;
    store1<F32>(p.cache, (slot * p.R + t % p.R) * p.D + d, load1<F32>(p.k, e) * load1<F32>(p.v, e));
}

template <typename K> int launch(K kernel, const StepParams &p, int64_t threads, void *stream) {
    const int64_t blocks = ceil_div(threads, 256);
    if (blocks > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, p);
    return launch_status();
}

int check_dtype(int dtype) {
    return dtype == HYENA_DTYPE_BF16 || dtype == HYENA_DTYPE_F32 ? HYENA_OK : HYENA_ERR_DTYPE;
}

}  // namespace
}  // namespace layer

using namespace layer;

extern "C" {

int hyena_scan_step(const void *q, const void *k, const void *v, const void *g, int64_t B, int64_t D, int64_t ld,
                    int gate, float *state, float *state_out, int64_t S, const int32_t *slots, void *y, int dtype,
                    void *stream) {
    int st = check_dtype(dtype);
    if (st != HYENA_OK) return st;
    if (gate != HYENA_GATE_SIGMOID && gate != HYENA_GATE_LOG) return HYENA_ERR_UNSUPPORTED;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (B < 0 || D < 0 || S < 0 || ld < D || !mul_fits(B, ld, eb, &n) || !mul_fits(S, D, 4, &n)) return HYENA_ERR_SHAPE;
    if (!slots && S < B) return HYENA_ERR_SHAPE;
    if (B == 0 || D == 0) return HYENA_OK;
    if (!q || !k || !v || !g || !y || (!state && S > 0)) return HYENA_ERR_NULL;
    if (!state_out) state_out = state;
    if (!aligned(q, eb) || !aligned(k, eb) || !aligned(v, eb) || !aligned(g, eb) || !aligned(y, eb) ||
        !aligned(state, 4) || !aligned(state_out, 4) || !aligned(slots, 4))
        return HYENA_ERR_ALIGN;
    const Rows in[5] = {{q, B, D * eb, ld * eb}, {k, B, D * eb, ld * eb}, {v, B, D * eb, ld * eb},
                        {g, B, D * eb, ld * eb}, {slots, B, 4, 4}};
    const Rows rs = {state, S, D * 4, D * 4}, ro = {state_out, S, D * 4, D * 4}, ry = {y, B, D * eb, D * eb};
    for (const Rows &r : in)
        if (overlap(ry, r) || overlap(ro, r)) return HYENA_ERR_ALIAS;
    if (overlap(ry, rs) || overlap(ry, ro) || (state != state_out && overlap(ro, rs))) return HYENA_ERR_ALIAS;
    StepParams p = {};
    p.q = q, p.k = k, p.v = v, p.g = g, p.state = state, p.state_out = state_out, p.slots = slots, p.y = y;
    p.B = B, p.D = D, p.ld = ld, p.S = S;
    const bool f32 = dtype == HYENA_DTYPE_F32, lg = gate == HYENA_GATE_LOG;
    return launch(f32 ? (lg ? scan_step_kernel<true, true> : scan_step_kernel<true, false>)
                      : (lg ? scan_step_kernel<false, true> : scan_step_kernel<false, false>), p, B * D, stream);
}

int hyena_conv_step(const void *q, const void *k, const void *v, const void *h, int64_t B, int64_t D, int64_t ld,
                    int64_t group_size, int64_t l_h, void *cache, int64_t S, int64_t R, const int64_t *pos,
                    const int32_t *slots, void *y, int dtype, void *stream) {
    int st = check_dtype(dtype);
    if (st != HYENA_OK) return st;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (B < 0 || D < 0 || S < 0 || ld < D || !mul_fits(B, ld, eb, &n)) return HYENA_ERR_SHAPE;
    if (group_size < 1 || D % group_size != 0) return HYENA_ERR_GROUP;
    if (l_h < 1 || l_h > 128) return HYENA_ERR_FILTER_LEN;
    if (R < l_h || !mul_fits(S, R, 1, &n) || !mul_fits(n, D, eb, &n)) return HYENA_ERR_SHAPE;
    if (!slots && S < B) return HYENA_ERR_SHAPE;
    if (B == 0 || D == 0) return HYENA_OK;
    if (!q || !k || !v || !h || !y || !pos || (!cache && S > 0)) return HYENA_ERR_NULL;
    if (!aligned(q, eb) || !aligned(k, eb) || !aligned(v, eb) || !aligned(h, eb) || !aligned(y, eb) ||
        !aligned(cache, eb) || !aligned(pos, 8) || !aligned(slots, 4))
        return HYENA_ERR_ALIGN;
    const Rows in[6] = {{q, B, D * eb, ld * eb}, {k, B, D * eb, ld * eb}, {v, B, D * eb, ld * eb},
                        {h, D / group_size, l_h * eb, l_h * eb}, {pos, B, 8, 8}, {slots, B, 4, 4}};
    const Rows rc = {cache, S * R, D * eb, D * eb}, ry = {y, B, D * eb, D * eb};
    for (const Rows &r : in)
        if (overlap(ry, r) || overlap(rc, r)) return HYENA_ERR_ALIAS;
    if (overlap(ry, rc)) return HYENA_ERR_ALIAS;
    StepParams p = {};
    p.q = q, p.k = k, p.v = v, p.h = h, p.cache = cache, p.pos = pos, p.slots = slots, p.y = y;
    p.B = B, p.D = D, p.ld = ld, p.S = S, p.R = R, p.group_size = group_size, p.l_h = l_h;
    return launch(dtype == HYENA_DTYPE_F32 ? conv_step_kernel<true> : conv_step_kernel<false>, p, B * D, stream);
}

int hyena_conv_cache_fill(const void *k, const void *v, int64_t B, int64_t L, int64_t D, int64_t ld, void *cache,
                          int64_t S, int64_t R, const int64_t *lens, const int32_t *slots, int dtype, void *stream) {
    int st = check_dtype(dtype);
    if (st != HYENA_OK) return st;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (B < 0 || L < 0 || D < 0 || S < 0 || R < 1 || ld < D || !mul_fits(B, L, 1, &n) || !mul_fits(n, ld, eb, &n) ||
        !mul_fits(S, R, 1, &n) || !mul_fits(n, D, eb, &n))
        return HYENA_ERR_SHAPE;
    if (!slots && S < B) return HYENA_ERR_SHAPE;
    if (B == 0 || D == 0 || L == 0) return HYENA_OK;
    if (!k || !v || (!cache && S > 0)) return HYENA_ERR_NULL;
    if (!aligned(k, eb) || !aligned(v, eb) || !aligned(cache, eb) || !aligned(lens, 8) || !aligned(slots, 4))
        return HYENA_ERR_ALIGN;
    const Rows in[4] = {{k, B * L, D * eb, ld * eb}, {v, B * L, D * eb, ld * eb}, {lens, B, 8, 8}, {slots, B, 4, 4}};
    const Rows rc = {cache, S * R, D * eb, D * eb};
    for (const Rows &r : in)
        if (overlap(rc, r)) return HYENA_ERR_ALIAS;
    StepParams p = {};
    p.k = k, p.v = v, p.cache = cache, p.pos = lens, p.slots = slots;
    p.B = B, p.L = L, p.D = D, p.ld = ld, p.S = S, p.R = R;
    return launch(dtype == HYENA_DTYPE_F32 ? cache_fill_kernel<true> : cache_fill_kernel<false>, p,
                  B * (R < L ? R : L) * D, stream);
}

const char *hyena_layer_strerror(int status) {
    switch (status) {
    case HYENA_OK: return "ok";
    case HYENA_ERR_NULL: return "a required pointer is NULL";
    case HYENA_ERR_SHAPE: return "a size is negative, too small for another or overflows, or a row stride is shorter than its row";
    case HYENA_ERR_GROUP: return "group_size must be >= 1 and divide D";
    case HYENA_ERR_FILTER_LEN: return "l_h must be in [1, 128]";
    case HYENA_ERR_ALIGN: return "a pointer is not aligned to its elements (workspaces: 16 bytes)";
    case HYENA_ERR_ALIAS: return "an output overlaps an input or another output";
    case HYENA_ERR_UNSUPPORTED: return "unknown gate or activation code, or a grid too large to launch";
    case HYENA_ERR_LAUNCH: return "kernel launch failed";
    case HYENA_ERR_DTYPE: return "unknown dtype code";
    case HYENA_ERR_WORKSPACE: return "workspace missing or smaller than the operator's workspace call reports";
    default: return "unknown status";
    }
}

}  // extern "C"
