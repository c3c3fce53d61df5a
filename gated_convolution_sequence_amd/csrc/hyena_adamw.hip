// An AdamW step and the norm of all gradients over a list of tensors, for
// MI355X (gfx950) (hyena_model.h has the formulas).
//
// Bound by memory: a bf16 weight with an fp32 master moves 28 bytes (16 with
// moments of 8 bits, and 2 more for the norm).  The tensors' addresses travel as
// kernel arguments, up to kTensors a launch, so that nothing is copied to the device
// beforehand and a captured call keeps its own; a workgroup finds its tensor by one
// comparison a lane.  688 million bf16 weights with masters: the step 3.50 ms (19.3 GB,
// 5.5 TB/s), the norm 0.20 (1.4 GB, 7.0 TB/s); 306 million with moments in 8 bits 0.90
// ms (4.9 GB, 5.4 TB/s; its arithmetic alone would take about half as long).

#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "hyena_model.h"
#include "layer_gemm.h"

namespace layer {
namespace {

constexpr int kTensors = 48;  // a launch: 3.5 KB of arguments
constexpr int kTurn = 2048;   // elements a workgroup takes at a time
constexpr int kBlock = 256;   // elements that share a scale

struct Entry {
    void *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale, *master;
    int64_t numel;
};
struct Table {
    Entry t[kTensors];
    uint32_t first[kTensors];  // each tensor's first workgroup
    uint32_t place[kTensors];  // its place in the list
    int n, blocks;             // tensors, workgroups of all of them
    int span;                  // elements a workgroup, whole turns
};

// The tensor of a workgroup, and the workgroup's place in it.
__device__ inline int find(const Table &p, int block) {
    const int lane = threadIdx.x & 63;
    const uint64_t at = __builtin_amdgcn_ballot_w64(lane < p.n && p.first[lane] <= (uint32_t)block);
    return __builtin_amdgcn_readfirstlane(__popcll(at) - 1);
}

// What a step multiplies by; from 64 bits, since 1 - beta^t cancels.  root is
// 1 / sqrt(1 - beta2^t).
struct Factors {
    float b1, c1, b2, c2, keep, size, root, eps;
};
__host__ __device__ inline double power(double x, int64_t n) {  // n >= 0
    double r = 1.0;
    for (; n > 0; n >>= 1, x *= x)
        if (n & 1) r *= x;
    return r;
}
struct AdamParams {
    double lr, beta1, beta2, weight_decay;
    int64_t step;
    const float *lr_dev;
    const int64_t *step_dev, *seed_dev;
    const float *scale;
    float eps;
    uint32_t seed;
    Factors given;  // of lr and step

    __host__ __device__ Factors factors(double lr, int64_t t) const {
        if (t < 1) t = 1;
        return Factors{(float)beta1, (float)(1.0 - beta1), (float)beta2, (float)(1.0 - beta2), (float)(1.0 - lr * weight_decay),
                       (float)(lr / (1.0 - power(beta1, t))), (float)(1.0 / sqrt(1.0 - power(beta2, t))), eps};
    }
};

// A workgroup's tensor and factors.
struct Work {
    Entry t;
    Factors f;
    float scale;
    uint32_t seed;  // of the tensor
    int64_t begin, end;
    bool skip;
};
__device__ __forceinline__ Work work_of(const Table &p, const AdamParams &a, int block) {
    __shared__ Factors shared;
    Work w;
    const int i = find(p, block);
    w.t = p.t[i];
    w.begin = (int64_t)((uint32_t)block - p.first[i]) * p.span, w.end = min(w.t.numel, w.begin + p.span);
    w.f = a.given;
    if (a.lr_dev || a.step_dev) {
        if (threadIdx.x == 0) shared = a.factors(a.lr_dev ? (double)*a.lr_dev : a.lr, a.step_dev ? *a.step_dev : a.step);
        __syncthreads();
        w.f = shared;
    }
    w.scale = a.scale ? *a.scale : 1.0f;
    w.skip = !(fabsf(w.scale) <= 3.402823466e38f);
    w.seed = (a.seed_dev ? (uint32_t)*a.seed_dev : a.seed) + 0x9E3779B9u * p.place[i];
    return w;
}

// The new m, v and r = sqrt(v) and the value that they move, V elements at a time.
// Products and sums of the moments are rounded one by one: codes of 8 bits then
// depend on the written formula alone, not on what a compiler fuses.
template <int V>
__device__ __forceinline__ void move(const Factors &f, float scale, const float (&g)[V], float (&m)[V], float (&v)[V],
                                     float (&r)[V], float (&w)[V]) {
#pragma clang fp contract(off)
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const float d = g[k] * scale;
        m[k] = f.b1 * m[k] + f.c1 * d;
        v[k] = f.b2 * v[k] + f.c2 * (d * d);
        r[k] = sqrtf(v[k]);
        // the hardware's reciprocal is off by one unit in its last place, of a move that is a part of w
        w[k] = w[k] * f.keep - f.size * m[k] * __builtin_amdgcn_rcpf(r[k] * f.root + f.eps);
    }
}
// V values from element e on, n of them where that is fewer (WHOLE: never), past the
// caches where a wave's accesses cover whole lines, at 16 bytes a lane or less (with 32,
// in two accesses that each touch half of every line, the step took 1.3 times as long).
template <bool F32, bool WHOLE, int V> __device__ __forceinline__ void read(const void *p, int64_t e, int n, float (&x)[V]) {
    const auto r = Pack<F32, V>::template load<Pack<F32, V>::PARTS == 1>(p, e, WHOLE ? V : n);
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = r.get(k);
}
template <bool F32, bool WHOLE, int V> __device__ __forceinline__ void write(void *p, int64_t e, int n, const float (&x)[V]) {
    Pack<F32, V>::template store<Pack<F32, V>::PARTS == 1>(p, e, WHOLE ? V : n, x);
}
template <bool F32, bool WHOLE, int V>
__device__ __forceinline__ void read_value(const Entry &t, int64_t e, int n, float (&w)[V]) {
    if (t.master) read<true, WHOLE, V>(t.master, e, n, w);
    else read<F32, WHOLE, V>(t.param, e, n, w);
}
template <bool F32, bool WHOLE, int V>
__device__ __forceinline__ void write_value(const Entry &t, int64_t e, int n, const float (&w)[V]) {
    if (t.master) write<true, WHOLE, V>(t.master, e, n, w);
    write<F32, WHOLE, V>(t.param, e, n, w);
}

// Four elements a lane, twice.
template <bool F32, bool WHOLE> __device__ __forceinline__ void step32(const Work &k, int64_t at) {
    constexpr int V = 4, U = kTurn / (256 * V);
    float g[U][V], m[U][V], v[U][V], r[V], w[U][V];
    int n[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = at + (u * 256 + threadIdx.x) * V;
        n[u] = WHOLE ? V : (int)min(k.end - e, (int64_t)V);
        if (!WHOLE && n[u] <= 0) continue;
        read<F32, WHOLE, V>(k.t.grad, e, n[u], g[u]);
        read<true, WHOLE, V>(k.t.m, e, n[u], m[u]);
        read<true, WHOLE, V>(k.t.v, e, n[u], v[u]);
        read_value<F32, WHOLE, V>(k.t, e, n[u], w[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = at + (u * 256 + threadIdx.x) * V;
        if (!WHOLE && n[u] <= 0) continue;
        move(k.f, k.scale, g[u], m[u], v[u], r, w[u]);
        write<true, WHOLE, V>(k.t.m, e, n[u], m[u]);
        write<true, WHOLE, V>(k.t.v, e, n[u], v[u]);
        write_value<F32, WHOLE, V>(k.t, e, n[u], w[u]);
    }
}
template <bool F32> __global__ __launch_bounds__(256) void adamw_kernel(Table p, AdamParams a) {
    const int block = block_of();
    if (block >= p.blocks) return;
    const Work k = work_of(p, a, block);
    if (k.skip) return;
    int64_t at = k.begin;
    for (; at + kTurn <= k.end; at += kTurn) step32<F32, true>(k, at);
    if (at < k.end) step32<F32, false>(k, at);
}

// ---- moments in 8 bits ----------------------------------------------------------------

// 32 bits well mixed: the last steps of murmur3.
__device__ inline uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

// Eight codes as they lie in memory, n of them where that is fewer.
struct Codes {
    typedef u32x2_t any __attribute__((aligned(1)));
    u32x2_t c;
    __device__ static Codes load(const void *p, int64_t e, int n) {
        const uint8_t *at = (const uint8_t *)p + e;
        if (n >= 8) return Codes{*(const any *)at};
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) w[k / 4] |= (uint32_t)at[k] << 8 * (k % 4);
        return Codes{u32x2_t{w[0], w[1]}};
    }
    __device__ void store(void *p, int64_t e, int n) const {
        uint8_t *at = (uint8_t *)p + e;
        if (n >= 8) {
            *(any *)at = c;
            return;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) at[k] = (uint8_t)(c[k / 4] >> 8 * (k % 4));
    }
    __device__ void get(float (&x)[8]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x[4 * h] = __builtin_amdgcn_cvt_f32_fp8(c[h], 0);
            x[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(c[h], 1);
            x[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(c[h], 2);
            x[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(c[h], 3);
        }
    }
    // of values that e4m3 holds
    __device__ static Codes of(const float (&x)[8]) {
        Codes r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h], x[4 * h + 1], 0, false);
            r.c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2], x[4 * h + 3], w, true);
        }
        return r;
    }
};

// The block's scale (32 lanes, eight values each) and the codes of t = |x| / scale:
// with the spacing 2^(e - 3) of the codes around it (2^-9 at least), floor(t /
// spacing + up) of them.  16 bits of `up` from each of h; it is 2^-16 below 1 at most, so
// that the largest x, 14 spacings of 32 but for roundings, stays at 14.
template <int SHIFT>
__device__ __forceinline__ Codes round_codes(const float (&x)[8], const uint32_t (&h)[8], float &scale) {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
    top = over_32(top, [](float a, float b) { return fmaxf(a, b); });
    scale = top < 0x1p-117f ? 0.0f : top * (1.0f / 448.0f);
    const float inverse = scale != 0.0f ? 1.0f / scale : 0.0f;
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // the quotient rounded as a division would, from the rounded reciprocal
        const float t0 = fabsf(x[k]) * inverse;
        const float t = fmaf(fmaf(-t0, scale, fabsf(x[k])), inverse, t0);
        const uint32_t e = max(__float_as_uint(t) & 0x7f800000u, 121u << 23);
        const float spacing = __uint_as_float(e - (3u << 23)), per = __uint_as_float((257u << 23) - e);
        const float up = (float)(h[k] >> SHIFT & 0xffffu);
        q[k] = copysignf(floorf(fmaf(up, 0x1p-16f, t * per)) * spacing, x[k]);
    }
    return Codes::of(q);
}

// A wave's halves take a block of 256 each, so that its largest is five steps between
// lanes.  Every lane comes along, with none of its own past the end.
template <bool F32, bool WHOLE> __device__ __forceinline__ void step8(const Work &k, int64_t e) {
    constexpr int V = 8;
    static_assert(kBlock == 32 * V && kTurn == 256 * V, "half a wave a block");
    const int n = WHOLE ? V : (int)max(min(k.end - e, (int64_t)V), (int64_t)0);
    const int64_t block = e / kBlock;
    float g[V] = {}, m[V] = {}, v[V] = {}, r[V], w[V] = {};
    if (WHOLE || n > 0) {
        const Codes cm = Codes::load(k.t.m, e, n), cv = Codes::load(k.t.v, e, n);
        const float sm = k.t.m_scale[block], sv = k.t.v_scale[block];
        read<F32, WHOLE, V>(k.t.grad, e, n, g);
        read_value<F32, WHOLE, V>(k.t, e, n, w);
        cm.get(m);
        cv.get(v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m[i] *= sm;
            v[i] *= sv;
            v[i] *= v[i];
        }
    }
    move(k.f, k.scale, g, m, v, r, w);
    if (WHOLE || n > 0) write_value<F32, WHOLE, V>(k.t, e, n, w);
    uint32_t h[V];
    const uint32_t key = mix(k.seed + (uint32_t)(e >> 32));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        h[i] = mix((uint32_t)(e + i) ^ key);  // e is a multiple of 8: the high half is the same
        if (!WHOLE && i >= n) m[i] = r[i] = 0.0f;
    }
    float sm, sv;
    const Codes cm = round_codes<0>(m, h, sm), cv = round_codes<16>(r, h, sv);
    if (!WHOLE && n <= 0) return;
    cm.store(k.t.m, e, n);
    cv.store(k.t.v, e, n);
    if ((threadIdx.x & 31) == 0) k.t.m_scale[block] = sm, k.t.v_scale[block] = sv;
}
template <bool F32> __global__ __launch_bounds__(256) void adamw8_kernel(Table p, AdamParams a) {
    const int block = block_of();
    if (block >= p.blocks) return;
    const Work k = work_of(p, a, block);
    if (k.skip) return;
    const int64_t e = k.begin + threadIdx.x * 8;
    if (k.end - k.begin == kTurn) step8<F32, true>(k, e);
    else step8<F32, false>(k, e);
}

// ---- norm of all gradients ------------------------------------------------------------

__device__ inline double block_sum(double s) {
    __shared__ double part[16];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) s += part[w];
    return s;
}

constexpr int kNormSpan = 32768;
template <bool F32> __global__ __launch_bounds__(256) void squares_kernel(Table p, double *partial) {
    constexpr int V = F32 ? 4 : 8, U = 4;  // loads in flight
    const int block = block_of();
    if (block >= p.blocks) return;
    const int i = find(p, block);
    const Entry t = p.t[i];
    const int64_t begin = (int64_t)((uint32_t)block - p.first[i]) * kNormSpan, end = min(t.numel, begin + kNormSpan);
    double s[V] = {};
    int64_t at = begin;
    for (; at + U * 256 * V <= end; at += U * 256 * V) {
        Pack<F32, V> g[U];
#pragma unroll
        for (int u = 0; u < U; ++u) g[u] = Pack<F32, V>::template load<true>(t.grad, at + (u * 256 + threadIdx.x) * V, V);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k) s[k] = fma((double)g[u].get(k), (double)g[u].get(k), s[k]);
    }
    for (int64_t e = at + threadIdx.x * V; e < end; e += 256 * V) {
        const auto g = Pack<F32, V>::load(t.grad, e, (int)min(end - e, (int64_t)V));
#pragma unroll
        for (int k = 0; k < V; ++k) s[k] = fma((double)g.get(k), (double)g.get(k), s[k]);
    }
#pragma unroll
    for (int k = 1; k < V; ++k) s[0] += s[k];
    s[0] = block_sum(s[0]);
    if (threadIdx.x == 0) partial[block] = s[0];
}

__global__ __launch_bounds__(1024) void norm_kernel(const double *partial, int64_t n, double max_norm, float *norm,
                                                    float *scale) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) s += partial[i];
    s = sqrt(block_sum(s));
    if (threadIdx.x == 0) {
        *norm = (float)s;
        // a norm that fp32 does not hold, or none: no step
        if (scale) *scale = !(s <= 3.402823466e38) ? __builtin_nanf("") : s > max_norm ? (float)(max_norm / s) : 1.0f;
    }
}

// ---- host --------------------------------------------------------------------------------

// The next launch's tensors: from `next` on, at most kTensors with elements.  A
// tensor below 2^40 elements has at most 2^29 workgroups (of kSpan8's 2048), 48 may have 2^34.6,
// so that a launch ends at 2^30.
constexpr int64_t kMostBlocks = (int64_t)1 << 30, kMostElements = (int64_t)1 << 40;
int64_t fill(Table &p, const hyena_tensor *ts, int64_t n, int64_t &next, int64_t span) {
    p.n = 0;
    p.span = (int)span;
    int64_t blocks = 0;
    for (; next < n && p.n < kTensors; ++next) {
        const hyena_tensor &t = ts[next];
        if (t.numel == 0) continue;
        const int64_t more = ceil_div(t.numel, span);
        if (blocks + more > kMostBlocks) break;
        p.t[p.n] = Entry{t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale, t.master, t.numel};
        p.first[p.n] = (uint32_t)blocks;
        p.place[p.n++] = (uint32_t)next;
        blocks += more;
    }
    p.blocks = (int)blocks;
    return blocks;
}

// The descriptors: with their gradients only (bits 0), or all of a step.
int check_tensors(const hyena_tensor *ts, int64_t n, int dtype, int bits, int64_t *numel) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    if (n < 0 || n >= (int64_t)1 << 31) return HYENA_ERR_SHAPE;
    if (n > 0 && !ts) return HYENA_ERR_NULL;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t all = 0;
    for (int64_t i = 0; i < n; ++i) {
        const hyena_tensor &t = ts[i];
        if (t.numel < 0 || t.numel >= kMostElements) return HYENA_ERR_SHAPE;
        all += t.numel;
        if (all >= (int64_t)1 << 56) return HYENA_ERR_SHAPE;
        if (t.numel == 0) continue;
        if (!t.grad) return HYENA_ERR_NULL;
        if (!aligned(t.grad, eb)) return HYENA_ERR_ALIGN;
        if (bits == 0) continue;
        if (!t.param || !t.exp_avg || !t.exp_avg_sq || (bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
            return HYENA_ERR_NULL;
        const int64_t sb = bits / 8;
        if (!aligned(t.param, eb) || !aligned(t.exp_avg, sb) || !aligned(t.exp_avg_sq, sb) || !aligned(t.master, 4) ||
            (bits == 8 && (!aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))))
            return HYENA_ERR_ALIGN;
    }
    if (numel) *numel = all;
    return HYENA_OK;
}

// Elements a workgroup.  Short spans, so that the workgroups of a moment touch few
// pages of each array: 688 million weights in 32 bits 3.50 ms with 2 turns, 3.52 with 1,
// 3.58 with 4, 3.8 with 16; 306 million in 8 bits 0.88 with 1, 0.93 with 4, 0.98 with 16.
constexpr int64_t kSpan32 = 2 * kTurn, kSpan8 = kTurn;

// Whether anything that a step writes overlaps something else of it, in one tensor or
// between two: all ranges in the order of their addresses.
struct Range {
    uintptr_t first, last;  // last: the first byte after it
    bool written;
};
int check_overlap(const hyena_tensor *ts, int64_t n, int64_t eb, int bits, const float *lr, const int64_t *step,
                  const int64_t *seed, const float *scale) {
    Range *r = (Range *)malloc((size_t)(7 * n + 4) * sizeof(Range));
    if (!r) return HYENA_ERR_UNSUPPORTED;
    int64_t k = 0;
    auto add = [&](const void *p, int64_t bytes, bool written) {
        if (p && bytes > 0) r[k++] = Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written};
    };
    for (int64_t i = 0; i < n; ++i) {
        const hyena_tensor &t = ts[i];
        const int64_t state = t.numel * (bits / 8), scales = bits == 8 ? ceil_div(t.numel, kBlock) * 4 : 0;
        add(t.param, t.numel * eb, true);
        add(t.grad, t.numel * eb, false);
        add(t.exp_avg, state, true);
        add(t.exp_avg_sq, state, true);
        add(t.exp_avg_scale, scales, true);
        add(t.exp_avg_sq_scale, scales, true);
        add(t.master, t.numel * 4, true);
    }
    add(lr, 4, false), add(step, 8, false), add(seed, 8, false), add(scale, 4, false);
    std::sort(r, r + k, [](const Range &a, const Range &b) { return a.first < b.first; });
    uintptr_t any = 0, written = 0;
    bool bad = false;
    for (int64_t i = 0; i < k && !bad; ++i) {
        bad = r[i].first < written || (r[i].written && r[i].first < any);
        if (r[i].last > any) any = r[i].last;
        if (r[i].written && r[i].last > written) written = r[i].last;
    }
    free(r);
    return bad ? HYENA_ERR_ALIAS : HYENA_OK;
}

int64_t norm_partials(int64_t n, int64_t numel) { return n + numel / kNormSpan; }

}  // namespace
}  // namespace layer

using namespace layer;

extern "C" {

int hyena_adamw_step(const hyena_tensor *tensors, int64_t n, double lr, double beta1, double beta2, double eps,
                     double weight_decay, int64_t step, int64_t seed, const float *lr_dev, const int64_t *step_dev,
                     const int64_t *seed_dev, const float *grad_scale, int state_bits, int dtype, void *stream) {
    if (state_bits != 32 && state_bits != 8) return HYENA_ERR_UNSUPPORTED;
    int st = check_tensors(tensors, n, dtype, state_bits, nullptr);
    if (st != HYENA_OK) return st;
    if ((!lr_dev && !isfinite(lr)) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) ||
        !isfinite(eps) || !isfinite(weight_decay) || (!step_dev && step < 1))
        return HYENA_ERR_UNSUPPORTED;
    if (!aligned(lr_dev, 4) || !aligned(step_dev, 8) || !aligned(seed_dev, 8) || !aligned(grad_scale, 4))
        return HYENA_ERR_ALIGN;
    const bool f32 = dtype == HYENA_DTYPE_F32;
    st = check_overlap(tensors, n, f32 ? 4 : 2, state_bits, lr_dev, step_dev, seed_dev, grad_scale);
    if (st != HYENA_OK) return st;
    AdamParams a = {};
    a.lr = lr, a.beta1 = beta1, a.beta2 = beta2, a.weight_decay = weight_decay, a.step = step, a.seed = (uint32_t)seed;
    a.lr_dev = lr_dev, a.step_dev = step_dev, a.seed_dev = seed_dev, a.scale = grad_scale, a.eps = (float)eps;
    a.given = a.factors(lr_dev ? 0.0 : lr, step_dev ? 1 : step);
    const auto kernel = state_bits == 8 ? (f32 ? adamw8_kernel<true> : adamw8_kernel<false>)
                                        : (f32 ? adamw_kernel<true> : adamw_kernel<false>);
    Table p;
    int64_t next = 0;
    while (const int64_t blocks = fill(p, tensors, n, next, state_bits == 8 ? kSpan8 : kSpan32)) {
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(256), 0, (hipStream_t)stream, p, a);
        if ((st = launch_status()) != HYENA_OK) return st;
    }
    return HYENA_OK;
}

int hyena_grad_norm_workspace(int64_t n, int64_t numel, int64_t *bytes_out) {
    if (n < 0 || numel < 0 || n >= (int64_t)1 << 56 || numel >= (int64_t)1 << 56) return HYENA_ERR_SHAPE;
    if (!bytes_out) return HYENA_ERR_NULL;
    *bytes_out = ceil_div(norm_partials(n, numel) * 8, 16) * 16;
    return HYENA_OK;
}

int hyena_grad_norm(const hyena_tensor *tensors, int64_t n, double max_norm, float *norm, float *scale, void *workspace,
                    int64_t workspace_bytes, int dtype, void *stream) {
    int64_t numel = 0, need = 0;
    int st = check_tensors(tensors, n, dtype, 0, &numel);
    if (st != HYENA_OK) return st;
    if (!norm) return HYENA_ERR_NULL;
    if (scale && !(max_norm >= 0)) return HYENA_ERR_UNSUPPORTED;
    if (!aligned(norm, 4) || !aligned(scale, 4) || !aligned(workspace, 16)) return HYENA_ERR_ALIGN;
    hyena_grad_norm_workspace(n, numel, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const bool f32 = dtype == HYENA_DTYPE_F32;
    const Rows out[3] = {{norm, 1, 4, 4}, {scale, 1, 4, 4}, {need > 0 ? workspace : nullptr, 1, need, need}};
    for (int a = 0; a < 3; ++a) {
        for (int b = 0; b < a; ++b)
            if (overlap(out[a], out[b])) return HYENA_ERR_ALIAS;
        for (int64_t i = 0; i < n; ++i) {
            const int64_t w = tensors[i].numel * (f32 ? 4 : 2);
            if (overlap(out[a], Rows{tensors[i].grad, 1, w, w})) return HYENA_ERR_ALIAS;
        }
    }
    double *partial = (double *)workspace;
    int64_t done = 0, next = 0;
    Table p;
    while (const int64_t blocks = fill(p, tensors, n, next, kNormSpan)) {
        hipLaunchKernelGGL((f32 ? squares_kernel<true> : squares_kernel<false>), grid_of(blocks), dim3(256), 0,
                           (hipStream_t)stream, p, partial + done);
        if ((st = launch_status()) != HYENA_OK) return st;
        done += blocks;
    }
    hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(1024), 0, (hipStream_t)stream, partial, done, max_norm, norm, scale);
    return launch_status();
}

const char *hyena_model_strerror(int status) {
    switch (status) {
    case HYENA_OK: return "ok";
    case HYENA_ERR_NULL: return "a required pointer is NULL";
    case HYENA_ERR_SHAPE: return "a size is negative, too small for another or overflows, or a row stride is shorter than its row";
    case HYENA_ERR_ALIGN: return "a pointer is not aligned to its elements (workspaces: 16 bytes)";
    case HYENA_ERR_ALIAS: return "an output overlaps an input or another output";
    case HYENA_ERR_UNSUPPORTED: return "unknown kind or state size, a mean for the rms kind, a scalar out of its range, or a size too large to launch";
    case HYENA_ERR_LAUNCH: return "kernel launch failed";
    case HYENA_ERR_DTYPE: return "unknown dtype code";
    case HYENA_ERR_WORKSPACE: return "workspace missing or smaller than the operator's workspace call reports";
    default: return "unknown status";
    }
}

}  // extern "C"
