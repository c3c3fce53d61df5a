// One token at a time for MI355X (gfx950): the recurrence of hyena_scan.hip
// and the gated convolution with a ring cache of past rows of x = k v
// (hyena_layer.h has the formulas and layouts).

#include "layer_common.h"

namespace layer {
namespace {

// A lane takes 16 bytes of a row (Lane), blockIdx.y counts sequences (or rows).

struct StepParams {
    const void *q, *k, *v, *g, *h;
    const float *state;
    float *state_out;
    void *cache, *y;
    const int64_t *pos;
    const int32_t *slots;
    int64_t B, L, D, ld, S, R, group_size, l_h;
};

// a / b and a % b for a >= 0, b > 0; the 64-bit division only where one is wanted.
__device__ inline int64_t quotient(int64_t a, int64_t b) {
    return a >> 32 | b >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
__device__ inline int64_t remainder_of(int64_t a, int64_t b) { return a < b ? a : a - quotient(a, b) * b; }

__device__ inline int64_t slot_of(const StepParams &p, int64_t b) { return p.slots ? p.slots[b] : b; }

// The lane's n channels at element e (n may be less than VEC at the right edge).
template <bool F32> __device__ inline typename Lane<F32>::raw load_row(const void *p, size_t e, int n) {
    return n == Lane<F32>::VEC ? Lane<F32>::load(p, e) : Lane<F32>::load_part(p, e, n);
}
template <bool F32>
__device__ inline void store_row(void *p, size_t e, const float (&x)[Lane<F32>::VEC], int n) {
    if (n == Lane<F32>::VEC) Lane<F32>::store(p, e, Lane<F32>::pack(x));
    else Lane<F32>::store_part(p, e, Lane<F32>::pack(x), n);
}

constexpr int kScanThreads = 64;

// The recurrence's token: a lane's channels are its own, so there is nothing to
// share; one wave a workgroup spreads even one sequence over the card.  Bound by
// the launch and one trip to memory: D = 4096 bf16 in 3 us for B = 1, 5 us for
// B = 256 (18.9 MB: 3.7 TB/s).
template <bool F32, bool LOG>
__global__ __launch_bounds__(kScanThreads) void scan_step_kernel(StepParams p) {
    using Ln = Lane<F32>;
    constexpr int VEC = Ln::VEC;
    const int64_t d0 = ((int64_t)blockIdx.x * kScanThreads + threadIdx.x) * VEC;
    const int n = (int)min((int64_t)VEC, p.D - d0);
    if (n <= 0) return;
    for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t slot = slot_of(p, b);
        float y[VEC] = {};
        if (slot >= 0 && slot < p.S) {
            const size_t e = b * p.ld + d0, at = slot * p.D + d0;
            const auto q = load_row<F32>(p.q, e, n), k = load_row<F32>(p.k, e, n), v = load_row<F32>(p.v, e, n),
                       g = load_row<F32>(p.g, e, n);
            f32x4_t s[VEC / 4];
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) s[i] = load_row<true>(p.state, at + 4 * i, max(0, min(4, n - 4 * i)));
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float a = decay<LOG>(Ln::get(g, i)), old = s[i / 4][i % 4];
                const float now = fmaf(a, a == 0.0f ? 0.0f : old, Ln::get(k, i) * Ln::get(v, i));
                s[i / 4][i % 4] = now;
                y[i] = Ln::get(q, i) * now;
            }
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float x[4] = {s[i][0], s[i][1], s[i][2], s[i][3]};
                store_row<true>(p.state_out, at + 4 * i, x, max(0, min(4, n - 4 * i)));
            }
        }
        store_row<F32>(p.y, b * p.D + d0, y, n);
    }
}

// N consecutive taps from element e on, `left` of them in the filter (the rest
// zero).
template <bool F32, int N> __device__ inline void load_taps(const void *h, size_t e, int left, float (&x)[N]) {
    if (left >= N) {
        constexpr int WORDS = F32 ? N : N / 2;
        typedef u32x2_t pair_any __attribute__((aligned(2)));
        u32x2_t r[WORDS / 2];
#pragma unroll
        for (int i = 0; i < WORDS / 2; ++i) r[i] = ((const pair_any *)((const char *)h + e * (F32 ? 4 : 2)))[i];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (F32) x[i] = __uint_as_float(r[i / 2][i % 2]);
            else x[i] = i & 1 ? bf_hi(r[i / 4][i / 2 % 2]) : bf_lo(r[i / 4][i / 2 % 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = i < left ? load1<F32>(h, e + i) : 0.0f;
    }
}

// The convolution's token: 8 lanes take 128 bytes of channels, and the taps of
// one sequence are cut between 8 W slices of such lanes (W waves), TAPS
// consecutive taps each, all their rows of the ring in flight at once; the
// slices' sums meet by shuffles and, over the waves, in LDS.  Bound by the
// ring's rows from memory (l_h - 1 of them a sequence; B = 64, l_h = 128, D =
// 4096 bf16: 69 MB in 14.5 us, 4.8 TB/s; fp32 139 MB in 25 us, 5.6 TB/s), or by
// latency for few sequences (B = 1: 4.7 us).  ONE: a lane's channels share a
// filter.  Where they do not, every sequence reads each channel's taps anew: B =
// 64 with a filter per channel 27 us (2.6 TB/s of the ring's rows).
template <bool F32, int W, int TAPS, bool ONE> __global__ __launch_bounds__(256) void conv_step_kernel(StepParams p) {
    using Ln = Lane<F32>;
    constexpr int VEC = Ln::VEC, EB = F32 ? 4 : 2, ITEMS = 4 / W;
    __shared__ float part[ITEMS][W][8 * VEC];
    const int wave = threadIdx.x >> 6, item = wave / W, c8 = threadIdx.x & 7;
    const int slice = (wave % W) * 8 + (threadIdx.x >> 3 & 7);
    const int first = slice * TAPS;
    const int64_t d0 = (((int64_t)blockIdx.x * ITEMS + item) * 8 + c8) * VEC;
    const int n = (int)min((int64_t)VEC, p.D - d0);
    for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int slot = __builtin_amdgcn_readfirstlane(slot_of(p, b) < p.S ? (int)slot_of(p, b) : -1);
        const int64_t pos = p.pos[b];
        const bool live = slot >= 0 && pos >= 0;
        float acc[VEC] = {}, x0[VEC] = {};
        typename Ln::raw q = {};
        if (live && n > 0) {
            const int now = (int)remainder_of(pos, p.R);           // R D elements of a ring are below 2^31 bytes
            const int most = (int)min(p.l_h - 1, pos);             // the longest lag there is
            const size_t ring = (size_t)slot * p.R * p.D;
            const uint32_t pitch = (uint32_t)p.D * EB;
            typename Ln::raw k = {}, v = {}, x[TAPS] = {};
            if (slice == 0) {
                const size_t e = b * p.ld + d0;
                q = load_row<F32>(p.q, e, n), k = load_row<F32>(p.k, e, n), v = load_row<F32>(p.v, e, n);
            }
            if (n == VEC) {
                // lags there are none of read past the ring's range: zero
                const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                    (char *)p.cache + ring * EB, (short)0, (int)((uint32_t)p.R * pitch), 0x00020000);
#pragma unroll
                for (int i = 0; i < TAPS; ++i) {
                    const int s = first + i, row = now - s + (s > now ? (int)p.R : 0);
                    const uint32_t off = s >= 1 && s <= most ? row * pitch + (uint32_t)d0 * EB : 0x80000000u;
                    x[i] = __builtin_bit_cast(typename Ln::raw, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 2));
                }
            } else {
#pragma unroll
                for (int i = 0; i < TAPS; ++i) {
                    const int s = first + i, row = now - s + (s > now ? (int)p.R : 0);
                    if (s >= 1 && s <= most) x[i] = Ln::load_part(p.cache, ring + (size_t)row * p.D + d0, n);
                }
            }
            if (slice == 0) {
#pragma unroll
                for (int c = 0; c < VEC; ++c) x0[c] = Ln::get(k, c) * Ln::get(v, c);
                store_row<F32>(p.cache, ring + (size_t)now * p.D + d0, x0, n);
            }
            // (a tap past the last lag may be anything: its x does not count)
            auto add = [&](int i, int c, float tap) {
                const float xi = i == 0 && first == 0 ? x0[c] : Ln::get(x[i], c);
                if (first + i <= most) acc[c] = fmaf(tap, xi, acc[c]);
            };
            float h[TAPS];
            // the scheduling barriers keep one tap's (channel's) values in
            // registers at a time, not all of them
            if constexpr (ONE) {
                load_taps<F32, TAPS>(p.h, quotient(d0, p.group_size) * p.l_h + first, (int)p.l_h - first, h);
#pragma unroll
                for (int i = 0; i < TAPS; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int c = 0; c < VEC; ++c) add(i, c, h[i]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (c < n)
                        load_taps<F32, TAPS>(p.h, quotient(d0 + c, p.group_size) * p.l_h + first, (int)p.l_h - first, h);
#pragma unroll
                    for (int i = 0; i < TAPS; ++i) add(i, c, h[i]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < VEC; ++c)
#pragma unroll
            for (int o = 8; o < 64; o *= 2) acc[c] += __shfl_xor(acc[c], o);
        if constexpr (W > 1) {
            __syncthreads();  // the sums before are taken
            if ((threadIdx.x & 63) < 8) {
#pragma unroll
                for (int c = 0; c < VEC; ++c) part[item][wave % W][c8 * VEC + c] = acc[c];
            }
            __syncthreads();
        }
        if (slice == 0 && n > 0) {
            float y[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                float sum = acc[c];
                if constexpr (W > 1) {
#pragma unroll
                    for (int w = 1; w < W; ++w) sum += part[item][w][c8 * VEC + c];
                }
                y[c] = live ? Ln::get(q, c) * sum : 0.0f;
            }
            store_row<F32>(p.y, b * p.D + d0, y, n);
        }
    }
}

// The last rows of a prompt's k v: read and written once, bound by memory (64
// sequences, 128 rows of 4096 channels: bf16 201 MB in 33 us, fp32 403 MB in 66
// us, 6.1 TB/s) and, for a few sequences, the launch (one: 3 us).  blockIdx.y counts the rows from the last one
// back, blockIdx.z the sequences.
template <bool F32> __global__ __launch_bounds__(kScanThreads) void cache_fill_kernel(StepParams p) {
    using Ln = Lane<F32>;
    constexpr int VEC = Ln::VEC;
    const int64_t d0 = ((int64_t)blockIdx.x * kScanThreads + threadIdx.x) * VEC;
    const int n = (int)min((int64_t)VEC, p.D - d0);
    if (n <= 0) return;
    const int64_t rows = min(p.R, p.L);
    for (int64_t b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int64_t slot = slot_of(p, b);
        if (slot < 0 || slot >= p.S) continue;
        int64_t len = p.pos ? p.pos[b] : p.L;
        len = len < 0 ? 0 : len > p.L ? p.L : len;
        for (int64_t r = blockIdx.y; r < rows && r < len; r += gridDim.y) {
            const int64_t t = len - 1 - r;
            const size_t e = (size_t)(b * p.L + t) * p.ld + d0;
            const auto k = load_row<F32>(p.k, e, n), v = load_row<F32>(p.v, e, n);
            float x[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) x[c] = Ln::get(k, c) * Ln::get(v, c);
            store_row<F32>(p.cache, ((size_t)slot * p.R + remainder_of(t, p.R)) * p.D + d0, x, n);
        }
    }
}

unsigned at_most(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

template <typename K> int launch(K kernel, const StepParams &p, dim3 grid, int threads, void *stream) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, (hipStream_t)stream, p);
    return launch_status();
}

// Blocks of `lanes` lanes over a row's channels.
int64_t row_blocks(int64_t D, bool f32, int64_t lanes) { return ceil_div(ceil_div(D, f32 ? 4 : 8), lanes); }

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
    const int64_t x = row_blocks(D, f32, kScanThreads);
    if (x > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    return launch(f32 ? (lg ? scan_step_kernel<true, true> : scan_step_kernel<true, false>)
                      : (lg ? scan_step_kernel<false, true> : scan_step_kernel<false, false>),
                  p, dim3((unsigned)x, at_most(B, 65535)), kScanThreads, stream);
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
    int64_t ring;
    if (R < l_h || !mul_fits(R, D, eb, &ring) || !mul_fits(S, ring, 1, &n)) return HYENA_ERR_SHAPE;
    if (!slots && S < B) return HYENA_ERR_SHAPE;
    if (B == 0 || D == 0) return HYENA_OK;
    // offsets in a ring are 31 bits, rings are counted in 32
    if (ring > 0x7fffffff || S > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
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
    // The cut of the taps.  Filters of up to 32 taps: one wave, 4 taps a lane.
    // Few sequences: as many lanes as there can be (B = 1, l_h = 128, D = 4096
    // bf16, one filter for 16 channels: 4.7 us).  Once that is more waves than the
    // card holds, 16 taps a lane (B = 64: 15.5 us against 19.0 with 4 and 17.7
    // with 8); 8 where a lane's channels have filters of their own, whose taps
    // take registers too (27.5 us against 33.1 with 16).
    const bool f32 = dtype == HYENA_DTYPE_F32, single = l_h <= 32;
    const bool one = group_size % (f32 ? 4 : 8) == 0;
    const bool many = !single && ceil_div(D, f32 ? 32 : 64) * B > 1024;
    const int64_t x = row_blocks(D, f32, single || (many && one) ? 32 : many ? 16 : 8);
    if (x > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)x, at_most(B, 65535));
#define CONV_STEP(W, TAPS, ONE) \
    launch(f32 ? conv_step_kernel<true, W, TAPS, ONE> : conv_step_kernel<false, W, TAPS, ONE>, p, grid, 256, stream)
    if (one) return single ? CONV_STEP(1, 4, true) : many ? CONV_STEP(1, 16, true) : CONV_STEP(4, 4, true);
    return single ? CONV_STEP(1, 4, false) : many ? CONV_STEP(2, 8, false) : CONV_STEP(4, 4, false);
#undef CONV_STEP
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
    const bool f32 = dtype == HYENA_DTYPE_F32;
    const int64_t x = row_blocks(D, f32, kScanThreads);
    if (x > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    return launch(f32 ? cache_fill_kernel<true> : cache_fill_kernel<false>, p,
                  dim3((unsigned)x, at_most(R < L ? R : L, 65535), at_most(B, 65535)), kScanThreads, stream);
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
    case HYENA_ERR_UNSUPPORTED: return "unknown gate or activation code, a ring of 2 GiB or more, or a grid too large to launch";
    case HYENA_ERR_LAUNCH: return "kernel launch failed";
    case HYENA_ERR_DTYPE: return "unknown dtype code";
    case HYENA_ERR_WORKSPACE: return "workspace missing or smaller than the operator's workspace call reports";
    default: return "unknown status";
    }
}

}  // extern "C"
