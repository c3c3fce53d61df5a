// Layer norm and root-mean-square norm over the channels of a row, forward and
// backward, for MI355X (gfx950) (hyena_model.h has the formulas and layouts).
//
// Both directions are bound by memory: the forward reads and writes a row once,
// the backward reads x and dy and writes dx.  A row is held in the registers of
// T lanes (a wave, a workgroup of 4 waves or one of 16, by the row's length), 16 bytes
// a lane and chunk, so that mean, deviations and output come from one read; the
// workgroups walk the rows with the next one's loads in flight, past the caches.
// 8192 x 4096 bf16: forward 23.5 us (134 MB, 5.7 TB/s; at 32768 rows 5.9), backward
// 43 us (201 MB, 4.7 TB/s; of it 4 to 5 us the launch that adds the workgroups' sums
// for dw and db; at 32768 rows 5.4).  The longest rows' forms do not hold w and b beside
// a row and the next one: the compiler keeps some 100 bytes a lane of them in scratch (bf16
// forward, 1024 x 4 chunks) or up to 48 (backward, 1024 x 2), and 2048 x 24576 takes 85 us
// forward (2.4 TB/s), 2048 x 16384 backward 53 (3.8).  Without the streaming accesses and the loads
// ahead the forward took 28.5 us.

#include "hyena_model.h"
#include "layer_gemm.h"

namespace layer {
namespace {

struct NormParams {
    const void *x, *w, *b, *dy;
    void *y;                 // forward: y, backward: dx
    float *mean, *rstd;      // forward: outputs or null
    const float *mean_in, *rstd_in;
    float *sums;             // backward: [blocks][2][D] partial sums of dw and db
    float *dots;             // backward of wide rows: [M][2]
    void *dw, *db;
    int64_t M, ldx, ldy, lddy;
    int64_t D;
    float eps;
    int rms, want_dw, want_db;
};

template <bool F32> constexpr int kVec = F32 ? 4 : 8;  // values of 16 bytes

// The sums over the T lanes that share a row.  `lds` is the row's own: [2][T /
// 64] values a call; calls alternate between two areas (`turn`), so that one barrier each
// is enough.
template <int T, int N> __device__ inline void row_sums(float (&s)[N], float *lds, int turn) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = wave_sum(s[k]);
    if constexpr (T > 64) {
        constexpr int W = T / 64;
        float *at = lds + (turn & 1) * N * W;
        const int wave = threadIdx.x / 64 % W;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) at[k * W + wave] = s[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            s[k] = 0.0f;
#pragma unroll
            for (int v = 0; v < W; ++v) s[k] += at[k * W + v];
        }
    }
}

// Chunk c of a lane of T: values (c T + lane) V .. of the row.  WHOLE: the row is
// T CH V values long, and no chunk needs a look at its end.
template <bool F32, int T, int CH, bool WHOLE> struct RowOf {
    static constexpr int V = kVec<F32>;
    Pack<F32, V> r[CH];
    // Values of chunk c that belong to the row.
    __device__ static int count(int c, int lane, int D) {
        return WHOLE ? V : max(min(D - (c * T + lane) * V, V), 0);
    }
    template <bool STREAM> __device__ void load(const void *p, int64_t at, int lane, int D) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = count(c, lane, D);
            r[c] = n > 0 ? Pack<F32, V>::template load<STREAM>(p, at + (c * T + lane) * V, n) : Pack<F32, V>::zero();
        }
    }
};

// The forward.  T lanes a row, NT / T rows a workgroup at a time; workgroups walk
// the rows and keep w and b in registers.
template <bool F32, int T, int CH, int NT, bool WHOLE> __global__ __launch_bounds__(NT) void norm_fwd_kernel(NormParams p) {
    using R = RowOf<F32, T, CH, WHOLE>;
    constexpr int V = kVec<F32>, ROWS = NT / T;
    __shared__ float lds[T > 64 ? 2 * ROWS * (T / 64) : 1];
    const int lane = threadIdx.x % T, sub = threadIdx.x / T, D = (int)p.D;
    float *area = lds + sub * 2 * (T / 64);
    R w, b;
    if (p.w) w.template load<false>(p.w, 0, lane, D);
    if (p.b) b.template load<false>(p.b, 0, lane, D);
    const float inv = 1.0f / (float)D;
    int turn = 0;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t m = (int64_t)blockIdx.x * ROWS + sub;
    R next;
    if (m < p.M) next.template load<true>(p.x, m * p.ldx, lane, D);
    // T > 64: one row a workgroup, so that every wave takes part in each barrier
    for (; m < p.M; m += step) {
        const R x = next;
        if (m + step < p.M) next.template load<true>(p.x, (m + step) * p.ldx, lane, D);
        float s[1] = {0.0f}, mean = 0.0f;
        if (!p.rms) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] += x.r[c].get(e);
            row_sums<T>(s, area, turn++);
            mean = s[0] * inv;
        }
        s[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = R::count(c, lane, D);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = WHOLE || e < n ? x.r[c].get(e) - mean : 0.0f;
                s[0] += d * d;
            }
        }
        row_sums<T>(s, area, turn++);
        const float rstd = 1.0f / sqrtf(s[0] * inv + p.eps);
        if (lane == 0) {
            if (p.mean) p.mean[m] = mean;
            if (p.rstd) p.rstd[m] = rstd;
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = R::count(c, lane, D);
            if (n <= 0) continue;
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[e] = (x.r[c].get(e) - mean) * rstd;
                if (p.w) y[e] *= w.r[c].get(e);
                if (p.b) y[e] += b.r[c].get(e);
            }
            Pack<F32, V>::template store<true>(p.y, m * p.ldy + (c * T + lane) * V, n, y);
        }
    }
}

// Rows longer than registers hold: read three times (the second and third come
// from the caches), a workgroup of 1024 a row.
constexpr int kWide = 1024;
template <bool F32> __global__ __launch_bounds__(kWide) void norm_fwd_wide_kernel(NormParams p) {
    constexpr int V = kVec<F32>;
    __shared__ float lds[2 * (kWide / 64)];
    const float inv = 1.0f / (float)p.D;
    int turn = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        float s[1] = {0.0f}, mean = 0.0f;
        if (!p.rms) {
            for (int64_t d = (int64_t)threadIdx.x * V; d < p.D; d += kWide * V) {
                const auto x = Pack<F32, V>::load(p.x, m * p.ldx + d, (int)min(p.D - d, (int64_t)V));
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] += x.get(e);
            }
            row_sums<kWide>(s, lds, turn++);
            mean = s[0] * inv;
        }
        s[0] = 0.0f;
        for (int64_t d = (int64_t)threadIdx.x * V; d < p.D; d += kWide * V) {
            const int n = (int)min(p.D - d, (int64_t)V);
            const auto x = Pack<F32, V>::load(p.x, m * p.ldx + d, n);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float t = e < n ? x.get(e) - mean : 0.0f;
                s[0] += t * t;
            }
        }
        row_sums<kWide>(s, lds, turn++);
        const float rstd = 1.0f / sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[m] = mean;
            if (p.rstd) p.rstd[m] = rstd;
        }
        for (int64_t d = (int64_t)threadIdx.x * V; d < p.D; d += kWide * V) {
            const int n = (int)min(p.D - d, (int64_t)V);
            const auto x = Pack<F32, V>::load(p.x, m * p.ldx + d, n);
            const auto w = p.w ? Pack<F32, V>::load(p.w, d, n) : Pack<F32, V>::zero();
            const auto b = p.b ? Pack<F32, V>::load(p.b, d, n) : Pack<F32, V>::zero();
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[e] = (x.get(e) - mean) * rstd;
                if (p.w) y[e] *= w.get(e);
                if (p.b) y[e] += b.get(e);
            }
            Pack<F32, V>::store(p.y, m * p.ldy + d, n, y);
        }
    }
}

// The backward.  As the forward, with the sums over rows that dw and db want kept
// in registers, a lane's columns being the same in every row, and written once a
// workgroup; column_sums_kernel adds the workgroups'.  A row's loads go out before the
// row before it is finished.
template <bool F32, int T, int CH, int NT, bool WHOLE> __global__ __launch_bounds__(NT) void norm_bwd_kernel(NormParams p) {
    using R = RowOf<F32, T, CH, WHOLE>;
    constexpr int V = kVec<F32>, ROWS = NT / T;
    __shared__ float lds[T > 64 ? 4 * ROWS * (T / 64) : 1];
    __shared__ float joint[ROWS > 1 ? T * V : 1];
    const int lane = threadIdx.x % T, sub = threadIdx.x / T, D = (int)p.D;
    float *area = lds + sub * 4 * (T / 64);
    R w;
    if (p.w) w.template load<false>(p.w, 0, lane, D);
    float dw[CH][V] = {}, db[CH][V] = {};
    const float inv = 1.0f / (float)D;
    int turn = 0;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t m = (int64_t)blockIdx.x * ROWS + sub;
    R x, dy;
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](int64_t m) {
        if (m >= p.M) return;
        x.template load<true>(p.x, m * p.ldx, lane, D);
        dy.template load<true>(p.dy, m * p.lddy, lane, D);
        mean = p.rms ? 0.0f : p.mean_in[m];
        rstd = p.rstd_in[m];
    };
    fetch(m);
    // T > 64: one row a workgroup, so that every wave takes part in each barrier
    for (; m < p.M; m += step) {
        float s[2] = {0.0f, 0.0f};
        float u[CH][V], g[CH][V];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = R::count(c, lane, D);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                u[c][e] = WHOLE || e < n ? (x.r[c].get(e) - mean) * rstd : 0.0f;
                const float d = dy.r[c].get(e);
                g[c][e] = p.w ? d * w.r[c].get(e) : d;
                s[0] += g[c][e];
                s[1] += g[c][e] * u[c][e];
                dw[c][e] += d * u[c][e];
                db[c][e] += d;
            }
        }
        const float r = rstd;
        fetch(m + step);
        if (!p.y) continue;
        row_sums<T>(s, area, turn++);
        const float c0 = p.rms ? 0.0f : s[0] * inv, c1 = s[1] * inv;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = R::count(c, lane, D);
            if (n <= 0) continue;
            float dx[V];
#pragma unroll
            for (int e = 0; e < V; ++e) dx[e] = r * (g[c][e] - c0 - u[c][e] * c1);
            Pack<F32, V>::template store<true>(p.y, m * p.ldy + (c * T + lane) * V, n, dx);
        }
    }
    if (!p.sums) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!(k ? p.want_db : p.want_dw)) continue;
        float *to = p.sums + ((int64_t)blockIdx.x * 2 + k) * p.D;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float (&mine)[V] = k ? db[c] : dw[c];
            if constexpr (ROWS > 1) {  // the row groups in turn, in a fixed order
                for (int r = 0; r < ROWS; ++r) {
                    __syncthreads();
                    if (sub == r) {
#pragma unroll
                        for (int e = 0; e < V; ++e) joint[lane * V + e] = (r ? joint[lane * V + e] : 0.0f) + mine[e];
                    }
                }
                __syncthreads();
                if (sub == 0) {
#pragma unroll
                    for (int e = 0; e < V; ++e) mine[e] = joint[lane * V + e];
                }
            }
            const int n = R::count(c, lane, D);
            if (sub == 0 && n > 0) Pack<true, V>::store(to, (c * T + lane) * V, n, mine);
        }
    }
}

// Long rows: the two sums of each row first (a workgroup a row) ...
template <bool F32> __global__ __launch_bounds__(kWide) void norm_dots_kernel(NormParams p) {
    constexpr int V = kVec<F32>;
    __shared__ float lds[4 * (kWide / 64)];
    int turn = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const float mean = p.rms ? 0.0f : p.mean_in[m], rstd = p.rstd_in[m];
        float s[2] = {0.0f, 0.0f};
        for (int64_t d = (int64_t)threadIdx.x * V; d < p.D; d += kWide * V) {
            const int n = (int)min(p.D - d, (int64_t)V);
            const auto x = Pack<F32, V>::load(p.x, m * p.ldx + d, n), dy = Pack<F32, V>::load(p.dy, m * p.lddy + d, n);
            const auto w = p.w ? Pack<F32, V>::load(p.w, d, n) : Pack<F32, V>::zero();
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float g = p.w ? dy.get(e) * w.get(e) : dy.get(e);
                s[0] += g;
                s[1] += e < n ? g * ((x.get(e) - mean) * rstd) : 0.0f;
            }
        }
        row_sums<kWide>(s, lds, turn++);
        if (threadIdx.x == 0) {
            p.dots[2 * m] = p.rms ? 0.0f : s[0] / (float)p.D;
            p.dots[2 * m + 1] = s[1] / (float)p.D;
        }
    }
}
// ... then dx and the sums over rows, 256 lanes of columns by a run of rows a workgroup.
template <bool F32> __global__ __launch_bounds__(256) void norm_bwd_wide_kernel(NormParams p) {
    constexpr int V = kVec<F32>;
    const int64_t d = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (d >= p.D) return;
    const int n = (int)min(p.D - d, (int64_t)V);
    const int64_t per = ceil_div(p.M, gridDim.y), first = blockIdx.y * per, last = min(p.M, first + per);
    const auto w = p.w ? Pack<F32, V>::load(p.w, d, n) : Pack<F32, V>::zero();
    float dw[V] = {}, db[V] = {};
    for (int64_t m = first; m < last; ++m) {
        const float mean = p.rms ? 0.0f : p.mean_in[m], rstd = p.rstd_in[m];
        const float c0 = p.y ? p.dots[2 * m] : 0.0f, c1 = p.y ? p.dots[2 * m + 1] : 0.0f;
        const auto x = Pack<F32, V>::load(p.x, m * p.ldx + d, n), dy = Pack<F32, V>::load(p.dy, m * p.lddy + d, n);
        float dx[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float u = (x.get(e) - mean) * rstd, t = dy.get(e);
            const float g = p.w ? t * w.get(e) : t;
            dx[e] = rstd * (g - c0 - u * c1);
            dw[e] += t * u;
            db[e] += t;
        }
        if (p.y) Pack<F32, V>::store(p.y, m * p.ldy + d, n, dx);
    }
    if (!p.sums) return;
    float *to = p.sums + (int64_t)blockIdx.y * 2 * p.D;
    if (p.want_dw) Pack<true, V>::store(to, d, n, dw);
    if (p.want_db) Pack<true, V>::store(to + p.D, d, n, db);
}

// dw and db from the workgroups' sums: 64 columns by 16 lanes each.
struct ColumnSums {
    const float *from;  // [n][2][D]
    void *to[2];
    int64_t D;
    int n;
};
template <bool F32> __global__ __launch_bounds__(1024) void column_sums_kernel(ColumnSums p) {
    __shared__ float part[16][64];
    void *to = p.to[blockIdx.z];
    if (!to) return;
    const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
    const int64_t d = (int64_t)block_of() * 64 + c;
    float s = 0.0f;
    if (d < p.D) {
#pragma unroll 8
        for (int i = r; i < p.n; i += 16) s += p.from[((int64_t)i * 2 + blockIdx.z) * p.D + d];
    }
    part[r][c] = s;
    __syncthreads();
    if (r == 0 && d < p.D) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][c];
        store1<F32>(to, d, s);
    }
}

// ---- host --------------------------------------------------------------------------------

// Lanes and chunks of a row of D values, and the workgroups that walk the rows; 0
// chunks: longer than registers hold.  us, bf16 unless said:
//   forward  8192 x 4096: 256 lanes x 2 chunks 24.3 with 768 workgroups, 24.6 with
//            1024, 27.2 with 2048, and 38 with a wave a row (275 registers); 8192 x
//            2048: a wave x 4 14.6, 256 lanes x 1 18.6; 8192 x 1024 fp32 13.7 against
//            17.8; 8192 x 8192: 256 x 4 46, 1024 x 1 50; 8192 x 16384: 256 x 8 and
//            1024 x 2 92 and 91
//   backward 8192 x 4096: 256 x 2 45.0 with 256 workgroups, 45.6 with 512, 48.7 with
//            768, 1000 x 4096: 14.6 with 256, 19.3 with 512 (each leaves a row of sums
//            to be read again); 1024 x 1 48.3; 8192 x 2048: 256 x 1 26.7 with 512, 34.8
//            with 256; 8192 x 1000: a wave x 2 18.3, 256 x 1 24.8; 8192 x 8192: 1024 x 1
//            with 256 74.7, 256 x 4 75.8
struct Form {
    int lanes, chunks, blocks;
};
Form form_of(int64_t D, bool f32, bool backward) {
    static const Form fwd[] = {{64, 1, 1024}, {64, 2, 1024}, {64, 4, 1024}, {256, 2, 768}, {256, 4, 768}, {256, 8, 768}, {1024, 4, 512}};
    static const Form bwd[] = {{64, 1, 256}, {64, 2, 256}, {256, 1, 512}, {256, 2, 256}, {1024, 1, 256}, {1024, 2, 256}};
    const int64_t n = ceil_div(D, f32 ? 4 : 8);
    if (backward) {
        for (const Form &f : bwd)
            if (n <= (int64_t)f.lanes * f.chunks) return f;
        return Form{kWide, 0, 256};
    }
    for (const Form &f : fwd)
        if (n <= (int64_t)f.lanes * f.chunks) return f;
    return Form{kWide, 0, 2048};
}
// Workgroups for M rows, four at a time where a row is a wave's.
int blocks_of(const Form &f, int64_t M) {
    const int64_t groups = ceil_div(M, f.lanes == 64 ? 4 : 1);
    return (int)(groups < f.blocks ? groups : f.blocks);
}

template <bool F32> int launch_fwd(const NormParams &p, hipStream_t stream) {
    const Form f = form_of(p.D, F32, false);
    const dim3 grid(blocks_of(f, p.M));
    const bool whole = p.D == (int64_t)f.lanes * f.chunks * kVec<F32>;
#define FWD(T, CH, NT)                                                                                                \
    if (f.lanes == T && f.chunks == CH) {                                                                             \
        hipLaunchKernelGGL((whole ? norm_fwd_kernel<F32, T, CH, NT, true> : norm_fwd_kernel<F32, T, CH, NT, false>),  \
                           grid, dim3(NT), 0, stream, p);                                                             \
        return launch_status();                                                                                       \
    }
    FWD(64, 1, 256) FWD(64, 2, 256) FWD(64, 4, 256) FWD(256, 2, 256) FWD(256, 4, 256) FWD(256, 8, 256) FWD(1024, 4, 1024)
#undef FWD
    hipLaunchKernelGGL(norm_fwd_wide_kernel<F32>, grid, dim3(kWide), 0, stream, p);
    return launch_status();
}

template <bool F32> int launch_bwd(NormParams p, char *ws, hipStream_t stream) {
    const Form f = form_of(p.D, F32, true);
    const bool sums = p.want_dw || p.want_db;
    int blocks = 0, st = HYENA_OK;
    if (p.M > 0) {
        if (f.chunks == 0) {
            p.dots = (float *)ws;
            ws += ceil_div(p.M * 8, 16) * 16;
            p.sums = sums ? (float *)ws : nullptr;
            if (p.y) {
                hipLaunchKernelGGL(norm_dots_kernel<F32>, dim3((unsigned)(p.M < 2048 ? p.M : 2048)), dim3(kWide), 0, stream, p);
                if ((st = launch_status()) != HYENA_OK) return st;
            }
            blocks = blocks_of(f, p.M);
            hipLaunchKernelGGL(norm_bwd_wide_kernel<F32>, dim3((unsigned)ceil_div(p.D, 256 * kVec<F32>), blocks), dim3(256), 0,
                               stream, p);
        } else {
            p.sums = sums ? (float *)ws : nullptr;
            blocks = blocks_of(f, p.M);
            const dim3 grid(blocks);
            const bool whole = p.D == (int64_t)f.lanes * f.chunks * kVec<F32>;
#define BWD(T, CH, NT)                                                                                                \
    if (f.lanes == T && f.chunks == CH)                                                                               \
        hipLaunchKernelGGL((whole ? norm_bwd_kernel<F32, T, CH, NT, true> : norm_bwd_kernel<F32, T, CH, NT, false>),  \
                           grid, dim3(NT), 0, stream, p);
            BWD(64, 1, 256) BWD(64, 2, 256) BWD(256, 1, 256) BWD(256, 2, 256) BWD(1024, 1, 1024) BWD(1024, 2, 1024)
#undef BWD
        }
        if ((st = launch_status()) != HYENA_OK) return st;
    }
    if (!sums) return HYENA_OK;
    ColumnSums c = {};
    c.from = p.sums, c.to[0] = p.want_dw ? p.dw : nullptr, c.to[1] = p.want_db ? p.db : nullptr;
    c.D = p.D, c.n = blocks;
    dim3 grid = grid_of(ceil_div(p.D, 64));
    grid.z = 2;
    hipLaunchKernelGGL(column_sums_kernel<F32>, grid, dim3(1024), 0, stream, c);
    return launch_status();
}

int check_norm(int64_t M, int64_t D, int dtype) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    int64_t n;
    // 64 columns a workgroup, and the sums of 512 workgroups, have to fit
    if (!mul_fits(M, D, 64, &n) || !mul_fits(D, 512 * 8, 16, &n) || D > (int64_t)1 << 31) return HYENA_ERR_SHAPE;
    return HYENA_OK;
}

}  // namespace
}  // namespace layer

using namespace layer;

extern "C" {

int hyena_norm_workspace(int64_t M, int64_t D, int dtype, int64_t *bytes_out) {
    const int st = check_norm(M, D, dtype);
    if (st != HYENA_OK) return st;
    if (!bytes_out) return HYENA_ERR_NULL;
    const Form f = form_of(D, dtype == HYENA_DTYPE_F32, true);
    const int64_t blocks = blocks_of(f, M);
    *bytes_out = D == 0 ? 0 : (f.chunks == 0 ? ceil_div(M * 8, 16) * 16 : 0) + ceil_div(blocks * D * 8, 16) * 16;
    return HYENA_OK;
}

int hyena_norm_fwd(const void *x, const void *w, const void *b, int64_t M, int64_t D, int64_t ldx, int64_t ldy,
                   int kind, float eps, void *y, float *mean, float *rstd, int dtype, void *stream) {
    int st = check_norm(M, D, dtype);
    if (st != HYENA_OK) return st;
    if (kind != HYENA_NORM_LAYER && kind != HYENA_NORM_RMS) return HYENA_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f) || eps > 3.4e38f || (kind == HYENA_NORM_RMS && mean)) return HYENA_ERR_UNSUPPORTED;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (ldx < D || ldy < D || !mul_fits(M, ldx, eb, &n) || !mul_fits(M, ldy, eb, &n)) return HYENA_ERR_SHAPE;
    if (M == 0 || D == 0) return HYENA_OK;
    if (!x || !y) return HYENA_ERR_NULL;
    if (!aligned(x, eb) || !aligned(w, eb) || !aligned(b, eb) || !aligned(y, eb) || !aligned(mean, 4) || !aligned(rstd, 4))
        return HYENA_ERR_ALIGN;
    const Rows in[3] = {{x, M, D * eb, ldx * eb}, {w, 1, D * eb, D * eb}, {b, 1, D * eb, D * eb}};
    const Rows out[3] = {{y, M, D * eb, ldy * eb}, {mean, 1, M * 4, M * 4}, {rstd, 1, M * 4, M * 4}};
    for (int i = 0; i < 3; ++i) {
        for (const Rows &r : in)
            if (overlap(out[i], r)) return HYENA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HYENA_ERR_ALIAS;
    }
    NormParams p = {};
    p.x = x, p.w = w, p.b = b, p.y = y, p.mean = mean, p.rstd = rstd;
    p.M = M, p.D = D, p.ldx = ldx, p.ldy = ldy, p.eps = eps, p.rms = kind == HYENA_NORM_RMS;
    return dtype == HYENA_DTYPE_F32 ? launch_fwd<true>(p, (hipStream_t)stream) : launch_fwd<false>(p, (hipStream_t)stream);
}

int hyena_norm_bwd(const void *x, const void *w, const void *dy, const float *mean, const float *rstd, int64_t M,
                   int64_t D, int64_t ldx, int64_t lddy, int64_t lddx, int kind, void *dx, void *dw, void *db,
                   void *workspace, int64_t workspace_bytes, int dtype, void *stream) {
    int st = check_norm(M, D, dtype);
    if (st != HYENA_OK) return st;
    if (kind != HYENA_NORM_LAYER && kind != HYENA_NORM_RMS) return HYENA_ERR_UNSUPPORTED;
    if (kind == HYENA_NORM_RMS && mean) return HYENA_ERR_UNSUPPORTED;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (ldx < D || lddy < D || (dx && lddx < D) || !mul_fits(M, ldx, eb, &n) || !mul_fits(M, lddy, eb, &n) ||
        (dx && !mul_fits(M, lddx, eb, &n)))
        return HYENA_ERR_SHAPE;
    if (D == 0) return HYENA_OK;
    if (!dx && !dw && !db) return M > 0 ? HYENA_ERR_NULL : HYENA_OK;
    if (M > 0 && (!x || !dy || !rstd || (kind == HYENA_NORM_LAYER && !mean))) return HYENA_ERR_NULL;
    if (!aligned(x, eb) || !aligned(w, eb) || !aligned(dy, eb) || !aligned(dx, eb) || !aligned(dw, eb) ||
        !aligned(db, eb) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
        return HYENA_ERR_ALIGN;
    int64_t need = 0;
    hyena_norm_workspace(M, D, dtype, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const Rows in[5] = {{x, M, D * eb, ldx * eb}, {w, 1, D * eb, D * eb}, {dy, M, D * eb, lddy * eb},
                        {mean, 1, M * 4, M * 4}, {rstd, 1, M * 4, M * 4}};
    const Rows out[4] = {{dx, M, D * eb, lddx * eb}, {dw, 1, D * eb, D * eb}, {db, 1, D * eb, D * eb},
                         {need > 0 ? workspace : nullptr, 1, need, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Rows &r : in)
            if (overlap(out[i], r)) return HYENA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HYENA_ERR_ALIAS;
    }
    NormParams p = {};
    p.x = x, p.w = w, p.dy = dy, p.y = dx, p.mean_in = mean, p.rstd_in = rstd, p.dw = dw, p.db = db;
    p.want_dw = dw != nullptr, p.want_db = db != nullptr;
    p.M = M, p.D = D, p.ldx = ldx, p.ldy = lddx, p.lddy = lddy, p.rms = kind == HYENA_NORM_RMS;
    return dtype == HYENA_DTYPE_F32 ? launch_bwd<true>(p, (char *)workspace, (hipStream_t)stream)
                                    : launch_bwd<false>(p, (char *)workspace, (hipStream_t)stream);
}

}  // extern "C"
