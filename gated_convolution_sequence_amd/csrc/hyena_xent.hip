// Softmax cross entropy of a readout over a vocabulary, without keeping the
// logits, and its gradients, for MI355X (gfx950) (hyena_model.h has the formulas
// and layouts).
//
// Bound by the matrix cores: one product (2 M K V) forward and three backward,
// since the logits are formed again.  The products are layer_gemm.h's tiles.
//   * Rows without a target are left out: rank_kernel numbers the others in order,
//     and every product after that reads the number of rows from memory.  So such
//     rows cost no products, and what their x holds (NaN from padding) meets no zero in
//     dw's sums.  The logits fetch the rows from where they are; dw's sum runs over
//     rows, so for it pack_kernel copies them together.  Where rows are no whole 16
//     bytes they are copied for the logits as well, and w where its are not.
//   * Forward: a tile keeps the maximum and the sum of exp(z - maximum) of its
//     columns for each row, from the registers that hold the sums; merge_kernel
//     joins the tiles.
//   * Backward, a piece of the vocabulary at a time: the logits again, with e = p -
//     [target] as their epilogue (in bf16 rounded, as the matrix cores take it; db sums
//     dloss e unrounded), then dx += e w in fp32, times dloss and rounded after the last
//     piece, and dw = c e^T (dloss / c x), or c (dloss / c e)^T x where the entries are few;
//     c is the largest |dloss|.  dloss stays out of dx's e, so that the -1 of a target,
//     the largest part of a gradient where p is small, is exact; inside, its rounding
//     would be that of whole rows, and with a mean's equal dloss one factor (to 0.4 %
//     off) for all gradients.  Equal dloss leave dw's operands as they are.
//   * No more than 16 rows forward: the weights stream once through rows_product.

#include <initializer_list>

#include "hyena_model.h"
#include "layer_gemm.h"

namespace layer {
namespace {

// ---- maxima and sums of a softmax ---------------------------------------------------

// (m, s) stands for the values' maximum m and the sum of exp(z - m); where m is
// infinite, of exp(z), which is 0 (m = -inf: no value can occur) or inf.  exp is the hardware's
// 2^x of a rounded product: off by (|z - m| + 2) 2^-23 of a term, most where the term is small; errors
// against 64 bits are the same with exp's own function.
struct Part {
    float m, s;
};
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ inline float shift_of(float m) { return fabsf(m) == __builtin_inff() ? 0.0f : m; }
__device__ inline void join(Part &a, const Part &b) {
    const float m = fmaxf(a.m, b.m);
    a.s = a.s * (a.m == m ? 1.0f : __expf(a.m - m)) + b.s * (b.m == m ? 1.0f : __expf(b.m - m));
    a.m = m;
}

// K of the logits is not cut between workgroups, so fp32 logits are summed in runs of 256 of it, at
// no cost in time.  Relative errors of db against 64 bits, in one chain, in runs, and of PyTorch's products in fp32:
// 32 x 4096 x 256 1.5e-6, 1.9e-7, 5.5e-7; 64 x 16384 x 300 2.0e-6, 1.8e-7, 6.4e-7; 1024 x 4096 x 4096
// 2.8e-7, 5.9e-8, 3.1e-7.
constexpr int kLogitRun = 256;

// What a forward tile does with its sums.
struct StatsEpi {
    static constexpr bool kSums = true;
    static constexpr int kRun = kLogitRun;
    const void *bias;
    const int *target;  // of each packed row
    Part *part;         // [tiles of columns][ldp rows]
    float *at;          // the target's logit of each row
    int64_t ldp;
    int M, N;

    // columns(), before(), finish() and close() are not reached
    template <bool F32, int V> __device__ Pack<F32, V> columns(int) const { return Pack<F32, V>::zero(); }
    template <bool F32, int V> __device__ int before(int64_t, int) const { return 0; }
    template <bool F32, int V> __device__ void finish(int64_t, int, float (&)[V], const Pack<F32, V> &, int) const {}
    template <bool F32, int V> __device__ void close(const Pack<F32, V> &, int, int, int) const {}

    // A lane holds columns 16 u + 4 j + e of rows 16 t + i of its wave's part of the
    // tile: its own 16 columns first, then the four lanes of a row, then the waves.
    template <class S, class G, int MT, int NTL>
    __device__ __forceinline__ void sums(const G &p, f32x4_t (&acc)[MT][NTL], int m0, int n0, int wm, int wn,
                                         LDS_PTR unsigned char *lds) const {
        constexpr bool F32 = S::CE == 4;
        constexpr int WN = S::BN / (NTL * 16);
        const int i = threadIdx.x & 15, j = (threadIdx.x >> 4) & 3;
        const int tn = n0 / S::BN;
        LDS_PTR f32x2_t *meet = (LDS_PTR f32x2_t *)lds;
        const int first = n0 + wn + j * 4;
        const bool edge = n0 + S::BN > N;  // columns past the vocabulary
        float b[NTL][4];
#pragma unroll
        for (int u = 0; u < NTL; ++u) {
            const int left = N - (first + u * 16);
            const auto r = bias && left > 0 ? Pack<F32, 4>::load(bias, first + u * 16, left) : Pack<F32, 4>::zero();
#pragma unroll
            for (int e = 0; e < 4; ++e) b[u][e] = r.get(e);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = m0 + wm + t * 16 + i;
            const int goal = m < M ? target[m] : -1;
            Part r = {-__builtin_inff(), 0.0f};
            float hit = 0.0f;
            bool here = false;
#pragma unroll
            for (int u = 0; u < NTL; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = first + u * 16 + e;
                    acc[t][u][e] += b[u][e];
                    if (edge && n >= N) acc[t][u][e] = -__builtin_inff();
                    r.m = fmaxf(r.m, acc[t][u][e]);
                    if (n == goal) hit = acc[t][u][e], here = true;
                }
            r.m = fmaxf(r.m, __shfl_xor(r.m, 16));
            r.m = fmaxf(r.m, __shfl_xor(r.m, 32));
            const float shift = shift_of(r.m);
#pragma unroll
            for (int u = 0; u < NTL; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) r.s += __expf(acc[t][u][e] - shift);
            r.s += __shfl_xor(r.s, 16);
            r.s += __shfl_xor(r.s, 32);
            if (here) at[m] = hit;
            if (j == 0) {
                if constexpr (WN == 1) {
                    if (m < M) part[tn * ldp + m] = r;
                } else {
                    meet[(wn / (NTL * 16)) * S::BM + wm + t * 16 + i] = f32x2_t{r.m, r.s};
                }
            }
        }
        if constexpr (WN > 1) {
            __syncthreads();
            for (int row = threadIdx.x; row < S::BM; row += S::NT) {
                f32x2_t o = meet[row];
                Part r = {o[0], o[1]};
#pragma unroll
                for (int w = 1; w < WN; ++w) {
                    o = meet[w * S::BM + row];
                    join(r, Part{o[0], o[1]});
                }
                if (m0 + row < M) part[tn * ldp + m0 + row] = r;
            }
        }
    }
};

// The rows of `count` take the place of the upper bound that the host planned with.  Whether
// there is a tile for workgroup `block`.
template <class S, class E> __device__ inline bool rows_from(Gemm<E> &p, const int *count, int block) {
    p.M = *count;
    p.e.M = p.M;
    p.tiles_m = (p.M + S::BM - 1) / S::BM;
    return block < p.tiles_m * p.tiles_n * p.splits;
}

// The forward's logits.  8192 x 4096 x 65536 bf16 3.2 to 3.4 ms (1.28 to 1.36 PFLOP/s),
// bound as layer_gemm.h's products are: the matrix cores are busy in 62 % of all cycles, L2 gives
// 10 TB/s, memory 2.
template <bool F32, bool DIRECT, bool GATHER, typename S>
__global__ __launch_bounds__(S::NT, S::WAVES) void stats_kernel(Gemm<StatsEpi> p, const int *count, const int *apart) {
    TILE_BUFFERS(S)
    const int block = block_of();
    if ((apart && (*apart != 0) == GATHER) || !rows_from<S>(p, count, block)) return;
    run_tile<false, false, DIRECT, S, GATHER>(p, block, a0, a1, a2, a3, b0, b1, b2, b3);
}

// Few rows: 16 columns a workgroup; columns of four lanes a row.  Bound by the weights:
// 8 rows against 65536 x 4096 bf16 111 to 116 us (537 MB, 4.7 TB/s); 1, 2 or 4 steps in
// flight and 4, 8 or 16 waves lie within 3 %.
struct RowStats {
    const void *bias;
    const int64_t *target;
    Part *part;  // [rows][ldp groups of 16 columns]
    float *at;
    int64_t ldp;
    int M, N;
    template <bool F32, int V> __device__ Pack<F32, V> columns(int n) const {
        return bias && n < N ? Pack<F32, V>::load(bias, n, N - n) : Pack<F32, V>::zero();
    }
    template <bool F32, int V> __device__ int64_t before(int64_t m, int) const { return m < M ? target[m] : -1; }
    template <bool F32, int V>
    __device__ void finish(int64_t m, int n, float (&z)[V], const Pack<F32, V> &bias, int64_t goal) const {
        Part r = {-__builtin_inff(), 0.0f};
#pragma unroll
        for (int e = 0; e < V; ++e) {
            z[e] = n + e < N ? z[e] + bias.get(e) : -__builtin_inff();
            r.m = fmaxf(r.m, z[e]);
            if (n + e == goal) at[m] = z[e];
        }
        r.m = fmaxf(r.m, __shfl_xor(r.m, 1));
        r.m = fmaxf(r.m, __shfl_xor(r.m, 2));
        const float shift = shift_of(r.m);
#pragma unroll
        for (int e = 0; e < V; ++e) r.s += __expf(z[e] - shift);
        r.s += __shfl_xor(r.s, 1);
        r.s += __shfl_xor(r.s, 2);
        if ((threadIdx.x & 3) == 0 && m < M) part[m * ldp + n / 16] = r;
    }
    template <bool F32, int V> __device__ void close(const Pack<F32, V> &, int, int, int) const {}
};
template <bool F32> __global__ __launch_bounds__(64 * kRowWaves) void rows_stats_kernel(RowsParams<RowStats> p) {
    __shared__ __attribute__((aligned(16))) float sums[kRowWaves][1][16][16];
    const int block = block_of();
    if ((int64_t)block * 16 >= p.N) return;
    rows_product<F32, 1>(p, block, sums);
}

// Loss and lse of each row from its tiles, by SLICES lanes a row: 8192 rows of 256
// tiles in 8.5 us (17 MB).
struct MergeParams {
    const Part *part;
    const float *at;
    const int *index, *count;  // the packed rows' places and their number, or null:
    const int64_t *target;     // every row in place, those without a target among them
    float *loss, *lse;
    int64_t tile, row;         // parts from one tile, and from one row, to the next
    int64_t V;
    int tiles, M;
};
template <int SLICES> __global__ __launch_bounds__(256) void merge_kernel(MergeParams p) {
    constexpr int ROWS = 256 / SLICES;
    __shared__ Part meet[SLICES][ROWS];
    const int row = threadIdx.x % ROWS, slice = threadIdx.x / ROWS;
    const int64_t m = (int64_t)block_of() * ROWS + row, rows = p.count ? *p.count : p.M;
    Part r = {-__builtin_inff(), 0.0f};
    if (m < rows) {
#pragma unroll 4
        for (int t = slice; t < p.tiles; t += SLICES) join(r, p.part[t * p.tile + m * p.row]);
    }
    meet[slice][row] = r;
    for (int n = SLICES / 2; n > 0; n /= 2) {
        __syncthreads();
        if (slice < n) join(meet[slice][row], meet[slice + n][row]);
    }
    if (slice != 0 || m >= rows) return;
    r = meet[0][row];
    const int64_t to = p.index ? p.index[m] : m;
    const bool on = p.index || (uint64_t)p.target[m] < (uint64_t)p.V;
    // the loss from the logits' difference, which is exact where they are close, and not from lse: of
    // a nearly certain token among logits of thousands, lse's rounding would be most of it
    const float shift = shift_of(r.m), log_s = logf(r.s);
    p.loss[to] = on ? shift - p.at[m] + log_s : 0.0f;
    p.lse[to] = on ? shift + log_s : 0.0f;
}

// ---- rows with a target ----------------------------------------------------------------

// Numbers the rows that have a target, in order, and brings what belongs to them
// together; the others' loss and lse are 0.  A workgroup takes 8192 rows, and more than
// those are counted by a launch before.  5 to 8 us at 8192 rows.
struct RankParams {
    const int64_t *target;
    const float *lse_in, *dloss;  // backward
    float *lse_out, *dloss_out;   // packed
    float *loss, *lse;            // forward: zeroed where there is no target
    int *rank, *index, *goal, *count;
    int *apart;                   // cleared, for apart_kernel; or null
    float *most;                  // backward: the largest |dloss| of them (NaN where one is NaN or -inf)
    int *alike;                   // backward: whether all of them are that
    int *counts;                  // of each workgroup's rows (more than one workgroup)
    float *tops;                  // backward: the largest |dloss| there, and the least dloss
    int64_t V;
    int M;
};
constexpr int kRankRows = 8192;

// The sum (largest) over 1024 threads, in all of them; `lds` of 16 is free again after
// the next barrier.
template <class T, class F> __device__ inline T over_1024(T x, T *lds, F f) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x = f(x, __shfl_xor(x, o));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int w = 1; w < 16; ++w) x = f(x, lds[w]);
    return x;
}
__device__ inline int add(int a, int b) { return a + b; }
__device__ inline float larger(float a, float b) { return fmaxf(a, b); }
__device__ inline float lesser(float a, float b) { return fminf(a, b); }
// The largest |d| but for NaN, and the least d, with -inf for a NaN.
__device__ inline void bounds(float d, float &top, float &low) {
    top = fmaxf(top, fabsf(d));
    low = fminf(low, d == d ? d : -__builtin_inff());
}

__global__ __launch_bounds__(1024) void count_kernel(RankParams p) {
    __shared__ int sums[16];
    __shared__ float tops[16], lows[16];
    int n = 0;
    float top = 0.0f, low = __builtin_inff();
#pragma unroll
    for (int k = 0; k < kRankRows / 1024; ++k) {
        const int64_t m = (int64_t)blockIdx.x * kRankRows + k * 1024 + threadIdx.x;
        const bool on = m < p.M && (uint64_t)p.target[m] < (uint64_t)p.V;
        n += on;
        if (p.most && on) bounds(p.dloss[m], top, low);
    }
    n = over_1024(n, sums, add);
    if (threadIdx.x == 0) p.counts[blockIdx.x] = n;
    if (!p.most) return;
    top = over_1024(top, tops, larger);
    low = over_1024(low, lows, lesser);
    if (threadIdx.x == 0) p.tops[2 * blockIdx.x] = top, p.tops[2 * blockIdx.x + 1] = low;
}

__global__ __launch_bounds__(1024) void rank_kernel(RankParams p) {
    __shared__ int ahead[128];  // rows in the waves before, of the workgroup's 8 times 16
    __shared__ int first_half, both, sums[16];
    __shared__ float tops[16], lows[16];
    float top = 0.0f, low = __builtin_inff();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = (int64_t)blockIdx.x * kRankRows;
    int goal[8], before[8], base = 0;
    float lse[8], d[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t m = first + k * 1024 + threadIdx.x;
        const int64_t t = m < p.M ? p.target[m] : -1;
        if (p.lse_in) lse[k] = m < p.M ? p.lse_in[m] : 0.0f, d[k] = m < p.M ? p.dloss[m] : 0.0f;
        goal[k] = (uint64_t)t < (uint64_t)p.V ? (int)t : -1;
    }
    if (gridDim.x > 1) {
        for (int i = threadIdx.x; i < (int)blockIdx.x; i += 1024) base += p.counts[i];
        base = over_1024(base, sums, add);
        if (blockIdx.x == 0 && p.most)
            for (int i = threadIdx.x; i < (int)gridDim.x; i += 1024)
                top = fmaxf(top, p.tops[2 * i]), low = fminf(low, p.tops[2 * i + 1]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint64_t on = __builtin_amdgcn_ballot_w64(goal[k] >= 0);
        before[k] = __popcll(on & (((uint64_t)1 << lane) - 1));
        if (lane == 0) ahead[k * 16 + wave] = __popcll(on);
        if (gridDim.x == 1 && goal[k] >= 0 && p.most) bounds(d[k], top, low);
    }
    __syncthreads();
    if (wave < 2) {  // running sums of the 128 counts, 64 a wave
        const int mine = ahead[threadIdx.x];
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int other = __shfl_up(sum, o);
            if (lane >= o) sum += other;
        }
        ahead[threadIdx.x] = sum - mine;
        if (threadIdx.x == 63) first_half = sum;
        if (threadIdx.x == 127) both = sum;
    }
    __syncthreads();
    const int half = first_half;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t m = first + k * 1024 + threadIdx.x;
        if (m >= p.M) continue;
        const int at = base + (k >= 4 ? half : 0) + ahead[k * 16 + wave] + before[k];
        p.rank[m] = goal[k] >= 0 ? at : -1;
        if (goal[k] >= 0) {
            p.index[at] = (int)m;
            p.goal[at] = goal[k];
            if (p.lse_in) p.lse_out[at] = lse[k], p.dloss_out[at] = d[k];
        } else if (p.loss) {
            p.loss[m] = 0.0f, p.lse[m] = 0.0f;
        }
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
        *p.count = base + half + both;
        if (p.apart) *p.apart = 0;
    }
    if (!p.most || blockIdx.x != 0) return;
    top = over_1024(top, tops, larger);
    low = over_1024(low, lows, lesser);
    // a NaN, of which only `low` tells, has to reach what `most` scales: with the others 0,
    // their largest would leave a dw of 0
    if (threadIdx.x == 0) *p.most = low == -__builtin_inff() ? __builtin_nanf("") : top, *p.alike = low == top;
}

// Where x is 2 GiB or more, a tile's rows may lie further apart than its 32-bit offsets
// reach (a few with a target among very many without): then the rows are packed, and the
// products that gather them leave at once; else those of packed rows do.
__global__ __launch_bounds__(256) void apart_kernel(const int *index, const int *count, int reach, int *apart) {
    const int n = *count;
    const int64_t first = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 256;
    if (first < n && index[min(first + 255, (int64_t)n - 1)] - index[first] > reach) *apart = 1;
}

// Rows of x with a target to rows of whole 16 bytes, zeros behind them; dx of the
// others to zero; and w to such rows where its own are not.  A wave a row, 64 chunks of
// one where the rows are few, or several rows a wave where they are short.  8192 x 4096 bf16, dloss x only: 22 us (134 MB).
struct PackParams {
    const void *from[2];  // x, w (null: as it is)
    void *to[2];          // null: only what follows is wanted
    void *scaled;         // backward: dloss / most x of the rows as well
    const float *dloss, *most;
    int64_t rows[2], ld[2];
    const int *rank;
    const int *apart;     // to[0] only where it says so, or null
    const int *count;     // where all rows[0] have a target (and are not apart), nothing is copied; or null
    void *dx;
    int64_t lddx;
    int K, chunks, parts;
    int lanes;  // a power of two: of a row, where a wave takes several
};
enum PackMode { kPackRow, kPackParts, kPackShort };
template <bool F32, int MODE> __global__ __launch_bounds__(256) void pack_kernel(PackParams p) {
    constexpr bool PARTS = MODE == kPackParts, SHORT = MODE == kPackShort;
    using T = typename El<F32>::type;
    constexpr int CE = El<F32>::CE;
    // SHORT: rows of no more chunks than lanes, 256 / lanes of them a workgroup
    const int lane = SHORT ? threadIdx.x & (p.lanes - 1) : threadIdx.x & 63;
    const int rows = SHORT ? 256 / p.lanes : 4;
    const int64_t step = (int64_t)gridDim.x * rows;
    const int64_t start = (int64_t)blockIdx.x * rows + (SHORT ? threadIdx.x / p.lanes : threadIdx.x >> 6);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (!p.from[g] || (g == 0 && p.count && *p.count == p.rows[0] && !(p.apart && *p.apart))) continue;
        for (int64_t id = start; id < p.rows[g] * p.parts; id += step) {
            const int64_t row = PARTS ? id / p.parts : id;
            const int first = PARTS ? (int)(id - row * p.parts) * 64 + lane : lane;
            const int end = PARTS || SHORT ? min(first + 1, p.chunks) : p.chunks;
            const int64_t at = g == 0 ? p.rank[row] : row;
            if (at < 0) {
                if (p.dx) {
                    const float none[CE] = {};
                    for (int c = first; c < end; c += 64)
                        Pack<F32, CE>::store(p.dx, row * p.lddx + c * CE, p.K - c * CE, none);
                }
                continue;
            }
            void *const whole = g == 0 && p.apart && !p.count && *p.apart == 0 ? nullptr : p.to[g];
            if (!whole && !(g == 0 && p.scaled)) continue;  // only dx of the others
            const T *from = (const T *)p.from[g] + row * p.ld[g];
            u32x4_t *to = whole ? (u32x4_t *)whole + at * p.chunks : nullptr;
            u32x4_t *scaled = g == 0 && p.scaled ? (u32x4_t *)p.scaled + at * p.chunks : nullptr;
            const float by = scaled && *p.most != 0.0f ? p.dloss[row] / *p.most : 0.0f;
            auto put = [&](int c, u32x4_t v) {
                if (to) to[c] = v;
                if (scaled) {
                    float y[CE];
                    const auto r = Pack<F32, CE>::from(v);
#pragma unroll
                    for (int e = 0; e < CE; ++e) y[e] = by * r.get(e);
                    scaled[c] = __builtin_bit_cast(u32x4_t, Pack<F32, CE>::of(y).w[0]);
                }
            };
            const int full = p.K / CE;  // chunks inside the row
            const int stop = min(end, full);
            constexpr int U = MODE == kPackRow ? 4 : 1;  // loads ahead of the stores
            for (int c = first; c < stop; c += 64 * U) {
                u32x4_t v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + 64 * u < stop) v[u] = *(const typename El<F32>::chunk_any *)(from + (c + 64 * u) * CE);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + 64 * u < stop) put(c + 64 * u, v[u]);
            }
            if (full < end && full >= first && (full - first) % 64 == 0) {
                T x[CE];
#pragma unroll
                for (int e = 0; e < CE; ++e) x[e] = full * CE + e < p.K ? from[full * CE + e] : (T)0.0f;
                put(full, __builtin_bit_cast(u32x4_t, x));
            }
        }
    }
}

// ---- gradients ------------------------------------------------------------------------

// The logits' epilogue in the backward: e = p - [target] of a piece, and the column
// sums of dloss e.
struct DzEpi {
    static constexpr bool kSums = false;
    static constexpr int kRun = kLogitRun;
    const void *bias;           // of the piece
    const float *lse, *dloss;   // packed
    const int *target;          // packed, of the whole vocabulary
    void *dz;                   // e: [rows][ld], ld whole 16 bytes, zeros behind the columns
    void *scaled;               // the same times dloss / most, where not all dloss are alike; or null
    const float *most;
    const int *alike;
    float *sums;                // [row blocks][N] or null
    int64_t ld;
    int v0;                     // the piece's first entry
    int M, N;

    template <bool F32, int V> struct Columns {
        Pack<F32, V> bias;
        float sum[V];
    };
    struct Row {
        float lse, dloss, by;
        int target;
    };
    template <bool F32, int V> __device__ __forceinline__ Columns<F32, V> columns(int n) const {
        Columns<F32, V> c = {bias && n < N ? Pack<F32, V>::load(bias, n, N - n) : Pack<F32, V>::zero(), {}};
        return c;
    }
    template <bool F32, int V> __device__ __forceinline__ Row before(int64_t m, int) const {
        if (m >= M) return Row{};
        return Row{lse[m], dloss[m], scaled && *most != 0.0f ? dloss[m] / *most : 0.0f, target[m] - v0};
    }
    template <bool F32, int V>
    __device__ __forceinline__ void finish(int64_t m, int n, float (&z)[V], Columns<F32, V> &c, const Row &r) const {
        if (m >= M || n >= ld) return;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float p = __expf(z[e] + c.bias.get(e) - r.lse);
            z[e] = n + e < N ? (n + e == r.target ? p - 1.0f : p) : 0.0f;
            c.sum[e] += r.dloss * z[e];
        }
        Pack<F32, V>::store(dz, m * ld + n, (int)(ld - n), z);
        if (!scaled || *alike) return;
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] *= r.by;
        Pack<F32, V>::store(scaled, m * ld + n, (int)(ld - n), z);
    }
    template <bool F32, int V> __device__ __forceinline__ void close(const Columns<F32, V> &c, int m, int block, int n) const {
        if (!sums || m >= M) return;  // eight lanes a row, the wave's eight rows at a time
        float s[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s[e] = c.sum[e];
#pragma unroll
            for (int o = 8; o < 64; o <<= 1) s[e] += __shfl_xor(s[e], o);
        }
        if ((threadIdx.x & 63) < 8 && n < N) Pack<true, V>::store(sums, (int64_t)block * N + n, N - n, s);
    }
};

// The gradients' epilogue.  ACC: pieces of the vocabulary are added up in fp32, and
// rows are scaled and put in place by `index` at last.
template <bool ACC> struct GradEpi {
    static constexpr bool kSums = false;
    static constexpr int kRun = 0;
    void *y;
    const float *from;   // what the pieces before gave, or null
    float *to;           // where the sum goes, or null: y
    const int *index;
    const float *scale;  // ACC: packed, one a row; else one for all
    int64_t ldy;
    int M, N;

    template <bool F32, int V> struct Row {
        Pack<true, V> sum;
        int64_t at;
        float scale;
    };
    struct None {};
    template <bool F32, int V> __device__ __forceinline__ float columns(int) const { return ACC ? 0.0f : *scale; }
    template <bool F32, int V> __device__ __forceinline__ auto before(int64_t m, int n) const {
        if constexpr (ACC) {
            Row<F32, V> r = {Pack<true, V>::zero(), 0, 0.0f};
            if (m < M && n < N) {
                if (from) r.sum = Pack<true, V>::load(from, m * N + n, N - n);
                if (!to) r.at = index[m], r.scale = scale[m];
            }
            return r;
        } else {
            return None{};
        }
    }
    template <bool F32, int V, class R>
    __device__ __forceinline__ void finish(int64_t m, int n, float (&z)[V], float by, const R &r) const {
        if (m >= M || n >= N) return;
        if constexpr (ACC) {
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] += r.sum.get(e);
            if (to) return Pack<true, V>::store(to, m * N + n, N - n, z);
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] *= r.scale;
            Pack<F32, V>::store(y, r.at * ldy + n, N - n, z);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] *= by;
            Pack<F32, V>::store(y, m * ldy + n, N - n, z);
        }
    }
    template <bool F32, int V> __device__ __forceinline__ void close(float, int, int, int) const {}
};
using DwEpi = GradEpi<false>;
using DxEpi = GradEpi<true>;

// The backward's logits.  6144 rows, 8192 entries, K = 4096 bf16 341 us (1.21 PFLOP/s).
template <bool F32, bool DIRECT, bool GATHER, typename S>
__global__ __launch_bounds__(S::NT, S::WAVES) void dz_kernel(Gemm<DzEpi> p, const int *count, const int *apart) {
    TILE_BUFFERS(S)
    const int block = block_of();
    if ((apart && (*apart != 0) == GATHER) || !rows_from<S>(p, count, block)) return;
    run_tile<false, false, DIRECT, S, GATHER>(p, block, a0, a1, a2, a3, b0, b1, b2, b3);
}

// What dw is formed from where dloss is in e (see xent_bwd), as the rows turn out: e
// itself or e times dloss, x in place or packed.
struct DwFrom {
    const void *scaled, *x;  // scaled null: as the product says
    const int *alike, *apart;
    int64_t ldx;
    int M;
};

// dw's sum runs over the rows: their number, cut anew between the splits.
template <bool F32> __device__ inline void sum_from(Gemm<DwEpi> &p, const int *count, const DwFrom &f) {
    constexpr int BK = 8 * El<F32>::CE;
    p.C = *count;
    if (f.scaled) {
        if (!*f.alike) p.a = f.scaled;
        if (p.C == f.M && !(f.apart && *f.apart)) p.b = f.x, p.ldb = f.ldx;
    }
    const int steps = (p.C + BK - 1) / BK;
    p.c_per_split = max((steps + p.splits - 1) / p.splits, 1) * BK;
}

// The first `blocks` workgroups form dw, the others dx.
template <bool F32, bool DIRECT, typename S>
__global__ __launch_bounds__(S::NT, S::WAVES) void grads_kernel(Gemm<DwEpi> dw, Gemm<DxEpi> dx, int blocks, DwFrom from,
                                                                const int *count) {
    TILE_BUFFERS(S)
    const int id = block_of();
    if (id < blocks) {
        sum_from<F32>(dw, count, from);
        run_tile<true, true, DIRECT, S>(dw, id, a0, a1, a2, a3, b0, b1, b2, b3);
    } else {
        dx.M = dx.e.M = *count;
        dx.tiles_m = (dx.M + S::BM - 1) / S::BM;
        const int block = id - blocks;
        if (block >= dx.tiles_m * dx.tiles_n * dx.splits) return;
        run_tile<false, true, DIRECT, S>(dx, block, a0, a1, a2, a3, b0, b1, b2, b3);
    }
}
// The same in tiles of 256 x 256, whichever walks more steps a tile first: what is left
// of its last round is then filled by the other's shorter tiles.  (6144 rows, a piece of
// 16384 entries, K = 4096: dx's 384 tiles alone take two rounds of 256 units, 971 us,
// and dw's 1024 another 671; together 1440.  A piece of 8192: 682, 1.21 PFLOP/s.)
template <typename S>
__global__ __launch_bounds__(S::NT, S::WAVES) void large_grads_kernel(Gemm<DwEpi> dw, Gemm<DxEpi> dx, int lead, int dx_first,
                                                                      DwFrom from, const int *count) {
    TILE_BUFFERS(S)
    const int id = block_of();
    const bool in_lead = id < lead;
    const int block = in_lead ? id : id - lead;
    if (in_lead != (dx_first != 0)) {
        if (block >= dw.tiles_m * dw.tiles_n * dw.splits) return;
        sum_from<false>(dw, count, from);
        run_tile<true, true, true, S>(dw, block, a0, a1, a2, a3, b0, b1, b2, b3);
    } else {
        dx.M = dx.e.M = *count;
        dx.tiles_m = (dx.M + S::BM - 1) / S::BM;
        if (block >= dx.tiles_m * dx.tiles_n * dx.splits) return;
        run_tile<false, true, true, S>(dx, block, a0, a1, a2, a3, b0, b1, b2, b3);
    }
}

// What remains of a piece: the sums of splits, and db from the row blocks' sums.
struct JoinParams {
    Gemm<DwEpi> dw;
    Gemm<DxEpi> dx;
    int64_t blocks[2];
    const float *sums;
    const int *count;
    int rows;     // rows of a row block of the sums
    int columns;  // of db a workgroup: 2 to this power
    int N;
    void *db;
};
template <bool F32> __global__ __launch_bounds__(256) void join_kernel(JoinParams p) {
    __shared__ float part[256];
    int64_t block = blockIdx.x;
    const int count = *p.count;
    if (block < p.blocks[0]) return sum_splits<F32>(p.dw, block * 256 + threadIdx.x);
    block -= p.blocks[0];
    if (block < p.blocks[1]) {
        p.dx.M = p.dx.e.M = count;
        return sum_splits<F32>(p.dx, block * 256 + threadIdx.x);
    }
    block -= p.blocks[1];
    // 2^`columns` of them, up to 64, by the other threads
    const int columns = 1 << p.columns, c = threadIdx.x & (columns - 1), r = threadIdx.x >> p.columns;
    const int lanes = 256 >> p.columns, n_sums = (count + p.rows - 1) / p.rows;
    const int64_t n = (block << p.columns) + c;
    float s = 0.0f;
    if (n < p.N) {
#pragma unroll 8
        for (int b = r; b < n_sums; b += lanes) s += p.sums[(int64_t)b * p.N + n];
    }
    part[threadIdx.x] = s;
    for (int o = 128; o >= columns; o /= 2) {
        __syncthreads();
        if ((int)threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
    }
    if (r == 0 && n < p.N) store1<F32>(p.db, n, part[threadIdx.x]);
}

// ---- host --------------------------------------------------------------------------------

enum Tile { kLarge, kDeep, kSmall, kFineDeep, kFine };
Tile tile_of(const Plan &p) { return p.large ? kLarge : p.fine ? (p.deep ? kFineDeep : kFine) : p.deep ? kDeep : kSmall; }
// Rows of one wave, which leave one row of column sums: of a tile's WM x MT x 16.
int wave_rows(const Plan &p) { return p.large ? 128 : p.fine ? 16 : 64; }

// A product whose epilogue wants whole sums: its c is not cut, so tiles that fill the
// last round of units count for more than in plan_of.  fp32: 64 x 64 always (us, with
// 128 x 128 and with 64 x 64: 1021 x 776 x 5000 115 and 81, 600 x 2048 x 8192 261 and
// 179, 3000 x 1024 x 4000 227 and 208, 8192 x 4096 x 4096 2040 and 2026).  bf16: 256 x
// 256 where that is no more than 2/5 of the rounds of 128 x 128 (3000 x 1024 x 4000 38
// against 43, 4000 x 2048 x 2500 56 against 69; but with 2 rounds against 1, 600 x 2048
// x 8192, 55 against 38).
Plan whole_plan(int64_t M, int64_t N, int64_t K, bool f32, bool direct) {
    const Size sz = {M, N, K};
    Plan p = plan_of(&sz, 1, f32, direct);
    const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128), t256 = ceil_div(M, 256) * ceil_div(N, 256);
    if (f32) p.fine = true, p.deep = false;
    else if (direct && t256 >= 128 && 5 * ceil_div(t256, 256) <= 2 * ceil_div(t128, 256)) p.large = true, p.deep = false;
    const int edge = p.large ? 256 : p.fine ? 64 : 128;
    p.tiles_m[0] = (int)ceil_div(M, edge), p.tiles_n[0] = (int)ceil_div(N, edge);
    p.splits[0] = 1;
    p.c_per_split[0] = (int)(ceil_div(K, f32 ? 32 : 64) * (f32 ? 32 : 64));
    p.blocks[0] = (int64_t)p.tiles_m[0] * p.tiles_n[0];
    p.partial[0] = 0;
    return p;
}

// What lies in the workspace begins on whole cache lines, wherever the workspace does:
// operands whose 128-byte rows straddled two lines took 6 % longer (a forward of 8192 x
// 4096 x 65536 3.63 against 3.36 ms).
constexpr int64_t kLine = 256;
int64_t lines(int64_t n) { return ceil_div(n, kLine) * kLine; }
char *first_line(void *ws) { return (char *)(((uintptr_t)ws + kLine - 1) & ~(uintptr_t)(kLine - 1)); }

constexpr int64_t kFewRows = 16;  // rows_product's

int64_t rank_blocks(int64_t M) { return M > kRankRows ? ceil_div(M, kRankRows) : 1; }

// The forward's workspace.
struct FwdSpace {
    int64_t count, counts, rank, index, goal, at, part, x, w, total;
};
FwdSpace fwd_space(int64_t M, int64_t K, int64_t V, bool f32) {
    const int64_t eb = f32 ? 4 : 2;
    FwdSpace s = {};
    int64_t n = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = n;
        n += lines(bytes);
        return at;
    };
    if (M <= kFewRows) {
        s.at = take(M * 4), s.part = take(ceil_div(V, 16) * M * 8);
    } else {
        // w may lie at any element, which the caller of hyena_xent_workspace does not say
        const int64_t tiles[2] = {whole_plan(M, V, K, f32, false).tiles_n[0], whole_plan(M, V, K, f32, true).tiles_n[0]};
        s.count = take(8), s.counts = take(rank_blocks(M) * 4);
        s.rank = take(M * 4), s.index = take(M * 4), s.goal = take(M * 4), s.at = take(M * 4);
        s.part = take((tiles[0] > tiles[1] ? tiles[0] : tiles[1]) * M * 8);
        s.x = take(M * whole(K, eb) * eb);
        s.w = take(whole(K, eb) != K ? V * whole(K, eb) * eb : 0);
    }
    s.total = n + kLine - 16;  // to the first whole line
    return s;
}

// Entries of the vocabulary a piece of the backward takes: e of a piece is some 128 MB
// and stays in the last cache for its two products, or 2048 entries where the rows are
// many.  8192 rows, V = 65536 bf16: K = 4096 10.83 ms (256 MB 10.98, 512 MB 10.90), K =
// 1024 3.08 ms (3.44, 3.15).
int64_t piece_of(int64_t M, int64_t V, int64_t eb) {
    int64_t most = ((int64_t)1 << 27) / ((M > 0 ? M : 1) * eb) / 256 * 256;
    if (most < 2048) most = 2048;
    if (most > (int64_t)1 << 18) most = (int64_t)1 << 18;
    const int64_t pieces = ceil_div(V, most);
    return pieces == 1 ? V : ceil_div(ceil_div(V, pieces), 256) * 256;
}

struct BwdSpace {
    int64_t count, counts, tops, rank, index, goal, lse, dloss, x, scaled, w, dz, sums, acc, partial, total;
    int64_t piece;
};
BwdSpace bwd_space(int64_t M, int64_t K, int64_t V, bool f32) {
    const int64_t eb = f32 ? 4 : 2;
    BwdSpace s = {};
    int64_t n = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = n;
        n += lines(bytes);
        return at;
    };
    s.piece = piece_of(M, V, eb);
    s.count = take(16), s.counts = take(rank_blocks(M) * 4), s.tops = take(rank_blocks(M) * 8);
    s.rank = take(M * 4), s.index = take(M * 4), s.goal = take(M * 4);
    s.lse = take(M * 4), s.dloss = take(M * 4);
    s.x = take(M * whole(K, eb) * eb), s.scaled = take(M * whole(K, eb) * eb);  // x, or e of few entries
    s.w = take(whole(K, eb) != K ? V * whole(K, eb) * eb : 0);
    s.dz = take(M * whole(s.piece, eb) * eb);
    int64_t sums = 0, partial = 0;
    for (int64_t v0 = 0; v0 < V; v0 += s.piece) {  // the first and the last piece
        const int64_t N = V - v0 < s.piece ? V - v0 : s.piece;
        for (bool direct : {false, true}) {  // w may lie at any element
            const int64_t b = ceil_div(M, wave_rows(whole_plan(M, N, K, f32, direct))) * N * 4;
            if (b > sums) sums = b;
        }
        const Size both[2] = {{N, K, M}, {M, K, N}};
        for (int64_t bytes : {partial_bytes(both, 2, f32), partial_bytes(both, 1, f32), partial_bytes(both + 1, 1, f32)})
            if (bytes > partial) partial = bytes;
        if (v0 == 0 && V > s.piece) v0 = (ceil_div(V, s.piece) - 2) * s.piece;
    }
    s.sums = take(sums), s.acc = take(V > s.piece ? M * K * 4 : 0), s.partial = take(partial);
    s.total = n + kLine - 16;  // to the first whole line
    return s;
}

int launch_rank(const RankParams &r, hipStream_t stream) {
    const dim3 grid((unsigned)rank_blocks(r.M));
    if (grid.x > 1) {
        hipLaunchKernelGGL(count_kernel, grid, dim3(1024), 0, stream, r);
        const int st = launch_status();
        if (st != HYENA_OK) return st;
    }
    hipLaunchKernelGGL(rank_kernel, grid, dim3(1024), 0, stream, r);
    return launch_status();
}

template <bool F32> int launch_pack(PackParams p, hipStream_t stream) {
    int64_t rows = p.from[0] ? p.rows[0] : 0;
    if (p.from[1] && p.rows[1] > rows) rows = p.rows[1];
    if (rows == 0 || p.chunks == 0) return HYENA_OK;
    p.parts = rows < 1024 ? (int)ceil_div(p.chunks, 64) : 1;
    for (p.lanes = 1; p.lanes < p.chunks && p.lanes < 64;) p.lanes *= 2;
    const bool several = p.lanes < 64;
    const int64_t blocks = several ? ceil_div(rows, 256 / p.lanes) : ceil_div(rows * p.parts, 4);
    hipLaunchKernelGGL((several       ? pack_kernel<F32, kPackShort>
                        : p.parts > 1 ? pack_kernel<F32, kPackParts>
                                      : pack_kernel<F32, kPackRow>),
                       dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, p);
    return launch_status();
}

// LAUNCH(DIRECT, GATHER, S) for whole_plan's tiles.
#define FOR_TILE(plan, direct, gather, LAUNCH)                                               \
    if constexpr (F32) {                                                                     \
        if (direct) { BOTH(gather, LAUNCH, Fine<true>) } else { LAUNCH(false, false, Fine<true>) } \
    } else {                                                                                 \
        switch (tile_of(plan)) {                                                             \
        case kLarge: BOTH(gather, LAUNCH, Large) break;                                      \
        case kDeep: BOTH(gather, LAUNCH, Deep<false>) break;                                 \
        case kFineDeep: BOTH(gather, LAUNCH, FineDeep) break;                                \
        case kSmall:                                                                         \
            if (direct) { BOTH(gather, LAUNCH, Small<false>) } else { LAUNCH(false, false, Small<false>) } \
            break;                                                                           \
        case kFine:                                                                          \
            LAUNCH(false, false, Fine<false>)                                                \
            break;                                                                           \
        }                                                                                    \
    }
#define BOTH(gather, LAUNCH, S)                                      \
    if (gather) { LAUNCH(true, true, S) } else { LAUNCH(true, false, S) }

// Whether the logits can fetch the rows of x from where they are: whole aligned 16
// bytes, w as well (rows are gathered straight into LDS); and whether all lie within
// their offsets, or apart_kernel has to look.
bool gather_ok(const void *x, int64_t ldx, int64_t K, int64_t eb, const void *w) {
    return direct_ok(x, ldx, K, eb) && direct_ok(w, K, K, eb);
}
constexpr int64_t kReach = ((int64_t)1 << 31) - ((int64_t)1 << 23);  // a row is below 2^23 bytes
bool all_near(int64_t M, int64_t ldx, int64_t eb) { return M * ldx * eb <= kReach; }
int launch_apart(const RankParams &r, int64_t ldx, int64_t eb, hipStream_t stream) {
    hipLaunchKernelGGL(apart_kernel, dim3((unsigned)ceil_div(r.M, 256 * 256)), dim3(256), 0, stream, r.index, r.count,
                       (int)(kReach / (ldx * eb)) - 1, r.apart);
    return launch_status();
}

template <bool F32>
int xent_fwd(const void *x, const void *w, const void *bias, const int64_t *target, int64_t M, int64_t K, int64_t V,
             int64_t ldx, float *loss, float *lse, char *ws, hipStream_t stream) {
    const int64_t eb = F32 ? 4 : 2;
    const FwdSpace sp = fwd_space(M, K, V, F32);
    MergeParams mp = {};
    mp.part = (Part *)(ws + sp.part), mp.at = (float *)(ws + sp.at), mp.V = V, mp.M = (int)M;
    mp.loss = loss, mp.lse = lse;
    int st;
    if (M <= kFewRows) {
        RowsParams<RowStats> p = {};
        p.x = x, p.w = w, p.ldx = ldx, p.M = (int)M, p.N = (int)V, p.K = (int)K;
        p.e.bias = bias, p.e.target = target, p.e.part = (Part *)(ws + sp.part), p.e.at = (float *)(ws + sp.at);
        mp.tiles = (int)ceil_div(V, 16), mp.target = target, mp.tile = 1, mp.row = mp.tiles;
        p.e.ldp = mp.tiles, p.e.M = p.M, p.e.N = p.N;
        hipLaunchKernelGGL(rows_stats_kernel<F32>, grid_of(mp.tiles), dim3(64 * kRowWaves), 0, stream, p);
        if ((st = launch_status()) != HYENA_OK) return st;
    } else {
        RankParams r = {};
        r.target = target, r.loss = loss, r.lse = lse, r.V = V, r.M = (int)M;
        r.rank = (int *)(ws + sp.rank), r.index = (int *)(ws + sp.index), r.goal = (int *)(ws + sp.goal);
        r.count = (int *)(ws + sp.count), r.counts = (int *)(ws + sp.counts);
        const bool gather = gather_ok(x, ldx, K, eb, w);
        if (gather && !all_near(M, ldx, eb)) r.apart = r.count + 1;
        if ((st = launch_rank(r, stream)) != HYENA_OK) return st;
        const int64_t ld = whole(K, eb);
        PackParams k = {};
        if (!gather || r.apart) {
            k.from[0] = x, k.to[0] = ws + sp.x, k.rows[0] = M, k.ld[0] = ldx, k.rank = r.rank, k.apart = r.apart;
            if (ld != K) k.from[1] = w, k.to[1] = ws + sp.w, k.rows[1] = V, k.ld[1] = K;
            k.K = (int)K, k.chunks = (int)(ld * eb / 16);
            if (r.apart && (st = launch_apart(r, ldx, eb, stream)) != HYENA_OK) return st;
            if ((st = launch_pack<F32>(k, stream)) != HYENA_OK) return st;
        }
        const bool direct = gather || k.from[1] || direct_ok(w, K, K, eb);
        const Plan pl = whole_plan(M, V, K, F32, direct);
        StatsEpi e = {};
        e.bias = bias, e.target = r.goal, e.part = (Part *)(ws + sp.part), e.at = (float *)(ws + sp.at), e.ldp = M;
        // of rows in place, of packed rows, or of whichever apart_kernel found
        for (const bool here : {true, false}) {
            if (here ? !gather : gather && !r.apart) continue;
            char *none = nullptr;
            Gemm<StatsEpi> p = gemm_params(pl, 0, Size{M, V, K}, here ? x : k.to[0], here ? ldx : ld,
                                           k.from[1] ? k.to[1] : w, k.from[1] ? ld : K, e, none);
            p.rows = r.index;
#define STATS(DIRECT, GATHER, S)                                                                                       \
    hipLaunchKernelGGL((stats_kernel<F32, DIRECT, GATHER, S>), grid_of(pl.blocks[0]), dim3(S::NT), 0, stream, p, r.count, \
                       r.apart);
            FOR_TILE(pl, direct, here, STATS)
#undef STATS
            if ((st = launch_status()) != HYENA_OK) return st;
        }
        mp.tiles = pl.tiles_n[0], mp.index = r.index, mp.count = r.count, mp.tile = M, mp.row = 1;
    }
    // a workgroup a row for few rows, whose tiles are many: 59 us at 8 rows of 4096 tiles
    // with eight lanes a row, 5 with 256
    if (M <= 256) hipLaunchKernelGGL(merge_kernel<256>, dim3((unsigned)M), dim3(256), 0, stream, mp);
    else hipLaunchKernelGGL(merge_kernel<8>, grid_of(ceil_div(M, 32)), dim3(256), 0, stream, mp);
    return launch_status();
}

template <bool F32>
int xent_bwd(const void *x, const void *w, const void *bias, const int64_t *target, const float *lse, const float *dloss,
             int64_t M, int64_t K, int64_t V, int64_t ldx, int64_t lddx, void *dx, void *dw, void *db, char *ws,
             hipStream_t stream) {
    const int64_t eb = F32 ? 4 : 2;
    const BwdSpace sp = bwd_space(M, K, V, F32);
    int st;
    RankParams r = {};
    r.target = target, r.lse_in = lse, r.dloss = dloss, r.V = V, r.M = (int)M;
    r.lse_out = (float *)(ws + sp.lse), r.dloss_out = (float *)(ws + sp.dloss);
    r.rank = (int *)(ws + sp.rank), r.index = (int *)(ws + sp.index), r.goal = (int *)(ws + sp.goal);
    r.count = (int *)(ws + sp.count), r.most = (float *)(ws + sp.count) + 1;
    r.counts = (int *)(ws + sp.counts), r.tops = (float *)(ws + sp.tops);
    const bool gather = gather_ok(x, ldx, K, eb, w);
    if (gather && !all_near(M, ldx, eb)) r.apart = r.count + 2;
    r.alike = r.count + 3;
    if ((st = launch_rank(r, stream)) != HYENA_OK) return st;
    const int64_t ld = whole(K, eb);
    // dw's dloss goes with e where the entries are few (x is then taken as it is where
    // every row has a target: 8192 x 4096 bf16 with V = 512 150 against 169 us, V = 4 74
    // against 98, though 148 against 141 with V = 512 and 0.3 of the rows masked), else
    // with x, once for all pieces (V = 4096 694 either way).
    const bool with_e = dw && gather && 2 * V <= K;
    PackParams k = {};
    k.from[0] = x, k.rows[0] = M, k.ld[0] = ldx, k.rank = r.rank, k.dx = dx, k.lddx = lddx, k.apart = r.apart;
    k.to[0] = gather && !r.apart && !with_e ? nullptr : ws + sp.x;
    if (with_e) k.count = r.count;
    else if (dw) k.scaled = ws + sp.scaled, k.dloss = dloss, k.most = r.most;
    const DwFrom from = with_e ? DwFrom{ws + sp.scaled, x, r.alike, r.apart, ldx, (int)M} : DwFrom{};
    if (ld != K) k.from[1] = w, k.to[1] = ws + sp.w, k.rows[1] = V, k.ld[1] = K;
    k.K = (int)K, k.chunks = (int)(ld * eb / 16);
    if (r.apart && (st = launch_apart(r, ldx, eb, stream)) != HYENA_OK) return st;
    if ((st = launch_pack<F32>(k, stream)) != HYENA_OK) return st;
    const char *wp = (const char *)(k.from[1] ? k.to[1] : w);
    const int64_t ldw = k.from[1] ? ld : K;
    const bool direct = k.from[1] || direct_ok(w, K, K, eb);  // of each piece, rows being whole 16 bytes
    for (int64_t v0 = 0; v0 < V; v0 += sp.piece) {
        const int64_t N = V - v0 < sp.piece ? V - v0 : sp.piece, ldz = whole(N, eb);
        const char *wv = wp + v0 * ldw * eb;
        const Plan pl = whole_plan(M, N, K, F32, direct);
        DzEpi e = {};
        e.bias = bias ? (const char *)bias + v0 * eb : nullptr, e.lse = r.lse_out, e.dloss = r.dloss_out, e.target = r.goal;
        e.dz = ws + sp.dz, e.ld = ldz, e.sums = db ? (float *)(ws + sp.sums) : nullptr, e.v0 = (int)v0;
        if (with_e) e.scaled = ws + sp.scaled, e.most = r.most, e.alike = r.alike;
        for (const bool here : {true, false}) {  // as in the forward
            if (M == 0 || (here ? !gather : gather && !r.apart)) continue;
            char *none = nullptr;
            Gemm<DzEpi> p = gemm_params(pl, 0, Size{M, N, K}, here ? x : k.to[0], here ? ldx : ld, wv, ldw, e, none);
            p.rows = r.index;
#define DZ(DIRECT, GATHER, S)                                                                                       \
    hipLaunchKernelGGL((dz_kernel<F32, DIRECT, GATHER, S>), grid_of(pl.blocks[0]), dim3(S::NT), 0, stream, p, r.count, \
                       r.apart);
            FOR_TILE(pl, direct, here, DZ)
#undef DZ
            if ((st = launch_status()) != HYENA_OK) return st;
        }

        JoinParams j = {};
        j.count = r.count;
        if (dw || dx) {
            Size sz[2];
            int n = 0;
            if (dw) sz[n++] = Size{N, K, M};
            if (dx) sz[n++] = Size{M, K, N};
            const Plan gp = plan_of(sz, n, F32, direct);
            const int64_t blocks = gp.blocks[0] + gp.blocks[1];
            char *at = ws + sp.partial;
            int g = 0;
            if (dw) {
                DwEpi o = {};
                o.y = (char *)dw + v0 * K * eb, o.ldy = K, o.scale = r.most;
                j.dw = gemm_params(gp, g, sz[g], e.dz, ldz, with_e ? k.to[0] : k.scaled, ld, o, at);
                if (j.dw.partial) j.blocks[0] = ceil_div(N * ceil_div(K, 4), 256);
                ++g;
            }
            if (dx) {
                DxEpi o = {};
                float *acc = (float *)(ws + sp.acc);
                o.y = dx, o.ldy = lddx, o.index = r.index, o.scale = r.dloss_out;
                o.from = v0 > 0 ? acc : nullptr, o.to = v0 + N < V ? acc : nullptr;
                j.dx = gemm_params(gp, g, sz[g], e.dz, ldz, wv, ldw, o, at);
                if (j.dx.partial) j.blocks[1] = ceil_div(M * ceil_div(K, 4), 256);
            }
            const int first = dw ? (int)gp.blocks[0] : 0;
            if (gp.large) {
                if constexpr (!F32) {
                    // whole rounds of the eight XCDs for the first, so that place() holds for both
                    const bool dx_first = N >= M;
                    const int64_t n_dw = dw ? gp.blocks[0] : 0, n_dx = blocks - n_dw;
                    const int64_t lead = ceil_div(dx_first ? n_dx : n_dw, 8) * 8;
                    hipLaunchKernelGGL((large_grads_kernel<Large>), grid_of(lead + (dx_first ? n_dw : n_dx)),
                                       dim3(Large::NT), 0, stream, j.dw, j.dx, (int)lead, (int)dx_first, from, r.count);
                }
            } else {
#define GRADS(DIRECT, S)                                                                                                \
    hipLaunchKernelGGL((grads_kernel<F32, DIRECT, S>), grid_of(blocks), dim3(S::NT), 0, stream, j.dw, j.dx, first, from, \
                       r.count);
                switch (tile_of(gp)) {
                case kDeep: GRADS(true, Deep<F32>) break;
                case kFineDeep: if constexpr (!F32) { GRADS(true, FineDeep) } break;
                case kSmall:
                    if (direct) { GRADS(true, Small<F32>) } else { GRADS(false, Small<F32>) }
                    break;
                default:
                    if (direct) { GRADS(true, Fine<F32>) } else { GRADS(false, Fine<F32>) }
                    break;
                }
#undef GRADS
            }
            if ((st = launch_status()) != HYENA_OK) return st;
        }
        int64_t blocks = j.blocks[0] + j.blocks[1];
        if (db) {
            j.sums = (float *)(ws + sp.sums), j.rows = wave_rows(pl), j.N = (int)N, j.db = (char *)db + v0 * eb;
            // few entries leave their lanes to the rows: 4 of them over 4 million rows 747 us with
            // 64 columns a workgroup
            // (16 columns where there are more: 128 sums of each are then eight a thread)
            for (j.columns = 0; (1 << j.columns) < N && j.columns < 4;) ++j.columns;
            blocks += ceil_div(N, 1 << j.columns);
        }
        if (blocks == 0) continue;
        hipLaunchKernelGGL(join_kernel<F32>, dim3((unsigned)blocks), dim3(256), 0, stream, j);
        if ((st = launch_status()) != HYENA_OK) return st;
    }
    return HYENA_OK;
}

int check_xent(int64_t M, int64_t K, int64_t V, int dtype) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    int64_t n;
    if (!mul_fits(M, V, 64, &n) || !mul_fits(M, K, 64, &n) || !mul_fits(V, K, 64, &n)) return HYENA_ERR_SHAPE;
    const int64_t most = ((int64_t)1 << 31) - 1024;  // tile coordinates are 32 bits
    if (M > most || V > most) return HYENA_ERR_SHAPE;
    if (K >= (int64_t)1 << 20) return HYENA_ERR_UNSUPPORTED;  // byte offsets inside a tile are 32 bits
    // tiles are numbered in 31 bits (grid_of): of whole_plan's and plan_of's least edge where they are
    // many, and some hundred of them may be cut into splits
    const int64_t edge = dtype == HYENA_DTYPE_F32 ? 64 : 128, tiles = ((int64_t)1 << 31) - ((int64_t)1 << 22);
    const int64_t m = ceil_div(M, edge), k = ceil_div(K, edge), v = ceil_div(V, edge);
    if (m * v > tiles || m * k + k * v > tiles) return HYENA_ERR_UNSUPPORTED;
    return HYENA_OK;
}

}  // namespace
}  // namespace layer

using namespace layer;

extern "C" {

int hyena_xent_workspace(int64_t M, int64_t K, int64_t V, int dtype, int backward, int64_t *bytes_out) {
    const int st = check_xent(M, K, V, dtype);
    if (st != HYENA_OK) return st;
    if (!bytes_out) return HYENA_ERR_NULL;
    const bool f32 = dtype == HYENA_DTYPE_F32;
    *bytes_out = V == 0 || (M == 0 && !backward) ? 0 : backward ? bwd_space(M, K, V, f32).total : fwd_space(M, K, V, f32).total;
    return HYENA_OK;
}

int hyena_xent_fwd(const void *x, const void *w, const void *bias, const int64_t *target, int64_t M, int64_t K, int64_t V,
                   int64_t ldx, float *loss, float *lse, void *workspace, int64_t workspace_bytes, int dtype, void *stream) {
    const int st = check_xent(M, K, V, dtype);
    if (st != HYENA_OK) return st;
    const bool f32 = dtype == HYENA_DTYPE_F32;
    const int64_t eb = f32 ? 4 : 2;
    int64_t n, need = 0;
    if (ldx < K || V < 1 || !mul_fits(M, ldx, eb, &n)) return HYENA_ERR_SHAPE;
    if (M == 0) return HYENA_OK;
    if (!target || !loss || !lse || (K > 0 && (!x || !w))) return HYENA_ERR_NULL;
    if (!aligned(x, eb) || !aligned(w, eb) || !aligned(bias, eb) || !aligned(target, 8) || !aligned(loss, 4) ||
        !aligned(lse, 4) || !aligned(workspace, 16))
        return HYENA_ERR_ALIGN;
    hyena_xent_workspace(M, K, V, dtype, 0, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const Rows in[4] = {{x, M, K * eb, ldx * eb}, {w, V, K * eb, K * eb}, {bias, 1, V * eb, V * eb}, {target, 1, M * 8, M * 8}};
    const Rows out[3] = {{loss, 1, M * 4, M * 4}, {lse, 1, M * 4, M * 4}, {workspace, 1, need, need}};
    for (int i = 0; i < 3; ++i) {
        for (const Rows &r : in)
            if (overlap(out[i], r)) return HYENA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HYENA_ERR_ALIAS;
    }
    return (f32 ? xent_fwd<true> : xent_fwd<false>)(x, w, bias, target, M, K, V, ldx, loss, lse,
                                                    first_line(workspace), (hipStream_t)stream);
}

int hyena_xent_bwd(const void *x, const void *w, const void *bias, const int64_t *target, const float *lse,
                   const float *dloss, int64_t M, int64_t K, int64_t V, int64_t ldx, int64_t lddx, void *dx, void *dw,
                   void *db, void *workspace, int64_t workspace_bytes, int dtype, void *stream) {
    const int st = check_xent(M, K, V, dtype);
    if (st != HYENA_OK) return st;
    const bool f32 = dtype == HYENA_DTYPE_F32;
    const int64_t eb = f32 ? 4 : 2;
    int64_t n, need = 0;
    if (ldx < K || V < 1 || !mul_fits(M, ldx, eb, &n) || (dx && (lddx < K || !mul_fits(M, lddx, eb, &n)))) return HYENA_ERR_SHAPE;
    if (!dx && !dw && !db) return M > 0 && K > 0 ? HYENA_ERR_NULL : HYENA_OK;
    if (M > 0 && (!target || !lse || !dloss || (K > 0 && (!x || !w)))) return HYENA_ERR_NULL;
    if (!aligned(x, eb) || !aligned(w, eb) || !aligned(bias, eb) || !aligned(target, 8) || !aligned(lse, 4) ||
        !aligned(dloss, 4) || !aligned(dx, eb) || !aligned(dw, eb) || !aligned(db, eb) || !aligned(workspace, 16))
        return HYENA_ERR_ALIGN;
    hyena_xent_workspace(M, K, V, dtype, 1, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    const Rows in[6] = {{x, M, K * eb, ldx * eb},  {w, V, K * eb, K * eb},  {bias, 1, V * eb, V * eb},
                        {target, 1, M * 8, M * 8}, {lse, 1, M * 4, M * 4}, {dloss, 1, M * 4, M * 4}};
    const Rows out[4] = {{dx, M, K * eb, lddx * eb}, {dw, V, K * eb, K * eb}, {db, 1, V * eb, V * eb},
                         {need > 0 ? workspace : nullptr, 1, need, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Rows &r : in)
            if (overlap(out[i], r)) return HYENA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HYENA_ERR_ALIAS;
    }
    if (M == 0 || K == 0) dx = nullptr;
    if (K == 0) dw = nullptr;
    if (!dx && !dw && !db) return HYENA_OK;
    return (f32 ? xent_bwd<true> : xent_bwd<false>)(x, w, bias, target, lse, dloss, M, K, V, ldx, lddx, dx, dw, db,
                                                    first_line(workspace), (hipStream_t)stream);
}

}  // extern "C"
