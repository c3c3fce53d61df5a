// Matrix product with bias, activation and residual in its epilogue, and its
// backward, for MI355X (gfx950) (hyena_layer.h has the formulas and layouts).
//
// The tiled products are layer_gemm.h's.
// Operands whose 16-byte chunks are not aligned (odd sizes, strides or
// pointers) cannot be fetched straight into LDS.  Where their sizes are odd and
// the product is long enough, they are copied to padded rows first; otherwise the
// same kernels take them through registers, a step ahead, with unaligned 16-byte
// loads.

#include <initializer_list>

#include "layer_gemm.h"

namespace layer {
namespace {

// sigmoid(z), and its slope e r^2 with e = exp(-|z|), r = 1 / (1 + e): finite
// for every z, and exact to rounding at both ends.
__device__ inline float sigmoid(float z, float &slope) {
    const float e = __expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
    slope = e * r * r;
    return z < 0.0f ? e * r : r;
}

template <int ACT> __device__ inline float act_value(float z) {
    if constexpr (ACT == HYENA_ACT_RELU) return z < 0.0f ? 0.0f : z;
    else if constexpr (ACT == HYENA_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    else if constexpr (ACT == HYENA_ACT_SILU) return z / (1.0f + __expf(-z));
    else if constexpr (ACT == HYENA_ACT_SIGMOID) return decay<false>(z);
    else return z;
}

template <int ACT> __device__ inline float act_slope(float z) {
    if constexpr (ACT == HYENA_ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == HYENA_ACT_GELU) {
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * __expf(-0.5f * z * z) * 0.39894228040143268f;
    } else if constexpr (ACT == HYENA_ACT_SILU) {
        float slope;
        const float p = sigmoid(z, slope);
        return p + z * slope;
    } else if constexpr (ACT == HYENA_ACT_SIGMOID) {
        float slope;
        sigmoid(z, slope);
        return slope;
    } else {
        return 1.0f;
    }
}

// f<ACT>() for the activation code.
#define FOR_ACT(act, F)                                     \
    switch (act) {                                          \
    case HYENA_ACT_RELU: F(HYENA_ACT_RELU); break;          \
    case HYENA_ACT_GELU: F(HYENA_ACT_GELU); break;          \
    case HYENA_ACT_SILU: F(HYENA_ACT_SILU); break;          \
    case HYENA_ACT_SIGMOID: F(HYENA_ACT_SIGMOID); break;    \
    default: F(HYENA_ACT_NONE); break;                      \
    }

struct Epilogue {
    static constexpr bool kSums = false;
    static constexpr int kRun = 0;
    const void *bias, *residual;
    void *y, *preact;
    int64_t ldr, ldy;
    int M, N;
    int act;

    template <bool F32, int V> __device__ __forceinline__ Pack<F32, V> columns(int n) const {
        return bias && n < N ? Pack<F32, V>::load(bias, n, N - n) : Pack<F32, V>::zero();
    }
    template <bool F32, int V> __device__ __forceinline__ Pack<F32, V> before(int64_t m, int n) const {
        return residual && m < M ? Pack<F32, V>::load(residual, m * ldr + n, N - n) : Pack<F32, V>::zero();
    }
    template <bool F32, int V>
    __device__ __forceinline__ void finish(int64_t m, int n, float (&z)[V], const Pack<F32, V> &bias,
                                           const Pack<F32, V> &residual) const {
        using Q = Pack<F32, V>;
        const int left = N - n;
        if (m >= M || left <= 0) return;
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] += bias.get(e);
        if (preact) Q::store(preact, m * N + n, left, z);
#define ACTIVATE(ACT) \
    _Pragma("unroll") for (int e = 0; e < V; ++e) z[e] = act_value<ACT>(z[e]);
        if (act != HYENA_ACT_NONE) FOR_ACT(act, ACTIVATE)
#undef ACTIVATE
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] += residual.get(e);
        Q::store(y, m * ldy + n, left, z);
    }
    template <bool F32, int V> __device__ __forceinline__ void close(const Pack<F32, V> &, int, int, int) const {}
};
using GemmParams = Gemm<Epilogue>;

// The forward's product.
template <bool F32, bool DIRECT, typename S> __global__ __launch_bounds__(S::NT, S::WAVES) void fwd_kernel(GemmParams p) {
    TILE_BUFFERS(S)
    run_tile<false, false, DIRECT, S>(p, blockIdx.x, a0, a1, a2, a3, b0, b1, b2, b3);
}

// The backward's products side by side: the first `blocks` workgroups form
// dw = dz^T x, the others dx = dz w.
template <bool F32, bool DIRECT, typename S>
__global__ __launch_bounds__(S::NT, S::WAVES) void bwd_kernel(GemmParams dw, GemmParams dx, int blocks) {
    TILE_BUFFERS(S)
    if ((int)blockIdx.x < blocks) run_tile<true, true, DIRECT, S>(dw, blockIdx.x, a0, a1, a2, a3, b0, b1, b2, b3);
    else run_tile<false, true, DIRECT, S>(dx, blockIdx.x - blocks, a0, a1, a2, a3, b0, b1, b2, b3);
}
// One of them (256 x 256 tiles fill the card alone, and have no registers to
// spare: dw's loads keep 11 of theirs in memory, two 16-byte reloads a step).
template <bool TALL_A, typename S> __global__ __launch_bounds__(S::NT, S::WAVES) void large_kernel(GemmParams p) {
    TILE_BUFFERS(S)
    run_tile<TALL_A, true, true, S>(p, blockIdx.x, a0, a1, a2, a3, b0, b1, b2, b3);
}

// What remains after the products: the sums of the splits with their epilogue
// (four columns a thread), and db from the row blocks' column sums.  Bound by its
// launch (4 to 5 us at N = 4096).  Atomics in the products would spare it and make
// the bits depend on their order.
struct FinishParams {
    GemmParams g[2];
    int64_t blocks[2];   // workgroups of each
    const float *sums;   // [n_sums][N] or null
    int n_sums, N;
    void *db;
};

template <bool F32> __global__ __launch_bounds__(256) void finish_kernel(FinishParams p) {
    __shared__ float part[4][64];
    int64_t block = blockIdx.x;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (block < p.blocks[g]) return sum_splits<F32>(p.g[g], block * 256 + threadIdx.x);
        block -= p.blocks[g];
    }
    // 64 columns, four lanes each
    const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
    const int64_t n = block * 64 + c;
    float s = 0.0f;
    if (n < p.N) {
#pragma unroll 8
        for (int b = r; b < p.n_sums; b += 4) s += p.sums[(int64_t)b * p.N + n];
    }
    part[r][c] = s;
    __syncthreads();
    if (r == 0 && n < p.N) store1<F32>(p.db, n, part[0][c] + part[1][c] + part[2][c] + part[3][c]);
}

// ---- few rows ----------------------------------------------------------------------

template <bool F32, int MT>
__global__ __launch_bounds__(64 * kRowWaves) void rows_kernel(RowsParams<Epilogue> p) {
    __shared__ __attribute__((aligned(16))) float sums[kRowWaves][MT][16][16];
    rows_product<F32, MT>(p, blockIdx.x, sums);
}

// ---- dz, db and padded rows ------------------------------------------------------------

// dz = dy act'(z) (rounded once, to the type the matrix cores take) and each
// block's column sums of the unrounded dz.  A block takes 32 lanes of four
// columns by `rows` rows.  Bound by memory: 8192 x 4096 bf16 in 41 us (201 MB,
// 4.9 TB/s).  Formed in the products' loads instead, dy and z would be read anew
// by every tile of a row and column of tiles, and straight loads into LDS lost.
//
// Where rows are no whole number of 16 bytes, x and w are copied to rows that
// are, zeros behind them, by further blocks of the same launch (and dz is written
// so), for the products to fetch straight into LDS: one pass over the operands
// instead of registers and element-wise edges in every tile.
struct Pads {
    const void *from[2];  // null: none
    void *to[2];          // rows of `chunks` 16-byte chunks
    int64_t ld[2];
    uint32_t rows[2];     // rows * chunks is below 2^31
    uint32_t n, chunks;
};
struct DzParams {
    const void *dy, *z;
    void *dz;         // null: only the sums
    float *sums;      // [row blocks][N], or null
    int64_t M, lddy, lddz;  // lddz: whole 16 bytes
    int N, rows;
    unsigned row_blocks;  // blockIdx.y from there on: padded rows
    Pads pads;
};

template <bool F32> __device__ inline void copy_rows(const Pads &p, uint32_t block, uint32_t blocks) {
    using T = typename El<F32>::type;
    constexpr int CE = El<F32>::CE;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (!p.from[g]) continue;
        const uint32_t total = p.rows[g] * p.chunks;
        for (uint32_t id = block * 256 + threadIdx.x; id < total; id += blocks * 256) {
            const uint32_t row = id / p.chunks, c = (id - row * p.chunks) * CE, left = p.n - c;
            const T *from = (const T *)p.from[g] + (int64_t)row * p.ld[g] + c;
            u32x4_t v;
            if (left >= CE) {
                v = *(const typename El<F32>::chunk_any *)from;
            } else {
                T x[CE];
#pragma unroll
                for (int e = 0; e < CE; ++e) x[e] = e < (int)left ? from[e] : (T)0.0f;
                v = __builtin_bit_cast(u32x4_t, x);
            }
            ((u32x4_t *)p.to[g])[id] = v;
        }
    }
}

template <bool F32, int ACT> __global__ __launch_bounds__(256) void dz_kernel(DzParams p) {
    __shared__ float part[8][128];
    if (blockIdx.y >= p.row_blocks)
        return copy_rows<F32>(p.pads, (blockIdx.y - p.row_blocks) * gridDim.x + blockIdx.x,
                              (gridDim.y - p.row_blocks) * gridDim.x);
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int n = (blockIdx.x * 32 + cl) * 4, left = p.N - n;
    const int64_t first = (int64_t)blockIdx.y * p.rows, last = min(p.M, first + p.rows);
    float sum[4] = {};
    const int wide = p.dz ? (int)(p.lddz - n) : left;  // dz has zeros behind its columns
    if (wide > 0) {
#pragma unroll 4
        for (int64_t m = first + rl; m < last; m += 8) {
            const auto rd = Pack<F32, 4>::load(p.dy, m * p.lddy + n, left);
            float d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = rd.get(e);
            if constexpr (ACT != HYENA_ACT_NONE) {
                const auto rz = Pack<F32, 4>::load(p.z, m * p.N + n, left);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] *= act_slope<ACT>(rz.get(e));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += d[e];
            if (p.dz) Pack<F32, 4>::store(p.dz, m * p.lddz + n, 4, d);
        }
    }
    if (!p.sums) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) part[rl][cl * 4 + e] = sum[e];
    __syncthreads();
    const int col = blockIdx.x * 128 + threadIdx.x;
    if (threadIdx.x >= 128 || col >= p.N) return;
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s += part[r][threadIdx.x];
    p.sums[(int64_t)blockIdx.y * p.N + col] = s;
}

// ---- host --------------------------------------------------------------------------------

// Whether rows_kernel takes the forward.  It cuts no c between workgroups, so long
// rows want enough columns, and every workgroup reads all of x, so more rows want
// short ones (us in bf16, rows_kernel and tiles):
//   M = 16: N x K = 1024 x 1024 5.3 / 8.0, 512 x 2048 6.6 / 7.3, 4096 x 4096
//           11.7 / 12.2, 4096 x 8192 20.1 / 21.3; but 1024 x 4096 10.6 / 9.2, 2048 x
//           8192 18.6 / 13.2
//   M = 32: 1024 x 1024 5.4 / 7.4, 4096 x 1024 6.2 / 8.6, 8192 x 1024 9.2 / 10.1;
//           but 16384 x 1024 15.1 / 10.0, 1024 x 4096 13.9 / 9.2, 4096 x 4096 15.0 / 12.8
bool few_rows(int64_t M, int64_t N, int64_t K) {
    return M <= 16 ? K <= 2048 || N >= 4096 : M <= 32 && K <= 1024 && N <= 8192;
}

// Products from which on padded rows are worth a launch (see pad_rows), measured
// against the way through registers.  Forward: 1300 x 1291 x 1293 (2.2e9) fp32 63
// against 67 us but bf16 25 against 21, 4091 x 2045 x 2045 (1.7e10) bf16 55 against
// 64.  Backward: 1300 x 1291 x 1293 bf16 37 against 51 us, 1021 x 777 x 521 (4e8)
// fp32 40 against 38; in a launch that is there anyway 41 against 45, and bf16 24
// against 31.  That holds for few rows too, though each copy then serves one row
// of tiles: N = K = 4095 with M = 8, 64 and 256 bf16 46, 48 and 63 us against 58,
// 64 and 89, fp32 106, 113 and 190 against 112, 131 and 256; 64 x 515 x 517 level.
constexpr double pad_forward(bool f32) { return f32 ? 2e9 : 7e9; }
constexpr double kPadBackward = 1e9;

// Whether rows of K values are padded for the products: where they are no whole
// 16 bytes, and the product is long enough to earn the copies (`least` products).
bool pad_rows(int64_t M, int64_t N, int64_t K, int64_t eb, double least) {
    const int64_t pitch = whole(K, eb), rows = M > N ? M : N;
    return pitch != K && pitch < (int64_t)1 << 21 && rows * (pitch * eb / 16) < (int64_t)1 << 31 &&
           (double)M * (double)N * (double)K >= least;
}

// Adds [rows, n] at `from` to the pads: at `at` from now on.
void add_pad(Pads &p, int g, const void *&from, int64_t &ld, int64_t rows, int64_t n, int64_t eb, char *&at) {
    p.from[g] = from, p.to[g] = at, p.ld[g] = ld, p.rows[g] = (uint32_t)rows;
    p.n = (uint32_t)n;
    ld = whole(n, eb);
    p.chunks = (uint32_t)(ld * eb / 16);
    from = at;
    at += rows * ld * eb;
}

template <bool F32> int launch_dz(const DzParams &p, int act, hipStream_t stream) {
    int64_t copies = 0;  // blocks, four chunks a thread or more
    for (int g = 0; g < 2; ++g)
        if (p.pads.from[g]) copies += ceil_div((int64_t)p.pads.rows[g] * p.pads.chunks, 1024);
    const int64_t x = ceil_div(p.N, 128), y = ceil_div(copies < 2048 ? copies : 2048, x);
    const dim3 grid((unsigned)x, (unsigned)(p.row_blocks + y));
#define DZ(ACT) hipLaunchKernelGGL((dz_kernel<F32, ACT>), grid, dim3(256), 0, stream, p);
    FOR_ACT(act, DZ)
#undef DZ
    return launch_status();
}

template <bool F32> int launch_finish(const GemmParams *g, int n, const float *sums, int n_sums, int N, void *db,
                                      hipStream_t stream) {
    FinishParams p = {};
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i)
        if (g[i].partial) {
            p.g[i] = g[i];
            p.blocks[i] = ceil_div((int64_t)g[i].M * ceil_div(g[i].N, 4), 256);
            blocks += p.blocks[i];
        }
    if (db) {
        p.sums = sums, p.n_sums = n_sums, p.N = N, p.db = db;
        blocks += ceil_div(N, 64);
    }
    if (blocks == 0) return HYENA_OK;
    if (blocks > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(finish_kernel<F32>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return launch_status();
}

template <bool F32>
int linear_fwd(const void *x, int64_t ldx, const void *w, int64_t M, int64_t N, int64_t K, Epilogue e, void *ws,
               hipStream_t stream) {
    const int64_t eb = F32 ? 4 : 2;
    if (few_rows(M, N, K)) {
        RowsParams<Epilogue> p = {};
        p.x = x, p.w = w, p.ldx = ldx, p.M = (int)M, p.N = (int)N, p.K = (int)K;
        p.e = e;
        p.e.M = p.M, p.e.N = p.N;
        hipLaunchKernelGGL((M <= 16 ? rows_kernel<F32, 1> : rows_kernel<F32, 2>), dim3((unsigned)ceil_div(N, 16)),
                           dim3(64 * kRowWaves), 0, stream, p);
        return launch_status();
    }
    const Size sz = {M, N, K};
    bool direct = direct_ok(x, ldx, K, eb) && direct_ok(w, K, K, eb);
    int64_t ldw = K;
    char *at = (char *)ws;
    if (pad_rows(M, N, K, eb, pad_forward(F32))) {
        DzParams p = {};
        p.N = (int)N;
        add_pad(p.pads, 0, x, ldx, M, K, eb, at);
        add_pad(p.pads, 1, w, ldw, N, K, eb, at);
        const int st = launch_dz<F32>(p, HYENA_ACT_NONE, stream);
        if (st != HYENA_OK) return st;
        direct = true;
    }
    const Plan pl = plan_of(&sz, 1, F32, direct);
    if (pl.blocks[0] > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    const GemmParams p = gemm_params(pl, 0, sz, x, ldx, w, ldw, e, at);
    const dim3 grid((unsigned)pl.blocks[0]);
    if (pl.large) {
        if constexpr (!F32) hipLaunchKernelGGL((fwd_kernel<F32, true, Large>), grid, dim3(Large::NT), 0, stream, p);
    } else if (pl.fine && pl.deep) {
        if constexpr (!F32)
            hipLaunchKernelGGL((fwd_kernel<F32, true, FineDeep>), grid, dim3(FineDeep::NT), 0, stream, p);
    } else if (pl.fine) {
        hipLaunchKernelGGL((direct ? fwd_kernel<F32, true, Fine<F32>> : fwd_kernel<F32, false, Fine<F32>>), grid,
                           dim3(Fine<F32>::NT), 0, stream, p);
    } else if (pl.deep) {
        hipLaunchKernelGGL((fwd_kernel<F32, true, Deep<F32>>), grid, dim3(Deep<F32>::NT), 0, stream, p);
    } else if (direct) {
        hipLaunchKernelGGL((fwd_kernel<F32, true, Small<F32>>), grid, dim3(Small<F32>::NT), 0, stream, p);
    } else {
        hipLaunchKernelGGL((fwd_kernel<F32, false, Small<F32>>), grid, dim3(Small<F32>::NT), 0, stream, p);
    }
    const int st = launch_status();
    return st != HYENA_OK ? st : launch_finish<F32>(&p, 1, nullptr, 0, 0, nullptr, stream);
}

// Row blocks of dz_kernel.
int64_t dz_blocks(int64_t M, int64_t N) {
    const int64_t blocks = ceil_div(1024, ceil_div(N, 128)), most = ceil_div(M, 32);
    return blocks < most ? blocks : most;
}

// Workspace of the forward: padded x and w, partial sums.
int64_t fwd_space(int64_t M, int64_t N, int64_t K, bool f32) {
    if (N == 0 || few_rows(M, N, K)) return 0;
    const int64_t eb = f32 ? 4 : 2;
    const Size sz = {M, N, K};
    return (pad_rows(M, N, K, eb, pad_forward(f32)) ? (M + N) * whole(K, eb) * eb : 0) + partial_bytes(&sz, 1, f32);
}

// Workspace of the backward: dz, the column sums, padded x and w, the products'
// partial sums.
struct BwdSpace {
    int64_t dz, sums, pads, partial;
};
BwdSpace bwd_space(int64_t M, int64_t N, int64_t K, int act, int dtype) {
    const bool f32 = dtype == HYENA_DTYPE_F32;
    const int64_t eb = f32 ? 4 : 2;
    BwdSpace s = {};
    if (act != HYENA_ACT_NONE || pad_rows(M, K, N, eb, 0)) s.dz = M * whole(N, eb) * eb;
    if (pad_rows(M, N, K, eb, 0)) s.pads = (M + N) * whole(K, eb) * eb;
    if (M == 0 || N == 0) return s;
    s.sums = (dz_blocks(M, N) * N * 4 + 15) / 16 * 16;
    if (K == 0) return s;
    // one product alone splits as much as both together, or more
    const Size both[2] = {{M, K, N}, {N, K, M}};
    for (int64_t b : {partial_bytes(both, 2, f32), partial_bytes(both, 1, f32), partial_bytes(both + 1, 1, f32)})
        if (b > s.partial) s.partial = b;
    return s;
}

template <bool F32>
int linear_bwd(const void *x, const void *w, const void *z, const void *dy, int64_t M, int64_t N, int64_t K,
               int64_t ldx, int64_t lddy, int64_t lddx, int act, void *dx, void *dw, void *db, char *ws,
               const BwdSpace &sp, hipStream_t stream) {
    const int64_t eb = F32 ? 4 : 2;
    if (M == 0 || K == 0) dx = nullptr;
    if (N == 0 || K == 0) dw = nullptr;
    if (N == 0) db = nullptr;
    const bool products = (dx || dw) && M > 0 && N > 0;
    // Padded rows earn their copies where there is a launch for dz or db anyway.
    const double least = act != HYENA_ACT_NONE || db ? 0 : kPadBackward;
    const bool pad = products && pad_rows(M, N, K, eb, least);
    const bool x_ok = !dw || pad || direct_ok(x, ldx, K, eb), w_ok = !dx || pad || direct_ok(w, K, K, eb);
    const bool make = products && (act != HYENA_ACT_NONE || (x_ok && w_ok && pad_rows(M, K, N, eb, least)));
    const bool direct = x_ok && w_ok && (make ? direct_ok(ws, whole(N, eb), whole(N, eb), eb) : direct_ok(dy, lddy, N, eb));
    const void *dz = make ? ws : dy;
    const int64_t lddz = make ? whole(N, eb) : lddy;
    int64_t ldw = K;
    const int64_t row_blocks = M > 0 && N > 0 ? dz_blocks(M, N) : 0;
    float *sums = (float *)(ws + sp.dz);
    int st = HYENA_OK;
    DzParams d = {};
    d.N = (int)N;
    if (pad && direct) {
        char *at = ws + sp.dz + sp.sums;
        if (dw) add_pad(d.pads, 0, x, ldx, M, K, eb, at);
        if (dx) add_pad(d.pads, 1, w, ldw, N, K, eb, at);
    }
    if ((make || db) && row_blocks > 0) {
        d.dy = dy, d.z = z, d.dz = make ? ws : nullptr, d.sums = db ? sums : nullptr;
        d.M = M, d.lddy = lddy, d.lddz = lddz;
        d.rows = (int)ceil_div(M, row_blocks), d.row_blocks = (unsigned)row_blocks;
    }
    if ((d.row_blocks > 0 || d.pads.from[0] || d.pads.from[1]) && (st = launch_dz<F32>(d, act, stream)) != HYENA_OK)
        return st;
    Size sz[2];
    GemmParams g[2] = {};
    int n = 0;
    if (dw) sz[n++] = Size{N, K, M};
    if (dx) sz[n++] = Size{M, K, N};
    if (n > 0) {
        const Plan pl = plan_of(sz, n, F32, direct);
        const int64_t blocks = pl.blocks[0] + pl.blocks[1];
        if (blocks > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
        char *at = ws + sp.dz + sp.sums + sp.pads;
        Epilogue e = {};
        int i = 0;
        if (dw) {
            e.y = dw, e.ldy = K;
            g[i] = gemm_params(pl, i, sz[i], dz, lddz, x, ldx, e, at);
            ++i;
        }
        if (dx) {
            e.y = dx, e.ldy = lddx;
            g[i] = gemm_params(pl, i, sz[i], dz, lddz, w, ldw, e, at);
        }
        const int first = dw ? (int)pl.blocks[0] : 0;
        const GemmParams &second = g[n - 1];
        const dim3 grid((unsigned)blocks);
        if (pl.large) {
            if constexpr (!F32) {
                if (dw) hipLaunchKernelGGL((large_kernel<true, Large>), dim3((unsigned)first), dim3(Large::NT), 0, stream, g[0]);
                if (dx)
                    hipLaunchKernelGGL((large_kernel<false, Large>), dim3((unsigned)(blocks - first)), dim3(Large::NT), 0,
                                       stream, second);
            }
        } else if (pl.fine && pl.deep) {
            if constexpr (!F32)
                hipLaunchKernelGGL((bwd_kernel<F32, true, FineDeep>), grid, dim3(FineDeep::NT), 0, stream, g[0], second,
                                   first);
        } else if (pl.fine) {
            hipLaunchKernelGGL((direct ? bwd_kernel<F32, true, Fine<F32>> : bwd_kernel<F32, false, Fine<F32>>), grid,
                               dim3(Fine<F32>::NT), 0, stream, g[0], second, first);
        } else if (pl.deep) {
            hipLaunchKernelGGL((bwd_kernel<F32, true, Deep<F32>>), grid, dim3(Deep<F32>::NT), 0, stream, g[0], second, first);
        } else if (direct) {
            hipLaunchKernelGGL((bwd_kernel<F32, true, Small<F32>>), grid, dim3(Small<F32>::NT), 0, stream, g[0], second,
                               first);
        } else {
            hipLaunchKernelGGL((bwd_kernel<F32, false, Small<F32>>), grid, dim3(Small<F32>::NT), 0, stream, g[0],
                               second, first);
        }
        if ((st = launch_status()) != HYENA_OK) return st;
    }
    return launch_finish<F32>(g, n, sums, (int)row_blocks, (int)N, db, stream);
}

int check_linear(int64_t M, int64_t N, int64_t K, int act, int dtype) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    if (act < HYENA_ACT_NONE || act > HYENA_ACT_SIGMOID) return HYENA_ERR_UNSUPPORTED;
    int64_t n;
    if (!mul_fits(M, N, 64, &n) || !mul_fits(M, K, 64, &n) || !mul_fits(N, K, 64, &n)) return HYENA_ERR_SHAPE;
    const int64_t most = ((int64_t)1 << 31) - 1024;  // tile coordinates are 32 bits
    if (M > most || N > most || K > most) return HYENA_ERR_SHAPE;
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
    if (backward) {
        const BwdSpace s = bwd_space(M, N, K, act, dtype);
        *bytes_out = s.dz + s.sums + s.pads + s.partial;
    } else {
        *bytes_out = fwd_space(M, N, K, dtype == HYENA_DTYPE_F32);
    }
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
    Epilogue e = {};
    e.bias = bias, e.residual = residual, e.ldr = ldr, e.ldy = ldy, e.y = y, e.preact = preact, e.act = act;
    hipStream_t s = (hipStream_t)stream;
    const bool f32 = dtype == HYENA_DTYPE_F32;
    return f32 ? linear_fwd<true>(x, ldx, w, M, N, K, e, workspace, s) : linear_fwd<false>(x, ldx, w, M, N, K, e, workspace, s);
}

int hyena_linear_bwd(const void *x, const void *w, const void *preact, const void *dy, int64_t M, int64_t N,
                     int64_t K, int64_t ldx, int64_t lddy, int64_t lddx, int act, void *dx, void *dw, void *db,
                     void *workspace, int64_t workspace_bytes, int dtype, void *stream) {
    const int st = check_linear(M, N, K, act, dtype);
    if (st != HYENA_OK) return st;
    const int64_t eb = dtype == HYENA_DTYPE_F32 ? 4 : 2;
    int64_t n;
    if (lddy < N || (dw && ldx < K) || (dx && lddx < K) || !mul_fits(M, lddy, eb, &n) ||
        (dw && !mul_fits(M, ldx, eb, &n)) || (dx && !mul_fits(M, lddx, eb, &n)))
        return HYENA_ERR_SHAPE;
    // an output of no elements may be NULL, also where it is the only one wanted
    if (!dx && !dw && !db) return M > 0 && N > 0 && K > 0 ? HYENA_ERR_NULL : HYENA_OK;
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
    const void *z = act != HYENA_ACT_NONE ? preact : nullptr;
    const BwdSpace sp = bwd_space(M, N, K, act, dtype);
    hipStream_t s = (hipStream_t)stream;
    return dtype == HYENA_DTYPE_F32
               ? linear_bwd<true>(x, w, z, dy, M, N, K, ldx, lddy, lddx, act, dx, dw, db, (char *)workspace, sp, s)
               : linear_bwd<false>(x, w, z, dy, M, N, K, ldx, lddy, lddx, act, dx, dw, db, (char *)workspace, sp, s);
}

}  // extern "C"
