// Matrix product with bias, activation and residual in its epilogue, and its
// backward, for MI355X (gfx950) (hyena_layer.h has the formulas and layouts).
//
// Every large product is C[m, n] = sum_c A(m, c) B(n, c), each operand lying in
// memory either with c contiguous ("flat": x and w of the forward, dz of dx)
// or with c as its rows ("tall": w of dx; dz and x of dw):
//   * A workgroup owns a BM x BN tile of C and walks c in steps of 128 bytes
//     of a flat row (64 bf16 or 32 fp32 values).  Each step's operand tiles go
//     from memory straight into LDS (16 bytes a lane, no registers), into one
//     of two buffers while the other is multiplied.
//   * LDS order.  The direct loads fill LDS in lane order, so the order is
//     chosen by which 16 bytes each lane fetches.  Flat tiles keep rows of 128
//     bytes whose eight 16-byte chunks are XOR-ed with the row's low bits: the
//     16 rows of a fragment then spread over all banks.  Tall tiles keep rows
//     of BM values whose 32-byte blocks (16 bf16 values, one fragment's width)
//     are XOR-ed with bits of the row for the same reason.
//   * bf16 fragments are 8 values of c a lane: one 16-byte read of a flat tile,
//     two transposing reads (ds_read_b64_tr_b16) of a tall one.  fp32
//     fragments are 4 values of c, each its own v_mfma_f32_16x16x4_f32; the
//     order of c inside a step differs from memory's, alike for both operands.
//   * The products are formed as B A^T, so a lane ends up with 4 consecutive n
//     of one m, which the epilogue turns into one 8- or 16-byte access.
// Sizes, pointers or strides that do not allow 16-byte fetches take the same
// kernel with a loader that fetches single elements.

#include "layer_common.h"

namespace layer {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
#define LDS_PTR __attribute__((address_space(3)))

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

// ---- epilogue -----------------------------------------------------------------

struct Epilogue {
    const void *bias, *residual;
    void *y, *preact;
    int64_t ldr, ldy;
    int N;
    int act;
    bool vec;  // four values at a time: N, strides and pointers allow it
};

template <bool F32> __device__ inline void load4(const void *p, size_t e, float (&x)[4]) {
    if constexpr (F32) {
        const f32x4_t r = *(const f32x4_t *)((const float *)p + e);
        x[0] = r[0], x[1] = r[1], x[2] = r[2], x[3] = r[3];
    } else {
        const u32x2_t r = *(const u32x2_t *)((const bf16_t *)p + e);
        x[0] = bf_lo(r[0]), x[1] = bf_hi(r[0]), x[2] = bf_lo(r[1]), x[3] = bf_hi(r[1]);
    }
}
template <bool F32> __device__ inline void store4(void *p, size_t e, const float (&x)[4]) {
    if constexpr (F32) *(f32x4_t *)((float *)p + e) = f32x4_t{x[0], x[1], x[2], x[3]};
    else *(u32x2_t *)((bf16_t *)p + e) = u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
}

// z of row m, columns n .. n+3 (those below N), n a multiple of 4.
template <bool F32, int ACT> __device__ inline void finish4(const Epilogue &p, int64_t m, int n, const float (&acc)[4]) {
    if (n >= p.N) return;
    float z[4], r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.vec) {
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (p.bias) load4<F32>(p.bias, n, b);
        if (p.residual) load4<F32>(p.residual, m * p.ldr + n, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = acc[i] + b[i];
        if (p.preact) store4<F32>(p.preact, m * p.N + n, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = act_value<ACT>(z[i]) + r[i];
        store4<F32>(p.y, m * p.ldy + n, z);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (n + i >= p.N) break;
            float v = acc[i];
            if (p.bias) v += load1<F32>(p.bias, n + i);
            if (p.preact) store1<F32>(p.preact, m * p.N + n + i, v);
            v = act_value<ACT>(v);
            if (p.residual) v += load1<F32>(p.residual, m * p.ldr + n + i);
            store1<F32>(p.y, m * p.ldy + n + i, v);
        }
    }
}

// ---- tiled product ---------------------------------------------------------------

struct GemmParams {
    const void *a, *b;
    int64_t lda, ldb;         // elements between memory rows of a and b
    int M, N, C;
    int tiles_m, tiles_n;
    int splits, c_per_split;  // c is cut into splits (a multiple of the step each, but the last)
    float *partial;           // splits > 1: [splits][M][N] sums for split_kernel; else null
    Epilogue e;
};

template <bool F32> struct El;
template <> struct El<false> {
    static constexpr int CE = 8;   // values per 16-byte chunk
    typedef bf16x8_t frag;
    typedef bf16_t type;
};
template <> struct El<true> {
    static constexpr int CE = 4;
    typedef f32x4_t frag;
    typedef float type;
};

// One operand's LDS tile of X values of m (or n) by one step of c.
template <bool F32, bool TALL, int X, int NT> struct Operand {
    static constexpr int CE = El<F32>::CE;
    static constexpr int BK = 8 * CE;
    static constexpr int BYTES = X * 128;
    static constexpr int CHUNKS = X * 8;
    static constexpr int LOADS = CHUNKS / NT;
    static constexpr int ROW_CHUNKS = TALL ? X / CE : 8;  // chunks per LDS row
    static constexpr int BLOCKS = X / 16;                 // tall: 16-value blocks per LDS row
    static constexpr int BC = 16 / CE;                    // chunks per block
    static_assert(CHUNKS % NT == 0, "whole loads");

    // XOR of a tall row's block index: the rows that one read touches are
    // 8 j + (0..3) (bf16; + 4 in the second read) or 4 j + i (fp32), j = 0..3.
    __device__ static int turn(int row) {
        const int t = F32 ? (row >> 2) & 3 : (row & 3) | (row >> 1 & 4);
        return t & (BLOCKS - 1);
    }
    // The chunk of memory (relative to the tile: row of memory, chunk in it)
    // that LDS chunk q holds.
    __device__ static void source(int q, int &row, int &chunk) {
        row = q / ROW_CHUNKS;
        const int c = q % ROW_CHUNKS;
        if constexpr (TALL) chunk = ((c / BC) ^ turn(row)) * BC + c % BC;
        else chunk = c ^ (row >> 1 & 7);
    }

    // Direct loads.  off[i]: the lane's byte offset in the tile, or past every
    // range where its m is outside the matrix.
    static constexpr uint32_t kOutside = 0x80000000u;
    __device__ static void plan(uint32_t (&off)[LOADS], int64_t ld, int x_left) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            int row, chunk;
            source(i * NT + threadIdx.x, row, chunk);
            const int x = TALL ? chunk * CE : row;
            off[i] = x < x_left ? (uint32_t)(row * ld + chunk * CE) * sizeof(typename El<F32>::type) : kOutside;
        }
    }
    __device__ static void fetch(const typename El<F32>::type *tile, const uint32_t (&off)[LOADS], int c_left,
                                 LDS_PTR unsigned char *lds) {
        // offsets stay below 2^31 (the host checks), so only kOutside is out of range
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void *)tile, (short)0, 0x7fffffff, 0x00020000);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if (c_left >= BK) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDS_PTR void *)(lds + (i * NT + wave * 64) * 16), 16,
                                                         off[i], 0, 0, 0);
        } else {  // the last step: zeros past the end of c
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                int row, chunk;
                source(i * NT + threadIdx.x, row, chunk);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDS_PTR void *)(lds + (i * NT + wave * 64) * 16), 16,
                                                         (TALL ? row : chunk * CE) < c_left ? off[i] : kOutside, 0, 0, 0);
            }
        }
    }
    // Single elements, through registers.
    __device__ static void fetch_narrow(const typename El<F32>::type *tile, int64_t ld, int x_left, int c_left,
                                        LDS_PTR unsigned char *lds) {
        for (int i = 0; i < LOADS; ++i) {
            int row, chunk;
            source(i * NT + threadIdx.x, row, chunk);
            union {
                typename El<F32>::type v[CE];
                u32x4_t r;
            } u;
            u.r = u32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < CE; ++e) {
                const int x = TALL ? chunk * CE + e : row, c = TALL ? row : chunk * CE + e;
                if (x < x_left && c < c_left) u.v[e] = tile[row * ld + chunk * CE + e];
            }
            *(LDS_PTR u32x4_t *)(lds + (i * NT + threadIdx.x) * 16) = u.r;
        }
    }

    // Fragment of the 16 values x0 .. x0+15 and the half `kk` of the step:
    // lane (i, j) holds value x0 + i and c = kk BK/2 + CE j + (0 .. CE-1).
    __device__ static typename El<F32>::frag read(LDS_PTR unsigned char *lds, int x0, int kk, int i, int j) {
        if constexpr (!TALL) {
            const int row = x0 + i;
            return *(LDS_PTR typename El<F32>::frag *)(lds + row * 128 + (((kk * 4 + j) ^ (row >> 1 & 7)) << 4));
        } else if constexpr (F32) {
            f32x4_t f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = kk * 16 + j * 4 + e;
                f[e] = *(LDS_PTR float *)(lds + row * X * 4 + (((x0 >> 4) ^ turn(row)) << 6) + i * 4);
            }
            return f;
        } else {
            // 16 lanes read a block of 4 rows by 16 values and get its columns
            const int row = kk * 32 + j * 8 + (i >> 2);
            LDS_PTR unsigned char *at = lds + row * X * 2 + (((x0 >> 4) ^ turn(row)) << 5) + (i & 3) * 8;
            // turn(row + 4) == turn(row)
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR s16x4_t *)at);
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR s16x4_t *)(at + 4 * X * 2));
            return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

template <bool F32> __device__ inline f32x4_t mma(typename El<F32>::frag b, typename El<F32>::frag a, f32x4_t acc) {
    if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(b[e], a[e], acc, 0, 0, 0);
        return acc;
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, acc, 0, 0, 0);
    }
}

// Tile of this workgroup.  Workgroups go round the 8 XCDs in turn; each XCD
// gets a run of neighbouring tiles (8 rows of tiles at a time), which share
// operand panels in its L2.
__device__ inline void place(const GemmParams &p, int &tm, int &tn, int &split) {
    const int total = gridDim.x, per = total / 8, rest = total % 8;
    const int xcd = blockIdx.x % 8, idx = blockIdx.x / 8;
    const int id = xcd * per + min(xcd, rest) + idx;
    const int tiles = p.tiles_m * p.tiles_n;
    split = id / tiles;
    const int t = id % tiles, band = 8 * p.tiles_n;
    const int first = t / band * 8, rows = min(p.tiles_m - first, 8);
    tm = first + t % band % rows;
    tn = t % band / rows;
}

// WM x WN waves, each MT x NTL tiles of 16 x 16.
template <bool F32, bool TALL_A, bool TALL_B, bool DIRECT, int WM, int WN, int MT, int NTL>
__global__ __launch_bounds__(64 * WM *WN, 2) void gemm_kernel(GemmParams p) {
    constexpr int NT = 64 * WM * WN, BM = WM * MT * 16, BN = WN * NTL * 16;
    using A = Operand<F32, TALL_A, BM, NT>;
    using B = Operand<F32, TALL_B, BN, NT>;
    using T = typename El<F32>::type;
    constexpr int BK = A::BK;
    // four variables, so that the compiler sees which one a direct load fills
    __shared__ __attribute__((aligned(16))) unsigned char a0[A::BYTES], a1[A::BYTES], b0[B::BYTES], b1[B::BYTES];

    int tm, tn, split;
    place(p, tm, tn, split);
    const int m0 = tm * BM, n0 = tn * BN;
    const int c_begin = split * p.c_per_split, c_end = min(p.C, c_begin + p.c_per_split);
    const T *a = (const T *)p.a + (TALL_A ? (int64_t)c_begin * p.lda + m0 : (int64_t)m0 * p.lda + c_begin);
    const T *b = (const T *)p.b + (TALL_B ? (int64_t)c_begin * p.ldb + n0 : (int64_t)n0 * p.ldb + c_begin);
    const int64_t step_a = TALL_A ? BK * p.lda : BK, step_b = TALL_B ? BK * p.ldb : BK;

    uint32_t off_a[A::LOADS], off_b[B::LOADS];
    if constexpr (DIRECT) {
        A::plan(off_a, p.lda, p.M - m0);
        B::plan(off_b, p.ldb, p.N - n0);
    }
    auto fetch = [&](unsigned char *la, unsigned char *lb, int c_left) {
        if constexpr (DIRECT) {
            A::fetch(a, off_a, c_left, (LDS_PTR unsigned char *)la);
            B::fetch(b, off_b, c_left, (LDS_PTR unsigned char *)lb);
        } else {
            A::fetch_narrow(a, p.lda, p.M - m0, c_left, (LDS_PTR unsigned char *)la);
            B::fetch_narrow(b, p.ldb, p.N - n0, c_left, (LDS_PTR unsigned char *)lb);
        }
        a += step_a;
        b += step_b;
    };

    const int wave = threadIdx.x >> 6, i = threadIdx.x & 15, j = (threadIdx.x >> 4) & 3;
    const int wm = wave / WN * MT * 16, wn = wave % WN * NTL * 16;
    f32x4_t acc[MT][NTL] = {};
    auto multiply = [&](unsigned char *la, unsigned char *lb) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            typename El<F32>::frag fa[MT], fb[NTL];
#pragma unroll
            for (int t = 0; t < NTL; ++t) fb[t] = B::read((LDS_PTR unsigned char *)lb, wn + t * 16, kk, i, j);
#pragma unroll
            for (int t = 0; t < MT; ++t) fa[t] = A::read((LDS_PTR unsigned char *)la, wm + t * 16, kk, i, j);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int u = 0; u < NTL; ++u) acc[t][u] = mma<F32>(fb[u], fa[t], acc[t][u]);
        }
    };

    // two steps a turn (past the end of c: zeros); a buffer is filled while the
    // other is multiplied, and the barrier (which waits for the fills) stands
    // between the two uses
    int left = c_end - c_begin;
    fetch(a0, b0, left);
    for (; left > 0; left -= 2 * BK) {
        __syncthreads();
        fetch(a1, b1, left - BK);
        multiply(a0, b0);
        __syncthreads();
        if (left > 2 * BK) fetch(a0, b0, left - 2 * BK);
        multiply(a1, b1);
    }

    if (p.partial) {
        float *out = p.partial + (int64_t)split * p.M * p.N;
        const bool vec = (p.N & 3) == 0;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = m0 + wm + t * 16 + i;
            if (m >= p.M) continue;
#pragma unroll
            for (int u = 0; u < NTL; ++u) {
                const int n = n0 + wn + u * 16 + j * 4;
                float *to = out + (int64_t)m * p.N + n;
                if (vec && n < p.N) {
                    *(f32x4_t *)to = acc[t][u];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < p.N) to[e] = acc[t][u][e];
                }
            }
        }
        return;
    }
#define FINISH(ACT)                                                                     \
    _Pragma("unroll") for (int t = 0; t < MT; ++t) {                                    \
        const int m = m0 + wm + t * 16 + i;                                             \
        if (m >= p.M) continue;                                                         \
        _Pragma("unroll") for (int u = 0; u < NTL; ++u) {                               \
            const float z[4] = {acc[t][u][0], acc[t][u][1], acc[t][u][2], acc[t][u][3]}; \
            finish4<F32, ACT>(p.e, m, n0 + wn + u * 16 + j * 4, z);                     \
        }                                                                               \
    }
    FOR_ACT(p.e.act, FINISH)
#undef FINISH
}

// Sums of the splits, then the epilogue: four columns a thread.
template <bool F32> __global__ __launch_bounds__(256) void split_kernel(GemmParams p) {
    const int quads = (p.N + 3) / 4;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= (int64_t)p.M * quads) return;
    const int64_t m = id / quads;
    const int n = (int)(id % quads) * 4;
    float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.splits; ++s) {
        const float *from = p.partial + ((int64_t)s * p.M + m) * p.N + n;
        if ((p.N & 3) == 0) {
            const f32x4_t v = *(const f32x4_t *)from;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] += v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) z[e] += from[e];
        }
    }
#define FINISH(ACT) finish4<F32, ACT>(p.e, m, n, z);
    FOR_ACT(p.e.act, FINISH)
#undef FINISH
}

// ---- few rows ----------------------------------------------------------------------

// For a few rows of x the weights stream through once and bound the time.  A
// workgroup owns 16 rows of w (16 columns of y) and MT x 16 rows of x; its
// waves cut c between them, and each loads its fragments of w and x straight
// from memory into the matrix cores' layout: lane (i, j) takes 32 bytes of row i
// at 128-byte steps, two chunks which serve two products (c is permuted alike
// for x and w).  The waves' sums meet in LDS.
struct RowsParams {
    const void *x, *w;
    int64_t ldx;
    int M, N, K;
    Epilogue e;
};

constexpr int kRowWaves = 8;

template <bool F32, bool WIDE, int MT>
__global__ __launch_bounds__(64 * kRowWaves) void rows_kernel(RowsParams p) {
    using T = typename El<F32>::type;
    using frag = typename El<F32>::frag;
    constexpr int CE = El<F32>::CE, BK = 8 * CE;
    __shared__ __attribute__((aligned(16))) float sums[kRowWaves][MT][16][16];
    const int wave = threadIdx.x >> 6, i = threadIdx.x & 15, j = (threadIdx.x >> 4) & 3;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * MT * 16;
    const bool n_in = n0 + i < p.N;
    const T *w = (const T *)p.w + (int64_t)(n_in ? n0 + i : 0) * p.K;

    auto load = [&](const T *row, bool in, int c) {
        union {
            u32x4_t r;
            T v[CE];
            frag f;
        } u;
        u.r = u32x4_t{0, 0, 0, 0};
        if constexpr (WIDE) {
            if (in && c < p.K) u.r = *(const u32x4_t *)(row + c);
        } else {
#pragma unroll
            for (int e = 0; e < CE; ++e)
                if (in && c + e < p.K) u.v[e] = row[c + e];
        }
        return u.f;
    };

    f32x4_t acc[MT] = {};
    // steps of BK in turn between the waves, two at a time
    for (int c0 = wave * BK; c0 < p.K; c0 += 2 * kRowWaves * BK) {
        frag fw[4], fx[MT][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) fw[s] = load(w, n_in, c0 + (s >> 1) * kRowWaves * BK + (j * 2 + (s & 1)) * CE);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = m0 + t * 16 + i;
            const T *x = (const T *)p.x + (int64_t)(m < p.M ? m : 0) * p.ldx;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                fx[t][s] = load(x, m < p.M, c0 + (s >> 1) * kRowWaves * BK + (j * 2 + (s & 1)) * CE);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[t] = mma<F32>(fw[s], fx[t][s], acc[t]);
    }
    // lane (i, j): row t 16 + i of x, columns 4 j .. 4 j + 3
#pragma unroll
    for (int t = 0; t < MT; ++t) *(f32x4_t *)&sums[wave][t][i][j * 4] = acc[t];
    __syncthreads();
    for (int id = threadIdx.x; id < MT * 64; id += 64 * kRowWaves) {
        const int t = id >> 6, r = id >> 2 & 15, q = (id & 3) * 4;
        const int64_t m = m0 + t * 16 + r;
        if (m >= p.M) continue;
        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kRowWaves; ++v) {
            const f32x4_t s = *(const f32x4_t *)&sums[v][t][r][q];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] += s[e];
        }
#define FINISH(ACT) finish4<F32, ACT>(p.e, m, n0 + q, z);
        FOR_ACT(p.e.act, FINISH)
#undef FINISH
    }
}

// ---- dz and db -----------------------------------------------------------------------

// dz = dy act'(z) (one element type rounding) and each block's column sums of
// the unrounded dz.  A block takes 32 lanes of V columns by `rows` rows.
struct DzParams {
    const void *dy, *z;
    void *dz;         // null: only the sums
    float *sums;      // [row blocks][N], or null
    int64_t M, lddy;
    int N, rows;
};

template <bool F32, int ACT, int V> __global__ __launch_bounds__(256) void dz_kernel(DzParams p) {
    __shared__ float part[8][32 * V];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int n = (blockIdx.x * 32 + cl) * V;
    const int64_t first = (int64_t)blockIdx.y * p.rows, last = min(p.M, first + p.rows);
    float sum[V] = {};
    if (n < p.N) {
#pragma unroll 4
        for (int64_t m = first + rl; m < last; m += 8) {
            float d[V], z[V];
            if constexpr (V == 4) {
                load4<F32>(p.dy, m * p.lddy + n, d);
                if constexpr (ACT != HYENA_ACT_NONE) load4<F32>(p.z, m * p.N + n, z);
            } else {
                d[0] = load1<F32>(p.dy, m * p.lddy + n);
                if constexpr (ACT != HYENA_ACT_NONE) z[0] = load1<F32>(p.z, m * p.N + n);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if constexpr (ACT != HYENA_ACT_NONE) d[e] *= act_slope<ACT>(z[e]);
                sum[e] += d[e];
            }
            if (p.dz) {
                if constexpr (V == 4) store4<F32>(p.dz, m * p.N + n, d);
                else store1<F32>(p.dz, m * p.N + n, d[0]);
            }
        }
    }
    if (!p.sums) return;
#pragma unroll
    for (int e = 0; e < V; ++e) part[rl][cl * V + e] = sum[e];
    __syncthreads();
    for (int c = threadIdx.x; c < 32 * V; c += 256) {
        const int col = blockIdx.x * 32 * V + c;
        if (col >= p.N) continue;
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += part[r][c];
        p.sums[(int64_t)blockIdx.y * p.N + col] = s;
    }
}

template <bool F32> __global__ __launch_bounds__(64) void db_kernel(const float *sums, int blocks, int N, void *db) {
    const int n = blockIdx.x * 64 + threadIdx.x;
    if (n >= N) return;
    float s = 0.0f;
    for (int b = 0; b < blocks; ++b) s += sums[(int64_t)b * N + n];
    store1<F32>(db, n, s);
}

// ---- host --------------------------------------------------------------------------------

constexpr int kRowsMost = 32;  // rows of x up to which rows_kernel is taken

struct Plan {
    bool large;  // 256 x 256 tiles (else 128 x 128)
    int tiles_m, tiles_n, splits, c_per_split;
};

// 256 x 256 tiles where they fill the card's 256 units about as well as 128 x
// 128 ones; c is split where there are too few tiles for all units.
Plan plan_of(int64_t M, int64_t N, int64_t C, bool f32, bool direct) {
    const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128), t256 = ceil_div(M, 256) * ceil_div(N, 256);
    const int64_t bk = f32 ? 32 : 64;
    Plan p;
    p.large = !f32 && direct && t256 >= 128 && 4 * ceil_div(t256, 256) <= ceil_div(t128, 256) * 5 / 4;
    const int64_t edge = p.large ? 256 : 128, tiles = p.large ? t256 : t128;
    p.tiles_m = (int)ceil_div(M, edge);
    p.tiles_n = (int)ceil_div(N, edge);
    int64_t splits = tiles >= 192 ? 1 : 256 / tiles;
    const int64_t most = ceil_div(C, 4 * bk);
    splits = splits < most ? splits : most;
    if (splits < 1) splits = 1;
    const int64_t steps = ceil_div(ceil_div(C, bk), splits);
    p.c_per_split = (int)(steps * bk);
    p.splits = C > 0 ? (int)ceil_div(C, steps * bk) : 1;
    if (C == 0) p.c_per_split = (int)bk;
    return p;
}

int64_t partial_bytes(int64_t M, int64_t N, int64_t C, bool f32) {
    int64_t most = 0;
    for (int direct = 0; direct < 2; ++direct) {
        const Plan p = plan_of(M, N, C, f32, direct);
        if (p.splits > 1 && p.splits * M * N * 4 > most) most = p.splits * M * N * 4;
    }
    return (most + 15) / 16 * 16;
}

bool epilogue_vec(const Epilogue &e, int64_t eb) {
    const int64_t b = 4 * eb;
    return e.N % 4 == 0 && e.ldy % 4 == 0 && aligned(e.y, b) && aligned(e.preact, b) && aligned(e.bias, b) &&
           (!e.residual || (e.ldr % 4 == 0 && aligned(e.residual, b)));
}

// C = A B^T with the epilogue, `partial` at least partial_bytes.
template <bool F32, bool TALL_A, bool TALL_B>
int gemm(const void *a, int64_t lda, const void *b, int64_t ldb, int64_t M, int64_t N, int64_t C, Epilogue e,
         float *partial, hipStream_t stream) {
    if (M == 0 || N == 0) return HYENA_OK;
    const int64_t eb = F32 ? 4 : 2, ce = 16 / eb;
    GemmParams p = {};
    p.a = a, p.b = b, p.lda = lda, p.ldb = ldb, p.M = (int)M, p.N = (int)N, p.C = (int)C;
    p.e = e;
    p.e.N = (int)N;
    p.e.vec = epilogue_vec(p.e, eb);
    // 16-byte chunks: aligned, none across an operand's edge, offsets in a tile below 2^31
    const bool direct = aligned(a, 16) && aligned(b, 16) && lda % ce == 0 && ldb % ce == 0 &&
                        (TALL_A ? M : C) % ce == 0 && (TALL_B ? N : C) % ce == 0 &&
                        lda < (int64_t)1 << 21 && ldb < (int64_t)1 << 21;
    const Plan pl = plan_of(M, N, C, F32, direct);
    p.tiles_m = pl.tiles_m, p.tiles_n = pl.tiles_n, p.splits = pl.splits, p.c_per_split = pl.c_per_split;
    p.partial = pl.splits > 1 ? partial : nullptr;
    const int64_t blocks = (int64_t)pl.tiles_m * pl.tiles_n * pl.splits;
    if (blocks > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks);
    if (pl.large) {
        if constexpr (!F32)
            hipLaunchKernelGGL((gemm_kernel<F32, TALL_A, TALL_B, true, 2, 4, 8, 4>), grid, dim3(512), 0, stream, p);
    } else if (direct) {
        hipLaunchKernelGGL((gemm_kernel<F32, TALL_A, TALL_B, true, 2, 2, 4, 4>), grid, dim3(256), 0, stream, p);
    } else {
        hipLaunchKernelGGL((gemm_kernel<F32, TALL_A, TALL_B, false, 2, 2, 4, 4>), grid, dim3(256), 0, stream, p);
    }
    if (p.partial) {
        const int64_t n = ceil_div(M * ceil_div(N, 4), 256);
        if (n > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
        hipLaunchKernelGGL(split_kernel<F32>, dim3((unsigned)n), dim3(256), 0, stream, p);
    }
    return launch_status();
}

template <bool F32>
int rows_product(const void *x, int64_t ldx, const void *w, int64_t M, int64_t N, int64_t K, Epilogue e,
                 hipStream_t stream) {
    const int64_t eb = F32 ? 4 : 2;
    RowsParams p = {};
    p.x = x, p.w = w, p.ldx = ldx, p.M = (int)M, p.N = (int)N, p.K = (int)K;
    p.e = e;
    p.e.N = (int)N;
    p.e.vec = epilogue_vec(p.e, eb);
    const bool wide = aligned(x, 16) && aligned(w, 16) && (ldx * eb) % 16 == 0 && (K * eb) % 16 == 0;
    const dim3 grid((unsigned)ceil_div(N, 16), 1), block(64 * kRowWaves);
    if (M <= 16)
        hipLaunchKernelGGL((wide ? rows_kernel<F32, true, 1> : rows_kernel<F32, false, 1>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((wide ? rows_kernel<F32, true, 2> : rows_kernel<F32, false, 2>), grid, block, 0, stream, p);
    return launch_status();
}

// Row blocks of dz_kernel.
int64_t dz_blocks(int64_t M, int64_t N) {
    const int64_t cols = ceil_div(N, 128);
    int64_t blocks = ceil_div(1024, cols);
    const int64_t most = ceil_div(M, 32);
    return blocks < most ? blocks : most;
}

template <bool F32>
int dz_and_db(const void *dy, int64_t lddy, const void *z, int act, int64_t M, int64_t N, void *dz, float *sums,
              void *db, hipStream_t stream) {
    if (N == 0) return HYENA_OK;
    const int64_t eb = F32 ? 4 : 2;
    const int64_t blocks = dz_blocks(M, N);
    if (M > 0) {
        DzParams p = {};
        p.dy = dy, p.z = z, p.dz = dz, p.sums = db ? sums : nullptr, p.M = M, p.lddy = lddy, p.N = (int)N;
        p.rows = (int)ceil_div(M, blocks);
        const bool vec = N % 4 == 0 && lddy % 4 == 0 && aligned(dy, 4 * eb) && aligned(z, 4 * eb);
        const dim3 grid((unsigned)ceil_div(N, vec ? 128 : 32), (unsigned)blocks);
#define DZ(ACT)                                                                                                    \
    hipLaunchKernelGGL((vec ? dz_kernel<F32, ACT, 4> : dz_kernel<F32, ACT, 1>), grid, dim3(256), 0, stream, p);
        FOR_ACT(act, DZ)
#undef DZ
    }
    if (db)
        hipLaunchKernelGGL(db_kernel<F32>, dim3((unsigned)ceil_div(N, 64)), dim3(64), 0, stream, sums,
                           M > 0 ? (int)blocks : 0, (int)N, db);
    return launch_status();
}

int check_linear(int64_t M, int64_t N, int64_t K, int act, int dtype) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    if (act < HYENA_ACT_NONE || act > HYENA_ACT_SIGMOID) return HYENA_ERR_UNSUPPORTED;
    int64_t n;
    if (!mul_fits(M, N, 4, &n) || !mul_fits(M, K, 4, &n) || !mul_fits(N, K, 4, &n)) return HYENA_ERR_SHAPE;
    const int64_t most = ((int64_t)1 << 31) - 1024;  // tile coordinates are 32 bits
    if (M > most || N > most || K > most) return HYENA_ERR_SHAPE;
    return HYENA_OK;
}

// Workspace of the backward: dz, the column sums, then a product's partials.
struct BwdSpace {
    int64_t dz, sums, partial;
};
BwdSpace bwd_space(int64_t M, int64_t N, int64_t K, int act, int dtype) {
    const bool f32 = dtype == HYENA_DTYPE_F32;
    BwdSpace s = {};
    if (act != HYENA_ACT_NONE) s.dz = (M * N * (f32 ? 4 : 2) + 15) / 16 * 16;
    if (M > 0 && N > 0) s.sums = (dz_blocks(M, N) * N * 4 + 15) / 16 * 16;
    if (M > 0 && N > 0 && K > 0) {
        const int64_t a = partial_bytes(M, K, N, f32), b = partial_bytes(N, K, M, f32);
        s.partial = a > b ? a : b;
    }
    return s;
}

template <bool F32>
int linear_bwd(const void *x, const void *w, const void *z, const void *dy, int64_t M, int64_t N, int64_t K,
               int64_t ldx, int64_t lddy, int64_t lddx, int act, void *dx, void *dw, void *db, char *ws,
               const BwdSpace &sp, hipStream_t stream) {
    const void *dz = dy;
    int64_t lddz = lddy;
    void *made = nullptr;
    if (act != HYENA_ACT_NONE && (dx || dw)) {
        dz = made = ws;
        lddz = N;
    }
    int st = HYENA_OK;
    if (made || db) st = dz_and_db<F32>(dy, lddy, z, act, M, N, made, (float *)(ws + sp.dz), db, stream);
    float *partial = (float *)(ws + sp.dz + sp.sums);
    Epilogue e = {};
    if (dx && st == HYENA_OK) {
        e.y = dx, e.ldy = lddx;
        st = gemm<F32, false, true>(dz, lddz, w, K, M, K, N, e, partial, stream);
    }
    if (dw && st == HYENA_OK) {
        e.y = dw, e.ldy = K;
        st = gemm<F32, true, true>(dz, lddz, x, ldx, N, K, M, e, partial, stream);
    }
    return st;
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
        *bytes_out = s.dz + s.sums + s.partial;
    } else {
        *bytes_out = M > kRowsMost && N > 0 ? partial_bytes(M, N, K, dtype == HYENA_DTYPE_F32) : 0;
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
    if (M <= kRowsMost)
        return f32 ? rows_product<true>(x, ldx, w, M, N, K, e, s) : rows_product<false>(x, ldx, w, M, N, K, e, s);
    return f32 ? gemm<true, false, false>(x, ldx, w, K, M, N, K, e, (float *)workspace, s)
               : gemm<false, false, false>(x, ldx, w, K, M, N, K, e, (float *)workspace, s);
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
    const void *z = act != HYENA_ACT_NONE ? preact : nullptr;
    const BwdSpace sp = bwd_space(M, N, K, act, dtype);
    hipStream_t s = (hipStream_t)stream;
    return dtype == HYENA_DTYPE_F32
               ? linear_bwd<true>(x, w, z, dy, M, N, K, ldx, lddy, lddx, act, dx, dw, db, (char *)workspace, sp, s)
               : linear_bwd<false>(x, w, z, dy, M, N, K, ldx, lddy, lddx, act, dx, dw, db, (char *)workspace, sp, s);
}

}  // extern "C"
