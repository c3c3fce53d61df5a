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
//     of one m, and the epilogue's way through LDS is in 16-byte accesses.
// Operands whose 16-byte chunks are not aligned (odd sizes, strides or
// pointers) cannot be fetched straight into LDS.  Where their sizes are odd and
// the product is long enough, they are copied to padded rows first; otherwise the
// same kernels take them through registers, a step ahead, with unaligned 16-byte
// loads.

#include <initializer_list>

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

// ---- V values of a row ------------------------------------------------------------

template <bool F32> struct El;
template <> struct El<false> {
    static constexpr int CE = 8;   // values per 16-byte chunk
    typedef bf16x8_t frag;
    typedef bf16_t type;
    typedef u32x4_t chunk_any __attribute__((aligned(2)));  // at any element's address
};
template <> struct El<true> {
    static constexpr int CE = 4;
    typedef f32x4_t frag;
    typedef float type;
    typedef u32x4_t chunk_any __attribute__((aligned(4)));
};

// V = 4 or 8 values as they lie in memory, read or written in as few accesses
// as possible at any element's address; n of them where that is fewer.
template <bool F32, int V> struct Pack {
    static constexpr int WORDS = F32 ? V : V / 2;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS > 4 ? 4 : WORDS)));
    typedef words words_any __attribute__((aligned(F32 ? 4 : 2)));
    static constexpr int PARTS = WORDS > 4 ? 2 : 1;
    words w[PARTS];

    __device__ static Pack zero() { return Pack{}; }
    __device__ uint32_t word(int i) const { return w[i / 4][i % 4]; }
    __device__ float get(int i) const {
        if constexpr (F32) return __uint_as_float(word(i));
        else return i & 1 ? bf_hi(word(i >> 1)) : bf_lo(word(i >> 1));
    }
    __device__ static Pack of(const float (&x)[V]) {
        Pack r;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.w[i / 4][i % 4] = F32 ? __float_as_uint(x[i]) : pack_bf16(x[2 * i % V], x[(2 * i + 1) % V]);
        return r;
    }
    __device__ static Pack load(const void *p, size_t e, int n) {
        using T = typename El<F32>::type;
        Pack r;
        if (n >= V) {
#pragma unroll
            for (int i = 0; i < PARTS; ++i) r.w[i] = *(const words_any *)((const T *)p + e + i * 4);
            return r;
        }
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < n ? load1<F32>(p, e + i) : 0.0f;
        return of(x);
    }
    __device__ static void store(void *p, size_t e, int n, const float (&x)[V]) {
        using T = typename El<F32>::type;
        if (n >= V) {
            const Pack r = of(x);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) *(words_any *)((T *)p + e + i * 4) = r.w[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) store1<F32>(p, e + i, x[i]);
        }
    }
};

struct Epilogue {
    const void *bias, *residual;
    void *y, *preact;
    int64_t ldr, ldy;
    int M, N;
    int act;
};

// The epilogue of columns n .. n + V - 1 of row m, z without its bias.
template <bool F32, int V>
__device__ __forceinline__ void finish(const Epilogue &p, int64_t m, int n, float (&z)[V], const Pack<F32, V> &bias,
                                       const Pack<F32, V> &residual) {
    using Q = Pack<F32, V>;
    const int left = p.N - n;
    if (m >= p.M || left <= 0) return;
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] += bias.get(e);
    if (p.preact) Q::store(p.preact, m * p.N + n, left, z);
#define ACTIVATE(ACT) \
    _Pragma("unroll") for (int e = 0; e < V; ++e) z[e] = act_value<ACT>(z[e]);
    if (p.act != HYENA_ACT_NONE) FOR_ACT(p.act, ACTIVATE)
#undef ACTIVATE
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] += residual.get(e);
    Q::store(p.y, m * p.ldy + n, left, z);
}
template <bool F32, int V> __device__ __forceinline__ Pack<F32, V> bias_of(const Epilogue &p, int n) {
    return p.bias ? Pack<F32, V>::load(p.bias, n, p.N - n) : Pack<F32, V>::zero();
}
template <bool F32, int V> __device__ __forceinline__ Pack<F32, V> residual_of(const Epilogue &p, int64_t m, int n) {
    return p.residual && m < p.M ? Pack<F32, V>::load(p.residual, m * p.ldr + n, p.N - n) : Pack<F32, V>::zero();
}

// ---- tiled product ---------------------------------------------------------------

struct GemmParams {
    const void *a, *b;
    int64_t lda, ldb;         // elements between memory rows of a and b
    int M, N, C;
    int tiles_m, tiles_n;
    int splits, c_per_split;  // c is cut into splits (a multiple of the step each, but the last)
    float *partial;           // splits > 1: [splits][M][N] sums for finish_kernel; else null
    Epilogue e;
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

    // Direct loads.  A lane's chunks are STEP rows of memory apart, and the XOR
    // repeats every 16 rows; off holds the byte offsets of the chunks before
    // that.  Values of m outside the matrix read zero: a flat tile's rows by the
    // descriptor's range, a tall tile's columns by an offset past every range.
    static constexpr uint32_t kOutside = 0x80000000u;
    static constexpr int STEP = NT / ROW_CHUNKS;
    static constexpr int PHASES = STEP >= 16 ? 1 : 16 / STEP;
    static_assert(NT % ROW_CHUNKS == 0 && (STEP % 16 == 0 || 16 % STEP == 0) && LOADS % PHASES == 0, "phases of the XOR");
    struct Lane {
        uint32_t off[PHASES], step, range;
    };
    __device__ static Lane plan(int64_t ld, int x_left) {
        const uint32_t pitch = (uint32_t)ld * sizeof(typename El<F32>::type);  // below 2^23 (the host checks)
        Lane l;
#pragma unroll
        for (int h = 0; h < PHASES; ++h) {
            int row, chunk;
            source(h * NT + threadIdx.x, row, chunk);
            l.off[h] = !TALL || chunk * CE < x_left ? row * pitch + chunk * 16 : kOutside;
        }
        l.step = STEP * pitch;
        l.range = TALL ? 0x7fffffffu : (uint32_t)min(x_left, X) * pitch;
        return l;
    }
    __device__ static void fetch(const typename El<F32>::type *tile, const Lane &l, int c_left,
                                 LDS_PTR unsigned char *lds) {
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void *)tile, (short)0, (int)l.range, 0x00020000);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        uint32_t at[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) at[i] = l.off[i % PHASES] + (i - i % PHASES) * l.step;
        if (c_left < BK) {  // the last step: zeros past the end of c
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                int row, chunk;
                source(i * NT + threadIdx.x, row, chunk);
                if ((TALL ? row : chunk * CE) >= c_left) at[i] = kOutside;
            }
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDS_PTR void *)(lds + (i * NT + wave * 64) * 16), 16, at[i], 0,
                                                     0, 0);
    }
    // The same chunks into registers, at any alignment ...
    __device__ static void pull(const typename El<F32>::type *tile, int64_t ld, int x_left, int c_left,
                                u32x4_t (&r)[LOADS]) {
        bool part = false;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            int row, chunk;
            source(i * NT + threadIdx.x, row, chunk);
            const int along = (TALL ? x_left : c_left) - chunk * CE;  // values left along memory's row
            r[i] = u32x4_t{0, 0, 0, 0};
            if (row < (TALL ? c_left : x_left)) {
                if (along >= CE) r[i] = *(const typename El<F32>::chunk_any *)(tile + row * ld + chunk * CE);
                else part |= along > 0;
            }
        }
        if (!any_lane(part)) return;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {  // chunks across the edge
            int row, chunk;
            source(i * NT + threadIdx.x, row, chunk);
            const int along = (TALL ? x_left : c_left) - chunk * CE;
            if (row < (TALL ? c_left : x_left) && along > 0 && along < CE) {
                typename El<F32>::type v[CE];
#pragma unroll
                for (int e = 0; e < CE; ++e)
                    v[e] = e < along ? tile[row * ld + chunk * CE + e] : (typename El<F32>::type)0.0f;
                r[i] = __builtin_bit_cast(u32x4_t, v);
            }
        }
    }
    // ... and from there into LDS.
    __device__ static void push(const u32x4_t (&r)[LOADS], LDS_PTR unsigned char *lds) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) *(LDS_PTR u32x4_t *)(lds + (i * NT + threadIdx.x) * 16) = r[i];
    }

    // Fragment t of the 16-value blocks from x0 on (a multiple of 16 times a
    // power of two no less than their number) and half kk of the step: lane (i,
    // j) holds value x0 + 16 t + i and c = kk BK/2 + CE j + (0 .. CE-1).  `at` is
    // start(x0, i, j); t and kk only enter as constants.
    __device__ static int start(int x0, int i, int j) {
        if constexpr (!TALL) {
            const int row = x0 + i;
            return row * 128 + ((j ^ (row >> 1 & 7)) << 4);
        } else if constexpr (F32) {
            const int row = j * 4;  // turn() is the same for the row's next three and 16 on
            return row * X * 4 + (((x0 >> 4) ^ turn(row)) << 6) + i * 4;
        } else {
            const int row = j * 8 + (i >> 2);  // turn() is the same 4 and 32 rows on
            return row * X * 2 + (((x0 >> 4) ^ turn(row)) << 5) + (i & 3) * 8;
        }
    }
    __device__ static typename El<F32>::frag read(LDS_PTR unsigned char *lds, int at, int t, int kk) {
        if constexpr (!TALL) {
            return *(LDS_PTR typename El<F32>::frag *)(lds + (at ^ kk << 6) + t * 2048);
        } else if constexpr (F32) {
            f32x4_t f;
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = *(LDS_PTR float *)(lds + (at ^ t << 6) + (kk * 16 + e) * X * 4);
            return f;
        } else {
            // 16 lanes read a block of 4 rows by 16 values and get its columns
            LDS_PTR unsigned char *from = lds + (at ^ t << 5) + kk * 32 * X * 2;
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR s16x4_t *)from);
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR s16x4_t *)(from + 4 * X * 2));
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

// Tile of workgroup `block` of `total`.  Workgroups go round the 8 XCDs in
// turn; each XCD gets a run of neighbouring tiles (8 rows of tiles at a time),
// which share operand panels in its L2.
__device__ inline void place(const GemmParams &p, int block, int &tm, int &tn, int &split) {
    const int tiles = p.tiles_m * p.tiles_n;
    const int total = tiles * p.splits, per = total / 8, rest = total % 8;
    const int xcd = block % 8, idx = block / 8;
    const int id = xcd * per + min(xcd, rest) + idx;
    split = id / tiles;
    const int t = id % tiles, band = 8 * p.tiles_n;
    const int first = t / band * 8, rows = min(p.tiles_m - first, 8);
    tm = first + t % band % rows;
    tn = t % band / rows;
}

// Waits until at most N of this wave's direct loads are on their way and for
// its LDS reads, then for the other waves.
template <int N> __device__ __forceinline__ void step_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | N >> 4 << 14);  // vmcnt(N) lgkmcnt(0), a form the compiler counts with
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A workgroup of WM x WN waves, each MT x NTL tiles of 16 x 16, with ST
// operand buffers: ST - 1 steps of c are on their way while one is multiplied.
// Bound by the matrix cores and the reads of LDS that feed them: at M = 8192, N
// = K = 4096 bf16, 256 x 256 tiles, the forward with bias and residual takes 236
// to 238 us in a row of calls (1.16 PFLOP/s), and in a trace of 30, where the
// clock falls under load, 243 us at least and 273 on average, dx = dz w 239 and
// 252, dw = dz^T x 227 and 240.
template <bool F32, int WM, int WN, int MT, int NTL, int ST> struct Shape {
    static constexpr int NT = 64 * WM * WN, BM = WM * MT * 16, BN = WN * NTL * 16;
    static constexpr int CE = El<F32>::CE, BK = 8 * CE;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGES = ST;
    static constexpr int LDS = ST * (A_BYTES + B_BYTES);
    static constexpr int WAVES = LDS > 80 * 1024 ? NT / 256 : LDS > 53 * 1024 ? NT / 128 : 3;  // a SIMD, by LDS

    // The workgroup's tile of one product; la and lb are the operands' buffers.
    template <bool TALL_A, bool TALL_B, bool DIRECT>
    __device__ __forceinline__ static void run(const GemmParams &p, int block, unsigned char *const (&la)[ST],
                                               unsigned char *const (&lb)[ST]) {
        using A = Operand<F32, TALL_A, BM, NT>;
        using B = Operand<F32, TALL_B, BN, NT>;
        using T = typename El<F32>::type;
        typedef LDS_PTR unsigned char *lds;
        int tm, tn, split;
        place(p, block, tm, tn, split);
        const int m0 = tm * BM, n0 = tn * BN;
        const int c_begin = split * p.c_per_split, c_end = min(p.C, c_begin + p.c_per_split);
        const T *a = (const T *)p.a + (TALL_A ? (int64_t)c_begin * p.lda + m0 : (int64_t)m0 * p.lda + c_begin);
        const T *b = (const T *)p.b + (TALL_B ? (int64_t)c_begin * p.ldb + n0 : (int64_t)n0 * p.ldb + c_begin);
        const int64_t step_a = TALL_A ? BK * p.lda : BK, step_b = TALL_B ? BK * p.ldb : BK;

        const int wave = threadIdx.x >> 6, i = threadIdx.x & 15, j = (threadIdx.x >> 4) & 3;
        const int wm = wave / WN * MT * 16, wn = wave % WN * NTL * 16;
        f32x4_t acc[MT][NTL] = {};
        const int start_a = A::start(wm, i, j), start_b = B::start(wn, i, j);
        auto multiply = [&](unsigned char *la, unsigned char *lb) {
            // hidden from the compiler, or it would keep the addresses of all
            // fragments in registers that the sums need
            int at_a = start_a, at_b = start_b;
            asm volatile("" : "+v"(at_a), "+v"(at_b));
            typename El<F32>::frag fa[2][MT], fb[2][NTL];
            auto read = [&](int kk) {
#pragma unroll
                for (int t = 0; t < NTL; ++t) fb[kk][t] = B::read((lds)lb, at_b, t, kk);
#pragma unroll
                for (int t = 0; t < MT; ++t) fa[kk][t] = A::read((lds)la, at_a, t, kk);
            };
            auto products = [&](int kk) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int u = 0; u < NTL; ++u) acc[t][u] = mma<F32>(fb[kk][u], fa[kk][t], acc[t][u]);
            };
            if constexpr (MT * NTL <= 16) {
                // registers for a whole step's fragments: all reads go out
                // first, and the second half's overlap the first's products
                read(0);
                read(1);
                __builtin_amdgcn_sched_barrier(0);
                products(0);
                products(1);
            } else {
                // the halves apart, so that their fragments share registers
                if (TALL_A) __builtin_amdgcn_sched_barrier(0);
                read(0);
                products(0);
                if (TALL_A) __builtin_amdgcn_sched_barrier(0);
                read(1);
                products(1);
            }
        };

        // ST steps a turn.  The barrier before a step waits for its fills, and
        // for every wave to be done with the buffer that is filled next.
        // Fills past the end of c are zeros, so that their number is the same.
        int left = c_end - c_begin;
        if constexpr (DIRECT) {
            constexpr int LOADS = A::LOADS + B::LOADS;
            const typename A::Lane lane_a = A::plan(p.lda, p.M - m0);
            const typename B::Lane lane_b = B::plan(p.ldb, p.N - n0);
            auto fetch = [&](int s, int c_left) {
                A::fetch(a, lane_a, c_left, (lds)la[s]);
                B::fetch(b, lane_b, c_left, (lds)lb[s]);
                a += step_a;
                b += step_b;
            };
#pragma unroll
            for (int s = 0; s < ST - 1; ++s) fetch(s, left - s * BK);
            for (; left > 0; left -= ST * BK) {
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    step_barrier<(ST - 2) * LOADS>();
                    fetch((s + ST - 1) % ST, left - (s + ST - 1) * BK);
                    if (ST == 2 || left > s * BK) multiply(la[s], lb[s]);
                }
            }
        } else {
            static_assert(DIRECT || ST == 2, "through registers: one step ahead");
            u32x4_t ra[A::LOADS], rb[B::LOADS];
            auto pull = [&](int c_left) {
                A::pull(a, p.lda, p.M - m0, c_left, ra);
                B::pull(b, p.ldb, p.N - n0, c_left, rb);
                a += step_a;
                b += step_b;
            };
            pull(left);
            A::push(ra, (lds)la[0]), B::push(rb, (lds)lb[0]);
            for (; left > 0; left -= 2 * BK) {
                __syncthreads();
                pull(left - BK);
                multiply(la[0], lb[0]);
                A::push(ra, (lds)la[1]), B::push(rb, (lds)lb[1]);
                __syncthreads();
                if (left > 2 * BK) pull(left - 2 * BK);
                multiply(la[1], lb[1]);
                A::push(ra, (lds)la[0]), B::push(rb, (lds)lb[0]);
            }
        }

        // The sums go through LDS, up to 64 rows by 64 columns a wave at a time in
        // a piece of its own, so that 8 lanes write a row's 64 columns: 16 bytes a
        // lane in bf16, whole 128-byte lines.  Rows are 256 bytes, their
        // 16-byte chunks XOR-ed with the row: no bank conflicts either way.
        constexpr int G = MT < 4 ? MT : 4, PIECE = G * 16 * 256;
        static_assert(NTL == 4 && MT % G == 0 && A_BYTES == B_BYTES && WM * WN * PIECE <= 4 * A_BYTES, "pieces of 64 columns");
        constexpr int PER = A_BYTES / PIECE;  // waves a buffer holds
        unsigned char *const buf[4] = {la[0], la[1], lb[0], lb[1]};
        lds piece = (lds)la[0];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (wave / PER == q) piece = (lds)buf[q] + wave % PER * PIECE;
        const int c8 = threadIdx.x & 7, r8 = (threadIdx.x >> 3) & 7;
        const int n = n0 + wn + c8 * 8;
        const Epilogue &ep = p.e;
        float *partial = p.partial ? p.partial + (int64_t)split * p.M * p.N : nullptr;
        const auto bias = partial ? Pack<F32, 8>::zero() : bias_of<F32, 8>(ep, n);
        // Every wave is done with the operands, and its fills past the end of c have
        // landed: the pieces lie where they go.
        step_barrier<0>();
#pragma unroll
        for (int g = 0; g < MT; g += G) {
            const int m = m0 + wm + g * 16 + r8;
            Pack<F32, 8> res[2 * G];
            if (!partial) {  // all fetched before the first store (y may be the residual)
#pragma unroll
                for (int r = 0; r < 2 * G; ++r) res[r] = residual_of<F32, 8>(ep, m + 8 * r, n);
            }
#pragma unroll
            for (int t = 0; t < G; ++t)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *(LDS_PTR f32x4_t *)(piece + (t * 16 + i) * 256 + (((u * 4 + j) ^ i) << 4)) = acc[g + t][u];
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the piece is this wave's own
#pragma unroll
            for (int r = 0; r < 2 * G; ++r) {
                const int row = r * 8 + r8;
                const f32x4_t lo = *(LDS_PTR f32x4_t *)(piece + row * 256 + (((c8 * 2) ^ (row & 15)) << 4));
                const f32x4_t hi = *(LDS_PTR f32x4_t *)(piece + row * 256 + (((c8 * 2 + 1) ^ (row & 15)) << 4));
                float z[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                if (partial) {
                    if (m + 8 * r < p.M && n < p.N)
                        Pack<true, 8>::store(partial, (int64_t)(m + 8 * r) * p.N + n, p.N - n, z);
                } else {
                    finish<F32, 8>(ep, m + 8 * r, n, z, bias, res[r]);
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    }
};

// an LDS variable for each buffer, so that the compiler sees which one a direct
// load fills and does not wait for it before it reads another
#define BUFFER(NAME, BYTES) __shared__ __attribute__((aligned(16))) unsigned char NAME[BYTES]
#define TILE_BUFFERS(S)                                                                                       \
    BUFFER(a0, S::A_BYTES); BUFFER(a1, S::A_BYTES); BUFFER(b0, S::B_BYTES); BUFFER(b1, S::B_BYTES);           \
    BUFFER(a2, S::STAGES > 2 ? S::A_BYTES : 16); BUFFER(b2, S::STAGES > 2 ? S::B_BYTES : 16);                 \
    BUFFER(a3, S::STAGES > 3 ? S::A_BYTES : 16); BUFFER(b3, S::STAGES > 3 ? S::B_BYTES : 16);

template <bool TALL_A, bool TALL_B, bool DIRECT, typename S>
__device__ __forceinline__ void run_tile(const GemmParams &p, int block, unsigned char *a0, unsigned char *a1,
                                         unsigned char *a2, unsigned char *a3, unsigned char *b0, unsigned char *b1,
                                         unsigned char *b2, unsigned char *b3) {
    if constexpr (S::STAGES == 2) S::template run<TALL_A, TALL_B, DIRECT>(p, block, {a0, a1}, {b0, b1});
    else if constexpr (S::STAGES == 3) S::template run<TALL_A, TALL_B, DIRECT>(p, block, {a0, a1, a2}, {b0, b1, b2});
    else S::template run<TALL_A, TALL_B, DIRECT>(p, block, {a0, a1, a2, a3}, {b0, b1, b2, b3});
}

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

template <bool F32> __device__ inline void sum_splits(const GemmParams &p, int64_t id) {
    const int quads = (p.N + 3) / 4;
    if (id >= (int64_t)p.M * quads) return;
    const int64_t m = id / quads;
    const int n = (int)(id % quads) * 4;
    const float *from = p.partial;
    float z[4] = {};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s, from += (int64_t)p.M * p.N) {
        const auto v = Pack<true, 4>::load(from, m * p.N + n, p.N - n);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] += v.get(e);
    }
    finish<F32, 4>(p.e, m, n, z, bias_of<F32, 4>(p.e, n), residual_of<F32, 4>(p.e, m, n));
}

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

// For a few rows of x the weights stream through once and bound the time.  A
// workgroup owns 16 rows of w (16 columns of y) and MT x 16 rows of x; its
// waves cut c between them, and each loads its fragments of w and x straight
// from memory into the matrix cores' layout: lane (i, j) takes two 16-byte chunks
// of row i at 128-byte steps, one of each 64 bytes, which serve two products.
// The waves' sums meet in LDS.  8 rows against 4096 x 4096 bf16 weights: 10.5 us
// (33.6 MB at 3.2 TB/s; a launch and one trip to memory are about 4.5 us of it).  A
// wave issues the next span's loads after it has multiplied the last one's, so a
// long row costs a trip to memory a span, four at K = 4096.
// 8 waves with 2 steps each in flight: 9.4 / 10.8 / 17.6 us for 1 row, 8 rows and
// 8 rows in fp32; 4 waves 11.2 / 11.2 / 20.3, 16 waves 10.1 / 11.1 / 19.1, 1 step
// 10.2 / 10.9 / 19.3, 4 steps 10.5 / 11.4 / 20.2.
struct RowsParams {
    const void *x, *w;
    int64_t ldx;
    int M, N, K;
    Epilogue e;
};

constexpr int kRowWaves = 8;
constexpr int kRowSteps = 2;  // steps of c in flight a wave

template <bool F32, int MT>
__global__ __launch_bounds__(64 * kRowWaves) void rows_kernel(RowsParams p) {
    using E = El<F32>;
    using T = typename E::type;
    using frag = typename E::frag;
    constexpr int CE = E::CE, BK = 8 * CE;
    __shared__ __attribute__((aligned(16))) float sums[kRowWaves][MT][16][16];
    const int wave = threadIdx.x >> 6, i = threadIdx.x & 15, j = (threadIdx.x >> 4) & 3;
    const int n0 = blockIdx.x * 16;
    const T *w = (const T *)p.w + (int64_t)(n0 + i) * p.K + j * CE;
    const T *x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) x[t] = (const T *)p.x + (int64_t)(t * 16 + i) * p.ldx + j * CE;

    f32x4_t acc[MT] = {};
    auto multiply = [&](const u32x4_t (&fw)[kRowSteps][2], const u32x4_t (&fx)[MT][kRowSteps][2]) {
#pragma unroll
        for (int s = 0; s < kRowSteps; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    acc[t] = mma<F32>(__builtin_bit_cast(frag, fw[s][h]), __builtin_bit_cast(frag, fx[t][s][h]), acc[t]);
    };
    // the waves take turns at spans of kRowSteps steps; c: the span's start
    const int span = kRowSteps * BK;
    int c = wave * span;
    for (; c + span <= p.K; c += kRowWaves * span) {
        u32x4_t fw[kRowSteps][2] = {}, fx[MT][kRowSteps][2] = {};
        if (n0 + i < p.N) {
#pragma unroll
            for (int s = 0; s < kRowSteps; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    fw[s][h] = __builtin_nontemporal_load((const typename E::chunk_any *)(w + c + s * BK + h * 4 * CE));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
            if (t * 16 + i < p.M) {
#pragma unroll
                for (int s = 0; s < kRowSteps; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) fx[t][s][h] = *(const typename E::chunk_any *)(x[t] + c + s * BK + h * 4 * CE);
            }
        multiply(fw, fx);
    }
    if (c < p.K) {  // the last span, cut short
        u32x4_t fw[kRowSteps][2] = {}, fx[MT][kRowSteps][2] = {};
        auto edge = [&](const T *row, int at) {
            const int left = p.K - at - j * CE;
            if (left >= CE) return (u32x4_t)*(const typename E::chunk_any *)(row + at);
            T v[CE];
#pragma unroll
            for (int e = 0; e < CE; ++e) v[e] = e < left ? row[at + e] : (T)0.0f;
            return __builtin_bit_cast(u32x4_t, v);
        };
#pragma unroll
        for (int s = 0; s < kRowSteps; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = c + s * BK + h * 4 * CE;
                if (n0 + i < p.N) fw[s][h] = edge(w, at);
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    if (t * 16 + i < p.M) fx[t][s][h] = edge(x[t], at);
            }
        multiply(fw, fx);
    }
    // lane (i, j): row t 16 + i of x, columns 4 j .. 4 j + 3
#pragma unroll
    for (int t = 0; t < MT; ++t) *(f32x4_t *)&sums[wave][t][i][j * 4] = acc[t];
    __syncthreads();
    if (threadIdx.x < MT * 64) {
        const int t = threadIdx.x >> 6, r = threadIdx.x >> 2 & 15, q = (threadIdx.x & 3) * 4;
        const int m = t * 16 + r, n = n0 + q;
        const auto bias = bias_of<F32, 4>(p.e, n), res = residual_of<F32, 4>(p.e, m, n);
        float z[4] = {};
#pragma unroll
        for (int v = 0; v < kRowWaves; ++v) {
            const f32x4_t x = *(const f32x4_t *)&sums[v][t][r][q];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] += x[e];
        }
        finish<F32, 4>(p.e, m, n, z, bias, res);
    }
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

template <bool F32> using Small = Shape<F32, 2, 2, 4, 4, 2>;  // 128 x 128 tiles, 4 waves, two workgroups a unit
template <bool F32> using Deep = Shape<F32, 2, 2, 4, 4, 4>;    // the same, three steps ahead, one workgroup a unit
template <bool F32> using Fine = Shape<F32, 4, 1, 1, 4, 2>;     // 64 x 64 tiles, 4 waves, up to five workgroups a unit
using FineDeep = Shape<false, 4, 1, 1, 4, 4>;                  // the same, three steps ahead, two workgroups a unit
using Large = Shape<false, 2, 4, 8, 4, 2>;                    // 256 x 256 tiles, 8 waves

// Products that run in one launch.
struct Plan {
    bool large, deep, fine;
    int tiles_m[2], tiles_n[2], splits[2], c_per_split[2];
    int64_t blocks[2], partial[2];  // workgroups; bytes of partial sums
};
struct Size {
    int64_t M, N, C;
};

// Steps of a split, and three times as many for c to be cut at all: the launch
// that adds the sums costs about as much as four.  (64 x 1024 x 1024, us in fp32
// and bf16: 9.2 / 7.1, with splits of 8 steps 10.7 / 7.8; cutting the 8 steps of
// 200 x 512 x 512 bf16 in two 7.0, uncut 5.2.)
constexpr int64_t kLeastSteps = 4;

// Tiles: 256 x 256 where they fill the card's 256 units about as well as 128 x
// 128 ones, 64 x 64 where there are fewer than 192 of 128 x 128 (forward at M =
// 1000, N = K = 1024 bf16 11 us, with split tiles of 128 x 128 20 us; at 500 x
// 1000 x 2000 15 against 20; fp32 at 1021 x 777 x 521 21 against 30 us, at 1024 x
// 768 x 512 14 against 23).
// Splits: c is cut where a workgroup would walk much more than its share of
// all steps.  One product is shared between 256 workgroups (in bf16 three steps
// ahead of its products where a unit has one); two products between 512, but two
// in fp32 of 64 x 64 tiles, whose blocks are of unlike length and few, between
// 1024.  (Backward at M = 256, N = K = 4096 bf16: 48 us with 512, 74 us with 256;
// forward 19 us with 256, 23 us with 512.  fp32 forward at 2048 x 2048 x 512 45 us
// with 256, 56 with 512.  fp32 backward of 64 x 64 tiles, with 512 and with 1024:
// 904 x 1100 x 600 50 and 40 us, 1021 x 777 x 521 44 and 40, 768 x 768 x 768 40
// and 35, 200 x 1500 x 1500 39.5 and 39, 300 x 300 x 300 and 640 x 1024 x 256 24
// and 24, but 500 x 700 x 900 28 and 30, 1500 x 500 x 400 29 and 31, 2000 x 400 x
// 400 29 and 33; of 128 x 128 tiles, 1300 x 1288 x 1288, 115 and 131.)
Plan plan_of(const Size *sz, int n, bool f32, bool direct) {
    int64_t t128 = 0, t256 = 0;
    const int64_t bk = f32 ? 32 : 64;
    for (int g = 0; g < n; ++g) {
        t128 += ceil_div(sz[g].M, 128) * ceil_div(sz[g].N, 128);
        t256 += ceil_div(sz[g].M, 256) * ceil_div(sz[g].N, 256);
    }
    Plan p = {};
    p.large = !f32 && direct && t256 >= 128 && 4 * ceil_div(t256, 256) <= ceil_div(t128, 256) * 5 / 4;
    p.fine = !p.large && t128 < 192;
    const int64_t edge = p.large ? 256 : p.fine ? 64 : 128;
    int64_t work = 0;
    for (int g = 0; g < n; ++g)
        work += ceil_div(sz[g].M, edge) * ceil_div(sz[g].N, edge) * (ceil_div(sz[g].C, bk) + 4);
    int64_t share = ceil_div(work, p.large ? 256 : f32 && p.fine && n == 2 ? 1024 : 256 * n);
    if (share < kLeastSteps) share = kLeastSteps;
    for (int g = 0; g < n; ++g) {
        p.tiles_m[g] = (int)ceil_div(sz[g].M, edge);
        p.tiles_n[g] = (int)ceil_div(sz[g].N, edge);
        const int64_t all = ceil_div(sz[g].C, bk);
        const int64_t splits = all * 2 > share * 3 && all >= 3 * kLeastSteps ? ceil_div(all, share) : 1;
        const int64_t steps = all > 0 ? ceil_div(all, splits) : 1;
        p.c_per_split[g] = (int)(steps * bk);
        p.splits[g] = all > 0 ? (int)ceil_div(all, steps) : 1;
        p.blocks[g] = (int64_t)p.tiles_m[g] * p.tiles_n[g] * p.splits[g];
        if (p.splits[g] > 1) p.partial[g] = (p.splits[g] * sz[g].M * sz[g].N * 4 + 15) / 16 * 16;
    }
    p.deep = direct && (p.fine ? !f32 && n == 1 : !p.large && p.blocks[0] + p.blocks[1] <= 256);
    return p;
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

// Workspace for the partial sums, whatever the operands' alignment.
int64_t partial_bytes(const Size *sz, int n, bool f32) {
    const Plan a = plan_of(sz, n, f32, false), b = plan_of(sz, n, f32, true);
    const int64_t x = a.partial[0] + a.partial[1], y = b.partial[0] + b.partial[1];
    return x > y ? x : y;
}

// Whether an operand can be fetched straight into LDS: aligned 16-byte chunks,
// none across its edge, offsets inside a tile below 2^31.
bool direct_ok(const void *p, int64_t ld, int64_t row, int64_t eb) {
    return aligned(p, 16) && (ld * eb) % 16 == 0 && (row * eb) % 16 == 0 && ld < (int64_t)1 << 21;
}

// Elements of n rounded up to whole 16 bytes.
int64_t whole(int64_t n, int64_t eb) { return ceil_div(n * eb, 16) * 16 / eb; }

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

GemmParams gemm_params(const Plan &pl, int g, const Size &sz, const void *a, int64_t lda, const void *b, int64_t ldb,
                       Epilogue e, char *&ws) {
    GemmParams p = {};
    p.a = a, p.b = b, p.lda = lda, p.ldb = ldb, p.M = (int)sz.M, p.N = (int)sz.N, p.C = (int)sz.C;
    p.tiles_m = pl.tiles_m[g], p.tiles_n = pl.tiles_n[g], p.splits = pl.splits[g], p.c_per_split = pl.c_per_split[g];
    p.e = e;
    p.e.M = p.M, p.e.N = p.N;
    if (pl.splits[g] > 1) {
        p.partial = (float *)ws;
        ws += pl.partial[g];
    }
    return p;
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
        RowsParams p = {};
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
