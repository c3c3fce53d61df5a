// Tiled matrix products on the matrix cores, with what happens to their sums as
// a parameter, for hyena_linear.hip and hyena_xent.hip.
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
#ifndef HYENA_LAYER_GEMM_H
#define HYENA_LAYER_GEMM_H

#include "layer_common.h"

namespace layer {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
#define LDS_PTR __attribute__((address_space(3)))

// ---- over the lanes of a wave --------------------------------------------------------

// x of the lane that a data-parallel move of the vector unit takes it from: without a
// trip through LDS, as a shuffle makes.
template <int CTRL> __device__ __forceinline__ float moved(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
// f of x over each 16 lanes, in all of them: pairs, fours, the other four of eight
// (mirrored: its lanes are alike by then), the other eight.
template <class F> __device__ __forceinline__ float over_16(float x, F f) {
    x = f(x, moved<0xB1>(x));
    x = f(x, moved<0x4E>(x));
    x = f(x, moved<0x141>(x));
    return f(x, moved<0x140>(x));
}
template <class F> __device__ __forceinline__ float over_32(float x, F f) {
    x = over_16(x, f);
    return f(x, __shfl_xor(x, 16));
}
__device__ __forceinline__ float wave_sum(float x) {
    const auto add = [](float a, float b) { return a + b; };
    x = over_32(x, add);
    return x + __shfl_xor(x, 32);
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
    __device__ static Pack from(u32x4_t v) {  // of 16 bytes
        static_assert(WORDS == 4, "16 bytes");
        return Pack{{__builtin_bit_cast(words, v)}};
    }
    __device__ static Pack of(const float (&x)[V]) {
        Pack r;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.w[i / 4][i % 4] = F32 ? __float_as_uint(x[i]) : pack_bf16(x[2 * i % V], x[(2 * i + 1) % V]);
        return r;
    }
    // STREAM: read (written) once, past the caches.
    template <bool STREAM = false> __device__ static Pack load(const void *p, size_t e, int n) {
        using T = typename El<F32>::type;
        Pack r;
        if (n >= V) {
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const words_any *at = (const words_any *)((const T *)p + e + i * 4);
                r.w[i] = STREAM ? __builtin_nontemporal_load(at) : *at;
            }
            return r;
        }
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < n ? load1<F32>(p, e + i) : 0.0f;
        return of(x);
    }
    template <bool STREAM = false> __device__ static void store(void *p, size_t e, int n, const float (&x)[V]) {
        using T = typename El<F32>::type;
        if (n >= V) {
            const Pack r = of(x);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                words_any *at = (words_any *)((T *)p + e + i * 4);
                if (STREAM) __builtin_nontemporal_store((words_any)r.w[i], at);
                else *at = r.w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) store1<F32>(p, e + i, x[i]);
        }
    }
};

// ---- tiled product ---------------------------------------------------------------

// E is what happens to the sums (the epilogue of V columns n .. of a row m):
//   e.columns<F32, V>(n)             what a lane holds for its columns,
//   e.before<F32, V>(m, n)           what it fetches for a row, all rows before the first store,
//   e.finish<F32, V>(m, n, z, c, r)  the sums z of one row with both,
//   e.close<F32, V>(c, m, block, n)  after the last row of row block `block`, the rows of one wave from m on,
// or, where E::kSums, e.sums<S>(...) on the sums as the matrix cores leave them.
// E::kRun: fp32 sums over c are formed in runs of so many values (0: in one), added up in
// order.  In fp32 the matrix cores round a sum once a product, so that one chain over a long c loses
// sqrt(c / 2) roundings' digits; bf16 products are summed 32 at a time.
template <class E> struct Gemm {
    const void *a, *b;
    const int *rows;          // GATHER: the memory row of each row of a, ascending; a tile's within 2^31 bytes
    int64_t lda, ldb;         // elements between memory rows of a and b
    int M, N, C;
    int tiles_m, tiles_n;
    int splits, c_per_split;  // c is cut into splits (a multiple of the step each, but the last)
    float *partial;           // splits > 1: [splits][M][N] sums for finish_kernel; else null
    E e;
};

// One operand's LDS tile of X values of m (or n) by one step of c.  GATHER (flat): its
// rows lie in memory where a list of row numbers says.
template <bool F32, bool TALL, int X, int NT, bool GATHER = false> struct Operand {
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
    static constexpr int PHASES = GATHER ? LOADS : STEP >= 16 ? 1 : 16 / STEP;
    static_assert(!GATHER || !TALL, "rows of a flat operand");
    static_assert(NT % ROW_CHUNKS == 0 && (STEP % 16 == 0 || 16 % STEP == 0) && LOADS % PHASES == 0, "phases of the XOR");
    struct Lane {
        uint32_t off[PHASES], step, range;
    };
    __device__ static Lane plan(int64_t ld, int x_left, const int *rows) {
        const uint32_t pitch = (uint32_t)ld * sizeof(typename El<F32>::type);  // below 2^23 (the host checks)
        Lane l;
#pragma unroll
        for (int h = 0; h < PHASES; ++h) {
            int row, chunk;
            source(h * NT + threadIdx.x, row, chunk);
            if constexpr (GATHER) l.off[h] = row < x_left ? (uint32_t)(rows[row] - rows[0]) * pitch + chunk * 16 : kOutside;
            else l.off[h] = !TALL || chunk * CE < x_left ? row * pitch + chunk * 16 : kOutside;
        }
        l.step = STEP * pitch;
        l.range = TALL || GATHER ? 0x7fffffffu : (uint32_t)min(x_left, X) * pitch;
        return l;
    }
    __device__ static void fetch(const typename El<F32>::type *tile, const Lane &l, int c_left,
                                 LDS_PTR unsigned char *lds) {
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void *)tile, (short)0, (int)l.range, 0x00020000);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        uint32_t at[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) at[i] = l.off[i % PHASES] + (i - i % PHASES) * l.step;  // (GATHER: off[i])
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
template <class E> __device__ inline void place(const Gemm<E> &p, int block, int &tm, int &tn, int &split) {
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
    template <bool TALL_A, bool TALL_B, bool DIRECT, bool GATHER, class E>
    __device__ __forceinline__ static void run(const Gemm<E> &p, int block, unsigned char *const (&la)[ST],
                                               unsigned char *const (&lb)[ST]) {
        using A = Operand<F32, TALL_A, BM, NT, GATHER>;
        using B = Operand<F32, TALL_B, BN, NT>;
        using T = typename El<F32>::type;
        typedef LDS_PTR unsigned char *lds;
        int tm, tn, split;
        place(p, block, tm, tn, split);
        const int m0 = tm * BM, n0 = tn * BN;
        const int c_begin = split * p.c_per_split, c_end = min(p.C, c_begin + p.c_per_split);
        const T *a = (const T *)p.a + (TALL_A   ? (int64_t)c_begin * p.lda + m0
                                       : GATHER ? (int64_t)p.rows[m0] * p.lda + c_begin
                                                : (int64_t)m0 * p.lda + c_begin);
        const T *b = (const T *)p.b + (TALL_B ? (int64_t)c_begin * p.ldb + n0 : (int64_t)n0 * p.ldb + c_begin);
        const int64_t step_a = TALL_A ? BK * p.lda : BK, step_b = TALL_B ? BK * p.ldb : BK;

        const int wave = threadIdx.x >> 6, i = threadIdx.x & 15, j = (threadIdx.x >> 4) & 3;
        const int wm = wave / WN * MT * 16, wn = wave % WN * NTL * 16;
        f32x4_t acc[MT][NTL] = {};
        constexpr bool RUNS = F32 && E::kRun > 0;
        f32x4_t before[RUNS ? MT : 1][RUNS ? NTL : 1] = {};
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
        // turn() while c is left, and the sums of each run to those before
        auto walk = [&](auto turn) {
            static_assert(E::kRun % (ST * BK) == 0, "runs of whole turns");
            if constexpr (RUNS) {
                while (left > E::kRun) {
#pragma unroll 1
                    for (int n = 0; n < E::kRun; n += ST * BK) turn();
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int u = 0; u < NTL; ++u) before[t][u] += acc[t][u], acc[t][u] = f32x4_t{};
                }
            }
            while (left > 0) turn();
        };
        if constexpr (DIRECT) {
            constexpr int LOADS = A::LOADS + B::LOADS;
            const typename A::Lane lane_a = A::plan(p.lda, p.M - m0, GATHER ? p.rows + m0 : nullptr);
            const typename B::Lane lane_b = B::plan(p.ldb, p.N - n0, nullptr);
            auto fetch = [&](int s, int c_left) {
                A::fetch(a, lane_a, c_left, (lds)la[s]);
                B::fetch(b, lane_b, c_left, (lds)lb[s]);
                a += step_a;
                b += step_b;
            };
#pragma unroll
            for (int s = 0; s < ST - 1; ++s) fetch(s, left - s * BK);
            walk([&] {
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    step_barrier<(ST - 2) * LOADS>();
                    fetch((s + ST - 1) % ST, left - (s + ST - 1) * BK);
                    if (ST == 2 || left > s * BK) multiply(la[s], lb[s]);
                }
                left -= ST * BK;
            });
        } else {
            static_assert(DIRECT || (ST == 2 && !GATHER), "through registers: one step ahead");
            u32x4_t ra[A::LOADS], rb[B::LOADS];
            auto pull = [&](int c_left) {
                A::pull(a, p.lda, p.M - m0, c_left, ra);
                B::pull(b, p.ldb, p.N - n0, c_left, rb);
                a += step_a;
                b += step_b;
            };
            pull(left);
            A::push(ra, (lds)la[0]), B::push(rb, (lds)lb[0]);
            walk([&] {
                __syncthreads();
                pull(left - BK);
                multiply(la[0], lb[0]);
                A::push(ra, (lds)la[1]), B::push(rb, (lds)lb[1]);
                __syncthreads();
                if (left > 2 * BK) pull(left - 2 * BK);
                multiply(la[1], lb[1]);
                A::push(ra, (lds)la[0]), B::push(rb, (lds)lb[0]);
                left -= 2 * BK;
            });
        }
        if constexpr (RUNS) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int u = 0; u < NTL; ++u) acc[t][u] += before[t][u];
        }

        if constexpr (E::kSums) {
            // Every wave is done with the operands, whose buffers the sums may use.
            step_barrier<0>();
            p.e.template sums<Shape>(p, acc, m0, n0, wm, wn, (lds)la[0]);
            return;
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
        const E &ep = p.e;
        float *partial = p.partial ? p.partial + (int64_t)split * p.M * p.N : nullptr;
        auto columns = ep.template columns<F32, 8>(partial ? p.N : n);
        // Every wave is done with the operands, and its fills past the end of c have
        // landed: the pieces lie where they go.
        step_barrier<0>();
#pragma unroll
        for (int g = 0; g < MT; g += G) {
            const int m = m0 + wm + g * 16 + r8;
            decltype(ep.template before<F32, 8>(0, 0)) res[2 * G];
            if (!partial) {  // all fetched before the first store (y may be the residual)
#pragma unroll
                for (int r = 0; r < 2 * G; ++r) res[r] = ep.template before<F32, 8>(m + 8 * r, n);
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
                    ep.template finish<F32, 8>(m + 8 * r, n, z, columns, res[r]);
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        if (!partial) ep.template close<F32, 8>(columns, m0 + wm, (m0 + wm) / (MT * 16), n);
    }
};

// an LDS variable for each buffer, so that the compiler sees which one a direct
// load fills and does not wait for it before it reads another
#define BUFFER(NAME, BYTES) __shared__ __attribute__((aligned(16))) unsigned char NAME[BYTES]
#define TILE_BUFFERS(S)                                                                                       \
    BUFFER(a0, S::A_BYTES); BUFFER(a1, S::A_BYTES); BUFFER(b0, S::B_BYTES); BUFFER(b1, S::B_BYTES);           \
    BUFFER(a2, S::STAGES > 2 ? S::A_BYTES : 16); BUFFER(b2, S::STAGES > 2 ? S::B_BYTES : 16);                 \
    BUFFER(a3, S::STAGES > 3 ? S::A_BYTES : 16); BUFFER(b3, S::STAGES > 3 ? S::B_BYTES : 16);

template <bool TALL_A, bool TALL_B, bool DIRECT, typename S, bool GATHER = false, class E>
__device__ __forceinline__ void run_tile(const Gemm<E> &p, int block, unsigned char *a0, unsigned char *a1,
                                         unsigned char *a2, unsigned char *a3, unsigned char *b0, unsigned char *b1,
                                         unsigned char *b2, unsigned char *b3) {
    if constexpr (S::STAGES == 2) S::template run<TALL_A, TALL_B, DIRECT, GATHER>(p, block, {a0, a1}, {b0, b1});
    else if constexpr (S::STAGES == 3) S::template run<TALL_A, TALL_B, DIRECT, GATHER>(p, block, {a0, a1, a2}, {b0, b1, b2});
    else S::template run<TALL_A, TALL_B, DIRECT, GATHER>(p, block, {a0, a1, a2, a3}, {b0, b1, b2, b3});
}

// The sums of the splits with their epilogue, four columns a thread.
template <bool F32, class E> __device__ inline void sum_splits(const Gemm<E> &p, int64_t id) {
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
    auto columns = p.e.template columns<F32, 4>(n);
    p.e.template finish<F32, 4>(m, n, z, columns, p.e.template before<F32, 4>(m, n));
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
template <class E> struct RowsParams {
    const void *x, *w;
    int64_t ldx;
    int M, N, K;
    E e;
};

constexpr int kRowWaves = 8;
constexpr int kRowSteps = 2;  // steps of c in flight a wave

template <bool F32, int MT, class E>
__device__ __forceinline__ void rows_product(const RowsParams<E> &p, int block, float (&sums)[kRowWaves][MT][16][16]) {
    using T = typename El<F32>::type;
    using frag = typename El<F32>::frag;
    using chunk_any = typename El<F32>::chunk_any;
    constexpr int CE = El<F32>::CE, BK = 8 * CE;
    const int wave = threadIdx.x >> 6, i = threadIdx.x & 15, j = (threadIdx.x >> 4) & 3;
    const int n0 = block * 16;
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
                    fw[s][h] = __builtin_nontemporal_load((const chunk_any *)(w + c + s * BK + h * 4 * CE));
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
            if (t * 16 + i < p.M) {
#pragma unroll
                for (int s = 0; s < kRowSteps; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) fx[t][s][h] = *(const chunk_any *)(x[t] + c + s * BK + h * 4 * CE);
            }
        multiply(fw, fx);
    }
    if (c < p.K) {  // the last span, cut short
        u32x4_t fw[kRowSteps][2] = {}, fx[MT][kRowSteps][2] = {};
        auto edge = [&](const T *row, int at) {
            const int left = p.K - at - j * CE;
            if (left >= CE) return (u32x4_t)*(const chunk_any *)(row + at);
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
        auto columns = p.e.template columns<F32, 4>(n);
        const auto before = p.e.template before<F32, 4>(m, n);
        float z[4] = {};
#pragma unroll
        for (int v = 0; v < kRowWaves; ++v) {
            const f32x4_t x = *(const f32x4_t *)&sums[v][t][r][q];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] += x[e];
        }
        p.e.template finish<F32, 4>(m, n, z, columns, before);
    }
}

// ---- host --------------------------------------------------------------------------------

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
inline Plan plan_of(const Size *sz, int n, bool f32, bool direct) {
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

// Workspace for the partial sums, whatever the operands' alignment.
inline int64_t partial_bytes(const Size *sz, int n, bool f32) {
    const Plan a = plan_of(sz, n, f32, false), b = plan_of(sz, n, f32, true);
    const int64_t x = a.partial[0] + a.partial[1], y = b.partial[0] + b.partial[1];
    return x > y ? x : y;
}

// Whether an operand can be fetched straight into LDS: aligned 16-byte chunks,
// none across its edge, offsets inside a tile below 2^31.
inline bool direct_ok(const void *p, int64_t ld, int64_t row, int64_t eb) {
    return aligned(p, 16) && (ld * eb) % 16 == 0 && (row * eb) % 16 == 0 && ld < (int64_t)1 << 21;
}

// Elements of n rounded up to whole 16 bytes.
inline int64_t whole(int64_t n, int64_t eb) { return ceil_div(n * eb, 16) * 16 / eb; }

template <class E>
Gemm<E> gemm_params(const Plan &pl, int g, const Size &sz, const void *a, int64_t lda, const void *b, int64_t ldb,
                    E e, char *&ws) {
    Gemm<E> p = {};
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

}  // namespace
}  // namespace layer

#endif
