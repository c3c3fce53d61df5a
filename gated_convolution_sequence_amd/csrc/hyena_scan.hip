// Gated linear recurrence along time for MI355X (gfx950):
//     s_t = a_t s_{t-1} + k_t v_t,   y_t = q_t s_t,   a = sigmoid(g) or exp(g),
// and its backward (hyena_layer.h has the formulas and layouts).
//
// Method.  A row maps the state by s -> a s + x, and such maps compose: over
// any run of rows s -> P s + S with P the product of the decays.  Time is cut
// into tiles of T rows; a workgroup owns one tile of C channels, keeps it in
// registers and works in three steps:
//   1. each lane composes its own R rows of each of its channels,
//   2. one lane per channel composes the tile's NS slices in LDS, publishes
//      the tile's (P, S), takes the state that enters the tile from the tiles
//      before it, and publishes the state that leaves it,
//   3. each lane walks its rows once more, from the state that enters them,
//      and writes its outputs.
// So every input is read once and every output written once (10 B a token and
// channel forward, 18 B backward in bf16), which is what bounds the kernels;
// two kernels with the tiles' maps in between would read g, k and v twice.
//
// Carries between workgroups (step 2).  Tile m of a chain publishes one 64-bit
// word per channel: first (P, S), then, once known, the state that leaves it.
// A tile reads the words of the kWindow tiles before it and walks forward from
// the nearest one that holds a state.  That state was reached by the same
// sequence of operations, so the result does not depend on which words were
// there yet: runs give the same bits.  The words are single relaxed atomics
// that carry their own readiness, so no fence is wanted.
// The waiting ends: tiles are handed out by a counter in chain order, so a
// workgroup only waits for workgroups that have started before it and the
// first unfinished one waits for none.
//
// P is held as m 2^e with an exponent of its own: over a tile it leaves the range
// of fp32 in ordinary use (128 gates of 0.5), and what it then makes of a large
// state, or with gates above 1 (gate "log", g > 0) of a small one, still counts.
//
// A gate of exactly 0 drops the state, whatever it holds: m is 0 exactly where a
// run holds such a gate.  A gate of NaN is not kept in m, which fmaxf would lose:
// S is NaN then, also where the run starts with it.

#include <float.h>

#include <type_traits>

#include "layer_common.h"

namespace layer {
namespace {

// Words a tile looks at in one go.  4, 8 or 16: level where there are many
// chains (forward at B = 1, L = 8192, D = 4096 bf16 68, 69 and 70 us); at D =
// 1024, where chains are few and carries wait, 30.1, 27.3 and 26.0 us; fp32 at 3
// x 1531 x 1000 28.4, 28.2 and 31.9 us.
constexpr int kWindow = 8;
constexpr int kMostCounters = 32;
constexpr int kCounterGap = 32;  // counters lie on lines of their own
constexpr uint32_t kEmpty = 0xffffffffu;  // high half of a word not yet written
constexpr uint32_t kState = 0xff800000u;  // high half of a word that holds a state (a map's exponent is less)
constexpr uint32_t kInfinite = 0xff7fffffu;  // high half of a map whose P is infinite

struct ScanParams {
    const void *q, *k, *v, *g, *dy;
    const float *s0, *ds_last, *states_in;
    void *y, *dq, *dk, *dv, *dg;
    float *s_last, *states, *ds0;
    int64_t B, L, D, ld, ldd;
    int64_t n_tiles, c_tiles;  // tiles of a chain, channel tiles of a row
    int64_t n_chains;          // B * c_tiles
    uint32_t *counters;        // tiles handed out so far, one every kCounterGap; null: one tile a chain, no carries
    int32_t n_counters;        // a power of two that divides n_chains
    uint64_t *words;           // [n_tiles][B][c_tiles * C]
};

// A product of decays.
struct Decay {
    float m;  // 0 or positive; infinite where a gate of the run is
    int e;    // of 2
};

// A run's gates lie between least and most.  Within these bounds the product P
// of a lane's rows (at most 8) is exact to rounding as it is.
__device__ inline bool plain(float least, float most) { return least >= 0x1p-15f && most <= 0x1p+15f; }

// m of a run that holds no gate of 0 (least = its smallest gate).
__device__ inline float keep_off_zero(float m, float least) {
    return least == 0.0f ? 0.0f : fmaxf(m, __uint_as_float(1u));
}

// s through a row, and through a run.
__device__ inline float apply(float a, float x, float s) { return a == 0.0f ? x : fmaf(a, s, x); }
__device__ inline float apply(Decay P, float S, float s) {
    return P.m == 0.0f ? S : S + __builtin_amdgcn_ldexpf(P.m * s, P.e);
}

// P with m in [0.5, 1), or 0.
__device__ inline Decay normal(Decay P) {
    return {__builtin_amdgcn_frexp_mantf(P.m), P.e + __builtin_amdgcn_frexp_expf(P.m)};
}

// Both runs one after the other; b normal.
template <bool LOG> __device__ inline Decay join(Decay a, Decay b) {
    const bool drops = LOG && (a.m == 0.0f || b.m == 0.0f);  // (a gate of 0 and an infinite one)
    return {drops ? 0.0f : a.m * b.m, a.e + b.e};
}

// P in the high half of a word: 9 bits of exponent (from 2^-254 to 2^254: past
// them it takes every fp32 to nothing or past the largest) and m's 23 bits.
template <bool LOG> __device__ inline uint32_t pack(Decay P) {
    const Decay n = normal(P);
    const uint32_t e = (uint32_t)(max(-254, min(254, n.e)) + 256);
    if (LOG && n.m > FLT_MAX) return kInfinite;
    return n.m == 0.0f ? 0u : e << 23 | (__float_as_uint(n.m) & 0x7fffffu);
}
template <bool LOG> __device__ inline Decay unpack(uint32_t hi) {
    Decay P = {hi == 0 ? 0.0f : __uint_as_float((hi & 0x7fffffu) | 0x3f000000u), (int)(hi >> 23) - 256};
    if (LOG && hi == kInfinite) P.m = __uint_as_float(0x7f800000u);
    return P;
}

// The state after a run's first row, taken from 0: x, or NaN where the gate is.
__device__ inline float from_zero(float a, float x) { return a == a ? x : a; }

__device__ inline void put_word(uint64_t *w, uint32_t hi, float lo) {
    __hip_atomic_store(w, ((uint64_t)hi << 32) | __float_as_uint(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that enters tile m of a chain whose words are `stride` apart;
// `first` enters tile 0.
template <bool LOG> __device__ inline float carry_in(uint64_t *words, int64_t stride, int64_t m, float first) {
    for (;;) {
        uint64_t w[kWindow];
#pragma unroll
        for (int i = 0; i < kWindow; ++i) {
            const int64_t at = m - 1 - i;
            w[i] = ((uint64_t)kState << 32) | __float_as_uint(first);
            if (at >= 0) w[i] = __hip_atomic_load(words + at * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        float s = 0.0f;
        bool known = false;
#pragma unroll
        for (int i = kWindow - 1; i >= 0; --i) {
            const uint32_t hi = (uint32_t)(w[i] >> 32);
            const float lo = __uint_as_float((uint32_t)w[i]);
            if (hi == kState) {
                s = lo;
                known = true;
            } else if (hi == kEmpty) {
                known = false;
            } else {
                s = apply(unpack<LOG>(hi), lo, s);
            }
        }
        if (known) return s;
        __builtin_amdgcn_s_sleep(1);
    }
}

// Empties the words and sets the counters back, in every call: the workspace
// may hold anything.  Bound by its launch (3 to 5 us; 8 us for the 34 MB of
// B = 4, L = 32768, D = 4096).
__global__ __launch_bounds__(256) void scan_init_kernel(uint32_t *counters, uint64_t *words, int64_t n) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) words[i] = ~(uint64_t)0;
    if (blockIdx.x == 0 && threadIdx.x < kMostCounters) counters[threadIdx.x * kCounterGap] = 0;
}

// No rows: the state that leaves is the one that enters.
__global__ __launch_bounds__(256) void scan_none_kernel(const float *from, float *to, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.0f;
}

// Geometry of a tile: R rows a lane, NS slices of them, LANES lanes a row.
template <bool F32, int THREADS, int ROWS, int LANES_> struct Tile {
    static constexpr int VEC = Lane<F32>::VEC, LANES = LANES_, NT = THREADS;
    static constexpr int R = ROWS;
    static constexpr int NS = NT / LANES;
    static constexpr int T = NS * R;
    static constexpr int C = LANES * VEC;
    static_assert(T % kStateRows == 0 && kStateRows % R == 0, "saved states lie on slices");
    static_assert(C <= NT, "a lane per channel");
};
// Rows of a wave's loads are 256 bytes in both.  The forward holds 4 x 8 x 8
// bf16 inputs a lane in flight, two workgroups a unit.  At B = 1, L = 8192 / B =
// 4, L = 32768, D = 4096 bf16 a call takes 69 / 928 us (separate q, k, v, g; 878 as
// slices of one buffer); with 4 rows a lane 77 / 1005, with 16 (which spill) 170
// / 2347, with 128-byte rows 73 / 871 but 35 against 28 us in fp32 at 3 x 1531 x
// 1000, with 512 threads 74 / 929.
// The backward holds five inputs: 4 rows a lane, three workgroups a unit (its 138
// registers do not let a fourth in), 131 / 1928 us (1708 with buffers placed
// otherwise); 8 rows spill (587 us), 128-byte rows 139 / 1936 (fp32 at 3 x 1531 x
// 1000 74 against 55 us), 512 threads 143 / 2195.
template <bool F32> using FwdTile = Tile<F32, 256, 8, 16>;
template <bool F32> using BwdTile = Tile<F32, 256, 4, 16>;

// Waits for this wave's LDS accesses and meets the others.  Loads from memory
// stay in flight (__syncthreads would wait for them).
__device__ inline void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Tiles in order: ticket i is tile i / n_chains of chain i % n_chains.
// Counter j hands out the tickets that are j modulo n_counters, so a chain's
// tiles come from one counter, in order.  One ticket a workgroup.
__device__ inline int64_t next_ticket(const ScanParams &p) {
    if (!p.counters) return blockIdx.x;
    const int j = blockIdx.x & (p.n_counters - 1);
    const uint32_t t = __hip_atomic_fetch_add(p.counters + j * kCounterGap, 1u, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
    return (int64_t)t * p.n_counters + j;
}

__device__ inline int64_t uniform(int64_t x) {
    return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32)) << 32) |
                     (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)x));
}

// Where a lane stands in the tile of a ticket.
template <typename G> struct Place {
    int64_t m, b, ct;    // chain position, batch row, channel tile
    int64_t t0, d0;      // the lane's first row and channel
    int n_ch;            // its channels; <= 0: none
    __device__ void set(const ScanParams &p, int64_t ticket, bool backward) {
        const int64_t chain = ticket % p.n_chains;
        m = ticket / p.n_chains;
        ct = chain % p.c_tiles;
        b = chain / p.c_tiles;
        t0 = (backward ? p.n_tiles - 1 - m : m) * G::T + threadIdx.x / G::LANES * G::R;
        d0 = ct * G::C + threadIdx.x % G::LANES * G::VEC;
        n_ch = (int)min((int64_t)G::VEC, p.D - d0);
    }
    // Row r of the lane in [B L]; rows past the end read the last one.
    __device__ size_t row(const ScanParams &p, int r) const {
        return (size_t)b * p.L + (t0 + r < p.L ? t0 + r : p.L - 1);
    }
};

// The gate of rows past the end, exactly 1.  Both factors of their products are
// cleared with it (the row they were read from may hold infinities), so that
// they pass the state and its gradient on unchanged.
template <bool F32, bool LOG> __device__ inline typename Lane<F32>::raw open_gate() {
    constexpr uint32_t one = LOG ? 0u : F32 ? 0x7f800000u : 0x7f807f80u;  // exp(0) or sigmoid(+inf)
    return __builtin_bit_cast(typename Lane<F32>::raw, u32x4_t{one, one, one, one});
}

// s -> a s + x; RESETS: where a may be 0 and must drop s.
template <bool RESETS> __device__ inline float walk(float a, float x, float s) {
    if constexpr (RESETS) return apply(a, x, s);
    else return fmaf(a, s, x);
}

// Forward: 8 bytes read and 2 written a token and channel in bf16, and bound by
// them: B = 1, L = 8192, D = 4096 in 68 us (5.0 TB/s: four rounds of workgroups,
// whose ends leave units idle), B = 4, L = 32768 in 870 to 890 us (6.1 TB/s).  fp32:
// 125 us (5.4 TB/s) at the first, 27 us (3.4 TB/s) at 3 x 1531 x 1000, whose 576
// workgroups are a round and a bit.
template <bool F32, bool LOG, bool PART>
__global__ __launch_bounds__(FwdTile<F32>::NT, 2) void scan_fwd_kernel(ScanParams p) {
    using G = FwdTile<F32>;
    using Ln = Lane<F32>;
    constexpr int VEC = G::VEC, R = G::R, NS = G::NS, C = G::C;
    __shared__ float sM[NS][C], sS[NS][C], sIn[C];
    __shared__ int sE[NS][C];
    __shared__ int64_t sTicket;

    if (threadIdx.x == 0) sTicket = next_ticket(p);
    __syncthreads();
    Place<G> at;
    at.set(p, uniform(sTicket), false);
    const int lane = threadIdx.x % G::LANES, slice = threadIdx.x / G::LANES;

    // 1. a and x of the lane's rows, and their composition
    float a[R][VEC], x[R][VEC];
    {
        typename Ln::raw g[R] = {}, k[R] = {}, v[R] = {};
        if (at.n_ch == VEC) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const size_t e = at.row(p, r) * p.ld + at.d0;
                g[r] = Ln::load(p.g, e);
                k[r] = Ln::load(p.k, e);
                v[r] = Ln::load(p.v, e);
            }
        } else if (PART && at.n_ch > 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const size_t e = at.row(p, r) * p.ld + at.d0;
                g[r] = Ln::load_part(p.g, e, at.n_ch);
                k[r] = Ln::load_part(p.k, e, at.n_ch);
                v[r] = Ln::load_part(p.v, e, at.n_ch);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                a[r][i] = decay<LOG>(Ln::get(g[r], i));
                x[r][i] = Ln::get(k[r], i) * Ln::get(v[r], i);
            }
        }
        if (at.t0 + R > p.L) {  // rows past the end pass the state on
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (at.t0 + r >= p.L) a[r][i] = 1.0f, x[r][i] = 0.0f;
        }
    }
    typename Ln::raw q[R] = {};
    if (p.y && at.n_ch == VEC) {
#pragma unroll
        for (int r = 0; r < R; ++r) q[r] = Ln::load(p.q, at.row(p, r) * p.ld + at.d0);
    } else if (PART && p.y && at.n_ch > 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) q[r] = Ln::load_part(p.q, at.row(p, r) * p.ld + at.d0, at.n_ch);
    }
    float P[VEC], S[VEC], least[VEC], least_of_all = 1.0f, most = 1.0f;
    int e[VEC] = {};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        least[i] = P[i] = a[0][i];
#pragma unroll
        for (int r = 1; r < R; ++r) {
            P[i] *= a[r][i];
            least[i] = fminf(least[i], a[r][i]);
        }
        least_of_all = fminf(least_of_all, least[i]);
        if constexpr (LOG) {
#pragma unroll
            for (int r = 0; r < R; ++r) most = fmaxf(most, a[r][i]);
        }
    }
    bool resets = false;
    if (any_lane(!plain(least_of_all, most))) {
        resets = any_lane(least_of_all == 0.0f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            P[i] = 1.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                P[i] *= __builtin_amdgcn_frexp_mantf(a[r][i]);
                e[i] += __builtin_amdgcn_frexp_expf(a[r][i]);
            }
        }
    }
    auto compose = [&](auto sel) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            S[i] = from_zero(a[0][i], x[0][i]);
#pragma unroll
            for (int r = 1; r < R; ++r) S[i] = walk<decltype(sel)::value>(a[r][i], x[r][i], S[i]);
        }
    };
    if (resets) compose(std::true_type());
    else compose(std::false_type());
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        sM[slice][lane * VEC + i] = keep_off_zero(P[i], least[i]);
        sE[slice][lane * VEC + i] = e[i];
        sS[slice][lane * VEC + i] = S[i];
    }
    lds_barrier();

    // 2. one lane per channel: the slices' maps from the tile's start on, and the carry
    if (threadIdx.x < C) {
        const int c = threadIdx.x;
        const int64_t d = at.ct * C + c;
        Decay P = {1.0f, 0};
        float S = 0.0f;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const Decay pj = normal({sM[j][c], sE[j][c]});
            const float sj = sS[j][c];
            sM[j][c] = P.m, sE[j][c] = P.e, sS[j][c] = S;
            P = join<LOG>(P, pj), S = apply(pj, sj, S);
        }
        const uint32_t word = pack<LOG>(P);
        P = unpack<LOG>(word);  // as the tiles after this one see it
        float in = p.s0 && d < p.D ? p.s0[at.b * p.D + d] : 0.0f;
        if (p.counters) {
            const int64_t pitch = p.c_tiles * C, stride = p.B * pitch;
            uint64_t *words = p.words + at.b * pitch + at.ct * C + c;
            if (at.m > 0) {
                if (at.m + 1 < p.n_tiles) put_word(words + at.m * stride, word, S);
                in = carry_in<LOG>(words, stride, at.m, in);
            }
            if (at.m + 1 < p.n_tiles) put_word(words + at.m * stride, kState, apply(P, S, in));
        }
        sIn[c] = in;
        if (p.s_last && at.m + 1 == p.n_tiles && d < p.D) p.s_last[at.b * p.D + d] = apply(P, S, in);
    }
    lds_barrier();

    // 3. the walk
    if (at.n_ch <= 0) return;
    float s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int c = lane * VEC + i;
        s[i] = apply(Decay{sM[slice][c], sE[slice][c]}, sS[slice][c], sIn[c]);
    }
    if (p.states && at.t0 % kStateRows == 0 && at.t0 < p.L) {
        const int64_t chunks = ceil_div(p.L, kStateRows);
        float *to = p.states + (at.b * chunks + at.t0 / kStateRows) * p.D + at.d0;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (!PART || i < at.n_ch) to[i] = s[i];
    }
    if (!p.y) return;
    auto outputs = [&](auto sel) {
        const size_t first = ((size_t)at.b * p.L + at.t0) * p.D + at.d0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[i] = walk<decltype(sel)::value>(a[r][i], x[r][i], s[i]);
                y[i] = Ln::get(q[r], i) * s[i];
            }
            if (at.t0 + r >= p.L) continue;
            if (!PART || at.n_ch == VEC) Ln::store(p.y, first + (size_t)r * p.D, Ln::pack(y));
            else Ln::store_part(p.y, first + (size_t)r * p.D, Ln::pack(y), at.n_ch);
        }
    };
    if (resets) outputs(std::true_type());
    else outputs(std::false_type());
}

// The backward walks chains from the end of time: c -> a (q dy + c) maps the
// gradient of a row's state to that of the row before, with the same decays.
// The states inside a tile are walked again from the saved state at its start:
// keeping all of them would be 4 more bytes a token and channel to write and read.
// 10 bytes read and 8 written a token and channel in bf16 and bound by them: B =
// 1, L = 8192, D = 4096 in 129 us (4.7 TB/s), B = 4, L = 32768 in 1.70 ms (5.7
// TB/s).  fp32: 235 us (5.1 TB/s) at the first.  3 x 1531 x 1000 in fp32 is 1152
// workgroups where 768 fit at three a unit, so half the card waits through the
// second round: 53 us (3.1 TB/s).
template <bool F32, bool LOG, bool PART>
__global__ __launch_bounds__(BwdTile<F32>::NT, PART ? 2 : 3) void scan_bwd_kernel(ScanParams p) {
    using G = BwdTile<F32>;
    using Ln = Lane<F32>;
    constexpr int VEC = G::VEC, R = G::R, NS = G::NS, C = G::C;
    __shared__ float sM[NS][C], sS[NS][C], sC[NS][C], sIn[C];
    __shared__ int sE[NS][C];
    __shared__ int64_t sTicket;

    if (threadIdx.x == 0) sTicket = next_ticket(p);
    __syncthreads();
    Place<G> at;
    at.set(p, uniform(sTicket), true);
    const int64_t n = p.n_tiles - 1 - at.m;  // the tile, counted in time
    const int lane = threadIdx.x % G::LANES, slice = threadIdx.x / G::LANES;

    // The inputs stay as they were loaded, and each channel's decays are
    // computed where they are wanted: twice, for a third of the registers.
    typename Ln::raw g[R] = {}, k[R] = {}, v[R] = {}, q[R] = {}, dy[R] = {};
    if (at.n_ch == VEC) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const size_t row = at.row(p, r), e = row * p.ld + at.d0;
            g[r] = Ln::load(p.g, e);
            k[r] = Ln::load(p.k, e);
            v[r] = Ln::load(p.v, e);
            q[r] = Ln::load(p.q, e);
            dy[r] = Ln::load(p.dy, row * p.D + at.d0);
        }
    } else if (PART && at.n_ch > 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const size_t row = at.row(p, r), e = row * p.ld + at.d0;
            g[r] = Ln::load_part(p.g, e, at.n_ch);
            k[r] = Ln::load_part(p.k, e, at.n_ch);
            v[r] = Ln::load_part(p.v, e, at.n_ch);
            q[r] = Ln::load_part(p.q, e, at.n_ch);
            dy[r] = Ln::load_part(p.dy, row * p.D + at.d0, at.n_ch);
        }
    }
    if (at.t0 + R > p.L) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (at.t0 + r >= p.L) {
                g[r] = open_gate<F32, LOG>();
                k[r] = v[r] = q[r] = dy[r] = typename Ln::raw{};
            }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float a[R], P, least, most = 1.0f, S, c = 0.0f;
        int e = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            a[r] = decay<LOG>(Ln::get(g[r], i));
            P = r == 0 ? a[0] : P * a[r];
            least = r == 0 ? a[0] : fminf(least, a[r]);
            if (LOG) most = fmaxf(most, a[r]);
        }
        if (any_lane(!plain(least, most))) {
            P = 1.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                P *= __builtin_amdgcn_frexp_mantf(a[r]);
                e += __builtin_amdgcn_frexp_expf(a[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float x = Ln::get(k[r], i) * Ln::get(v[r], i);
            S = r == 0 ? from_zero(a[0], x) : apply(a[r], x, S);
        }
#pragma unroll
        for (int r = R - 1; r >= 0; --r) c = apply(a[r], 0.0f, fmaf(Ln::get(q[r], i), Ln::get(dy[r], i), c));
        sM[slice][lane * VEC + i] = keep_off_zero(P, least);
        sE[slice][lane * VEC + i] = e;
        sS[slice][lane * VEC + i] = S;
        sC[slice][lane * VEC + i] = c;
    }
    lds_barrier();

    if (threadIdx.x < C) {
        const int c = threadIdx.x;
        const int64_t d = at.ct * C + c;
        // the maps from the tile's end back to the end of each slice
        Decay P = {1.0f, 0}, pj[NS];
        float S = 0.0f;
#pragma unroll
        for (int j = NS - 1; j >= 0; --j) {
            pj[j] = normal({sM[j][c], sE[j][c]});
            const float cj = sC[j][c];
            sM[j][c] = P.m, sE[j][c] = P.e, sC[j][c] = S;
            P = join<LOG>(P, pj[j]), S = apply(pj[j], cj, S);
        }
        const uint32_t word = pack<LOG>(P);
        P = unpack<LOG>(word);  // as the tiles after this one see it
        const int64_t pitch = p.c_tiles * C, stride = p.B * pitch;
        uint64_t *words = p.words + at.b * pitch + at.ct * C + c;
        if (p.counters && at.m > 0 && at.m + 1 < p.n_tiles) put_word(words + at.m * stride, word, S);
        // the state that enters each slice
        float s = 0.0f;
        if (d < p.D) s = p.states_in[(at.b * ceil_div(p.L, kStateRows) + n * (G::T / kStateRows)) * p.D + d];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const float sj = sS[j][c];
            sS[j][c] = s;
            s = apply(pj[j], sj, s);
        }
        float in = p.ds_last && d < p.D ? p.ds_last[at.b * p.D + d] : 0.0f;
        if (p.counters) {
            if (at.m > 0) in = carry_in<LOG>(words, stride, at.m, in);
            if (at.m + 1 < p.n_tiles) put_word(words + at.m * stride, kState, apply(P, S, in));
        }
        sIn[c] = in;
        if (p.ds0 && at.m + 1 == p.n_tiles && d < p.D) p.ds0[at.b * p.D + d] = apply(P, S, in);
    }
    lds_barrier();
    if (at.n_ch <= 0) return;

    // Or the compiler would keep what it computed from them above in registers.
#pragma unroll
    for (int r = 0; r < R; ++r) asm volatile("" : "+v"(g[r]), "+v"(k[r]), "+v"(v[r]), "+v"(q[r]), "+v"(dy[r]));
    // Two channels at a time (one, in fp32): their gradients take the place of
    // their inputs, dq of q, dk of k, dv of v and dg of g.
    constexpr int PAIR = F32 ? 1 : 2;
#pragma unroll
    for (int h = 0; h < VEC / PAIR; ++h) {
        float dq[R][PAIR], dk[R][PAIR], dv[R][PAIR], dg[R][PAIR];
#pragma unroll
        for (int w = 0; w < PAIR; ++w) {
            const int i = h * PAIR + w, ch = lane * VEC + i;
            float a[R], s[R + 1];  // s[r]: before row r
            s[0] = sS[slice][ch];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                a[r] = decay<LOG>(Ln::get(g[r], i));
                s[r + 1] = apply(a[r], Ln::get(k[r], i) * Ln::get(v[r], i), s[r]);
            }
            float c = apply(Decay{sM[slice][ch], sE[slice][ch]}, sC[slice][ch], sIn[ch]);
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                const float dyi = Ln::get(dy[r], i), ds = fmaf(Ln::get(q[r], i), dyi, c);
                dq[r][w] = dyi * s[r + 1];
                dk[r][w] = ds * Ln::get(v[r], i);
                dv[r][w] = ds * Ln::get(k[r], i);
                dg[r][w] = ds * s[r] * decay_slope<LOG>(Ln::get(g[r], i), a[r]);
                c = a[r] * ds;
                if (a[r] == 0.0f) dg[r][w] = c = 0.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Ln::put(q[r], h, dq[r]);
            Ln::put(k[r], h, dk[r]);
            Ln::put(v[r], h, dv[r]);
            Ln::put(g[r], h, dg[r]);
        }
    }
    // Computed here, not sunk into the branches of the stores with all it takes.
#pragma unroll
    for (int r = 0; r < R; ++r) asm volatile("" : "+v"(g[r]), "+v"(k[r]), "+v"(v[r]), "+v"(q[r]));
    const size_t to = ((size_t)at.b * p.L + at.t0) * p.ldd + at.d0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (at.t0 + r >= p.L) break;
        const size_t o = to + (size_t)r * p.ldd;
        if (!PART || at.n_ch == VEC) {
            if (p.dq) Ln::store(p.dq, o, q[r]);
            if (p.dk) Ln::store(p.dk, o, k[r]);
            if (p.dv) Ln::store(p.dv, o, v[r]);
            if (p.dg) Ln::store(p.dg, o, g[r]);
        } else {
            if (p.dq) Ln::store_part(p.dq, o, q[r], at.n_ch);
            if (p.dk) Ln::store_part(p.dk, o, k[r], at.n_ch);
            if (p.dv) Ln::store_part(p.dv, o, v[r], at.n_ch);
            if (p.dg) Ln::store_part(p.dg, o, g[r], at.n_ch);
        }
    }
}

// Rows and channels of the smallest tile of any variant bound the words.
constexpr int64_t kLeastRows = 64, kMostChannels = 128;
constexpr int64_t kHeader = kMostCounters * kCounterGap * 4;

int check_sizes(int64_t B, int64_t L, int64_t D, int gate, int dtype) {
    if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_DTYPE;
    if (gate != HYENA_GATE_SIGMOID && gate != HYENA_GATE_LOG) return HYENA_ERR_UNSUPPORTED;
    int64_t n;
    if (B < 0 || L < 0 || D < 0) return HYENA_ERR_SHAPE;
    if (L > (int64_t)1 << 40 || D > (int64_t)1 << 30 || B > (int64_t)1 << 30) return HYENA_ERR_SHAPE;
    if (!mul_fits(B, L, 1, &n) || !mul_fits(n, D + kMostChannels, 4, &n)) return HYENA_ERR_SHAPE;
    return HYENA_OK;
}

int64_t workspace_bytes(int64_t B, int64_t L, int64_t D) {
    if (L <= kLeastRows || B == 0 || D == 0) return 0;
    return kHeader + 8 * ceil_div(L, kLeastRows) * B * (ceil_div(D, kMostChannels) * kMostChannels);
}

template <typename G, typename K> int launch(K kernel, ScanParams p, void *workspace, void *stream) {
    static_assert(G::T >= kLeastRows && kMostChannels % G::C == 0, "the workspace holds every variant's words");
    p.n_tiles = ceil_div(p.L, G::T);
    p.c_tiles = ceil_div(p.D, G::C);
    p.n_chains = p.B * p.c_tiles;
    int64_t blocks;
    if (!mul_fits(p.n_tiles, p.n_chains, 1, &blocks) || blocks > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    hipStream_t s = (hipStream_t)stream;
    if (p.n_tiles > 1) {
        p.counters = (uint32_t *)workspace;
        p.words = (uint64_t *)((char *)workspace + kHeader);
        // Several counters spare the first workgroups the wait for one (B = 1, L =
        // 8192: 69 against 71 us; 3 x 1531 x 1000 fp32: 28 against 33 us); one
        // keeps the tiles in flight closer together in memory, which counts once
        // there are many rounds of them (B = 4, L = 32768: 928 against 1018 us).
        p.n_counters = 1;
        while (blocks <= 8192 && p.n_counters < kMostCounters && p.n_chains % (2 * p.n_counters) == 0) p.n_counters *= 2;
        const int64_t words = p.n_tiles * p.n_chains * G::C;
        const int64_t grid = ceil_div(words, 1024);
        hipLaunchKernelGGL(scan_init_kernel, dim3((unsigned)(grid < 2048 ? grid : 2048)), dim3(256), 0, s, p.counters,
                           p.words, words);
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(G::NT), 0, s, p);
    return launch_status();
}

int launch_none(const float *from, float *to, int64_t n, void *stream) {
    if (!to) return HYENA_OK;
    if (ceil_div(n, 256) > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(scan_none_kernel, dim3((unsigned)ceil_div(n, 256)), dim3(256), 0, (hipStream_t)stream, from, to, n);
    return launch_status();
}

// PART: some lane at the right edge of D has less than its channels.
template <bool F32, bool LOG> int launch_fwd(const ScanParams &p, void *ws, void *stream) {
    const bool part = p.D % Lane<F32>::VEC != 0;
    return launch<FwdTile<F32>>(part ? scan_fwd_kernel<F32, LOG, true> : scan_fwd_kernel<F32, LOG, false>, p, ws, stream);
}
template <bool F32, bool LOG> int launch_bwd(const ScanParams &p, void *ws, void *stream) {
    const bool part = p.D % Lane<F32>::VEC != 0;
    return launch<BwdTile<F32>>(part ? scan_bwd_kernel<F32, LOG, true> : scan_bwd_kernel<F32, LOG, false>, p, ws, stream);
}

}  // namespace
}  // namespace layer

using namespace layer;

extern "C" {

int hyena_scan_workspace(int64_t B, int64_t L, int64_t D, int dtype, int64_t *bytes_out) {
    const int st = check_sizes(B, L, D, HYENA_GATE_SIGMOID, dtype);
    if (st != HYENA_OK) return st;
    if (!bytes_out) return HYENA_ERR_NULL;
    *bytes_out = workspace_bytes(B, L, D);
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
    if (!y && !s_last && !states) return L > 0 ? HYENA_ERR_NULL : HYENA_OK;
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
    if (L == 0) return launch_none(s0, s_last, B * D, stream);
    if (f32) return lg ? launch_fwd<true, true>(p, workspace, stream) : launch_fwd<true, false>(p, workspace, stream);
    return lg ? launch_fwd<false, true>(p, workspace, stream) : launch_fwd<false, false>(p, workspace, stream);
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
    if (!dq && !dk && !dv && !dg && !ds0) return L > 0 ? HYENA_ERR_NULL : HYENA_OK;
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
    if (L == 0) return launch_none(ds_last, ds0, B * D, stream);
    if (f32) return lg ? launch_bwd<true, true>(p, workspace, stream) : launch_bwd<true, false>(p, workspace, stream);
    return lg ? launch_bwd<false, true>(p, workspace, stream) : launch_bwd<false, false>(p, workspace, stream);
}

}  // extern "C"
