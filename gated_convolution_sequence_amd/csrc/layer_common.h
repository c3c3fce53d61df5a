// What the sequence-layer kernels (hyena_scan.hip, hyena_step.hip,
// hyena_linear.hip) share: element access, gates, buffer descriptors and the
// host's argument checks.
#ifndef HYENA_LAYER_COMMON_H
#define HYENA_LAYER_COMMON_H

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "hyena_layer.h"

namespace layer {

typedef __bf16 bf16_t;
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStateRows = 64;  // rows between saved states (hyena_layer.h)

// ---- device -----------------------------------------------------------------

__device__ inline float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ inline uint32_t pack_bf16(float a, float b) {
    bf16x2_t r = {(__bf16)a, (__bf16)b};  // round to nearest even
    return __builtin_bit_cast(uint32_t, r);
}

// One element of a bf16 or fp32 array.
template <bool F32> __device__ inline float load1(const void *p, size_t i) {
    if constexpr (F32) return ((const float *)p)[i];
    else return (float)((const bf16_t *)p)[i];
}
template <bool F32> __device__ inline void store1(void *p, size_t i, float x) {
    if constexpr (F32) ((float *)p)[i] = x;
    else ((bf16_t *)p)[i] = (bf16_t)x;
}

// Whether any lane of the wave says so.
__device__ inline bool any_lane(bool x) { return __builtin_amdgcn_ballot_w64(x) != 0; }

// The decay a of a gate, and da/dg.  With e = exp(-g), sigmoid(g) = 1 / (1 + e)
// and its slope is e a^2, which keeps 1 - a exact to rounding where a is near
// 1.  a is 0 for g = -inf and for a finite g below -87.3, where it is below the
// least normal fp32; the slope of those is not used (nor a number where e
// overflows).
template <bool LOG> __device__ inline float decay(float g) {
    if constexpr (LOG) return __expf(g);
    else return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}
template <bool LOG> __device__ inline float decay_slope(float g, float a) {
    if constexpr (LOG) return a;
    else return __expf(-g) * a * a;
}

// What one lane reads and writes at a time: 16 bytes at any element's address
// (the hardware takes global accesses of any alignment), or the first n
// channels of them at the right edge of D.
template <bool F32> struct Lane;
template <> struct Lane<false> {
    static constexpr int VEC = 8;
    typedef u32x4_t raw;
    typedef u32x4_t raw_any __attribute__((aligned(2)));
    __device__ static raw load(const void *p, size_t e) {
        return __builtin_nontemporal_load((const raw_any *)((const bf16_t *)p + e));
    }
    __device__ static raw load_part(const void *p, size_t e, int n) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < n ? load1<false>(p, e + i) : 0.0f;
        return pack(x);
    }
    __device__ static float get(const raw &r, int i) { return i & 1 ? bf_hi(r[i >> 1]) : bf_lo(r[i >> 1]); }
    __device__ static raw pack(const float (&x)[8]) {
        return raw{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
    __device__ static void put(raw &r, int h, const float (&x)[2]) { r[h] = pack_bf16(x[0], x[1]); }  // channels 2 h, 2 h + 1
    __device__ static void store(void *p, size_t e, const raw &r) {
        __builtin_nontemporal_store(r, (raw_any *)((bf16_t *)p + e));
    }
    __device__ static void store_part(void *p, size_t e, const raw &r, int n) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) ((uint16_t *)p)[e + i] = (uint16_t)(r[i >> 1] >> (i & 1 ? 16 : 0));
    }
};
template <> struct Lane<true> {
    static constexpr int VEC = 4;
    typedef f32x4_t raw;
    typedef f32x4_t raw_any __attribute__((aligned(4)));
    __device__ static raw load(const void *p, size_t e) {
        return __builtin_nontemporal_load((const raw_any *)((const float *)p + e));
    }
    __device__ static raw load_part(const void *p, size_t e, int n) {
        raw r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = i < n ? load1<true>(p, e + i) : 0.0f;
        return r;
    }
    __device__ static float get(const raw &r, int i) { return r[i]; }
    __device__ static raw pack(const float (&x)[4]) { return raw{x[0], x[1], x[2], x[3]}; }
    __device__ static void put(raw &r, int h, const float (&x)[1]) { r[h] = x[0]; }
    __device__ static void store(void *p, size_t e, const raw &r) {
        __builtin_nontemporal_store(r, (raw_any *)((float *)p + e));
    }
    __device__ static void store_part(void *p, size_t e, const raw &r, int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) ((float *)p)[e + i] = r[i];
    }
};

// ---- host -------------------------------------------------------------------

// Rows of `width` bytes, `pitch` bytes apart.
struct Rows {
    const void *p;
    int64_t rows, width, pitch;
};

inline bool same_range(const Rows &a, const Rows &b) {
    return a.p == b.p && a.rows == b.rows && a.width == b.width && a.pitch == b.pitch;
}

// Whether two strided arrays share a byte.  Column slices of one buffer have
// the same pitch and interleave without sharing any; arrays of different
// pitch count as overlapping where their address ranges meet.
inline bool overlap(const Rows &a, const Rows &b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uint64_t a0 = (uint64_t)(uintptr_t)a.p, b0 = (uint64_t)(uintptr_t)b.p;
    const uint64_t an = (uint64_t)(a.rows - 1) * (uint64_t)a.pitch + (uint64_t)a.width;
    const uint64_t bn = (uint64_t)(b.rows - 1) * (uint64_t)b.pitch + (uint64_t)b.width;
    if (a0 < b0 ? b0 - a0 >= an : a0 - b0 >= bn) return false;
    if (a.pitch != b.pitch || (a.rows == 1 && b.rows == 1)) return true;
    const uint64_t pitch = (uint64_t)a.pitch;
    const uint64_t d = a0 <= b0 ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
    return d < (uint64_t)a.width || d + (uint64_t)b.width > pitch;
}

// bytes = a b c, false where that passes 2^62 or a factor is negative.
inline bool mul_fits(int64_t a, int64_t b, int64_t c, int64_t *out) {
    if (a < 0 || b < 0 || c < 0) return false;
    int64_t r;
    if (__builtin_mul_overflow(a, b, &r) || __builtin_mul_overflow(r, c, &r)) return false;
    if (r >= (int64_t)1 << 62) return false;
    *out = r;
    return true;
}

inline bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int launch_status() { return hipGetLastError() == hipSuccess ? HYENA_OK : HYENA_ERR_LAUNCH; }

}  // namespace layer

#endif
