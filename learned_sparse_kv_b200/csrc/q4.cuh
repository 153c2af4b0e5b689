// q4.cuh -- the 4-bit chunk pools: layout and conversions.
//
// A row of W values (one head of one token) is W / 16 groups of 16 consecutive values.  A
// value is an e2m1 code (0, .5, 1, 1.5, 2, 3, 4, 6 with a sign), a group has one e4m3 scale s,
// the pool one fp32 scale g:  value = e2m1 * s * g.  9 bits for two values: 0.5625 byte each.
// A chunk of one head is 36 W contiguous bytes: 64 code rows of W / 2 bytes (low nibble: even
// column), then 64 scale rows of W / 16 bytes, so that a window chunk is one contiguous block
// and a single row two pieces.  A pool is [n_slots, heads, 36 W].
//
// e2m1 * e4m3 has at most 6 significant bits and lies between 2^-10 and 2688, so every value
// (before g) is exact in f16 and in bf16: dequantising rounds nothing.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace lsa {
namespace q4 {

constexpr int GROUP = 16;
constexpr float E2M1_MAX = 6.f, E4M3_MAX = 448.f;

__host__ __device__ constexpr int64_t chunk_bytes(int W) { return 36 * (int64_t)W; }
__host__ __device__ constexpr int code_row(int W) { return W / 2; }
__host__ __device__ constexpr int scale_row(int W) { return W / GROUP; }
__host__ __device__ constexpr int scale_base(int W) { return LSA_CHUNK * (W / 2); }

// Eight e2m1 codes (nibble 2i and 2i + 1 in byte i) -> four f16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 bytes -> an f16 pair (low byte in the low half).
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The low / high half of an f16 pair in both halves.
__device__ __forceinline__ uint32_t dup_lo(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t h) { return __byte_perm(h, h, 0x3232); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// The 17 highest significant bits (16 of them stored).
__device__ __forceinline__ float cut17(float x) { return __uint_as_float(__float_as_uint(x) & ~0x7fu); }

// Half a group: eight values as four code bytes and, in scale_byte, the scale of the whole group, whose other half
// is with the neighbouring lane (lane ^ 1; both call together).
//   s = e4m3(min(amax / (6 g), 448)),  code = e2m1(x / (s g)), both to nearest even and
//   saturating; s = 0 stores zeros.  A NaN in the group gives a NaN scale: the whole group reads as NaN.
//   An infinity saturates the scale; the finite values of its group then read as they round.
// amax / 6 and x / s often lie exactly halfway between two codes, so a product with a rounded
// reciprocal will not do.  EXACT divides.  Otherwise (x of at most 11 significant bits, g a power of two, so
// s g has 4): a quotient X / S 2^k that is not the halfway point T 2^m is off it by at least 2^-11 of its
// size, because X 2^a and S T are whole numbers below 2^11 when both are scaled to the same size
// (T <= 7 and S <= 15 for the codes, T <= 31 and S = 6 for the scale).  The product with the approximate
// reciprocal is off by less than 2^-22; made larger by 2^-17 and cut to 17 significant bits it is the
// halfway point again where the quotient is (a halfway point is at most 31/16 of a power of two, and 31/16 (2^-17 +
// 2^-22) < 2^-16), and nothing else crosses one.
template <bool EXACT>
__device__ __forceinline__ uint32_t quantise_half(const float (&x)[8], float g, float g6, uint32_t &scale_byte) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(x[i]));
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    constexpr float UP = 1.f + 0x1p-17f;
    float t;
    if constexpr (EXACT) t = __fdiv_rn(amax, g6);
    else t = cut17(amax * (UP * g6));           // g6: 1 / (6 g) here
    uint16_t e;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e) : "f"(0.f), "f"(fminf(t, E4M3_MAX)));
    const float sg = __half2float(__ushort_as_half((uint16_t)e4m3x2_to_f16(e))) * g;
    scale_byte = amax != amax ? 0x7fu : (e & 0xffu);
    if (!(sg > 0.f)) return 0u;
    float y[8];
    if constexpr (EXACT) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], sg);
    } else {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sg));
        r *= UP;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = cut17(x[i] * r);
    }
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return w;
}

}  // namespace q4

// Element types of the entry points that take more than bf16 (LSA_DTYPE_*).
template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N consecutive elements as one or more aligned vector accesses of up to 16 bytes.
template <class T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Vec {
    T v[N];
};

// Pairs of elements: two from a 32-bit word (16-bit types), and back, rounding to nearest even.
template <class T> struct Two;
template <> struct Two<__nv_bfloat16> {
    static __device__ __forceinline__ float2 get(const Vec<__nv_bfloat16, 2> &v) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&v);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ void put(Vec<__nv_bfloat16, 2> &v, float a, float b) {
        *reinterpret_cast<uint32_t *>(&v) = pack_bf16x2(a, b);
    }
};
template <> struct Two<__half> {
    static __device__ __forceinline__ float2 get(const Vec<__half, 2> &v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    static __device__ __forceinline__ void put(Vec<__half, 2> &v, float a, float b) {
        *reinterpret_cast<uint32_t *>(&v) = q4::pack_f16x2(a, b);
    }
};
template <> struct Two<float> {
    static __device__ __forceinline__ float2 get(const Vec<float, 2> &v) { return make_float2(v.v[0], v.v[1]); }
    static __device__ __forceinline__ void put(Vec<float, 2> &v, float a, float b) { v.v[0] = a; v.v[1] = b; }
};
template <class T, int V>
__device__ __forceinline__ void widen(const Vec<T, V> &v, float (&x)[V]) {
    if constexpr (V == 1) {
        x[0] = to_f32(v.v[0]);
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 f = Two<T>::get(*reinterpret_cast<const Vec<T, 2> *>(&v.v[j]));
            x[j] = f.x;
            x[j + 1] = f.y;
        }
    }
}
template <class T, int V>
__device__ __forceinline__ Vec<T, V> narrow(const float (&x)[V]) {
    Vec<T, V> v;
    if constexpr (V == 1) {
        v.v[0] = from_f32<T>(x[0]);
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) Two<T>::put(*reinterpret_cast<Vec<T, 2> *>(&v.v[j]), x[j], x[j + 1]);
    }
    return v;
}

inline int dtype_size(int dtype) { return dtype == LSA_DTYPE_F32 ? 4 : 2; }
inline bool dtype_known(int dtype) { return dtype >= LSA_DTYPE_BF16 && dtype <= LSA_DTYPE_F32; }

}  // namespace lsa
