// Values held in 8 or 4 bits: device helpers.  Included by .hip sources only.
//
// A group of 32 values has one bf16 scale s, the smallest with TOP s >= the largest
// magnitude (TOP = 127 or 7; 0 where that is below 2^-100; NaN where a value is
// infinite or NaN).  A value v has the code nearest to v / s, ties to even, and
// stands for code * s.  TOP s and code * s are exact in fp32 (8 + 7 bits), so every
// decision below is an exact one and the codes do not depend on how the quotient
// was approximated.  A bf16 scale instead of an fp32 one costs the codes nothing
// (they are taken against the rounded scale) and half the bytes; rounding it up
// keeps every code inside [-TOP, TOP].
#pragma once

#include "gdn_layer_device.h"

namespace gdn {
namespace dev {

constexpr float kHeldTiny = 7.888609052210118e-31f;   // 2^-100

// The scale, from the largest magnitude's bits (as an integer: above 0x7f7fffff is
// an infinity or a NaN).
template <int TOP> __device__ __forceinline__ float held_scale(uint32_t high_bits) {
    const float high = __uint_as_float(high_bits);
    uint32_t b = __float_as_uint(high * (1.f / TOP)) & 0xffff0000u;
    // the product is off by at most 2^-23, far less than a bf16 step: at most two steps up
    b += TOP * __uint_as_float(b) < high ? 0x10000u : 0u;
    b += TOP * __uint_as_float(b) < high ? 0x10000u : 0u;
    b = high < kHeldTiny ? 0u : b;
    return __uint_as_float(high_bits > 0x7f7fffffu ? 0x7fc00000u : b);
}
// 1 / s for held_code; 0 for the scales 0 and NaN, which gives the code 0.
__device__ __forceinline__ float held_inverse(float s) { return s > 0.f ? __builtin_amdgcn_rcpf(s) : 0.f; }

// 1.5 * 2^23: adding it rounds to the nearest integer, ties to even, and leaves that
// integer in the low bits.
constexpr float kRoundBias = 12582912.f;

// The code of v as two's complement in the low bits.  q = v / s to fp32's precision:
// one correction of v * (1/s).
//   bf16 v: where v / s is a tie, q is it exactly; elsewhere it is at least 2^-17
//   (relative) away from one, and q is on the right side.
//   fp32 v: v / s may be nearer to a tie than q's precision.  With k the integer
//   nearest to q, v - k s is exact (k s has 15 bits) and says which side it is.
template <typename E> __device__ __forceinline__ uint32_t held_code(float v, float s, float inv) {
    float q = v * inv;
    if constexpr (sizeof(E) == 2) {
        q = fmaf(fmaf(-q, s, v), inv, q);
        q = inv == 0.f ? 0.f : q;
        return __float_as_uint(q + kRoundBias);
    } else {
        float k = (q + kRoundBias) - kRoundBias;
        const float e = 2.f * fmaf(-k, s, v);          // twice what is left: within [-s, s] if k is right
        const bool odd = __float_as_uint(k + kRoundBias) & 1u;
        k = e > s || (odd && e == s) ? k + 1.f : e < -s || (odd && e == -s) ? k - 1.f : k;
        k = inv == 0.f ? 0.f : k;
        return __float_as_uint(k + kRoundBias);
    }
}

// Eight codes of 8 bits as two words.
__device__ __forceinline__ uint32_t pack4(const uint32_t *c) {
    const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(c[3], c[2], 0x04000c0c);
    return lo | hi;
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32u __attribute__((aligned(1)));
typedef uint16_t u16u __attribute__((aligned(1)));
// Eight codes of 8 bits, or the first n of them, at any address; S: past the caches.
template <bool S = false> __device__ __forceinline__ void store_codes(uint8_t *p, uint32_t a, uint32_t b, int n) {
    if (n == 8) {
        if constexpr (S)
            __builtin_nontemporal_store(u32x2{a, b}, (u32x2u *)p);
        else
            *(u32x2u *)p = u32x2u{a, b};
        return;
    }
    if (n & 4) {
        *(u32u *)p = a;
        a = b;
    }
    if (n & 2) {
        *(u16u *)(p + (n & 4)) = (uint16_t)a;
        a >>= 16;
    }
    if (n & 1) p[n - 1] = (uint8_t)a;
}
template <bool S = false> __device__ __forceinline__ u32x2 load_codes(const uint8_t *p, int n) {
    if (n == 8) {
        if constexpr (S) return __builtin_nontemporal_load((const u32x2u *)p);
        return *(const u32x2u *)p;
    }
    uint32_t a = 0, b = 0;
    if (n & 1) a = p[n - 1];
    if (n & 2) a = a << 16 | *(const u16u *)(p + (n & 4));
    if (n & 4) {
        b = a;
        a = *(const u32u *)p;
    }
    return u32x2{a, b};
}
// Code e of a word of four, as fp32.
__device__ __forceinline__ float held_byte(uint32_t w, int e) { return (float)(int)(int8_t)(w >> (8 * e)); }

}  // namespace dev
}  // namespace gdn
