// Device-side helpers of the operators around the delta rule.  Included by
// their .hip sources only.
#pragma once

#include "gdn_device.h"
#include "gdn_layer.h"

namespace gdn {
namespace dev {

// Eight consecutive elements at an address aligned to one element: the
// hardware takes 16-byte accesses at any address, so rows of an odd length or
// stride need no path of their own.
typedef bf16 bf16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
struct f32x8p {
    f32x4 a, b;
};
template <typename E> struct Raw8;
template <> struct Raw8<bf16> {
    typedef bf16x8 T;
    static __device__ __forceinline__ T load(const bf16 *p) { return *(const bf16x8u *)p; }
    static __device__ __forceinline__ T zero() { return T{}; }
    static __device__ __forceinline__ float get(const T &r, int e) { return (float)r[e]; }
    static __device__ __forceinline__ void set(T &r, int e, float x) { r[e] = (bf16)x; }
    static __device__ __forceinline__ void store(bf16 *p, const T &r) { *(bf16x8u *)p = r; }
};
template <> struct Raw8<float> {
    typedef f32x8p T;
    static __device__ __forceinline__ T load(const float *p) {
        return T{*(const f32x4u *)p, *(const f32x4u *)(p + 4)};
    }
    static __device__ __forceinline__ T zero() { return T{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}; }
    static __device__ __forceinline__ float get(const T &r, int e) { return e < 4 ? r.a[e] : r.b[e - 4]; }
    static __device__ __forceinline__ void set(T &r, int e, float x) {
        if (e < 4)
            r.a[e] = x;
        else
            r.b[e - 4] = x;
    }
    static __device__ __forceinline__ void store(float *p, const T &r) {
        *(f32x4u *)p = r.a;
        *(f32x4u *)(p + 4) = r.b;
    }
};

// Elements p[0 .. n-1] (n <= 8, zeros behind them).
template <typename E> __device__ __forceinline__ typename Raw8<E>::T load_n(const E *p, int n) {
    if (n >= 8) return Raw8<E>::load(p);
    typename Raw8<E>::T r = Raw8<E>::zero();
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) Raw8<E>::set(r, e, to_f(p[e]));
    return r;
}
template <typename E> __device__ __forceinline__ void store_n(E *p, const typename Raw8<E>::T &r, int n) {
    if (n >= 8) {
        Raw8<E>::store(p, r);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = to_e<E>(Raw8<E>::get(r, e));
}
// The same of a weight that is fp32 or of type E.
template <typename E> __device__ __forceinline__ void load_w8(const void *w, int64_t at, int n, int f32, float *r) {
    if (f32) {
        const Raw8<float>::T v = load_n<float>((const float *)w + at, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = Raw8<float>::get(v, e);
    } else {
        const typename Raw8<E>::T v = load_n<E>((const E *)w + at, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = Raw8<E>::get(v, e);
    }
}

// 1 / (1 + e^-x) on the hardware exponential and reciprocal (about one ulp
// each); 0 and 1 in the tails.
__device__ __forceinline__ float sigmoid_f(float x) { return gate_beta(x); }

// First token and one past the last of sequence n, inside [0, T_tot].
__device__ __forceinline__ void seq_range(const int32_t *cu, int n, int T, int T_tot, int &t0, int &t1) {
    if (cu) {
        t0 = cu_at(cu, n, T_tot);
        t1 = max(t0, cu_at(cu, n + 1, T_tot));
    } else {
        t0 = n * T;
        t1 = t0 + T;
    }
}

}  // namespace dev
}  // namespace gdn
