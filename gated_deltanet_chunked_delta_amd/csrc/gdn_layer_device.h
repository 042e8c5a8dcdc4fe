// Device-side helpers of the operators around the delta rule.  Included by
// their .hip sources only.
#pragma once

#include "gdn_device.h"
#include "gdn_layer.h"

namespace gdn {
namespace dev {

// N = 4 or 8 consecutive elements, as loaded, at an address aligned to one
// element: the hardware takes 16-byte accesses at any address, so rows of an odd
// length or stride need no path of their own.
typedef bf16 bf16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef bf16 bf16x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x2u __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2u __attribute__((ext_vector_type(2), aligned(4)));
struct f32x8p {
    f32x4 a, b;
};
// S: past the caches, for passes over more than they hold.
template <typename E, int N> struct Raw;
template <> struct Raw<bf16, 8> {
    typedef bf16x8 T;
    template <bool S = false> static __device__ __forceinline__ T load(const bf16 *p) {
        if constexpr (S)
            return __builtin_nontemporal_load((const bf16x8u *)p);
        else
            return *(const bf16x8u *)p;
    }
    template <bool S = false> static __device__ __forceinline__ void store(bf16 *p, const T &r) {
        if constexpr (S)
            __builtin_nontemporal_store(r, (bf16x8u *)p);
        else
            *(bf16x8u *)p = r;
    }
    static __device__ __forceinline__ T zero() { return T{}; }
    static __device__ __forceinline__ float get(const T &r, int e) { return (float)r[e]; }
    static __device__ __forceinline__ void set(T &r, int e, float x) { r[e] = (bf16)x; }
};
template <> struct Raw<bf16, 4> {
    typedef bf16x4 T;
    template <bool S = false> static __device__ __forceinline__ T load(const bf16 *p) {
        if constexpr (S)
            return __builtin_nontemporal_load((const bf16x4u *)p);
        else
            return *(const bf16x4u *)p;
    }
    template <bool S = false> static __device__ __forceinline__ void store(bf16 *p, const T &r) {
        if constexpr (S)
            __builtin_nontemporal_store(r, (bf16x4u *)p);
        else
            *(bf16x4u *)p = r;
    }
    static __device__ __forceinline__ T zero() { return T{}; }
    static __device__ __forceinline__ float get(const T &r, int e) { return (float)r[e]; }
    static __device__ __forceinline__ void set(T &r, int e, float x) { r[e] = (bf16)x; }
};
template <> struct Raw<float, 4> {
    typedef f32x4 T;
    template <bool S = false> static __device__ __forceinline__ T load(const float *p) {
        if constexpr (S)
            return __builtin_nontemporal_load((const f32x4u *)p);
        else
            return *(const f32x4u *)p;
    }
    template <bool S = false> static __device__ __forceinline__ void store(float *p, const T &r) {
        if constexpr (S)
            __builtin_nontemporal_store(r, (f32x4u *)p);
        else
            *(f32x4u *)p = r;
    }
    static __device__ __forceinline__ T zero() { return T{}; }
    static __device__ __forceinline__ float get(const T &r, int e) { return r[e]; }
    static __device__ __forceinline__ void set(T &r, int e, float x) { r[e] = x; }
};
template <> struct Raw<float, 8> {
    typedef f32x8p T;
    template <bool S = false> static __device__ __forceinline__ T load(const float *p) {
        return T{Raw<float, 4>::load<S>(p), Raw<float, 4>::load<S>(p + 4)};
    }
    template <bool S = false> static __device__ __forceinline__ void store(float *p, const T &r) {
        Raw<float, 4>::store<S>(p, r.a);
        Raw<float, 4>::store<S>(p + 4, r.b);
    }
    static __device__ __forceinline__ T zero() { return T{f32x4{}, f32x4{}}; }
    static __device__ __forceinline__ float get(const T &r, int e) { return e < 4 ? r.a[e] : r.b[e - 4]; }
    static __device__ __forceinline__ void set(T &r, int e, float x) {
        if (e < 4)
            r.a[e] = x;
        else
            r.b[e - 4] = x;
    }
};
template <typename E> using Raw8 = Raw<E, 8>;
template <typename E> struct Two;
template <> struct Two<bf16> {
    typedef bf16x2 T;
    typedef bf16x2u U;
};
template <> struct Two<float> {
    typedef f32x2 T;
    typedef f32x2u U;
};

// Elements p[0 .. n-1] (n <= N, zeros behind them), and their store: whole, or by
// fours, twos and one.  tails (uniform): some lane of the wave has 0 < n < N.
template <typename E, int N = 8, bool S = false>
__device__ __forceinline__ typename Raw<E, N>::T load_n(const E *p, int n, bool tails) {
    if (n >= N) return Raw<E, N>::template load<S>(p);
    if (!tails) return Raw<E, N>::zero();
    E v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = to_e<E>(0.f);
    // the last part first, moved up as the parts before it come in
    if (n & 1) v[0] = p[n - 1];
    if (n & 2) {
        const typename Two<E>::T h = *(const typename Two<E>::U *)(p + (n & 4));
        v[2] = v[0];
        v[0] = h[0];
        v[1] = h[1];
    }
    if (N == 8 && (n & 4)) {
        const typename Raw<E, 4>::T h = Raw<E, 4>::load(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[(e + 4) % N] = v[e];
            v[e] = h[e];
        }
    }
    typename Raw<E, N>::T r;
#pragma unroll
    for (int e = 0; e < N; ++e) Raw<E, N>::set(r, e, to_f(v[e]));
    return r;
}
template <typename E, int N = 8, bool S = false>
__device__ __forceinline__ void store_n(E *p, const typename Raw<E, N>::T &r, int n, bool tails) {
    if (n >= N) {
        Raw<E, N>::template store<S>(p, r);
        return;
    }
    if (!tails || n <= 0) return;
    E v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = to_e<E>(Raw<E, N>::get(r, e));
    if (N == 8 && (n & 4)) {
        typename Raw<E, 4>::T h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[e] = v[e];
            v[e] = v[(e + 4) % N];
        }
        Raw<E, 4>::store(p, h);
    }
    if (n & 2) {
        *(typename Two<E>::U *)(p + (n & 4)) = typename Two<E>::T{v[0], v[1]};
        v[0] = v[2];
    }
    if (n & 1) p[n - 1] = v[0];
}
// The same of a weight that is fp32 or of type E, as fp32.
template <typename E, int N = 8>
__device__ __forceinline__ void load_w(const void *w, int64_t at, int n, bool tails, int f32, float *r) {
    if (f32) {
        const typename Raw<float, N>::T v = load_n<float, N>((const float *)w + at, n, tails);
#pragma unroll
        for (int e = 0; e < N; ++e) r[e] = Raw<float, N>::get(v, e);
    } else {
        const typename Raw<E, N>::T v = load_n<E, N>((const E *)w + at, n, tails);
#pragma unroll
        for (int e = 0; e < N; ++e) r[e] = Raw<E, N>::get(v, e);
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
