// The gated delta rule over a few tokens per sequence with the states in a
// pool, for gfx950: a token and its drafts to verify, or the rest of a prompt.
// Per sequence and value head, token by token,
//
//   a = S^T k,  b = S^T q,  u = v - e^g rk a
//   S <- e^g S + k (beta rk u)^T
//   out = scale (e^g rq b + beta rk rq (k . q) u)
//
// (rk, rq the L2 norm factors, 1 without the norm): the one-token step of
// gdn_recurrent.hip repeated, with both inner products taken on the state before
// the token.  The state after each token can be kept in a slot of its own, so
// that the next step may start behind any accepted token.
//
// Bound by HBM: a state is read once and written once per kept token; the
// arithmetic is 8 K V operations a token.  A column of the state depends on the
// other columns only through k and q, so a wave owns 32 columns of one head's
// state, in registers from the first token to the last, and needs no other
// wave: no LDS and no barrier between tokens.  A lane holds four columns (16
// bytes in fp32) of K/8 consecutive rows, so that its part of k and q is one
// run of loads; the inner products are summed over the eight row groups by
// lane permutes.  The next token's inputs are loaded while one is computed.
#include "gdn_layer_device.h"

namespace gdn {
namespace {

using namespace dev;

// Sum over the lanes that differ in bits 3, 4 and 5, in each of them.
__device__ __forceinline__ float rows_sum(float x) {
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, true));   // row_ror:8
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Four state elements as fp32, streamed past the caches.
template <typename S> struct Quad;
template <> struct Quad<float> {
    static __device__ __forceinline__ f32x4 load(const float *p) { return __builtin_nontemporal_load((const f32x4 *)p); }
    static __device__ __forceinline__ void store(float *p, f32x4 x) { __builtin_nontemporal_store(x, (f32x4 *)p); }
};
template <> struct Quad<bf16> {
    static __device__ __forceinline__ f32x4 load(const bf16 *p) {
        const bf16x4 x = __builtin_nontemporal_load((const bf16x4 *)p);
        return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
    }
    static __device__ __forceinline__ void store(bf16 *p, f32x4 x) {
        __builtin_nontemporal_store(bf16x4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]}, (bf16x4 *)p);
    }
};

// One token's inputs as loaded.
template <typename E, int RN> struct Token {
    typename Raw8<E>::T k[RN / 8], q[RN / 8];
    E v __attribute__((ext_vector_type(4)));
    float g, beta;
};

template <typename E, typename SE, int K, int V>
__global__ void __launch_bounds__(64 * (V / 32)) steps_kernel(StepsParams p) {
    constexpr int RN = K / 8;                          // state rows of a lane
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = blockIdx.x / p.HV, j = blockIdx.x % p.HV, jk = j / (p.HV / p.H);
    const int c = wv * 32 + (lane & 7) * 4, r0 = (lane >> 3) * RN;
    int t0, t1;
    seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
    if (t0 == t1) return;
    const StepSlots &sl = p.slots;
    const int32_t *idx = sl.indices + (int64_t)n * sl.cols;
    const int acc = sl.accepted ? min(max(sl.accepted[n], 1), sl.cols) : 1;
    const int slot = idx[acc - 1];
    E *__restrict__ out = (E *)p.out;
    typedef E E4 __attribute__((ext_vector_type(4), aligned(sizeof(E))));
    if (slot < 0 || slot >= sl.pool_size) {            // padding row
        if (r0 == 0)
            for (int t = t0; t < t1; ++t)
                *(E4 *)(out + ((int64_t)t * p.HV + j) * V + c) = E4{to_e<E>(0.f), to_e<E>(0.f), to_e<E>(0.f), to_e<E>(0.f)};
        return;
    }
    // this lane's part of a slot
    auto at = [&](int s) { return (SE *)sl.data + (((int64_t)s * p.HV + j) * K + r0) * V + c; };
    f32x4 S[RN];
    {
        const SE *src = at(slot);
#pragma unroll
        for (int i = 0; i < RN; ++i) S[i] = Quad<SE>::load(src + i * V);
    }
    const bool raw = p.gates.A_log != nullptr;
    const float negA = raw ? -expf(p.gates.A_log[j]) : 0.f, dtb = raw ? p.gates.dt_bias[j] : 0.f;
    auto fetch = [&](int t) {
        Token<E, RN> x;
        const E *kp = (const E *)p.k + ((int64_t)t * p.H + jk) * K + r0, *qp = (const E *)p.q + ((int64_t)t * p.H + jk) * K + r0;
#pragma unroll
        for (int i = 0; i < RN / 8; ++i) {
            x.k[i] = Raw8<E>::load(kp + 8 * i);
            x.q[i] = Raw8<E>::load(qp + 8 * i);
        }
        const int64_t th = (int64_t)t * p.HV + j;
        const E *vp = (const E *)p.v + th * V + c;
        x.v = *(const E4 *)vp;
        if (raw) {
            x.g = to_f(((const E *)p.gates.a)[th]);
            x.beta = to_f(((const E *)p.gates.b)[th]);
        } else {
            x.g = p.g[th];
            x.beta = p.beta[th];
        }
        return x;
    };
    Token<E, RN> x = fetch(t0);
    for (int t = t0; t < t1; ++t) {
        Token<E, RN> y;
        if (t + 1 < t1) y = fetch(t + 1);
        f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int i = 0; i < RN; ++i) {
            const float kv = Raw8<E>::get(x.k[i / 8], i % 8), qv = Raw8<E>::get(x.q[i / 8], i % 8);
            a += S[i] * kv;
            b += S[i] * qv;
            kk = fmaf(kv, kv, kk);
            qq = fmaf(qv, qv, qq);
            kq = fmaf(kv, qv, kq);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = rows_sum(a[e]);
            b[e] = rows_sum(b[e]);
        }
        kq = rows_sum(kq);
        float rk = 1.f, rq = 1.f;
        if (p.use_l2norm) {
            rk = rsqrtf(rows_sum(kk) + 1e-6f);
            rq = rsqrtf(rows_sum(qq) + 1e-6f);
        }
        const float gv = raw ? gate_g(x.g, negA, dtb) : x.g, bt = raw ? gate_beta(x.beta) : x.beta;
        const float eg = __expf(gv);
        f32x4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = to_f(x.v[e]) - eg * rk * a[e];
        const f32x4 bu = u * (bt * rk);
        if (r0 == 0) {
            const float cq = bt * kq * rk * rq, cb = eg * rq;
            E4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = to_e<E>(p.scale * (cb * b[e] + cq * u[e]));
            *(E4 *)(out + ((int64_t)t * p.HV + j) * V + c) = o;
        }
#pragma unroll
        for (int i = 0; i < RN; ++i) S[i] = S[i] * eg + bu * Raw8<E>::get(x.k[i / 8], i % 8);
        const int col = min(t - t0, sl.cols - 1);
        if (col < sl.cols - 1 || t == t1 - 1) {
            const int to = idx[col];
            if (to >= 0 && to < sl.pool_size) {
                SE *dst = at(to);
#pragma unroll
                for (int i = 0; i < RN; ++i) Quad<SE>::store(dst + i * V, S[i]);
            }
        }
        x = y;
    }
}

template <typename E, typename SE, int K, int V>
hipError_t launch_cfg(const StepsParams &p, hipStream_t st) {
    steps_kernel<E, SE, K, V><<<(unsigned)((int64_t)p.N * p.HV), 64 * (V / 32), 0, st>>>(p);
    return hipGetLastError();
}

template <typename E, typename SE>
hipError_t launch_kv(const StepsParams &p, hipStream_t st) {
    if (p.K == 64 && p.V == 64) return launch_cfg<E, SE, 64, 64>(p, st);
    if (p.K == 64 && p.V == 128) return launch_cfg<E, SE, 64, 128>(p, st);
    if (p.K == 128 && p.V == 64) return launch_cfg<E, SE, 128, 64>(p, st);
    return launch_cfg<E, SE, 128, 128>(p, st);
}

}  // namespace

hipError_t launch_steps(const StepsParams &p, int dtype, hipStream_t stream, Profiler *prof) {
    if (p.N == 0 || p.T_tot == 0) return hipSuccess;
    if (prof) prof->begin(kStepsKernel, stream);
    const hipError_t err = dtype == 0 ? (p.state_bf16 ? launch_kv<bf16, bf16>(p, stream) : launch_kv<bf16, float>(p, stream))
                                      : (p.state_bf16 ? launch_kv<float, bf16>(p, stream) : launch_kv<float, float>(p, stream));
    if (prof) prof->end(kStepsKernel, stream);
    return err;
}

}  // namespace gdn
