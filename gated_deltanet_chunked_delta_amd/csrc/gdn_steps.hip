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
// other columns only through k and q, so a wave owns 4 CL columns of one head's
// state, in registers from the first token to the last; a lane holds four
// columns (16 bytes in fp32) of K CL/64 rows.
//
// The token loop waits for nothing but itself: the rows of eight tokens are
// staged in LDS at a time, normalised and in fp32, with their gates (each token by
// one of the workgroup's waves, the next eight tokens' loads in flight
// meanwhile; one barrier every eight tokens).  The sums over the row groups of
// four columns at once leave one column in a lane (lane swaps, two registers a
// swap), u and out are then one operation a lane, and u goes back to all row
// groups by three swaps.  The decay is kept as one factor, S = f S', so that the
// update is one multiply-add an element; f is multiplied in when a state is
// stored, and into S' when it gets small.
//
// HV = 32, K = V = 128: 64 sequences of four tokens, a slot for each, 114 us, 5.7
// TB/s; 256 of 0 to 8 tokens on a bf16 pool in place 108 us, 4.5 TB/s with the vector
// units 70 % busy; one sequence of four tokens 7.7 us.
#include "gdn_layer_device.h"

namespace gdn {
namespace {

using namespace dev;

__device__ __forceinline__ float swap16_sum(float x, float y) {   // rows of 16 lanes: x0+x1, y0+y1, x2+x3, y2+y3
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap32_sum(float x, float y) {   // halves: x0+x1, y0+y1
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int CTRL> __device__ __forceinline__ float dpp_add(float x) {
    return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// Sums of x[0..3] over the row groups (lanes of equal lane % CL): row r of
// sixteen lanes gets the sum of x[r].
template <int CL> __device__ __forceinline__ float groups_sum(float x0, float x1, float x2, float x3) {
    float w = swap32_sum(swap16_sum(x0, x1), swap16_sum(x2, x3));
    if constexpr (CL <= 8) w = dpp_add<0x128>(w);   // row_ror:8
    if constexpr (CL <= 4) w = dpp_add<0x124>(w);   // row_ror:4
    return w;
}
// The way back: lane row r holds element r of every lane's result.
__device__ __forceinline__ f32x4 spread(float w) {
    const unsigned u = __float_as_uint(w);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);            // rows 0 1 0 1 and 2 3 2 3
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    return f32x4{__uint_as_float(a[0]), __uint_as_float(a[1]), __uint_as_float(b[0]), __uint_as_float(b[1])};
}
__device__ __forceinline__ float lane_of(float x, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
}

// Four state elements as fp32.  Stores are streamed past the caches, and so are
// the loads of a state that is updated in place (256 sequences, HV = 32, fp32: 200
// against 216 us); where a slot is kept for every token the pass is mostly
// writes, and plain loads beside them are faster (64 sequences of four tokens,
// four slots: 118 against 143 us).
template <typename S> struct Quad;
template <> struct Quad<float> {
    template <bool STREAM> static __device__ __forceinline__ f32x4 load(const float *p) {
        if constexpr (STREAM) return __builtin_nontemporal_load((const f32x4 *)p);
        return *(const f32x4 *)p;
    }
    static __device__ __forceinline__ void store(float *p, f32x4 x) { __builtin_nontemporal_store(x, (f32x4 *)p); }
};
template <> struct Quad<bf16> {
    template <bool STREAM> static __device__ __forceinline__ f32x4 load(const bf16 *p) {
        bf16x4 x;
        if constexpr (STREAM)
            x = __builtin_nontemporal_load((const bf16x4 *)p);
        else
            x = *(const bf16x4 *)p;
        return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
    }
    static __device__ __forceinline__ void store(bf16 *p, f32x4 x) {
        __builtin_nontemporal_store(bf16x4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]}, (bf16x4 *)p);
    }
};

constexpr int kTok = 8;                            // tokens staged at a time
constexpr float kSmall = 9.5367431640625e-07f;   // 2^-20: the decay factor goes into the state below it

// Eight tokens' inputs: k and q normalised, the workgroup's columns of v, the
// decay, the write strength and the inner product of k and q.
template <int K, int VW> struct Stage {
    float k[kTok][K], q[kTok][K], v[kTok][VW], eg[kTok], beta[kTok], kq[kTok];
};

// NW waves of 4 CL columns each; V / (4 CL NW) workgroups a head.
template <typename E, typename SE, int K, int V, int CL, int NW>
__global__ void __launch_bounds__(64 * NW) steps_kernel(StepsParams p) {
    constexpr int RG = 64 / CL;                        // row groups
    constexpr int RB = K / (4 * RG);                   // blocks of four rows of a lane, 4 RG rows apart
    constexpr int VW = 4 * CL * NW, WPH = V / VW;      // columns of the workgroup, workgroups of a head
    constexpr int KE = K / 64, VE = (VW + 63) / 64;    // elements of a token's rows a lane stages
    constexpr int TW = kTok / NW;                      // tokens a wave stages
    static_assert(RB >= 1 && TW * NW == kTok && WPH * VW == V, "unsupported split");
    __shared__ __attribute__((aligned(16))) Stage<K, VW> stage[2];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nj = blockIdx.x / WPH, n = nj / p.HV, j = nj % p.HV, jk = j / (p.HV / p.H);
    const int w0 = (blockIdx.x % WPH) * VW, c = w0 + wv * 4 * CL + (lane % CL) * 4, r0 = (lane / CL) * 4;
    const int cv = c + (lane >> 4);                    // the column whose sums this lane ends up with
    const StepSlots &sl = p.slots;
    const int32_t *idx = sl.indices + (int64_t)n * sl.cols;
    // the first 64 slots of the row in the lanes
    const int slots = idx[min(lane, sl.cols - 1)];
    const int acc = sl.accepted ? min(max(sl.accepted[n], 1), sl.cols) : 1;
    int t0, t1;
    seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
    if (t0 == t1) return;
    auto slot_of = [&](int col) { return col < 64 ? __builtin_amdgcn_readlane(slots, col) : idx[col]; };
    E *__restrict__ out = (E *)p.out + (int64_t)j * V + cv;
    const bool raw = p.gates.A_log != nullptr;
    const float negA = raw ? -expf(p.gates.A_log[j]) : 0.f, dtb = raw ? p.gates.dt_bias[j] : 0.f;

    // this wave's tokens of a chunk as loaded
    E ek[TW][KE], eq[TW][KE], ev[TW][VE];
    float eg[TW], eb[TW];
    auto load = [&](int tc) {
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int t = tc + wv * TW + i;
            if (t >= t1) break;
            const int64_t th = (int64_t)t * p.HV + j;
            const E *kp = (const E *)p.k + ((int64_t)t * p.H + jk) * K + lane * KE;
            const E *qp = (const E *)p.q + ((int64_t)t * p.H + jk) * K + lane * KE;
            const E *vp = (const E *)p.v + th * V + w0;
#pragma unroll
            for (int e = 0; e < KE; ++e) {
                ek[i][e] = kp[e];
                eq[i][e] = qp[e];
            }
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (VW >= 64 || lane < VW) ev[i][e] = vp[lane * VE + e];
            eg[i] = raw ? to_f(((const E *)p.gates.a)[th]) : p.g[th];
            eb[i] = raw ? to_f(((const E *)p.gates.b)[th]) : p.beta[th];
        }
    };
    auto put = [&](int tc, Stage<K, VW> &st) {
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int s = wv * TW + i;
            if (tc + s >= t1) break;
            float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
            for (int e = 0; e < KE; ++e) {
                const float kv = to_f(ek[i][e]), qv = to_f(eq[i][e]);
                kk = fmaf(kv, kv, kk);
                qq = fmaf(qv, qv, qq);
                kq = fmaf(kv, qv, kq);
            }
            float n2 = groups_sum<4>(kk, qq, kq, 0.f);
            n2 = dpp_add<0x122>(n2);                   // row_ror:2, row_ror:1: the rest of the row
            n2 = dpp_add<0x121>(n2);
            const float rn = rsqrtf(n2 + 1e-6f);
            const float rk = p.use_l2norm ? lane_of(rn, 0) : 1.f, rq = p.use_l2norm ? lane_of(rn, 16) : 1.f;
#pragma unroll
            for (int e = 0; e < KE; ++e) {
                st.k[s][lane * KE + e] = to_f(ek[i][e]) * rk;
                st.q[s][lane * KE + e] = to_f(eq[i][e]) * rq;
            }
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (VW >= 64 || lane < VW) st.v[s][lane * VE + e] = to_f(ev[i][e]);
            st.eg[s] = __expf(raw ? gate_g(eg[i], negA, dtb) : eg[i]);
            st.beta[s] = raw ? gate_beta(eb[i]) : eb[i];
            st.kq[s] = lane_of(n2, 32) * rk * rq;
        }
    };
    load(t0);                                          // on its way while the slot is looked up
    const int slot = slot_of(__builtin_amdgcn_readfirstlane(acc) - 1);
    const bool writes = (lane & 15) < CL;              // one of the lanes of a column
    if (slot < 0 || slot >= sl.pool_size) {            // padding row
        if (writes)
            for (int t = t0; t < t1; ++t) out[(int64_t)t * p.HV * V] = to_e<E>(0.f);
        return;
    }
    // this lane's part of a slot
    auto at = [&](int s) { return (SE *)sl.data + (((int64_t)s * p.HV + j) * K + r0) * V + c; };
    f32x4 S[RB][4];
    {
        const SE *src = at(slot);
        auto read = [&](auto stream) {
#pragma unroll
            for (int m = 0; m < RB; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][e] = Quad<SE>::template load<decltype(stream)::value>(src + (m * 4 * RG + e) * V);
        };
        if (sl.cols > 1) {   // the empty statements keep the two kinds of load from being merged into one
            asm volatile("");
            read(std::false_type{});
            asm volatile("");
        } else {
            read(std::true_type{});
        }
    }
    float f = 1.f;                                     // the state is f S
    for (int tc = t0, turn = 0; tc < t1; tc += kTok, turn ^= 1) {
        const Stage<K, VW> &st = stage[turn];
        put(tc, stage[turn]);
        lds_barrier();
        if (tc + kTok < t1) load(tc + kTok);
        const int m1 = min(kTok, t1 - tc);
        for (int s = 0; s < m1; ++s) {
            const int t = tc + s;
            f32x4 kv[RB], a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
            for (int m = 0; m < RB; ++m) {
                kv[m] = *(const f32x4 *)&st.k[s][m * 4 * RG + r0];
                const f32x4 qv = *(const f32x4 *)&st.q[s][m * 4 * RG + r0];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a += S[m][e] * kv[m][e];
                    b += S[m][e] * qv[e];
                }
            }
            const float fn = st.eg[s] * f, bt = st.beta[s];
            const float as = groups_sum<CL>(a[0], a[1], a[2], a[3]), bs = groups_sum<CL>(b[0], b[1], b[2], b[3]);
            const float u = bt * (st.v[s][cv - w0] - fn * as);
            if (writes) out[(int64_t)t * p.HV * V] = to_e<E>(p.scale * (fn * bs + st.kq[s] * u));
            f = fn;
            if (__builtin_amdgcn_readfirstlane(fn < kSmall)) {
#pragma unroll
                for (int m = 0; m < RB; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[m][e] *= fn;
                f = 1.f;
            }
            const f32x4 d = spread(u * __builtin_amdgcn_rcpf(f));
#pragma unroll
            for (int m = 0; m < RB; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][e] += d * kv[m][e];
            const int col = min(t - t0, sl.cols - 1);
            if (col < sl.cols - 1 || t == t1 - 1) {
                const int to = slot_of(col);
                if (to >= 0 && to < sl.pool_size) {
                    SE *dst = at(to);
#pragma unroll
                    for (int m = 0; m < RB; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) Quad<SE>::store(dst + (m * 4 * RG + e) * V, S[m][e] * f);
                }
            }
        }
    }
}

template <typename E, typename SE, int K, int V, int CL, int NW>
hipError_t launch_cols(const StepsParams &p, hipStream_t st) {
    steps_kernel<E, SE, K, V, CL, NW><<<(unsigned)((int64_t)p.N * p.HV * (V / (4 * CL * NW))), 64 * NW, 0, st>>>(p);
    return hipGetLastError();
}

// A wave's columns, one MI355X, four tokens, HV = 32, K = V = 128:
// - With fewer heads than CUs latency counts: 16 columns a wave put twice as many
//   SIMDs to work as 32 (64 heads 6.8 against 8.0 us; 256 heads 10.3 against
//   10.7; 512 heads 15.3 against 14.6: half rows of 64 bytes cost the memory more).
// - Else a wave takes 128 bytes of each row: 32 columns in fp32, 64 in bf16 (8192
//   heads 120 against 135 us with 32). 64 columns are 128 state registers a
//   lane, which pays only with many heads to hide it (512 heads 15.1 against 12.2
//   us, 1024 heads 18.8 against 19.2, 1536 heads 33.4 against 31.9).
template <typename E, typename SE, int K, int V>
hipError_t launch_cfg(const StepsParams &p, hipStream_t st) {
    const int64_t heads = (int64_t)p.N * p.HV;
    if (heads < 256) return launch_cols<E, SE, K, V, 4, 4>(p, st);
    if (sizeof(SE) == 2 && heads >= 2048) return launch_cols<E, SE, K, V, 16, V / 64>(p, st);
    return launch_cols<E, SE, K, V, 8, V / 32>(p, st);
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
