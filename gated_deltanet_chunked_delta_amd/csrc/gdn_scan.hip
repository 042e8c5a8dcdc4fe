// The gated linear recurrence for gfx950: per channel
//   h_t = e^(g_t) h_(t-1) + beta_t x_t,    y_t = h_t,
// the state in fp32, and its gradients
//   dh_t = dy_t + e^(g_(t+1)) dh_(t+1)     (dht added at a sequence's last token)
//   dx = beta dh,  dbeta = x dh,  dg_t = e^(g_t) h_(t-1) dh_t,  dh0 = e^(g_1) dh_1
// with h_(t-1) the forward's y_(t-1) as it was rounded, or the initial state.
#include "gdn_quant_device.h"

namespace gdn {
namespace {

using namespace dev;

// e^g for g <= 0 within 1.05 ulp, and 0.51 near 0: n = the integer nearest to
// g / ln 2, r = g - n ln 2 in two parts, e^r = 1 + r + r^2 p(r) with p of degree 4
// interpolating at Chebyshev's nodes (2e-9 off on |r| <= ln 2 / 2).  The hardware
// exponential is off by an ulp of e^g however small g is, which a channel with
// gates near 0 sums over all the tokens that it remembers.
__device__ __forceinline__ float decay(float g) {
    g = g < -104.f ? -104.f : g;                       // e^-104 is below the smallest subnormal
    const float n = rintf(g * 1.4426950408889634f);
    float r = fmaf(n, -0.693145751953125f, g);
    r = fmaf(n, -1.428606765330187e-06f, r);
    float q = fmaf(r, 0.0013926184f, 0.008363179f);
    q = fmaf(r, q, 0.041666556f);
    q = fmaf(r, q, 0.16666576f);
    q = fmaf(r, q, 0.5f);
    q = fmaf(r * r, q, r);
    return ldexpf(1.f + q, (int)n);
}

__device__ __forceinline__ float load_state(const void *s, int64_t at, int b16) {
    return b16 ? (float)((const bf16 *)s)[at] : ((const float *)s)[at];
}
__device__ __forceinline__ void store_state(void *s, int64_t at, int b16, float h) {
    if (b16)
        ((bf16 *)s)[at] = (bf16)h;
    else
        ((float *)s)[at] = h;
}

// One channel of one sequence a thread.
template <typename E, typename G> __global__ void __launch_bounds__(256) scan_kernel(ScanParams p, int cblocks) {
    const int n = blockIdx.x / cblocks, c = blockIdx.x % cblocks * 256 + threadIdx.x;
    if (c >= p.D) return;
    int t0, t1;
    seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
    int64_t at = (int64_t)n * p.D + c;
    bool kept = true;
    if (p.indices) {
        const int slot = p.indices[n];
        kept = slot >= 0 && slot < p.pool_size;
        at = (int64_t)slot * p.D + c;
    }
    float h = p.initial && kept ? load_state(p.initial, at, p.state_bf16) : 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        float u = to_f(((const E *)p.x)[t * p.x_stride + c]);
        if (p.beta) u *= to_f(((const G *)p.beta)[t * p.beta_stride + c]);
        h = fmaf(decay(to_f(((const G *)p.g)[t * p.g_stride + c])), h, u);
        ((E *)p.y)[t * p.D + c] = to_e<E>(h);
    }
    if (p.final_state && kept) store_state(p.final_state, at, p.state_bf16, h);
}

template <typename E, typename G> __global__ void __launch_bounds__(256) scan_bwd_kernel(ScanParams p, int cblocks) {
    const int n = blockIdx.x / cblocks, c = blockIdx.x % cblocks * 256 + threadIdx.x;
    if (c >= p.D) return;
    int t0, t1;
    seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
    const int64_t at = (int64_t)n * p.D + c;
    const int groups = (p.D + kGroup - 1) / kGroup;
    auto held = [&](const Held &h8, int64_t t) {
        return (float)((const int8_t *)h8.codes)[t * p.D + c] *
               (float)((const bf16 *)h8.scales)[t * groups + c / kGroup];
    };
    float carry = p.dht ? p.dht[at] : 0.f;
    for (int64_t t = t1 - 1; t >= t0; --t) {
        const float a = decay(to_f(((const G *)p.g)[t * p.g_stride + c]));
        const float dh = to_f(((const E *)p.dy)[t * p.D + c]) + carry;
        carry = a * dh;
        const float before = t == t0 ? (p.initial ? ((const float *)p.initial)[at] : 0.f)
                             : p.y8.codes ? held(p.y8, t - 1) : to_f(((const E *)p.y)[(t - 1) * p.D + c]);
        ((G *)p.dg)[t * p.D + c] = to_e<G>(carry * before);
        float dx = dh;
        if (p.beta) {
            const float x = p.x8.codes ? held(p.x8, t) : to_f(((const E *)p.x)[t * p.x_stride + c]);
            ((G *)p.dbeta)[t * p.D + c] = to_e<G>(x * dh);
            dx *= to_f(((const G *)p.beta)[t * p.beta_stride + c]);
        }
        ((E *)p.dx)[t * p.D + c] = to_e<E>(dx);
    }
    if (p.dinitial) p.dinitial[at] = carry;
}

// A few tokens per sequence, states in a pool: see StepSlots.
template <typename E, typename G> __global__ void __launch_bounds__(256) scan_steps_kernel(ScanParams p, int cblocks) {
    const int n = blockIdx.x / cblocks, c = blockIdx.x % cblocks * 256 + threadIdx.x;
    if (c >= p.D) return;
    int t0, t1;
    seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
    const int32_t *idx = p.slots.indices + (int64_t)n * p.slots.cols;
    const int a = p.slots.accepted ? min(max(p.slots.accepted[n], 1), p.slots.cols) : 1;
    const int first = idx[a - 1];
    if (first < 0 || first >= p.slots.pool_size) {
        for (int64_t t = t0; t < t1; ++t) ((E *)p.y)[t * p.D + c] = to_e<E>(0.f);
        return;
    }
    float h = load_state(p.slots.data, (int64_t)first * p.D + c, p.state_bf16);
    for (int64_t t = t0; t < t1; ++t) {
        float u = to_f(((const E *)p.x)[t * p.x_stride + c]);
        if (p.beta) u *= to_f(((const G *)p.beta)[t * p.beta_stride + c]);
        h = fmaf(decay(to_f(((const G *)p.g)[t * p.g_stride + c])), h, u);
        ((E *)p.y)[t * p.D + c] = to_e<E>(h);
        const int j = (int)(t - t0), col = min(j, p.slots.cols - 1);
        if (col == p.slots.cols - 1 && t != t1 - 1) continue;
        const int slot = idx[col];
        if (slot >= 0 && slot < p.slots.pool_size) store_state(p.slots.data, (int64_t)slot * p.D + c, p.state_bf16, h);
    }
}

enum Pass { kForward, kBackward, kSteps };
template <typename E, typename G> void launch_e(const ScanParams &p, Pass pass, hipStream_t st) {
    const int cblocks = (p.D + 255) / 256;
    const unsigned grid = (unsigned)((int64_t)p.N * cblocks);
    if (pass == kForward)
        scan_kernel<E, G><<<grid, 256, 0, st>>>(p, cblocks);
    else if (pass == kBackward)
        scan_bwd_kernel<E, G><<<grid, 256, 0, st>>>(p, cblocks);
    else
        scan_steps_kernel<E, G><<<grid, 256, 0, st>>>(p, cblocks);
}
hipError_t launch_any(const ScanParams &p, Pass pass, int dtype, int gate_f32, hipStream_t st, Profiler *prof) {
    if (p.N == 0) return hipSuccess;
    const int kind = pass == kForward ? kScanKernel : pass == kBackward ? kScanBwdKernel : kScanStepsKernel;
    if (prof) prof->begin(kind, st);
    if (dtype != 0)
        launch_e<float, float>(p, pass, st);
    else if (gate_f32)
        launch_e<bf16, float>(p, pass, st);
    else
        launch_e<bf16, bf16>(p, pass, st);
    const hipError_t err = hipGetLastError();
    if (prof) prof->end(kind, st);
    return err;
}

}  // namespace

size_t scan_workspace_bytes(int64_t, int, int, int, bool) { return 0; }
int64_t scan_grid(int64_t, int64_t D, int64_t N) { return N * ((D + 255) / 256); }

hipError_t launch_scan(const ScanParams &p, int dtype, int gate_f32, hipStream_t stream, Profiler *prof) {
    return launch_any(p, kForward, dtype, gate_f32, stream, prof);
}
hipError_t launch_scan_bwd(const ScanParams &p, int dtype, int gate_f32, hipStream_t stream, Profiler *prof) {
    return launch_any(p, kBackward, dtype, gate_f32, stream, prof);
}
hipError_t launch_scan_steps(const ScanParams &p, int dtype, int gate_f32, hipStream_t stream, Profiler *prof) {
    return launch_any(p, kSteps, dtype, gate_f32, stream, prof);
}

}  // namespace gdn
