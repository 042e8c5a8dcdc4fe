// RMS norms of a GDN layer for gfx950, forward and backward.
//
// gated (after the delta rule, per value head):  y = x r w silu(z)
// add   (before a block, per hidden row):        h = residual + alpha x,  y = h r (w + offset)
// with r = (mean of squares + eps)^-1/2, all in fp32, each output rounded once
// (add: y comes from the unrounded h).
//
// Backward, with n = x r (h r) the normalised row and u = dy w silu(z)
// (dy (w + offset)) the gradient of n:
//   dx = r (u - n mean(n u)),                dw = sum over rows of dy n silu(z)
//   gated: dz = dy n w s (1 + z (1 - s)),    s = sigmoid(z), silu' = s (1 + z (1 - s))
//   add:   d_residual = dx + dhidden,        d_x = alpha d_residual
// r is computed again from the row (it is being read anyway), so nothing but
// the forward's inputs has to be kept.
//
// Bound by HBM: every tensor is read or written once.  A row lives in the
// registers of a group of L lanes, eight elements a lane and vector, NV vectors:
// L = 8 .. 64 lanes of a wave up to 512 elements (1024 with two vectors), a
// workgroup of 256 .. 1024 threads above.  Groups walk the rows in strides, the
// weight (and in the backward pass its gradient's sums) staying in registers,
// and load the next row before they reduce the current one.  16,384 rows of 5120 in
// bf16 take 110 us forward, 524,288 gated rows of 128 67, their gradients 111, those
// of 16,383 rows of 4096 114: 5.9 to 6.1 TB/s.  Gradients of rows above 8192 spill (300
// bytes a lane of the 1024): 4096 rows of 16,384 390 us, 1.7 TB/s, forward 96.
#include "gdn_norm_device.h"

namespace gdn {
namespace {

using namespace dev;

// Elements [at, at + n) of a row: a lane's vector.  The last one of a row of an
// odd length ends with the row and begins `dup` elements inside its neighbour's,
// so that every access is a whole vector (rows of fewer than eight elements
// aside): both lanes compute and store the same values there, after the whole row
// has been read, and the sums leave them to the neighbour (131,072 gated rows of
// 187 with the last elements by fours, twos and one instead: 49 against 31 us,
// their gradients 146 against 62; 9000 rows of 5001 117 against 81).
struct Part {
    int at, n, dup;
    Part() = default;
    __device__ __forceinline__ Part(int D, int v) {
        const int left = D - v * 8;
        dup = left > 0 && left < 8 && D >= 8 ? 8 - left : 0;
        at = v * 8 - dup;
        n = min(max(D - at, 0), 8);
    }
};
// Sum of a b over the lane's own elements (chosen, not multiplied by zero: an infinity
// among the others is the neighbour's).
template <int NV> __device__ __forceinline__ float sum_own(const float (*a)[8], const float (*b)[8], const Part *pt, bool odd) {
    float s = 0.f;
    if (odd) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = e >= pt[i].dup ? fmaf(a[i][e], b[i][e], s) : s;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(a[i][e], b[i][e], s);
    }
    return s;
}

template <typename E, int L, int NV, bool GATED, bool STREAM>
__global__ void __launch_bounds__(threads_of(L)) norm_kernel(NormParams p) {
    typedef Raw8<E> R;
    typedef typename R::T V;
    constexpr int GPB = threads_of(L) / L;             // groups of a workgroup
    __shared__ float red[2][16];
    const int l = threadIdx.x % L;
    const int64_t groups = (int64_t)gridDim.x * GPB;
    const E *__restrict__ x = (const E *)p.x, *__restrict__ z = (const E *)p.z;
    const E *res = (const E *)p.residual;              // hidden may be the residual's buffer
    E *__restrict__ y = (E *)p.y;
    E *hid = (E *)p.hidden;
    const int D = p.D;
    const float inv = 1.f / (float)D;
    const bool odd = D % 8 != 0, tails = D < 8;
    float w[NV][8];
    Part pt[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        pt[i] = Part(D, i * L + l);
        load_w<E>(p.weight, pt[i].at, pt[i].n, tails, p.w_f32, w[i]);
        if (!GATED)
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i][e] += p.offset;
    }
    V xa[NV], za[NV];
    auto load = [&](int64_t row) {
        const int64_t at = row * D;
        const int64_t zat = !GATED ? 0 : p.heads == 1 ? row * p.z_stride
                                      : (int64_t)((uint32_t)row / (uint32_t)p.heads) * p.z_stride +
                                            (int64_t)((uint32_t)row % (uint32_t)p.heads) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xa[i] = load_n<E, 8, STREAM>(x + at + pt[i].at, pt[i].n, tails);
            if (GATED)
                za[i] = load_n<E, 8, STREAM>(z + zat + pt[i].at, pt[i].n, tails);
            else if (res)
                za[i] = load_n<E, 8, STREAM>(res + at + pt[i].at, pt[i].n, tails);
        }
    };
    int64_t row = (int64_t)blockIdx.x * GPB + threadIdx.x / L;
    if (row < p.rows) load(row);
    for (int turn = 0; row < p.rows; row += groups, turn ^= 1) {
        float h[NV][8], g[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = R::get(xa[i], e);
                g[i][e] = GATED || res ? R::get(za[i], e) : 0.f;
                if (!GATED) h[i][e] = fmaf(p.alpha, h[i][e], g[i][e]);
            }
        const float ss = sum_own<NV>(h, h, pt, odd);
        if (row + groups < p.rows) load(row + groups);
        const float r = rsqrtf(group_sum<L>(ss, red, turn) * inv + p.eps);
        const int64_t at = row * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V o, ho;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = h[i][e] * r * w[i][e];
                if (GATED) v *= g[i][e] * sigmoid_f(g[i][e]);
                R::set(o, e, v);
                if (!GATED) R::set(ho, e, h[i][e]);
            }
            store_n<E, 8, STREAM>(y + at + pt[i].at, o, pt[i].n, tails);
            if (!GATED)
                if (hid) store_n<E, 8, STREAM>(hid + at + pt[i].at, ho, pt[i].n, tails);
        }
    }
}

template <typename E, int L, int NV, bool GATED, bool STREAM>
__global__ void __launch_bounds__(threads_of(L)) norm_bwd_kernel(NormParams p) {
    typedef Raw8<E> R;
    typedef typename R::T V;
    constexpr int NT = threads_of(L), GPB = NT / L;
    __shared__ float red[2][16];
    __shared__ float red2[2][16];
    const int l = threadIdx.x % L;
    const int64_t groups = (int64_t)gridDim.x * GPB;
    const E *__restrict__ x = (const E *)(GATED ? p.x : p.hidden), *__restrict__ dy = (const E *)p.dy;
    const E *__restrict__ z = (const E *)(GATED ? p.z : p.dhidden);
    E *__restrict__ dx = (E *)p.dx, *__restrict__ dz = (E *)(GATED ? p.dz : p.dresidual);
    const int D = p.D;
    const float inv = 1.f / (float)D;
    const bool odd = D % 8 != 0, tails = D < 8;
    float w[NV][8], dw[NV][8];
    Part pt[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        pt[i] = Part(D, i * L + l);
        load_w<E>(p.weight, pt[i].at, pt[i].n, tails, p.w_f32, w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!GATED) w[i][e] += p.offset;
            dw[i][e] = 0.f;
        }
    }
    V xa[NV], da[NV], za[NV];
    auto load = [&](int64_t row) {
        const int64_t at = row * D;
        const int64_t zat = !GATED ? at : p.heads == 1 ? row * p.z_stride
                                      : (int64_t)((uint32_t)row / (uint32_t)p.heads) * p.z_stride +
                                            (int64_t)((uint32_t)row % (uint32_t)p.heads) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xa[i] = load_n<E, 8, STREAM>(x + at + pt[i].at, pt[i].n, tails);
            da[i] = load_n<E, 8, STREAM>(dy + at + pt[i].at, pt[i].n, tails);
            if (GATED || z) za[i] = load_n<E, 8, STREAM>(z + zat + pt[i].at, pt[i].n, tails);
        }
    };
    // the longest rows have no registers left for the next row's loads (128 a thread)
    constexpr bool AHEAD = L * NV <= 1024;
    int64_t row = (int64_t)blockIdx.x * GPB + threadIdx.x / L;
    if (AHEAD && row < p.rows) load(row);
    for (int turn = 0; row < p.rows; row += groups, turn ^= 1) {
        float h[NV][8], u[NV][8], g[NV][8];
        float ss = 0.f, sh = 0.f;
        if (!AHEAD) load(row);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = R::get(xa[i], e);
                u[i][e] = R::get(da[i], e);
                g[i][e] = GATED || z ? R::get(za[i], e) : 0.f;
                const float t = GATED ? u[i][e] * w[i][e] * (g[i][e] * sigmoid_f(g[i][e])) : u[i][e] * w[i][e];
                if (odd && e < pt[i].dup) continue;
                ss = fmaf(h[i][e], h[i][e], ss);
                sh = fmaf(t, h[i][e], sh);
            }
        if (AHEAD && row + groups < p.rows) load(row + groups);
        const float r = rsqrtf(group_sum<L>(ss, red, turn) * inv + p.eps);
        const float c = group_sum<L>(sh, red2, turn) * r * inv;       // mean(n u)
        const int64_t at = row * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V o, oz;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float nv = h[i][e] * r;
                if (GATED) {
                    const float s = sigmoid_f(g[i][e]), sl = g[i][e] * s;
                    const float dn = u[i][e] * sl;                     // dy silu(z)
                    dw[i][e] = fmaf(dn, nv, dw[i][e]);
                    R::set(oz, e, u[i][e] * nv * w[i][e] * (s * fmaf(g[i][e], 1.f - s, 1.f)));
                    R::set(o, e, r * (dn * w[i][e] - nv * c));
                } else {
                    dw[i][e] = fmaf(u[i][e], nv, dw[i][e]);
                    const float d = fmaf(r, u[i][e] * w[i][e] - nv * c, g[i][e]);
                    R::set(oz, e, d);
                    R::set(o, e, p.alpha * d);
                }
            }
            if (GATED || dx) store_n<E, 8, STREAM>(dx + at + pt[i].at, o, pt[i].n, tails);
            if (GATED || dz) store_n<E, 8, STREAM>(dz + at + pt[i].at, oz, pt[i].n, tails);
        }
    }
    // the workgroup's sums of dw: over its groups in order
    float *part = p.part + (int64_t)blockIdx.x * D;
    if constexpr (GPB == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= pt[i].dup && e < pt[i].n) part[pt[i].at + e] = dw[i][e];
    } else {
        __shared__ float acc[GPB][L * NV * 8];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= pt[i].dup && e < pt[i].n) acc[threadIdx.x / L][pt[i].at + e] = dw[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += NT) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < GPB; ++q) s += acc[q][c];
            part[c] = s;
        }
    }
}

// Sum of n rows of `cols` floats: CL columns by RL row lanes a workgroup; each row
// lane adds its rows in order, then the row lanes are added in a tree, so the
// result does not depend on scheduling.
template <int CL, int RL>
__global__ void __launch_bounds__(CL * RL) column_sum_kernel(const float *__restrict__ part, int n, int64_t cols,
                                                             float *__restrict__ out, int D, int W,
                                                             float *__restrict__ out2) {
    __shared__ float red[RL][CL + 1];
    const int cl = threadIdx.x % CL, rl = threadIdx.x / CL;
    const int64_t c = (int64_t)blockIdx.x * CL + cl;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int i = rl; i < n; i += RL) s += part[i * cols + c];
    }
    red[rl][cl] = s;
    __syncthreads();
#pragma unroll
    for (int h = RL / 2; h >= 1; h >>= 1) {
        if (rl < h) red[rl][cl] += red[rl + h][cl];
        __syncthreads();
    }
    if (rl == 0 && c < cols) {
        if (W == 0) {
            out[c] = red[0][cl];
        } else {
            const int plane = (int)(c / D), d = (int)(c % D);
            if (plane < W)
                out[(int64_t)d * W + plane] = red[0][cl];
            else if (out2)
                out2[d] = red[0][cl];
        }
    }
}

template <typename E, int L, int NV, bool GATED>
void launch_cfg(const NormParams &p, bool bwd, hipStream_t st) {
    if (bwd) {
        const int grid = norm_bwd_blocks(p.rows, p.D);
        if (streams(p, sizeof(E), 5))
            norm_bwd_kernel<E, L, NV, GATED, true><<<grid, threads_of(L), 0, st>>>(p);
        else
            norm_bwd_kernel<E, L, NV, GATED, false><<<grid, threads_of(L), 0, st>>>(p);
    } else {
        const int grid = norm_blocks(p.rows, p.D);
        if (streams(p, sizeof(E), GATED ? 3 : 4))
            norm_kernel<E, L, NV, GATED, true><<<grid, threads_of(L), 0, st>>>(p);
        else
            norm_kernel<E, L, NV, GATED, false><<<grid, threads_of(L), 0, st>>>(p);
    }
}

template <typename E, bool GATED>
void launch_e(const NormParams &p, bool bwd, hipStream_t st) {
    const Split s = split_of(p.D);
    if (s.L == 8) return launch_cfg<E, 8, 1, GATED>(p, bwd, st);
    if (s.L == 16) return launch_cfg<E, 16, 1, GATED>(p, bwd, st);
    if (s.L == 32) return launch_cfg<E, 32, 1, GATED>(p, bwd, st);
    if (s.L == 64 && s.NV == 1) return launch_cfg<E, 64, 1, GATED>(p, bwd, st);
    if (s.L == 64) return launch_cfg<E, 64, 2, GATED>(p, bwd, st);
    if constexpr (!GATED) {
        if (s.L == 256) return launch_cfg<E, 256, 1, GATED>(p, bwd, st);
        if (s.L == 512) return launch_cfg<E, 512, 1, GATED>(p, bwd, st);
        if (s.NV == 1) return launch_cfg<E, 1024, 1, GATED>(p, bwd, st);
        return launch_cfg<E, 1024, 2, GATED>(p, bwd, st);
    }
}

hipError_t launch_any(const NormParams &p, bool gated, int dtype, bool bwd, hipStream_t st) {
    if (dtype == 0)
        gated ? launch_e<bf16, true>(p, bwd, st) : launch_e<bf16, false>(p, bwd, st);
    else
        gated ? launch_e<float, true>(p, bwd, st) : launch_e<float, false>(p, bwd, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_column_sum(const float *part, int n, int64_t cols, float *out, int D, int W, float *out2,
                             hipStream_t stream, Profiler *prof) {
    if (cols == 0) return hipSuccess;
    if (prof) prof->begin(kColumnSumKernel, stream);
    // few columns: many row lanes, so that the rows are not a long chain of loads
    if (cols <= 8192)
        column_sum_kernel<16, 64><<<(unsigned)((cols + 15) / 16), 1024, 0, stream>>>(part, n, cols, out, D, W, out2);
    else
        column_sum_kernel<64, 4><<<(unsigned)((cols + 63) / 64), 256, 0, stream>>>(part, n, cols, out, D, W, out2);
    const hipError_t err = hipGetLastError();
    if (prof) prof->end(kColumnSumKernel, stream);
    return err;
}

hipError_t launch_norm(const NormParams &p, bool gated, int dtype, hipStream_t stream, Profiler *prof) {
    if (p.rows == 0) return hipSuccess;
    if (prof) prof->begin(kNormKernel, stream);
    const hipError_t err = launch_any(p, gated, dtype, false, stream);
    if (prof) prof->end(kNormKernel, stream);
    return err;
}

size_t norm_bwd_workspace_bytes(int64_t rows, int D) { return (size_t)norm_bwd_blocks(rows, D) * D * 4; }

hipError_t launch_norm_bwd(const NormParams &p, bool gated, int dtype, hipStream_t stream, Profiler *prof) {
    if (p.rows > 0) {
        if (prof) prof->begin(kNormBwdKernel, stream);
        const hipError_t err = launch_any(p, gated, dtype, true, stream);
        if (prof) prof->end(kNormBwdKernel, stream);
        if (err != hipSuccess) return err;
    }
    return launch_column_sum(p.part, p.rows > 0 ? norm_bwd_blocks(p.rows, p.D) : 0, p.D, p.dweight, p.D, 0, nullptr,
                             stream, prof);
}

const char *layer_kernel_name(int kind) {
    switch (kind) {
        case kStepsKernel: return "steps_kernel";
        case kConvKernel: return "conv_kernel";
        case kConvUpdateKernel: return "conv_update_kernel";
        case kConvBwdKernel: return "conv_bwd_kernel";
        case kNormKernel: return "norm_kernel";
        case kNormBwdKernel: return "norm_bwd_kernel";
        case kColumnSumKernel: return "column_sum_kernel";
        case kScanClearKernel: return "scan_clear_kernel";
        case kScanKernel: return "scan_kernel";
        case kScanStepsKernel: return "scan_steps_kernel";
        case kScanBwdKernel: return "scan_bwd_kernel";
        case kQuantKernel: return "quant_kernel";
        case kDequantKernel: return "dequant_kernel";
        default: return "unknown";
    }
}

}  // namespace gdn
