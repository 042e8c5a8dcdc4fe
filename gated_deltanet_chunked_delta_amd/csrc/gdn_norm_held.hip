// The gated RMS norm of a GDN layer that keeps its inputs in 8 bits for gfx950:
//   y = x r w silu(z),   r = (mean of squares + eps)^-1/2
// forward with the codes of x and z written beside y in the one pass that reads
// them, backward from the codes.  The arithmetic is that of gdn_norm.hip, on the
// values that the codes stand for; the format that of gdn_quant_device.h.
//
// Bound by HBM.  Against the norm that keeps x and z as they are the forward pass
// writes two bytes more an element (bf16: 8.1 instead of 6) and the backward pass
// reads two less (8.1 instead of 10); what lives from one to the other is halved.
// 524,288 rows of 128 in bf16 take 100 us forward (5.5 TB/s) and 117 us backward (4.7
// TB/s, 5 more for the sums of dweight); the backward pass does 36 instructions an
// element, two thirds of its time.  Rows that are not of whole eights load and store
// their last elements by fours, twos and one: 32,752 rows of 100 backward 13 us.
#include <algorithm>

#include "gdn_norm_device.h"
#include "gdn_quant_device.h"

namespace gdn {
namespace {

using namespace dev;

// A lane's vectors are the row's eights in order, so that four neighbours make a
// group of the format; the last one of a row may be short.
template <typename E, int L, int NV, bool STREAM>
__global__ void __launch_bounds__(threads_of(L)) norm_held_kernel(NormParams p, Held x8, Held z8) {
    typedef Raw8<E> R;
    typedef typename R::T V;
    constexpr int GPB = threads_of(L) / L;
    __shared__ float red[2][16];
    const int l = threadIdx.x % L;
    const int64_t rows_a_turn = (int64_t)gridDim.x * GPB;
    const E *__restrict__ x = (const E *)p.x, *__restrict__ z = (const E *)p.z;
    E *__restrict__ y = (E *)p.y;
    const int D = p.D, groups = (D + kGroup - 1) / kGroup;
    const float inv = 1.f / (float)D;
    const bool tails = D % 8 != 0;
    float w[NV][8];
    int cnt[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        cnt[i] = min(max(D - (i * L + l) * 8, 0), 8);
        load_w<E>(p.weight, (i * L + l) * 8, cnt[i], tails, p.w_f32, w[i]);
    }
    V xa[NV], za[NV];
    auto load = [&](int64_t row) {
        const int64_t at = row * D;
        const int64_t zat = p.heads == 1 ? row * p.z_stride
                                         : (int64_t)((uint32_t)row / (uint32_t)p.heads) * p.z_stride +
                                               (int64_t)((uint32_t)row % (uint32_t)p.heads) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xa[i] = load_n<E, 8, STREAM>(x + at + (i * L + l) * 8, cnt[i], tails);
            za[i] = load_n<E, 8, STREAM>(z + zat + (i * L + l) * 8, cnt[i], tails);
        }
    };
    auto keep = [&](const float *v, const Held &to, int64_t row, int i) {
        uint32_t high = 0, c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) high = max(high, __float_as_uint(v[e]) & 0x7fffffffu);
        high = max(high, (uint32_t)__shfl_xor((int)high, 1));
        high = max(high, (uint32_t)__shfl_xor((int)high, 2));
        const float s = held_scale<127>(high), si = held_inverse(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = held_code<E>(v[e], s, si);
        const int col = (i * L + l) * 8;
        const uint32_t a = pack4(c), b = pack4(c + 4);
        uint8_t *dst = (uint8_t *)to.codes + row * D + col;
        if (cnt[i] == 8 || tails) store_codes<STREAM>(dst, a, b, cnt[i]);
        if (l % 4 == 0 && cnt[i] > 0) ((bf16 *)to.scales)[row * groups + col / kGroup] = (bf16)s;
    };
    int64_t row = (int64_t)blockIdx.x * GPB + threadIdx.x / L;
    if (row < p.rows) load(row);
    for (int turn = 0; row < p.rows; row += rows_a_turn, turn ^= 1) {
        float h[NV][8], g[NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = R::get(xa[i], e);
                g[i][e] = R::get(za[i], e);
                ss = fmaf(h[i][e], h[i][e], ss);
            }
        if (row + rows_a_turn < p.rows) load(row + rows_a_turn);
        const float r = rsqrtf(group_sum<L>(ss, red, turn) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V o;
#pragma unroll
            for (int e = 0; e < 8; ++e) R::set(o, e, h[i][e] * r * w[i][e] * (g[i][e] * sigmoid_f(g[i][e])));
            store_n<E, 8, STREAM>(y + row * D + (i * L + l) * 8, o, cnt[i], tails);
            keep(h[i], x8, row, i);
            keep(g[i], z8, row, i);
        }
    }
}

// Workgroups of 512 threads: twice the waves of the norm's backward pass for as many
// rows of partial sums, as there is more arithmetic for fewer bytes (524,288 rows of
// 128: 117 us; with 256 threads, the next row's loads the only ones in flight, 174; with
// 1024 119).  Two of them a CU leave a lane 128 registers: bf16 rows above 128 and fp32 rows up
// to 512 keep 12 to 40 bytes in scratch memory.  Without the limit a CU has one workgroup
// (bf16 rows of 256 115 -> 174 us, 131,072 fp32 rows of 256 117 -> 114, 65,536 of 512 127 -> 114).
constexpr int kBwdThreads = 512;
template <typename E, int L, int NV, bool STREAM>
__global__ void __launch_bounds__(kBwdThreads, NV == 1 ? 4 : 2) norm_held_bwd_kernel(NormParams p, Held x8, Held z8) {
    typedef Raw8<E> R;
    typedef typename R::T V;
    constexpr int NT = kBwdThreads, GPB = NT / L;
    __shared__ float red[2][16];
    __shared__ float red2[2][16];
    __shared__ float acc[GPB][L * NV * 8];
    const int l = threadIdx.x % L;
    const int64_t rows_a_turn = (int64_t)gridDim.x * GPB;
    const E *__restrict__ dy = (const E *)p.dy;
    E *__restrict__ dx = (E *)p.dx, *__restrict__ dz = (E *)p.dz;
    const int D = p.D, groups = (D + kGroup - 1) / kGroup;
    const float inv = 1.f / (float)D;
    const bool tails = D % 8 != 0;
    float w[NV][8], dw[NV][8];
    int cnt[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        cnt[i] = min(max(D - (i * L + l) * 8, 0), 8);
        load_w<E>(p.weight, (i * L + l) * 8, cnt[i], tails, p.w_f32, w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    }
    auto fetch = [&](const Held &h, int64_t row, int i, u32x2 &codes, float &scale) {
        const int col = (i * L + l) * 8;
        const uint8_t *src = (const uint8_t *)h.codes + row * D + col;
        codes = u32x2{0, 0};
        scale = 0.f;
        if (cnt[i] > 0) scale = (float)((const bf16 *)h.scales)[row * groups + col / kGroup];
        if (cnt[i] == 8 || tails) codes = load_codes<STREAM>(src, cnt[i]);
    };
    V da[NV];
    u32x2 xc[NV], zc[NV];
    float xs[NV], zs[NV];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            da[i] = load_n<E, 8, STREAM>(dy + row * D + (i * L + l) * 8, cnt[i], tails);
            fetch(x8, row, i, xc[i], xs[i]);
            fetch(z8, row, i, zc[i], zs[i]);
        }
    };
    int64_t row = (int64_t)blockIdx.x * GPB + threadIdx.x / L;
    if (row < p.rows) load(row);
    for (int turn = 0; row < p.rows; row += rows_a_turn, turn ^= 1) {
        float h[NV][8], u[NV][8], g[NV][8];
        float ss = 0.f, sh = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = held_byte(xc[i][e / 4], e % 4) * xs[i];
                g[i][e] = held_byte(zc[i][e / 4], e % 4) * zs[i];
                u[i][e] = R::get(da[i], e);
                ss = fmaf(h[i][e], h[i][e], ss);
                sh = fmaf(u[i][e] * w[i][e] * (g[i][e] * sigmoid_f(g[i][e])), h[i][e], sh);
            }
        if (row + rows_a_turn < p.rows) load(row + rows_a_turn);
        const float r = rsqrtf(group_sum<L>(ss, red, turn) * inv + p.eps);
        const float c = group_sum<L>(sh, red2, turn) * r * inv;       // mean(n u)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V o, oz;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float nv = h[i][e] * r, s = sigmoid_f(g[i][e]);
                const float dn = u[i][e] * (g[i][e] * s);             // dy silu(z)
                dw[i][e] = fmaf(dn, nv, dw[i][e]);
                R::set(oz, e, u[i][e] * nv * w[i][e] * (s * fmaf(g[i][e], 1.f - s, 1.f)));
                R::set(o, e, r * (dn * w[i][e] - nv * c));
            }
            store_n<E, 8, STREAM>(dx + row * D + (i * L + l) * 8, o, cnt[i], tails);
            store_n<E, 8, STREAM>(dz + row * D + (i * L + l) * 8, oz, cnt[i], tails);
        }
    }
    // the workgroup's sums of dw: over its rows' lane groups in order
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[threadIdx.x / L][(i * L + l) * 8 + e] = dw[i][e];
    __syncthreads();
    float *part = p.part + (int64_t)blockIdx.x * D;
    for (int c = threadIdx.x; c < D; c += NT) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < GPB; ++q) s += acc[q][c];
        part[c] = s;
    }
}

// At most as many as norm_bwd_workspace_bytes has rows for; one for rows of two turns,
// whose sums are dweight then, without a launch for them (32 rows of 128 3.9 us and with
// two launches 6.1, 64 rows 5.3 and 6.1; 128 rows would take 7.9 and 6.1).
constexpr int kFewTurns = 2;
int held_bwd_blocks(int64_t rows, int D) {
    const int gpb = kBwdThreads / split_of(D).L;
    if (rows <= kFewTurns * gpb) return 1;
    return (int)std::min<int64_t>((rows + gpb - 1) / gpb, norm_bwd_blocks(rows, D));
}
template <typename E, int L, int NV, bool STREAM>
void launch_stream(const NormParams &p, const Held &x8, const Held &z8, bool bwd, hipStream_t st) {
    if (bwd)
        norm_held_bwd_kernel<E, L, NV, STREAM><<<held_bwd_blocks(p.rows, p.D), kBwdThreads, 0, st>>>(p, x8, z8);
    else
        norm_held_kernel<E, L, NV, STREAM><<<norm_blocks(p.rows, p.D), threads_of(L), 0, st>>>(p, x8, z8);
}
template <typename E, int L, int NV> void launch_cfg(const NormParams &p, const Held &x8, const Held &z8, bool bwd, hipStream_t st) {
    if (streams(p, sizeof(E), 4))                      // three tensors and two of codes
        launch_stream<E, L, NV, true>(p, x8, z8, bwd, st);
    else
        launch_stream<E, L, NV, false>(p, x8, z8, bwd, st);
}
template <typename E> void launch_e(const NormParams &p, const Held &x8, const Held &z8, bool bwd, hipStream_t st) {
    const Split s = split_of(p.D);
    if (s.L == 8) return launch_cfg<E, 8, 1>(p, x8, z8, bwd, st);
    if (s.L == 16) return launch_cfg<E, 16, 1>(p, x8, z8, bwd, st);
    if (s.L == 32) return launch_cfg<E, 32, 1>(p, x8, z8, bwd, st);
    if (s.NV == 1) return launch_cfg<E, 64, 1>(p, x8, z8, bwd, st);
    launch_cfg<E, 64, 2>(p, x8, z8, bwd, st);
}
hipError_t launch_any(const NormParams &p, const Held &x8, const Held &z8, int dtype, bool bwd, hipStream_t st) {
    if (dtype == 0)
        launch_e<bf16>(p, x8, z8, bwd, st);
    else
        launch_e<float>(p, x8, z8, bwd, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_held(const NormParams &p, const Held &x8, const Held &z8, int dtype, hipStream_t stream,
                            Profiler *prof) {
    if (p.rows == 0) return hipSuccess;
    if (prof) prof->begin(kNormKernel, stream);
    const hipError_t err = launch_any(p, x8, z8, dtype, false, stream);
    if (prof) prof->end(kNormKernel, stream);
    return err;
}

hipError_t launch_norm_held_bwd(const NormParams &q, const Held &x8, const Held &z8, int dtype, hipStream_t stream,
                                Profiler *prof) {
    NormParams p = q;
    const bool one = p.rows > 0 && held_bwd_blocks(p.rows, p.D) == 1;
    if (one) p.part = p.dweight;
    if (p.rows > 0) {
        if (prof) prof->begin(kNormBwdKernel, stream);
        const hipError_t err = launch_any(p, x8, z8, dtype, true, stream);
        if (prof) prof->end(kNormBwdKernel, stream);
        if (err != hipSuccess || one) return err;
    }
    return launch_column_sum(p.part, p.rows > 0 ? held_bwd_blocks(p.rows, p.D) : 0, p.D, p.dweight, p.D, 0, nullptr,
                             stream, prof);
}

}  // namespace gdn
