// How the RMS norms lay rows over lanes (gdn_norm.hip, gdn_norm_held.hip).  Included
// by .hip sources only.
#pragma once

#include "gdn_layer_device.h"

namespace gdn {
namespace {

constexpr int threads_of(int L) { return L <= 64 ? 256 : L; }

// Sum over the L lanes of a group, in every lane of it.  red: two rows of 16
// floats, used in turn so that one barrier a call is enough.
template <int L> __device__ __forceinline__ float group_sum(float x, float (*red)[16], int turn) {
#pragma unroll
    for (int o = (L < 64 ? L : 64) / 2; o >= 1; o >>= 1) x += __shfl_xor(x, o);
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = x;
        dev::lds_barrier();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < L / 64; ++w) x += red[turn][w];
    }
    return x;
}

// Lanes of a row's group and vectors a lane for D elements.
struct Split {
    int L, NV;
};
inline Split split_of(int D) {
    if (D <= 64) return {8, 1};
    if (D <= 128) return {16, 1};
    if (D <= 256) return {32, 1};
    if (D <= 512) return {64, 1};
    if (D <= 1024) return {64, 2};
    if (D <= 2048) return {256, 1};
    if (D <= 4096) return {512, 1};
    if (D <= 8192) return {1024, 1};
    return {1024, 2};
}

// Workgroups of `waves` waves in all, fewer for few rows.
inline int blocks_of(int64_t rows, int D, int waves) {
    const int L = split_of(D).L, t = threads_of(L), gpb = t / L;
    const int64_t b = (rows + gpb - 1) / gpb, most = waves * 64 / t;
    return (int)(b < most ? b : most);
}
// Forward: many short-lived waves (16,384 x 32 gated rows of 128: 32768 waves 68
// us, 8192 74), but few of the 1024-thread workgroups (8192 rows of 8192: 4096
// waves 94 us, 8192 97, 32768 100).
inline int norm_blocks(int64_t rows, int D) { return blocks_of(rows, D, split_of(D).L == 1024 ? 4096 : 32768); }
// Backward: two waves a SIMD, walking the rows with the next one loading, keep the
// memory busiest and leave the fewest partial sums (16,383 rows of 4096: 2048
// waves 114 us, 4096 125, 1024 157; gated rows of 128 111, 125 and 135), and every
// CU has a workgroup.
inline int norm_bwd_blocks(int64_t rows, int D) { return blocks_of(rows, D, split_of(D).L == 1024 ? 4096 : 2048); }

// Passes over more than the 256 MiB of the last cache are streamed past it: 16,384
// rows of 5120 forward 110 against 122 us (with plain loads 117), 16,383 of 4096
// backward 114 against 127; 16,384 x 32 gated rows of 128 forward 67 against 77,
// backward 111 against 129.  Smaller outputs stay there for their reader.
inline bool streams(const NormParams &p, size_t elem, int tensors) { return (size_t)p.rows * p.D * elem * tensors > (256u << 20); }

}  // namespace
}  // namespace gdn
