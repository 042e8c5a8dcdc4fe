// Values held in 8 and 4 bits for gfx950: rows of values to codes and scales, and
// back.  The rows are a state pool's slots (a cache of states between requests) or a
// saved activation's rows.
//
// Bound by HBM: each value is read once and 8.5 or 4.5 bits of it are written, or
// the other way.
#include "gdn_quant_device.h"

namespace gdn {
namespace {

using namespace dev;

typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32u __attribute__((aligned(1)));

constexpr int kThreads = 256, kTile = kThreads * 8;

// Rows of a tensor, or -1 for a row that is skipped.
__device__ __forceinline__ int64_t row_at(const int32_t *index, int64_t i, int rows) {
    if (!index) return i;
    const int r = index[i];
    return r >= 0 && r < rows ? r : -1;
}

// Eight values a thread, four threads a group; one tile of a row a workgroup.
template <typename E, int BITS> __global__ void __launch_bounds__(kThreads) quant_kernel(QuantParams p, int tiles) {
    constexpr int TOP = BITS == 8 ? 127 : 7;
    const int64_t i = blockIdx.x / tiles;
    const int64_t from = row_at(p.value_index, i, p.value_rows), to = row_at(p.held_index, i, p.held_rows);
    if (from < 0 || to < 0) return;
    const int64_t at = (int64_t)(blockIdx.x % tiles) * kTile + threadIdx.x * 8;
    const int n = (int)min(max(p.D - at, (int64_t)0), (int64_t)8);
    const E *src = (const E *)p.values + from * p.stride + at;
    const typename Raw8<E>::T r = load_n<E>(src, n, true);
    float v[8];
    uint32_t high = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = Raw8<E>::get(r, e);
        high = max(high, __float_as_uint(v[e]) & 0x7fffffffu);
    }
    high = max(high, (uint32_t)__shfl_xor((int)high, 1));
    high = max(high, (uint32_t)__shfl_xor((int)high, 2));
    const float s = held_scale<TOP>(high), inv = held_inverse(s);
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = held_code<E>(v[e], s, inv);
    if (n > 0 && threadIdx.x % 4 == 0)
        ((bf16 *)p.held.scales)[to * ((p.D + kGroup - 1) / kGroup) + at / kGroup] = (bf16)s;
    if constexpr (BITS == 8) {
        uint8_t *dst = (uint8_t *)p.held.codes + to * p.D + at;
        const uint32_t w[2] = {pack4(c), pack4(c + 4)};
        if (n == 8) {
            *(u32x2u *)dst = u32x2u{w[0], w[1]};
        } else {
            for (int e = 0; e < n; ++e) dst[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
        }
    } else {
        uint8_t *dst = (uint8_t *)p.held.codes + to * ((p.D + 1) / 2) + at / 2;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= (c[e] & 15u) << (4 * e);
        if (n == 8) {
            *(u32u *)dst = w;
        } else {
            for (int e = 0; e < n; e += 2) dst[e / 2] = (uint8_t)(w >> (4 * e));
        }
    }
}

template <typename E, int BITS> __global__ void __launch_bounds__(kThreads) dequant_kernel(QuantParams p, int tiles) {
    const int64_t i = blockIdx.x / tiles;
    const int64_t to = row_at(p.value_index, i, p.value_rows), from = row_at(p.held_index, i, p.held_rows);
    if (from < 0 || to < 0) return;
    const int64_t at = (int64_t)(blockIdx.x % tiles) * kTile + threadIdx.x * 8;
    const int n = (int)min(max(p.D - at, (int64_t)0), (int64_t)8);
    if (n == 0) return;
    const float s = (float)((const bf16 *)p.held.scales)[from * ((p.D + kGroup - 1) / kGroup) + at / kGroup];
    typename Raw8<E>::T r = Raw8<E>::zero();
    if constexpr (BITS == 8) {
        const uint8_t *src = (const uint8_t *)p.held.codes + from * p.D + at;
        uint32_t w[2] = {0, 0};
        if (n == 8) {
            const u32x2u t = *(const u32x2u *)src;
            w[0] = t[0];
            w[1] = t[1];
        } else {
            for (int e = 0; e < n; ++e) w[e / 4] |= (uint32_t)src[e] << (8 * (e % 4));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) Raw8<E>::set(r, e, held_byte(w[e / 4], e % 4) * s);
    } else {
        const uint8_t *src = (const uint8_t *)p.held.codes + from * ((p.D + 1) / 2) + at / 2;
        uint32_t w = 0;
        if (n == 8) {
            w = *(const u32u *)src;
        } else {
            for (int e = 0; e < n; e += 2) w |= (uint32_t)src[e / 2] << (4 * e);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) Raw8<E>::set(r, e, (float)((int)(w << (28 - 4 * e)) >> 28) * s);
    }
    store_n<E>((E *)p.values + to * p.stride + at, r, n, true);
}

template <typename E, int BITS> void launch_e(const QuantParams &p, bool back, hipStream_t st) {
    const int tiles = (int)((p.D + kTile - 1) / kTile);
    const unsigned grid = (unsigned)(p.n * tiles);
    if (back)
        dequant_kernel<E, BITS><<<grid, kThreads, 0, st>>>(p, tiles);
    else
        quant_kernel<E, BITS><<<grid, kThreads, 0, st>>>(p, tiles);
}

}  // namespace

int64_t quant_grid(int64_t n, int64_t D) { return n * ((D + kTile - 1) / kTile); }

hipError_t launch_quant(const QuantParams &p, int dtype, int bits, bool back, hipStream_t stream, Profiler *prof) {
    if (p.n == 0 || p.D == 0) return hipSuccess;
    const int kind = back ? kDequantKernel : kQuantKernel;
    if (prof) prof->begin(kind, stream);
    if (dtype == 0)
        bits == 8 ? launch_e<bf16, 8>(p, back, stream) : launch_e<bf16, 4>(p, back, stream);
    else
        bits == 8 ? launch_e<float, 8>(p, back, stream) : launch_e<float, 4>(p, back, stream);
    const hipError_t err = hipGetLastError();
    if (prof) prof->end(kind, stream);
    return err;
}

}  // namespace gdn
