// Values held in 8 and 4 bits for gfx950: rows of values to codes and scales, and
// back.  The rows are a state pool's slots (a cache of states between requests) or a
// saved activation's rows.
//
// Bound by HBM: each value is read once and 8.5 or 4.5 bits of it are written, or
// the other way.  256 delta-rule states of 2^19 bf16 elements take 66 us to 4 bits (5.2
// TB/s) and 77 us back (4.5 TB/s); one of them in fp32 to 8 bits 3.7 us and 3.3, a
// launch's time.
#include "gdn_quant_device.h"

namespace gdn {
namespace {

using namespace dev;

// Eight values a thread and part, U parts in flight; four threads a group.
constexpr int kThreads = 256, kPart = kThreads * 8;

// Rows of a tensor, or -1 for a row that is skipped.
__device__ __forceinline__ int64_t row_at(const int32_t *index, int64_t i, int rows) {
    if (!index) return i;
    const int r = index[i];
    return r >= 0 && r < rows ? r : -1;
}

template <typename E, int BITS, int U, bool STREAM>
__global__ void __launch_bounds__(kThreads) quant_kernel(QuantParams p, int tiles) {
    constexpr int TOP = BITS == 8 ? 127 : 7;
    const int64_t i = blockIdx.x / tiles;
    const int64_t from = row_at(p.value_index, i, p.value_rows), to = row_at(p.held_index, i, p.held_rows);
    if (from < 0 || to < 0) return;
    const int64_t at = (int64_t)(blockIdx.x % tiles) * (U * kPart) + threadIdx.x * 8;
    const bool tails = p.D % 8 != 0;
    const E *src = (const E *)p.values + from * p.stride;
    typename Raw8<E>::T r[U];
    int n[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        n[k] = (int)min(max(p.D - at - k * kPart, (int64_t)0), (int64_t)8);
        r[k] = load_n<E, 8, STREAM>(src + at + k * kPart, n[k], tails);
    }
    const int64_t groups = (p.D + kGroup - 1) / kGroup;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t col = at + k * kPart;
        float v[8];
        uint32_t high = 0, c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = Raw8<E>::get(r[k], e);
            high = max(high, __float_as_uint(v[e]) & 0x7fffffffu);
        }
        high = max(high, (uint32_t)__shfl_xor((int)high, 1));
        high = max(high, (uint32_t)__shfl_xor((int)high, 2));
        const float s = held_scale<TOP>(high), inv = held_inverse(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = held_code<E>(v[e], s, inv);
        if (n[k] > 0 && threadIdx.x % 4 == 0) ((bf16 *)p.held.scales)[to * groups + col / kGroup] = (bf16)s;
        if constexpr (BITS == 8) {
            if (n[k] == 8 || tails)
                store_codes<STREAM>((uint8_t *)p.held.codes + to * p.D + col, pack4(c), pack4(c + 4), n[k]);
        } else {
            uint8_t *dst = (uint8_t *)p.held.codes + to * ((p.D + 1) / 2) + col / 2;
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) w |= (c[e] & 15u) << (4 * e);
            if (n[k] == 8) {
                if constexpr (STREAM)
                    __builtin_nontemporal_store(w, (u32u *)dst);
                else
                    *(u32u *)dst = w;
            } else {
                for (int e = 0; e < n[k]; e += 2) dst[e / 2] = (uint8_t)(w >> (4 * e));
            }
        }
    }
}

template <typename E, int BITS, int U, bool STREAM>
__global__ void __launch_bounds__(kThreads) dequant_kernel(QuantParams p, int tiles) {
    const int64_t i = blockIdx.x / tiles;
    const int64_t to = row_at(p.value_index, i, p.value_rows), from = row_at(p.held_index, i, p.held_rows);
    if (from < 0 || to < 0) return;
    const int64_t at = (int64_t)(blockIdx.x % tiles) * (U * kPart) + threadIdx.x * 8;
    const bool tails = p.D % 8 != 0;
    const bf16 *scales = (const bf16 *)p.held.scales + from * ((p.D + kGroup - 1) / kGroup);
    const uint8_t *src = (const uint8_t *)p.held.codes + from * (BITS == 8 ? p.D : (p.D + 1) / 2);
    u32x2 w[U];
    float s[U];
    int n[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t col = at + k * kPart;
        n[k] = (int)min(max(p.D - col, (int64_t)0), (int64_t)8);
        s[k] = n[k] > 0 ? (float)scales[col / kGroup] : 0.f;
        w[k] = u32x2{0, 0};
        if constexpr (BITS == 8) {
            if (n[k] == 8 || tails) w[k] = load_codes<STREAM>(src + col, n[k]);
        } else if (n[k] == 8) {
            if constexpr (STREAM)
                w[k][0] = __builtin_nontemporal_load((const u32u *)(src + col / 2));
            else
                w[k][0] = *(const u32u *)(src + col / 2);
        } else {
            for (int e = 0; e < n[k]; e += 2) w[k][0] |= (uint32_t)src[(col + e) / 2] << (4 * e);
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        typename Raw8<E>::T r = Raw8<E>::zero();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            Raw8<E>::set(r, e, (BITS == 8 ? held_byte(w[k][e / 4], e % 4) : (float)((int)(w[k][0] << (28 - 4 * e)) >> 28)) * s[k]);
        store_n<E, 8, STREAM>((E *)p.values + to * p.stride + at + k * kPart, r, n[k], tails);
    }
}

int64_t tiles_of(int64_t D, int U) { return (D + U * kPart - 1) / (U * kPart); }

// Four parts a workgroup where that leaves every CU eight workgroups, for the loads in
// flight (the 256 states there and back 140 us, with one part and through the cache
// 168, with eight parts 139); one part for few rows, which then have the more
// workgroups.  Passes over more than the 256 MiB of the last cache are streamed past
// it, smaller ones stay there for their reader.
template <typename E, int BITS, int U, bool STREAM> void launch_u(const QuantParams &p, bool back, hipStream_t st) {
    const int tiles = (int)tiles_of(p.D, U);
    const unsigned grid = (unsigned)(p.n * tiles);
    if (back)
        dequant_kernel<E, BITS, U, STREAM><<<grid, kThreads, 0, st>>>(p, tiles);
    else
        quant_kernel<E, BITS, U, STREAM><<<grid, kThreads, 0, st>>>(p, tiles);
}
template <typename E, int BITS> void launch_e(const QuantParams &p, bool back, hipStream_t st) {
    if (p.D < 4 * kPart || p.n * tiles_of(p.D, 4) < 2048)
        launch_u<E, BITS, 1, false>(p, back, st);
    else if ((double)p.n * p.D * (sizeof(E) + BITS / 8.0) > (256 << 20))
        launch_u<E, BITS, 4, true>(p, back, st);
    else
        launch_u<E, BITS, 4, false>(p, back, st);
}

}  // namespace

int64_t quant_grid(int64_t n, int64_t D) { return n * tiles_of(D, 1); }

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
