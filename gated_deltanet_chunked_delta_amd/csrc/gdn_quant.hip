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

// Eight values a thread, four threads a group; U of these parts a thread in flight.
constexpr int kThreads = 256, kPart = kThreads * 8;

// Rows of a tensor, or -1 for a row that is skipped.
__device__ __forceinline__ int64_t row_at(const int32_t *index, int64_t i, int rows) {
    if (!index) return i;
    const int r = index[i];
    return r >= 0 && r < rows ? r : -1;
}

// A thread's parts: U parts of one row (split: workgroups a row), or, ROWS, a part of each
// of U rows that it shares with 2^split - 1 others.
struct Part {
    int64_t from, to, col;                             // rows of the tensor read and the one written, the first value
    int n;                                             // values, 0 for a row that is skipped
};
// False where there is nothing to do.  Four neighbours stay together: they share a row.
template <int U, bool ROWS>
__device__ __forceinline__ bool parts_of(const QuantParams &p, int split, const int32_t *read, int read_rows,
                                         const int32_t *written, int written_rows, Part (&q)[U]) {
    if constexpr (ROWS && U > 1) {
        const int per = kThreads >> split;             // rows a workgroup and part
        const int64_t first = (int64_t)blockIdx.x * (U * per) + (threadIdx.x >> split);
        const int64_t col = (threadIdx.x & ((1 << split) - 1)) * 8;
        const int n = (int)min(max(p.D - col, (int64_t)0), (int64_t)8);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t i = first + k * per;
            q[k] = {-1, -1, col, 0};
            if (i >= p.n) continue;
            q[k].from = row_at(read, i, read_rows);
            q[k].to = row_at(written, i, written_rows);
            q[k].n = q[k].from >= 0 && q[k].to >= 0 ? n : 0;
        }
        return true;
    } else {
        int64_t i, at;
        if constexpr (ROWS) {
            i = (int64_t)blockIdx.x * (kThreads >> split) + (threadIdx.x >> split);
            at = (threadIdx.x & ((1 << split) - 1)) * 8;
            if (i >= p.n) return false;
        } else {
            i = blockIdx.x / split;
            at = (int64_t)(blockIdx.x % split) * (U * kPart) + threadIdx.x * 8;
        }
        const int64_t from = row_at(read, i, read_rows), to = row_at(written, i, written_rows);
#pragma unroll
        for (int k = 0; k < U; ++k)
            q[k] = {from, to, at + k * kPart, (int)min(max(p.D - at - k * kPart, (int64_t)0), (int64_t)8)};
        return from >= 0 && to >= 0;
    }
}

template <typename E, int BITS, int U, bool STREAM, bool ROWS>
__global__ void __launch_bounds__(kThreads) quant_kernel(QuantParams p, int split) {
    constexpr int TOP = BITS == 8 ? 127 : 7;
    Part q[U];
    if (!parts_of<U, ROWS>(p, split, p.value_index, p.value_rows, p.held_index, p.held_rows, q)) return;
    const bool tails = p.D % 8 != 0;
    typename Raw8<E>::T r[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
        r[k] = load_n<E, 8, STREAM>((const E *)p.values + q[k].from * p.stride + q[k].col, q[k].n, tails);
    const int64_t groups = (p.D + kGroup - 1) / kGroup;
#pragma unroll
    for (int k = 0; k < U; ++k) {
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
        if (q[k].n > 0 && threadIdx.x % 4 == 0) ((bf16 *)p.held.scales)[q[k].to * groups + q[k].col / kGroup] = (bf16)s;
        if constexpr (BITS == 8) {
            if (q[k].n == 8 || tails)
                store_codes<STREAM>((uint8_t *)p.held.codes + q[k].to * p.D + q[k].col, pack4(c), pack4(c + 4), q[k].n);
        } else {
            uint8_t *dst = (uint8_t *)p.held.codes + q[k].to * ((p.D + 1) / 2) + q[k].col / 2;
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) w |= (c[e] & 15u) << (4 * e);
            if (q[k].n == 8) {
                if constexpr (STREAM)
                    __builtin_nontemporal_store(w, (u32u *)dst);
                else
                    *(u32u *)dst = w;
            } else {
                for (int e = 0; e < q[k].n; e += 2) dst[e / 2] = (uint8_t)(w >> (4 * e));
            }
        }
    }
}

template <typename E, int BITS, int U, bool STREAM, bool ROWS>
__global__ void __launch_bounds__(kThreads) dequant_kernel(QuantParams p, int split) {
    Part q[U];
    if (!parts_of<U, ROWS>(p, split, p.held_index, p.held_rows, p.value_index, p.value_rows, q)) return;
    const bool tails = p.D % 8 != 0;
    const int64_t groups = (p.D + kGroup - 1) / kGroup, row = BITS == 8 ? p.D : (p.D + 1) / 2;
    u32x2 w[U];
    float s[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const uint8_t *src = (const uint8_t *)p.held.codes + q[k].from * row + (BITS == 8 ? q[k].col : q[k].col / 2);
        s[k] = q[k].n > 0 ? (float)((const bf16 *)p.held.scales)[q[k].from * groups + q[k].col / kGroup] : 0.f;
        w[k] = u32x2{0, 0};
        if constexpr (BITS == 8) {
            if (q[k].n == 8 || tails) w[k] = load_codes<STREAM>(src, q[k].n);
        } else if (q[k].n == 8) {
            if constexpr (STREAM)
                w[k][0] = __builtin_nontemporal_load((const u32u *)src);
            else
                w[k][0] = *(const u32u *)src;
        } else {
            for (int e = 0; e < q[k].n; e += 2) w[k][0] |= (uint32_t)src[e / 2] << (4 * e);
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        typename Raw8<E>::T r = Raw8<E>::zero();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            Raw8<E>::set(r, e, (BITS == 8 ? held_byte(w[k][e / 4], e % 4) : (float)((int)(w[k][0] << (28 - 4 * e)) >> 28)) * s[k]);
        store_n<E, 8, STREAM>((E *)p.values + q[k].to * p.stride + q[k].col, r, q[k].n, tails);
    }
}

// What a call of these sizes launches.  Rows that follow each other in both tensors and
// are of whole groups are one long row (524,288 rows of 128 to 8 bits 33 us, a workgroup
// each 313); others of up to 1024 values share a workgroup.
//
// Of long rows four parts a thread where that leaves every CU eight workgroups, for the
// loads in flight (256 states there and back 139 us, with one part and through the cache
// 168, with eight parts 139); one part for few rows, which then have the more
// workgroups.  Passes over more than the 256 MiB of the last cache are streamed past
// it, smaller ones stay there for their reader.
//
// Of short rows, four or one a thread, 8 bits, us:
//   to codes from the cache one (35M values: 346,030 rows of 100 25 against 28, 34,603 of 1000
//     19.5 against 24), else four, streamed from bf16 (300M values: rows of 33 311 against 327, of
//     129 317 against 356, of 1000 172 against 176), not from fp32 (rows of 33 405, streamed 415, one a
//     thread 456);
//   back four (35M values in bf16, rows of 33 24 against 31, of 129 24 against 32, of 1000 18
//     and 18; 300M: 274 against 405, 264 against 422, 158 against 201), streamed where a row
//     fills a line (4 bits, slots in any order: rows of 1000 261 against 325, of 48 634 against 473);
//   fp32 rows of whole vectors one both ways (300M values, rows of 1000 258 against 284, back 303
//     against 348), but four back from 4 bits (392 against 500); rows of less than a group one to and
//     from 4 bits (300M fp32 values, rows of 7 3.3 ms against 4.1).
struct Plan {
    QuantParams p;
    bool rows, four, stream;
    int split;                                         // see Part
    int64_t grid;
};
Plan plan_of(const QuantParams &q, int elem, int bits, bool back) {
    Plan f{q, false, false, false, 0, 0};
    QuantParams &p = f.p;
    if (!p.value_index && !p.held_index && (p.n == 1 || (p.stride == p.D && p.D % kGroup == 0))) {
        p.D *= p.n;
        p.n = 1;
        p.stride = p.D;
    }
    f.rows = p.D <= kPart / 2 && p.n > 1;
    f.split = 2;
    while (f.rows && (8 << f.split) < p.D) ++f.split;
    const int64_t per = kThreads >> f.split;
    auto grid = [&](int U) { return f.rows ? (p.n + U * per - 1) / (U * per) : p.n * ((p.D + U * kPart - 1) / (U * kPart)); };
    const bool large = (double)p.n * p.D * (elem + bits / 8.0) > (256 << 20);
    if (f.rows) {
        const bool whole = elem == 4 && p.D % 4 == 0;
        f.four = (back ? !whole || bits == 4 : large && !whole) && (bits == 8 || p.D >= kGroup) && grid(4) >= 2048;
        f.stream = f.four && large && (back ? p.D * elem >= 128 : elem == 2 && bits == 8);
    } else {
        f.four = p.D >= 4 * kPart && grid(4) >= 2048;
        f.stream = f.four && large;
    }
    f.grid = grid(f.four ? 4 : 1);
    if (!f.rows) f.split = (int)(f.grid / p.n);
    return f;
}

template <typename E, int BITS, int U, bool STREAM, bool ROWS> void launch(const Plan &f, bool back, hipStream_t st) {
    if (back)
        dequant_kernel<E, BITS, U, STREAM, ROWS><<<(unsigned)f.grid, kThreads, 0, st>>>(f.p, f.split);
    else if constexpr (!ROWS || U == 1 || STREAM == (sizeof(E) == 2 && BITS == 8))
        quant_kernel<E, BITS, U, STREAM, ROWS><<<(unsigned)f.grid, kThreads, 0, st>>>(f.p, f.split);
}
template <typename E, int BITS, bool ROWS> void launch_rows(const Plan &f, bool back, hipStream_t st) {
    if (!f.four)
        launch<E, BITS, 1, false, ROWS>(f, back, st);
    else if (f.stream)
        launch<E, BITS, 4, true, ROWS>(f, back, st);
    else
        launch<E, BITS, 4, false, ROWS>(f, back, st);
}
template <typename E, int BITS> void launch_e(const Plan &f, bool back, hipStream_t st) {
    f.rows ? launch_rows<E, BITS, true>(f, back, st) : launch_rows<E, BITS, false>(f, back, st);
}

}  // namespace

int64_t quant_grid(const QuantParams &p, int dtype, int bits, bool back) {
    return plan_of(p, dtype == 0 ? 2 : 4, bits, back).grid;
}

hipError_t launch_quant(const QuantParams &p, int dtype, int bits, bool back, hipStream_t stream, Profiler *prof) {
    if (p.n == 0 || p.D == 0) return hipSuccess;
    const Plan f = plan_of(p, dtype == 0 ? 2 : 4, bits, back);
    const int kind = back ? kDequantKernel : kQuantKernel;
    if (prof) prof->begin(kind, stream);
    if (dtype == 0)
        bits == 8 ? launch_e<bf16, 8>(f, back, stream) : launch_e<bf16, 4>(f, back, stream);
    else
        bits == 8 ? launch_e<float, 8>(f, back, stream) : launch_e<float, 4>(f, back, stream);
    const hipError_t err = hipGetLastError();
    if (prof) prof->end(kind, stream);
    return err;
}

}  // namespace gdn
