// The gated linear recurrence for gfx950: per channel
//   h_t = e^(g_t) h_(t-1) + beta_t x_t,    y_t = h_t,
// the state in fp32, and its gradients
//   dh_t = dy_t + e^(g_(t+1)) dh_(t+1)     (dht added at a sequence's last token)
//   dx = beta dh,  dbeta = x dh,  dg_t = e^(g_t) h_(t-1) dh_t,  dh0 = e^(g_1) dh_1
// with h_(t-1) the forward's y_(t-1) as it was rounded, or the initial state.
//
// Bound by HBM where there are tokens enough: each input is read once and each output
// written once.  The recurrence is serial in the tokens, but what a run of tokens does
// to a state is a map h -> A h + b, and maps compose: workgroups take tiles of tokens
// and channels, keep them in registers, hand their maps on to the later ones (see
// carry_in) and run through their tokens again with the state that comes in, so that
// nothing is read twice: a single-pass scan with decoupled look-back (Merrill and
// Garland 2016) of maps, composed in an order that the sizes fix.  A pass over the data for the maps and another for the
// outputs would read x and the gates twice.
//
// A product of decays may underflow to zero where no decay is zero: an infinite state
// then becomes a NaN behind it, never a finite number.  To keep the infinity (products no
// smaller than 2^-149 while no factor is zero) took 2 to 10 % of the passes (64 packed
// prompts 650 -> 662 us, gradients of 64 x 4096 tokens of 32 channels 86 -> 94).
//
// Measured (the call, workspace cleared): 131,072 tokens of 4096 channels with bf16 gates
// and no beta 653 us (4.9 TB/s of x, g and y; one thread a channel 106 ms); 64 packed
// prompts, 74,000 tokens of 4096, fp32 g and beta 648 us (5.6 TB/s; 2.66 ms); gradients of
// 16,384 tokens of 4096 with fp32 gates 279 us (5.8 TB/s; 5.7 ms), of the packed prompts
// with bf16 gates and x and y in 8 bits 905 us (4.7 TB/s; 3.3 ms).  Few tokens or channels
// are bound by the latency of a tile, about 15 us: loads 3, decays and sums 3, maps
// of other tiles 4, stores 2 (2042 tokens of 1001 channels in fp32 15 us, and 2 for
// the workspace); long sequences of few channels by the states' way from block to
// block (131,072 tokens of 256 channels 126 us, floor 68; 2^20 of 64 177, floor 68).
#include <algorithm>
#include <type_traits>

// Products and sums are fused where fmaf says so and nowhere else: two lanes that
// share a channel (see lane_of) compute it at different places of their vectors and
// have to get the same bits.
#pragma clang fp contract(off)

#include "gdn_quant_device.h"

namespace gdn {
namespace {

using namespace dev;

// e^g for g <= 0, with a relative error of at most 0.62 2^-24 down to -0.1 and 1.4 2^-24
// to -87, and 0 below: n = the integer nearest to g / ln 2, r = g - n ln 2 with ln 2 in
// two parts (rounded to one the error grows with n, to 5.1 2^-24), e^r = 1 + r + r^2 p(r)
// with p of degree 4 interpolating at Chebyshev's nodes (2e-9 off on |r| <= ln 2 / 2), n
// added to the exponent.  The sum g / ln 2 + 1.5 2^23 has n in its low bits.  ldexp adds
// it: NaN for a NaN whatever its payload (which an integer sum would carry into the
// exponent), infinity for a gate above 88.7, which has no business here.  13 instructions;
// the hardware exponential takes the time of 5, but near 0 it is low by 0.12 2^-24 on
// average, which a channel sums over all the tokens that it remembers (it would save 1
// to 5 %).
__device__ __forceinline__ float decay(float g) {
    const float t = fmaf(g, 1.4426950408889634f, kRoundBias), n = t - kRoundBias;
    const float r = fmaf(n, 1.9046543e-9f, fmaf(n, -0.6931471805599453f, g));
    float q = fmaf(r, 0.0013926184f, 0.008363179f);
    q = fmaf(r, q, 0.041666556f);
    q = fmaf(r, q, 0.16666576f);
    q = fmaf(r, q, 0.5f);
    q = fmaf(r, q, 1.f);
    q = fmaf(r, q, 1.f);
    return g < -87.f ? 0.f : __builtin_amdgcn_ldexpf(q, (int)(__float_as_uint(t) - __float_as_uint(kRoundBias)));
}

// VC = 1, 2 or 4 consecutive elements, as loaded, at any address.  S: past the caches.
template <typename E, int VC> struct Vector : Raw<E, VC> {};
template <typename E> struct Vector<E, 2> {
    typedef typename Two<E>::T T;
    typedef typename Two<E>::U U;
    template <bool S = false> static __device__ __forceinline__ T load(const E *p) {
        if constexpr (S)
            return __builtin_nontemporal_load((const U *)p);
        else
            return *(const U *)p;
    }
    template <bool S = false> static __device__ __forceinline__ void store(E *p, T r) {
        if constexpr (S)
            __builtin_nontemporal_store(r, (U *)p);
        else
            *(U *)p = r;
    }
    static __device__ __forceinline__ T zero() { return T{}; }
    static __device__ __forceinline__ float get(T r, int e) { return to_f(r[e]); }
    static __device__ __forceinline__ void set(T &r, int e, float x) { r[e] = to_e<E>(x); }
};
template <typename E> struct Vector<E, 1> {
    typedef E T;
    template <bool S = false> static __device__ __forceinline__ T load(const E *p) { return *p; }
    template <bool S = false> static __device__ __forceinline__ void store(E *p, T r) { *p = r; }
    static __device__ __forceinline__ T zero() { return to_e<E>(0.f); }
    static __device__ __forceinline__ float get(T r, int) { return to_f(r); }
    static __device__ __forceinline__ void set(T &r, int, float x) { r = to_e<E>(x); }
};

// A value that the compiler takes to be another one, so that what was computed from it
// is computed again instead of being kept: two widened bf16 values take two registers,
// the pair as loaded one.
template <typename T> __device__ __forceinline__ void forget(T &r) {
    typedef std::conditional_t<sizeof(T) == 8, unsigned long long, std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>> U;
    U v = __builtin_bit_cast(U, r);
    asm("" : "+v"(v));
    r = __builtin_bit_cast(T, v);
}

template <int VC> __device__ __forceinline__ void load_states(const void *s, int64_t at, int b16, float *h) {
    if (b16) {
        const typename Vector<bf16, VC>::T r = Vector<bf16, VC>::load((const bf16 *)s + at);
#pragma unroll
        for (int e = 0; e < VC; ++e) h[e] = Vector<bf16, VC>::get(r, e);
    } else {
        const typename Vector<float, VC>::T r = Vector<float, VC>::load((const float *)s + at);
#pragma unroll
        for (int e = 0; e < VC; ++e) h[e] = Vector<float, VC>::get(r, e);
    }
}
template <int VC> __device__ __forceinline__ void store_states(void *s, int64_t at, int b16, const float *h) {
    if (b16) {
        typename Vector<bf16, VC>::T r;
#pragma unroll
        for (int e = 0; e < VC; ++e) Vector<bf16, VC>::set(r, e, h[e]);
        Vector<bf16, VC>::store((bf16 *)s + at, r);
    } else {
        typename Vector<float, VC>::T r;
#pragma unroll
        for (int e = 0; e < VC; ++e) Vector<float, VC>::set(r, e, h[e]);
        Vector<float, VC>::store((float *)s + at, r);
    }
}
// ---------------------------------------------------------------------------
// Tiles.  The tokens of all sequences lie on one axis, which is cut into tiles of
// W * R * S tokens; a workgroup of W waves takes one tile of up to 64 / R * VC
// channels, every strip of 64 / R lanes S of its tokens, every lane VC channels.  All
// of it is loaded once, into registers; what a strip's tokens do to a state is
// h -> A h + b, and such maps compose.  The backward pass is the same with tiles,
// strips and tokens in reverse.  R = 1, and 4 for up to 64 channels, which a wave
// has not lanes enough for otherwise.
// ---------------------------------------------------------------------------
constexpr int kGroupTiles = 8, kBlockGroups = 8;   // tiles of a group, groups of a block

// What is the same in all lanes of a strip, as a scalar where the strip is the wave.
template <int R> __device__ __forceinline__ int strip_int(int x) { return R == 1 ? __builtin_amdgcn_readfirstlane(x) : x; }

// Channels of a lane.  The vectors of VC channels are shared out evenly among the
// column blocks, 16 at a time, so that blocks meet where lines or halves of them do
// (gradients of 96,712 tokens of 720 channels with fp32 gates 398 -> 355 us); the last
// vector of an odd row ends with it and overlaps its neighbour, which is in the same
// strip: both compute and store the same values.
struct Lane {
    uint32_t c;                                        // unsigned: a 32-bit offset from a row in scalar registers
    bool live;
};
template <typename E> __device__ __forceinline__ const E *at(const void *base, int64_t row, int64_t stride, uint32_t c) {
    return (const E *)((const char *)((const E *)base + row * stride) + c * (uint32_t)sizeof(E));
}
template <typename E> __device__ __forceinline__ E *at(void *base, int64_t row, int64_t stride, uint32_t c) {
    return (E *)((char *)((E *)base + row * stride) + c * (uint32_t)sizeof(E));
}
// Token s of a strip that begins at token tw.  Where a wave has several strips their rows
// differ from lane to lane, and an address of its own for each token would take more
// registers than there are (gradients of 16 sequences of 16,384 tokens of 32 channels in
// fp32 152 us, with one address a strip 131).
template <int R, typename E>
__device__ __forceinline__ const E *token(const void *base, int tw, int s, int64_t stride, uint32_t c) {
    return R == 1 ? at<E>(base, tw + s, stride, c) : at<E>(base, tw, stride, c) + s * stride;
}
template <int R, typename E> __device__ __forceinline__ E *token(void *base, int tw, int s, int64_t stride, uint32_t c) {
    return R == 1 ? at<E>(base, tw + s, stride, c) : at<E>(base, tw, stride, c) + s * stride;
}
template <int VC> __device__ __forceinline__ Lane lane_of(int D, int ncb, int cb, int lane) {
    const int nv = (D + VC - 1) / VC, units = (nv + 15) / 16, each = units / ncb, more = units % ncb;
    const int v = 16 * (cb * each + min(cb, more)) + lane;
    return {(uint32_t)min(v * VC, D - VC), v < nv && lane < 16 * (each + (cb < more ? 1 : 0))};
}
template <int VC> __host__ __device__ __forceinline__ int column_blocks(int D) { return ((D + VC - 1) / VC + 63) / 64; }

// Workspace: a counter (16 bytes), then words, a channel of a column block each: what a
// tile does to a state, for all tiles; what a group does; the state before a block
// of groups.  A tile's words lie in the order of its lanes' vectors, so that 64 lanes
// move 512 bytes at a time.
struct Handed {
    unsigned long long *tiles, *groups, *states;
    int64_t row;                                       // words of one tile, all column blocks
};
__host__ __device__ __forceinline__ int64_t groups_of(int64_t tiles) { return (tiles + kGroupTiles - 1) / kGroupTiles; }
__host__ __device__ __forceinline__ int64_t handed_words(int64_t tiles, int64_t row) {
    const int64_t groups = groups_of(tiles);
    return 2 + (tiles + groups + (groups + kBlockGroups - 1) / kBlockGroups) * row;
}
// The words of column block cb, this lane's first.
template <int VC, int LR> __device__ __forceinline__ Handed handed_of(void *ws, int64_t tiles, int ncb, int cb, int lane) {
    const int64_t row = (int64_t)ncb * VC * LR;
    unsigned long long *w = (unsigned long long *)ws + 2 + cb * VC * LR + lane;
    return {w, w + tiles * row, w + (tiles + groups_of(tiles)) * row, row};
}

// A word carries its own flag, the sign of its upper half (decays are not negative),
// so that it is handed on without a fence: one 64-bit store and loads that repeat
// until the flag is there, past the caches that are not shared.  The wait is bounded:
// only where another call writes the same workspace meanwhile does a word fail to come,
// and then, after some seconds, NaNs are taken for it.
constexpr int kMaxPolls = 1 << 22;
__device__ __forceinline__ void put(unsigned long long *w, float A, float h) {
    __hip_atomic_store(w, (unsigned long long)(__float_as_uint(A) | 0x80000000u) << 32 | __float_as_uint(h),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <int VC, int LR> __device__ __forceinline__ void await(const unsigned long long *w, float2 (*to)[LR]) {
    unsigned long long v[VC];
    int polls = 0;
    for (;;) {                                         // the wave's lanes wait together
        bool all = true;
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            v[e] = __hip_atomic_load(w + e * LR, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            all = all && (long long)v[e] < 0;
        }
        if (__ballot(!all) == 0 || polls == kMaxPolls) break;
        ++polls;
        __builtin_amdgcn_s_sleep(1);
    }
    if (polls == kMaxPolls)
#pragma unroll
        for (int e = 0; e < VC; ++e)
            if ((long long)v[e] >= 0) v[e] = 0x7fc000007fc00000ull;
#pragma unroll
    for (int e = 0; e < VC; ++e)
        to[e][0] = float2{__uint_as_float((uint32_t)(v[e] >> 32) & 0x7fffffffu), __uint_as_float((uint32_t)v[e])};
}

// The words' flags, before any tile sets one, and the counter.
__global__ void __launch_bounds__(256) scan_clear_kernel(uint4 *w, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) w[i] = uint4{0, 0, 0, 0};
}

// Number of entries of cu[0 .. n-1] (not decreasing) that are at most t: a search by
// 64 lanes, 64 places a step.
__device__ __forceinline__ int count_to(const int32_t *cu, int n, int t, int lane) {
    int lo = 0, len = n;                               // the answer lies in [lo, lo + len]
    while (len > 0) {
        const int step = (len + 63) / 64, at = lo + (lane + 1) * step - 1;
        const bool in = at < lo + len && cu[at] <= t;
        const int k = __popcll(__ballot(in));
        const int end = lo + len;
        lo += k * step;
        len = min(step - 1, end - lo);
    }
    return lo;
}

// The sequences of a tile, in LDS: start[i] is the sequence that begins at its token i
// (the last, non-empty one of those that do), or -1; one token more than the tile's.
template <int TT> struct Sequences {
    int start[TT + 1];
    int first, first_token;                            // sequence of the tile's first token, its first token
};
template <int TT, int NT>
__device__ __forceinline__ void find_sequences(Sequences<TT> &q, const ScanParams &p, int t0, int t_end) {
    const int tid = threadIdx.x, lane = tid & 63;
    if (!p.cu_seqlens) {
        for (int i = tid; i <= TT; i += NT) q.start[i] = (t0 + i) % p.T == 0 ? (t0 + i) / p.T : -1;
        if (tid == 0) {
            q.first = t0 / p.T;
            q.first_token = q.first * p.T;
        }
        lds_barrier();
        return;
    }
    for (int i = tid; i <= TT; i += NT) q.start[i] = -1;
    const int n0 = min(max(count_to(p.cu_seqlens, p.N + 1, t0, lane) - 1, 0), p.N - 1);
    if (tid == 0) {
        q.first = n0;
        q.first_token = cu_at(p.cu_seqlens, n0, p.T_tot);
    }
    lds_barrier();
    for (int n = n0 + tid; n < p.N; n += NT) {
        const int at = cu_at(p.cu_seqlens, n, p.T_tot) - t0;
        if (at > TT) break;
        if (at >= 0) atomicMax(&q.start[at], n);
    }
    lds_barrier();
}

// Rows of sequences without tokens, shared out over the tiles: the final state is the
// initial one.
template <int VC, int W>
__device__ __forceinline__ void empty_sequences(const ScanParams &p, int tile, int tiles, uint32_t c, bool live) {
    if (!p.final_state || (p.indices && p.initial) || !live) return;   // a pool's slots keep what they hold
    const int lo = (int)((int64_t)p.N * tile / tiles), hi = (int)((int64_t)p.N * (tile + 1) / tiles);
    for (int n = lo + (threadIdx.x >> 6); n < hi; n += W) {
        int t0, t1;
        seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
        if (t0 != t1) continue;
        int64_t at = (int64_t)n * p.D + c;
        if (p.indices) {
            const int slot = p.indices[n];
            if (slot < 0 || slot >= p.pool_size) continue;
            at = (int64_t)slot * p.D + c;
        }
        float h[VC];
#pragma unroll
        for (int e = 0; e < VC; ++e) h[e] = 0.f;
        if (p.initial) load_states<VC>(p.initial, at, p.state_bf16, h);
        store_states<VC>(p.final_state, at, p.state_bf16, h);
    }
}

// Sequence of the token before token i of the tile (of the tile's first where i = 0).
template <int R, int TT> __device__ __forceinline__ int sequence_before(const Sequences<TT> &q, int i, int lane) {
    constexpr int LR = 64 / R;
    int n = q.first;
    for (int j = lane; j < i; j += LR) n = max(n, q.start[j]);
#pragma unroll
    for (int o = LR / 2; o >= 1; o >>= 1) n = max(n, __shfl_xor(n, o));
    return strip_int<R>(n);
}

// Tiles are taken in the order of a counter, so that whatever tile a workgroup waits
// for is with a workgroup that runs already; as each hands its map on before it
// waits, and the earliest one waits for none, every wait ends.  A number past the last
// tile's, which only a workspace that another call uses meanwhile can give, is none's.
__device__ __forceinline__ int next_tile(void *ws, int tiles, int *ticket) {
    if (tiles == 1) return blockIdx.x;
    if (threadIdx.x == 0) *ticket = (int)atomicAdd((uint32_t *)ws, 1u);
    lds_barrier();
    return __builtin_amdgcn_readfirstlane(*ticket);
}

template <int VC, int W, int R> struct Exchange {
    static constexpr int LR = 64 / R;                  // lanes of a strip
    float2 maps[W * R][VC][LR];                        // what each strip's tokens do to a state
    float2 before[kGroupTiles + kBlockGroups - 1][VC][LR];   // tiles and groups before this tile, the state before them
    int cut[W * R];                                    // a state begins anew in the strip's tokens
};
// Maps lo .. hi - 1 of those that a tile waits for, one a strip: nt of tiles from `from`
// on, ng of groups from gfrom on, the state before the block.
template <int VC, int W, int R>
__device__ __forceinline__ void fetch(Exchange<VC, W, R> &x, const Handed &hand, int lane, int rank, int lo, int hi, int from,
                                      int nt, int gfrom, int ng, int block) {
#pragma unroll 1
    for (int k = lo + rank; k < hi; k += W * R) {
        const unsigned long long *src = k < nt        ? hand.tiles + (from + k) * hand.row
                                        : k < nt + ng ? hand.groups + (gfrom + k - nt) * hand.row
                                                      : hand.states + block * hand.row;
        await<VC, 64 / R>(src, (float2 (*)[64 / R])&x.before[k][0][lane]);
    }
}
// The state that comes into a strip's tokens.  rank: the strip's place in its tile, tile:
// the tile's place in the order of the pass; A, b: the strip's map, fresh: whether a
// state begins anew in it (its map is then b alone); waits: whether a state comes
// into the tile, since: the place of the tile where it began.
//
// It is the state before the block of 64 tiles, then the maps of the block's groups
// of 8 tiles before this one, then those of the tiles before this one in its group:
// an order that depends on the sizes alone.  The last tile of a group hands on the
// group's map, the last one of a block the state.  A state handed on from one
// workgroup to another takes 2.8 us (a store, a load that meets it, the sum between);
// with one level, from group to group, 131,072 tokens of 256 channels took 700 us.
template <int VC, int W, int R>
__device__ __forceinline__ void carry_in(Exchange<VC, W, R> &x, const Handed &hand, int lane, int rank, int tile, int tiles,
                                         bool waits, int since, bool fresh, const float *A, const float *b, float *h) {
#pragma unroll
    for (int e = 0; e < VC; ++e) x.maps[rank][e][lane] = float2{A[e], b[e]};
    if (lane == 0) x.cut[rank] = fresh;
    lds_barrier();
    bool own = false;                                  // the state began in the tile, before the strip
    float Ae[VC], he[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        Ae[e] = 1.f;
        he[e] = 0.f;
    }
#pragma unroll 1
    for (int k = 0; k < rank; ++k) {
        const bool anew = x.cut[k] != 0;
        own = own || anew;
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            const float2 m = x.maps[k][e][lane];
            he[e] = anew ? m.y : fmaf(m.x, he[e], m.y);
            Ae[e] *= m.x;
        }
    }
    const bool last = rank == W * R - 1;               // the strip whose end is the tile's
    if (tiles > 1 && last) {
#pragma unroll
        for (int e = 0; e < VC; ++e)
            put(hand.tiles + tile * hand.row + e * (64 / R), Ae[e] * A[e], fresh ? b[e] : fmaf(A[e], he[e], b[e]));
    }
    const int group = tile / kGroupTiles, base = group * kGroupTiles, block = group / kBlockGroups;
    const int from = max(base, since), nt = waits ? tile - from : 0;
    const int gfrom = max(block * kBlockGroups, since / kGroupTiles), ng = waits && since < base ? group - gfrom : 0;
    const bool further = waits && since < block * kBlockGroups * kGroupTiles;
    const bool ends_group = tile % kGroupTiles == kGroupTiles - 1 && tile + 1 < tiles;
    const int all = nt + ng + (further ? 1 : 0);
    float At[VC], ht[VC], hin[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        At[e] = 1.f;
        ht[e] = hin[e] = 0.f;
    }
    if (waits) {
        fetch<VC, W, R>(x, hand, lane, rank, 0, ends_group ? nt : all, from, nt, gfrom, ng, block);
        lds_barrier();
#pragma unroll 1
        for (int k = 0; k < nt; ++k)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const float2 m = x.before[k][e][lane];
                ht[e] = since == from + k ? m.y : fmaf(m.x, ht[e], m.y);
                At[e] *= m.x;
            }
    }
    if (ends_group && last) {
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            const float T = Ae[e] * A[e], v = fresh ? b[e] : fmaf(A[e], he[e], b[e]);
            put(hand.groups + group * hand.row + e * (64 / R), At[e] * T, fresh || own ? v : fmaf(T, ht[e], v));
        }
    }
    if (waits) {
        if (ends_group) {
            fetch<VC, W, R>(x, hand, lane, rank, nt, all, from, nt, gfrom, ng, block);
            lds_barrier();
        }
        if (further)
#pragma unroll
            for (int e = 0; e < VC; ++e) hin[e] = x.before[nt + ng][e][lane].y;
#pragma unroll 1
        for (int k = 0; k < ng; ++k)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const float2 m = x.before[nt + k][e][lane];
                hin[e] = since / kGroupTiles == gfrom + k ? m.y : fmaf(m.x, hin[e], m.y);
            }
#pragma unroll
        for (int e = 0; e < VC; ++e) hin[e] = since < base ? fmaf(At[e], hin[e], ht[e]) : ht[e];
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) h[e] = own ? he[e] : fmaf(Ae[e], hin[e], he[e]);
    if (ends_group && group % kBlockGroups == kBlockGroups - 1 && last) {
#pragma unroll
        for (int e = 0; e < VC; ++e)
            put(hand.states + (block + 1) * hand.row + e * (64 / R), 0.f, fresh ? b[e] : fmaf(A[e], h[e], b[e]));
    }
}

template <typename E, typename G, bool BETA, bool STREAM, int VC, int W, int S, int R>
__global__ void __launch_bounds__(W * 64, 4) scan_kernel(ScanParams p, int ncb, int tiles) {
    constexpr int NT = W * 64, LR = 64 / R, TT = W * R * S;
    static_assert(S <= LR, "a strip looks at its tokens with a lane each");
    __shared__ Sequences<TT> q;
    __shared__ Exchange<VC, W, R> x;
    __shared__ int ticket;
    const int lane = threadIdx.x % LR, w = strip_int<R>(threadIdx.x / LR);   // in the strip; the strip
    const int id = next_tile(p.ws, tiles, &ticket);
    if ((uint32_t)id >= (uint32_t)(tiles * ncb)) return;
    const Handed hand = handed_of<VC, LR>(p.ws, tiles, ncb, id % ncb, lane);
    const int tile = id / ncb, t0 = tile * TT;
    const Lane ln = lane_of<VC>(p.D, ncb, id % ncb, lane);
    const int t_end = p.cu_seqlens ? cu_at(p.cu_seqlens, p.N, p.T_tot) : p.T_tot;
    empty_sequences<VC, W>(p, tile, tiles, ln.c, ln.live);
    if (t0 >= t_end) return;
    const int tw = t0 + w * S, nv = min(max(t_end - tw, 0), S);   // the strip's tokens

    typedef Vector<E, VC> RE;
    typedef Vector<G, VC> RG;
    // Inputs stay as they were loaded where that takes fewer registers (bf16 gates), and
    // are widened twice; decays are taken once.
    constexpr bool RAW = sizeof(G) == 2;
    typename RE::T xr[S];
    typename RG::T gr[S], br[S];
    float a[S][VC], u[RAW ? 1 : S][VC];
    // With a strip a wave every lane loads, those without channels another's and those
    // without tokens the last token, so that the loads are issued in one run; with several
    // only those that have both.
    const int last = R == 1 ? t_end - 1 - tw : S;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if constexpr (R > 1) {
            xr[s] = RE::zero();
            gr[s] = RG::zero();
            if (BETA) br[s] = RG::zero();
            if (s >= nv || !ln.live) continue;
        }
        const int t = min(s, last);
        xr[s] = RE::template load<STREAM>(token<R, E>(p.x, tw, t, p.x_stride, ln.c));
        gr[s] = RG::template load<STREAM>(token<R, G>(p.g, tw, t, p.g_stride, ln.c));
        if (BETA) br[s] = RG::template load<STREAM>(token<R, G>(p.beta, tw, t, p.beta_stride, ln.c));
    }
    find_sequences<TT, NT>(q, p, t0, t_end);
    if (R == 1 && nv < S)                              // no token: a = 1, u = 0, the state stays
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (s >= nv) {
                xr[s] = RE::zero();
                gr[s] = RG::zero();
            }
    auto input = [&](int s, int e) {
        const float v = RE::get(xr[s], e);
        return BETA ? v * RG::get(br[s], e) : v;
    };
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            a[s][e] = decay(RG::get(gr[s], e));
            if constexpr (!RAW) u[s][e] = input(s, e);
        }
    auto taken = [&](int s, int e) {
        if constexpr (RAW)
            return input(s, e);
        else
            return u[s][e];
    };
    // sequences that begin at, or end with, the strip's tokens
    const bool is = lane < nv;
    const int mine = w * S + min(lane, S - 1);
    const int strip = threadIdx.x % 64 / LR * LR;      // its first lane
    const uint32_t mask = LR == 64 ? ~0u : (1u << (LR % 32)) - 1;
    const uint32_t starts = (uint32_t)(__ballot(is && q.start[mine] >= 0) >> strip) & mask;
    const uint32_t ends = (uint32_t)(__ballot(is && (q.start[mine + 1] >= 0 || t0 + mine + 1 == t_end)) >> strip) & mask;
    auto initial = [&](int n, float *h) {
        int64_t from = (int64_t)n * p.D + ln.c;
        bool has = p.initial != nullptr && ln.live;
        if (p.indices) {
            const int slot = p.indices[n];
            has = has && slot >= 0 && slot < p.pool_size;
            from = (int64_t)slot * p.D + ln.c;
        }
#pragma unroll
        for (int e = 0; e < VC; ++e) h[e] = 0.f;
        if (has) load_states<VC>(p.initial, from, p.state_bf16, h);
    };
    float A[VC], h[VC], b[VC], h0[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        A[e] = 1.f;
        b[e] = h0[e] = 0.f;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (starts >> s & 1) {                         // what came in is replaced
            initial(strip_int<R>(q.start[w * S + s]), h0);
#pragma unroll
            for (int e = 0; e < VC; ++e) b[e] = h0[e];
        }
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            b[e] = fmaf(a[s][e], b[e], taken(s, e));
            A[e] *= a[s][e];
        }
    }
    carry_in<VC, W, R>(x, hand, lane, w, tile, tiles, q.first_token < t0, q.first_token / TT, starts != 0, A, b, h);
    if constexpr (RAW)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            forget(xr[s]);
            if (BETA) forget(br[s]);
        }
    const int stored = ln.live ? nv : 0;               // tokens that this lane stores
    int seq = ends ? sequence_before<R>(q, w * S, lane) : 0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (starts >> s & 1) {
            // The last sequence that begins here may end with another strip, which may have
            // stored its final state where its initial state was: that one is h0 still.
            // The others end here.
            seq = strip_int<R>(q.start[w * S + s]);
            if (starts >> s != 1)
                initial(seq, h);
            else
#pragma unroll
                for (int e = 0; e < VC; ++e) h[e] = h0[e];
        }
        typename RE::T o = RE::zero();
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            h[e] = fmaf(a[s][e], h[e], taken(s, e));
            RE::set(o, e, h[e]);
        }
        if (s < stored) RE::template store<STREAM>(token<R, E>(p.y, tw, s, p.D, ln.c), o);
        if ((ends >> s & 1) && p.final_state && ln.live) {
            int64_t to = (int64_t)seq * p.D + ln.c;
            bool kept = true;
            if (p.indices) {
                const int slot = p.indices[seq];
                kept = slot >= 0 && slot < p.pool_size;
                to = (int64_t)slot * p.D + ln.c;
            }
            if (kept) store_states<VC>(p.final_state, to, p.state_bf16, h);
        }
    }
}

// VC values of a row as they are, or in 8 bits: as loaded, and as fp32.  Of held ones
// those of a lane lie in two groups where vectors overlap (two, see lane_of).
template <typename E, int VC, bool HELD, bool STREAM> struct Saved {
    typename Vector<E, VC>::T r;
    __device__ __forceinline__ void clear() { r = Vector<E, VC>::zero(); }
    __device__ __forceinline__ void load(const void *v, const Held &, int64_t row, int64_t stride, int, uint32_t c, bool) {
        r = Vector<E, VC>::template load<STREAM>(at<E>(v, row, stride, c));
    }
    __device__ __forceinline__ float get(int e, uint32_t, bool) const { return Vector<E, VC>::get(r, e); }
};
template <typename E, int VC, bool STREAM> struct Saved<E, VC, true, STREAM> {
    uint32_t codes, scales;                            // scales: of the first value's group low, of the last one's high
    __device__ __forceinline__ void clear() { codes = scales = 0; }
    __device__ __forceinline__ void load(const void *, const Held &h, int64_t row, int64_t, int D, uint32_t c, bool two) {
        const uint8_t *src = at<uint8_t>(h.codes, row, D, c);
        const int groups = (D + kGroup - 1) / kGroup;
        codes = VC == 4 ? *(const u32u *)src : VC == 2 ? *(const u16u *)src : *src;
        scales = *at<uint16_t>(h.scales, row, groups, c / kGroup);
        if (two) scales |= (uint32_t)*at<uint16_t>(h.scales, row, groups, (c + VC - 1) / kGroup) << 16;
    }
    __device__ __forceinline__ float get(int e, uint32_t c, bool two) const {
        const uint32_t s = two && (c + e) / kGroup != c / kGroup ? scales & 0xffff0000u : scales << 16;
        return held_byte(codes, e) * __uint_as_float(s);
    }
};

template <typename E, typename G, bool BETA, bool HELD, bool STREAM, int VC, int W, int S, int R>
__global__ void __launch_bounds__(W * 64, 4) scan_bwd_kernel(ScanParams p, int ncb, int tiles) {
    constexpr int NT = W * 64, LR = 64 / R, TT = W * R * S;
    static_assert(S <= LR, "a strip looks at its tokens with a lane each");
    __shared__ Sequences<TT> q;
    __shared__ Exchange<VC, W, R> x;
    __shared__ int ticket;
    const int lane = threadIdx.x % LR, w = strip_int<R>(threadIdx.x / LR);   // in the strip; the strip
    const int id = next_tile(p.ws, tiles, &ticket);
    if ((uint32_t)id >= (uint32_t)(tiles * ncb)) return;
    const Handed hand = handed_of<VC, LR>(p.ws, tiles, ncb, id % ncb, lane);
    const int place = id / ncb, tile = tiles - 1 - place, t0 = tile * TT;
    const Lane ln = lane_of<VC>(p.D, ncb, id % ncb, lane);
    const int t_end = p.cu_seqlens ? cu_at(p.cu_seqlens, p.N, p.T_tot) : p.T_tot;
    {
        // the gradient of an empty sequence's initial state is that of its final state
        ScanParams e = p;
        e.initial = p.dht;
        e.final_state = p.dinitial;
        empty_sequences<VC, W>(e, tile, tiles, ln.c, ln.live);
    }
    if (t0 >= t_end) return;
    const int tw = t0 + w * S, nv = min(max(t_end - tw, 0), S);   // the strip's tokens
    const bool two = p.D % VC != 0;

    typedef Vector<E, VC> RE;
    typedef Vector<G, VC> RG;
    typedef Saved<E, VC, HELD, STREAM> SV;
    constexpr bool RAW = sizeof(G) == 2;               // see scan_kernel
    typename RE::T dr[S];
    typename RG::T gr[S], br[S];
    float a[RAW ? 1 : S][VC];
    const int ahead = R == 1 ? t_end - 1 - tw : S;
#pragma unroll
    for (int s = 0; s < S; ++s) {                      // see scan_kernel
        if constexpr (R > 1) {
            dr[s] = RE::zero();
            gr[s] = RG::zero();
            if (s >= nv || !ln.live) continue;
        }
        const int t = min(s, ahead);
        dr[s] = RE::template load<STREAM>(token<R, E>(p.dy, tw, t, p.D, ln.c));
        gr[s] = RG::template load<STREAM>(token<R, G>(p.g, tw, t, p.g_stride, ln.c));
    }
    find_sequences<TT, NT>(q, p, t0, t_end);
    if (R == 1 && nv < S)
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (s >= nv) {
                dr[s] = RE::zero();
                gr[s] = RG::zero();
            }
    if constexpr (!RAW)
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int e = 0; e < VC; ++e) a[s][e] = decay(RG::get(gr[s], e));
    auto decay_of = [&](int s, int e) {
        if constexpr (RAW)
            return decay(RG::get(gr[s], e));
        else
            return a[s][e];
    };
    // what the gradients of the gates take, on its way while the tiles wait
    SV yr[S], xr[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if constexpr (R > 1) {
            yr[s].clear();
            if (BETA) {
                xr[s].clear();
                br[s] = RG::zero();
            }
            if (s >= nv || !ln.live) continue;
        }
        const int t = min(s, ahead);
        yr[s].load(p.y, p.y8, max(tw + t - 1, 0), p.D, p.D, ln.c, two);
        if (BETA) {
            xr[s].load(p.x, p.x8, tw + t, p.x_stride, p.D, ln.c, two);
            br[s] = RG::template load<STREAM>(token<R, G>(p.beta, tw, t, p.beta_stride, ln.c));
        }
    }
    const bool is = lane < nv;
    const int mine = w * S + min(lane, S - 1);
    const int strip = threadIdx.x % 64 / LR * LR;      // its first lane
    const uint32_t mask = LR == 64 ? ~0u : (1u << (LR % 32)) - 1;
    const uint32_t starts = (uint32_t)(__ballot(is && q.start[mine] >= 0) >> strip) & mask;
    const uint32_t ends = (uint32_t)(__ballot(is && (q.start[mine + 1] >= 0 || t0 + mine + 1 == t_end)) >> strip) & mask;
    const int seq = ends ? sequence_before<R>(q, w * S, lane) : 0;   // of the wave's first token, unless one begins with it
    // the gradient of the final state of the sequence that ends with token s
    auto final_gradient = [&](int s, float *c) {
        const uint32_t up_to = starts & ((2u << s) - 1);
        const int n = up_to ? strip_int<R>(q.start[w * S + 31 - __builtin_clz(up_to)]) : seq;
#pragma unroll
        for (int e = 0; e < VC; ++e) c[e] = 0.f;
        if (p.dht && ln.live) load_states<VC>(p.dht, (int64_t)n * p.D + ln.c, 0, c);
    };
    float A[VC], c[VC], b[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        A[e] = 1.f;
        b[e] = 0.f;
    }
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
        if (ends >> s & 1) final_gradient(s, b);       // in the place of what came in
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            const float av = decay_of(s, e);
            b[e] = av * (RE::get(dr[s], e) + b[e]);
            A[e] *= av;
        }
    }
    // whether a gradient comes into the tile, and from where on
    const int count = min(TT, t_end - t0), last = sequence_before<R>(q, count, lane);
    const bool waits = q.start[count] < 0 && t0 + count < t_end;
    const int end = p.cu_seqlens ? min(cu_at(p.cu_seqlens, last + 1, p.T_tot), t_end) : (last + 1) * p.T;
    carry_in<VC, W, R>(x, hand, lane, W * R - 1 - w, place, tiles, waits, tiles - 1 - (max(end, t0 + count) - 1) / TT, ends != 0, A, b, c);
    if constexpr (RAW)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            forget(gr[s]);
            forget(dr[s]);
        }
    const int stored = ln.live ? nv : 0;               // tokens that this lane stores
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
        const bool first = starts >> s & 1;
        int n = 0;
        float h0[VC];
        if (first) {
            n = strip_int<R>(q.start[w * S + s]);
#pragma unroll
            for (int e = 0; e < VC; ++e) h0[e] = 0.f;
            if (p.initial && ln.live) load_states<VC>(p.initial, (int64_t)n * p.D + ln.c, 0, h0);
        }
        if (ends >> s & 1) final_gradient(s, c);
        typename RE::T ox = RE::zero();
        typename RG::T og = RG::zero(), ob = RG::zero();
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            const float dh = RE::get(dr[s], e) + c[e];
            c[e] = decay_of(s, e) * dh;
            RG::set(og, e, c[e] * (first ? h0[e] : yr[s].get(e, ln.c, two)));
            if (BETA) {
                RG::set(ob, e, xr[s].get(e, ln.c, two) * dh);
                RE::set(ox, e, RG::get(br[s], e) * dh);
            } else {
                RE::set(ox, e, dh);
            }
        }
        if (s < stored) {
            RE::template store<STREAM>(token<R, E>(p.dx, tw, s, p.D, ln.c), ox);
            RG::template store<STREAM>(token<R, G>(p.dg, tw, s, p.D, ln.c), og);
            if (BETA) RG::template store<STREAM>(token<R, G>(p.dbeta, tw, s, p.D, ln.c), ob);
        }
        if (first && p.dinitial && ln.live) store_states<VC>(p.dinitial, (int64_t)n * p.D + ln.c, 0, c);
    }
}

// A few tokens per sequence, states in a pool: see StepSlots.  A wave takes the
// channels of a column block of one sequence; kAhead tokens are loaded before the
// first of them is used, as the wave's own stores are in the way of later loads.
// Bound by the launch and two trips to memory, slots then states: one sequence of four
// tokens of 4096 channels 5.2 us, 64 of them with a slot a token 7.8 us (a call from
// Python takes 10).
constexpr int kAhead = 4;
template <typename E, typename G, bool BETA, int VC> __global__ void __launch_bounds__(64) scan_steps_kernel(ScanParams p, int ncb) {
    typedef Vector<E, VC> RE;
    typedef Vector<G, VC> RG;
    const int n = blockIdx.x / ncb;
    const Lane ln = lane_of<VC>(p.D, ncb, blockIdx.x % ncb, threadIdx.x);
    if (!ln.live) return;
    int t0, t1;
    seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
    const int32_t *idx = p.slots.indices + (int64_t)n * p.slots.cols;
    const int a = p.slots.accepted ? min(max(p.slots.accepted[n], 1), p.slots.cols) : 1;
    const int first = idx[a - 1];
    const bool row = first >= 0 && first < p.slots.pool_size;
    float h[VC];
    if (row) load_states<VC>(p.slots.data, (int64_t)first * p.D + ln.c, p.state_bf16, h);
    for (int64_t t = t0; t < t1; t += kAhead) {
        typename RE::T xr[kAhead];
        typename RG::T gr[kAhead], br[kAhead];
        int slot[kAhead];
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
            if (t + s >= t1) break;
            const int j = (int)(t - t0) + s, col = min(j, p.slots.cols - 1);
            slot[s] = col == p.slots.cols - 1 && t + s != t1 - 1 ? -1 : idx[col];   // the last column: the last token's
            if (!row) continue;
            xr[s] = RE::load((const E *)p.x + (t + s) * p.x_stride + ln.c);
            gr[s] = RG::load((const G *)p.g + (t + s) * p.g_stride + ln.c);
            if (BETA) br[s] = RG::load((const G *)p.beta + (t + s) * p.beta_stride + ln.c);
        }
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
            if (t + s >= t1) break;
            typename RE::T o = RE::zero();
            if (row) {
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    float u = RE::get(xr[s], e);
                    if (BETA) u *= RG::get(br[s], e);
                    h[e] = fmaf(decay(RG::get(gr[s], e)), h[e], u);
                    RE::set(o, e, h[e]);
                }
                if (slot[s] >= 0 && slot[s] < p.slots.pool_size)
                    store_states<VC>(p.slots.data, (int64_t)slot[s] * p.D + ln.c, p.state_bf16, h);
            }
            RE::store((E *)p.y + (t + s) * p.D + ln.c, o);
        }
    }
}

constexpr int kStepsVec = 4;
int steps_blocks(int D) { return D < kStepsVec ? column_blocks<1>(D) : column_blocks<kStepsVec>(D); }
template <typename E, typename G, bool BETA> void launch_steps_vc(const ScanParams &p, hipStream_t st) {
    const int ncb = steps_blocks(p.D);
    const unsigned grid = (unsigned)((int64_t)p.N * ncb);
    if (p.D < kStepsVec)
        scan_steps_kernel<E, G, BETA, 1><<<grid, 64, 0, st>>>(p, ncb);
    else
        scan_steps_kernel<E, G, BETA, kStepsVec><<<grid, 64, 0, st>>>(p, ncb);
}

enum Pass { kForward, kBackward, kSteps };
// Channels of a lane, waves of a workgroup, tokens of a strip and strips of a wave: as
// many tokens as two workgroups a CU have registers for (128 a lane), so that one
// loads while the other waits or computes, and as few tiles as that gives to hand
// states through.  Measured beside their neighbours:
//   131,072 x 4096, bf16 gates, no beta: 28 tokens 643 us, 24 663, 32 694 (spilled), 16
//     737, four channels by 12 tokens 701, by 8 788
//   with beta: 20 tokens 801, 16 831, four channels by 8 893
//   packed prompts, fp32 g and beta: four channels by 8 tokens 644, by 9 659, by 7 660, two
//     by 16 (one workgroup a CU) 904
//   backward, fp32 gates: two channels by 10 tokens 280, by 8 336, four by 4 290; fp32
//     tensors two by 8 374, by 10 413; held four by 4 276, two by 10 425
//   backward, bf16 gates: two channels by 14 tokens 732, four by 8 758; held four by 6
//     896, by 5 962, by 7 959; without beta four by 10 265, by 8 274, two by 16 270
//   up to 64 channels, 2^20 tokens of 64 or 8 channels, and 16 sequences of 16,384 of 32:
//     forward, bf16 gates, 10 tokens 179, 175 and 57, 8 203, 186 and 61; fp32 gates 8 tokens (8
//     channels) 193 and 66, 7 221 and 62
//     backward, bf16 gates with beta 5 tokens 191 (64 channels) and 89, 8 195 and 97, from 8 bits 92
//     and 101; without beta 8 tokens 242, 193 and 63, 5 314, 286 and 73 (8 sequences of 2048 of 64
//     channels 22.5 and 20.9); below 4 channels 8 tokens 128 and without beta 122, 5 166 and 167
// Some tiles keep a few values in scratch memory all the same: with fp32 gates and beta above 64
// channels 8 bytes a lane, from 4 to 64 channels 20 to 100 forward and, but without beta and with
// fp32 gates, 8 to 100 backward.
struct Tile {
    int VC, W, S, R;
    constexpr int tokens() const { return W * R * S; }
};
// By the number of channels: one a lane below 4, four strips a wave up to 64 (2^20
// tokens of 8 channels with one strip a wave: 715 against 193 us, of 64 274 against 177).
enum Width { kOne, kNarrow, kWide };
Width width_of(int D) { return D < 4 ? kOne : D <= 64 ? kNarrow : kWide; }
// What a call's tensors are, as far as its tiles go by it.
struct Kind {
    bool backward, f32, gate_f32, beta, held;
};
constexpr Tile tile_of(Width width, Kind k) {
    if (width == kOne) return {1, 8, k.backward ? (k.gate_f32 ? 4 : 8) : k.gate_f32 ? 8 : 10, 4};
    if (width == kNarrow) return {4, 8, k.backward ? (k.gate_f32 ? 4 : k.beta ? 5 : 8) : k.gate_f32 ? 8 : 10, 4};
    if (!k.backward)
        return k.gate_f32 ? (k.beta ? Tile{4, 8, 8, 1} : Tile{2, 8, 20, 1}) : Tile{2, 8, k.beta ? 20 : 28, 1};
    if (k.gate_f32) return k.held ? Tile{4, 8, 4, 1} : Tile{2, 8, k.f32 ? 8 : 10, 1};
    return !k.beta ? Tile{4, 8, 10, 1} : k.held ? Tile{4, 8, 6, 1} : Tile{2, 8, 14, 1};
}
int tiles_of(int64_t T_tot, const Tile &t) { return (int)std::max<int64_t>((T_tot + t.tokens() - 1) / t.tokens(), 1); }
int blocks_of(int D, const Tile &t) { return t.R > 1 ? 1 : t.VC == 2 ? column_blocks<2>(D) : column_blocks<4>(D); }
int64_t row_words(int D, const Tile &t) { return (int64_t)blocks_of(D, t) * t.VC * (64 / t.R); }

// Passes over more than the 256 MiB of the last cache are streamed past it: packed
// prompts 645 against 699 us, gradients of 16,384 tokens 286 against 311; smaller ones
// lose by it (2042 tokens of 1001 channels 22.4 against 21.2 us).  So do rows that are
// not of whole lines, of which two workgroups read and write a part each: 96,712 tokens
// of 721 channels with bf16 gates 183 against 171 us, backward 350 against 304, with fp32
// gates 433 against 398 (720 channels: 170 and 169, 298 and 278, 356 and 358); only the
// forward pass with fp32 gates keeps a gain (213 against 217, 204 against 211).
template <typename E, typename G> bool streams(const ScanParams &p, Pass pass) {
    const int gates = p.beta ? 2 : 1, kept = p.y8.codes ? gates : gates * (int)sizeof(E);
    const int token = pass == kForward ? 2 * sizeof(E) + gates * sizeof(G) : 2 * sizeof(E) + 2 * gates * sizeof(G) + kept;
    const bool lines = p.D * sizeof(E) % 128 == 0 || (pass == kForward && sizeof(G) == 4);
    return lines && (int64_t)p.T_tot * p.D * token > 256 << 20;
}
template <typename E, typename G, bool BETA, bool HELD, Width WIDTH> void launch_tiles(const ScanParams &p, Pass pass, hipStream_t st, Profiler *prof) {
    constexpr Tile f = tile_of(WIDTH, {false, sizeof(E) == 4, sizeof(G) == 4, BETA, HELD});
    constexpr Tile b = tile_of(WIDTH, {true, sizeof(E) == 4, sizeof(G) == 4, BETA, HELD});
    constexpr bool wide = WIDTH == kWide;
    const Tile t = pass == kForward ? f : b;
    const int tiles = tiles_of(p.T_tot, t), ncb = blocks_of(p.D, t);
    if (tiles > 1) {
        const int64_t n = handed_words(tiles, row_words(p.D, t)) / 2;
        if (prof) prof->begin(kScanClearKernel, st);
        scan_clear_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0, st>>>((uint4 *)p.ws, n);
        if (prof) prof->end(kScanClearKernel, st);
    }
    const int kind = pass == kForward ? kScanKernel : kScanBwdKernel;
    if (prof) prof->begin(kind, st);
    const unsigned grid = (unsigned)(tiles * ncb);
    const bool stream = wide && streams<E, G>(p, pass);
    if (pass == kBackward) {
        if (stream)
            scan_bwd_kernel<E, G, BETA, HELD, wide, b.VC, b.W, b.S, b.R><<<grid, b.W * 64, 0, st>>>(p, ncb, tiles);
        else
            scan_bwd_kernel<E, G, BETA, HELD, false, b.VC, b.W, b.S, b.R><<<grid, b.W * 64, 0, st>>>(p, ncb, tiles);
    } else if constexpr (!HELD) {
        if (stream)
            scan_kernel<E, G, BETA, wide, f.VC, f.W, f.S, f.R><<<grid, f.W * 64, 0, st>>>(p, ncb, tiles);
        else
            scan_kernel<E, G, BETA, false, f.VC, f.W, f.S, f.R><<<grid, f.W * 64, 0, st>>>(p, ncb, tiles);
    }
    if (prof) prof->end(kind, st);
}
template <typename E, typename G, bool BETA, bool HELD> void launch_width(const ScanParams &p, Pass pass, hipStream_t st, Profiler *prof) {
    switch (width_of(p.D)) {
        case kOne: return launch_tiles<E, G, BETA, HELD, kOne>(p, pass, st, prof);
        case kNarrow: return launch_tiles<E, G, BETA, HELD, kNarrow>(p, pass, st, prof);
        case kWide: return launch_tiles<E, G, BETA, HELD, kWide>(p, pass, st, prof);
    }
}
template <typename E, typename G, bool HELD> void launch_beta(const ScanParams &p, Pass pass, hipStream_t st, Profiler *prof) {
    p.beta ? launch_width<E, G, true, HELD>(p, pass, st, prof) : launch_width<E, G, false, HELD>(p, pass, st, prof);
}
template <typename E, typename G> void launch_e(const ScanParams &p, Pass pass, hipStream_t st, Profiler *prof) {
    if (pass != kSteps) {
        p.y8.codes ? launch_beta<E, G, true>(p, pass, st, prof) : launch_beta<E, G, false>(p, pass, st, prof);
        return;
    }
    if (prof) prof->begin(kScanStepsKernel, st);
    p.beta ? launch_steps_vc<E, G, true>(p, st) : launch_steps_vc<E, G, false>(p, st);
    if (prof) prof->end(kScanStepsKernel, st);
}
hipError_t launch_any(const ScanParams &p, Pass pass, int dtype, int gate_f32, hipStream_t st, Profiler *prof) {
    if (p.N == 0) return hipSuccess;
    if (dtype != 0)
        launch_e<float, float>(p, pass, st, prof);
    else if (gate_f32)
        launch_e<bf16, float>(p, pass, st, prof);
    else
        launch_e<bf16, bf16>(p, pass, st, prof);
    return hipGetLastError();
}

}  // namespace

// Over the tiles that calls of these sizes and types take: f(tile).
template <typename F> void each_tile(int D, int gate_f32, bool backward, F f) {
    for (int i = 0; i < 8; ++i) f(tile_of(width_of(D), {backward, gate_f32 && (i & 4), gate_f32 != 0, (i & 1) != 0, (i & 2) != 0}));
}
size_t scan_workspace_bytes(int64_t T_tot, int D, int gate_f32, bool backward) {
    size_t most = 0;
    each_tile(D, gate_f32, backward, [&](const Tile &t) {
        const int tiles = tiles_of(T_tot, t);
        if (tiles > 1) most = std::max(most, (size_t)handed_words(tiles, row_words(D, t)) * 8);
    });
    return most;
}
int64_t scan_grid(int64_t T_tot, int D, int dtype, int gate_f32, bool beta, bool held, bool backward) {
    const Tile t = tile_of(width_of(D), {backward, dtype != 0, gate_f32 != 0, beta, held});
    return (int64_t)tiles_of(T_tot, t) * blocks_of(D, t) * (t.W * 64 / 256);
}
int64_t scan_steps_grid(int64_t N, int D) { return N * steps_blocks(D); }

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
