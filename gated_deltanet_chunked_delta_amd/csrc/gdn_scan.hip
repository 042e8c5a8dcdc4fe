// The gated linear recurrence for gfx950: per channel
//   h_t = e^(g_t) h_(t-1) + beta_t x_t,    y_t = h_t,
// the state in fp32, and its gradients
//   dh_t = dy_t + e^(g_(t+1)) dh_(t+1)     (dht added at a sequence's last token)
//   dx = beta dh,  dbeta = x dh,  dg_t = e^(g_t) h_(t-1) dh_t,  dh0 = e^(g_1) dh_1
// with h_(t-1) the forward's y_(t-1) as it was rounded, or the initial state.
#include <algorithm>

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

// One element as Raw has four and eight.
template <typename E> struct RawOne {
    typedef E T;
    static __device__ __forceinline__ T load(const E *p) { return *p; }
    static __device__ __forceinline__ void store(E *p, T r) { *p = r; }
    static __device__ __forceinline__ T zero() { return to_e<E>(0.f); }
    static __device__ __forceinline__ float get(T r, int) { return to_f(r); }
    static __device__ __forceinline__ void set(T &r, int, float x) { r = to_e<E>(x); }
};
template <typename E, int VC> struct Vector : Raw<E, VC> {};
template <typename E> struct Vector<E, 1> : RawOne<E> {};

__device__ __forceinline__ float load_state(const void *s, int64_t at, int b16) {
    return b16 ? (float)((const bf16 *)s)[at] : ((const float *)s)[at];
}
__device__ __forceinline__ void store_state(void *s, int64_t at, int b16, float h) {
    if (b16)
        ((bf16 *)s)[at] = (bf16)h;
    else
        ((float *)s)[at] = h;
}

// ---------------------------------------------------------------------------
// Tiles.  The tokens of all sequences lie on one axis, which is cut into tiles of
// W * S tokens; a workgroup takes one tile of up to 64 * VC channels, every wave S
// of its tokens, every lane VC channels.  All of it is loaded once, into registers;
// what a wave's tokens do to a state is h -> A h + b, and such maps compose.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8, kGroupTiles = 8;

// Channels of a lane.  The vectors of VC channels are shared out evenly among the
// column blocks; the last one of an odd row ends with it and overlaps its neighbour,
// which is in the same wave: both compute and store the same values.
struct Lane {
    int c;
    bool live;
};
template <int VC> __device__ __forceinline__ Lane lane_of(int D, int ncb, int cb, int lane) {
    const int nv = (D + VC - 1) / VC, each = nv / ncb, more = nv % ncb;
    const int v = cb * each + min(cb, more) + lane;
    return {min(v * VC, D - VC), lane < each + (cb < more ? 1 : 0)};
}
template <int VC> __host__ __device__ __forceinline__ int column_blocks(int D) { return ((D + VC - 1) / VC + 63) / 64; }

// Workspace: a counter (16 bytes), then a word a tile and channel, what the tile does
// to a state, then a word a group of tiles and channel, the state before the group.
struct Handed {
    uint32_t *counter;
    unsigned long long *maps, *states;
};
__host__ __device__ __forceinline__ Handed handed_of(void *ws, int64_t tiles, int D) {
    unsigned long long *w = (unsigned long long *)ws;
    return {(uint32_t *)w, w + 2, w + 2 + tiles * D};
}
int64_t handed_words(int64_t tiles, int D) { return 2 + (tiles + (tiles + kGroupTiles - 1) / kGroupTiles) * D; }

// A word carries its own flag, the sign of its upper half (decays are not negative),
// so that it is handed on without a fence: one 64-bit store and loads that repeat
// until the flag is there, past the caches that are not shared.
__device__ __forceinline__ void put(unsigned long long *w, float A, float h) {
    __hip_atomic_store(w, (unsigned long long)(__float_as_uint(A) | 0x80000000u) << 32 | __float_as_uint(h),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <int VC> __device__ __forceinline__ void await(const unsigned long long *w, float *A, float *h) {
    unsigned long long v[VC];
    for (;;) {
        bool all = true;
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            v[e] = __hip_atomic_load(w + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            all = all && (long long)v[e] < 0;
        }
        if (all) break;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        A[e] = __uint_as_float((uint32_t)(v[e] >> 32) & 0x7fffffffu);
        h[e] = __uint_as_float((uint32_t)v[e]);
    }
}

__global__ void __launch_bounds__(256) clear_kernel(uint4 *w, int64_t n) {
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
        __syncthreads();
        return;
    }
    for (int i = tid; i <= TT; i += NT) q.start[i] = -1;
    const int n0 = min(max(count_to(p.cu_seqlens, p.N + 1, t0, lane) - 1, 0), p.N - 1);
    if (tid == 0) {
        q.first = n0;
        q.first_token = cu_at(p.cu_seqlens, n0, p.T_tot);
    }
    __syncthreads();
    for (int n = n0 + tid; n < p.N; n += NT) {
        const int at = cu_at(p.cu_seqlens, n, p.T_tot) - t0;
        if (at > TT) break;
        if (at >= 0) atomicMax(&q.start[at], n);
    }
    __syncthreads();
}

// Rows of sequences without tokens, shared out over the tiles: the final state is the
// initial one.
template <int VC>
__device__ __forceinline__ void empty_sequences(const ScanParams &p, int tile, int tiles, int c, bool live) {
    if (!p.final_state || (p.indices && p.initial) || !live) return;   // a pool's slots keep what they hold
    const int lo = (int)((int64_t)p.N * tile / tiles), hi = (int)((int64_t)p.N * (tile + 1) / tiles);
    for (int n = lo + (threadIdx.x >> 6); n < hi; n += kWaves) {
        int t0, t1;
        seq_range(p.cu_seqlens, n, p.T, p.T_tot, t0, t1);
        if (t0 != t1) continue;
        int64_t at = (int64_t)n * p.D + c;
        if (p.indices) {
            const int slot = p.indices[n];
            if (slot < 0 || slot >= p.pool_size) continue;
            at = (int64_t)slot * p.D + c;
        }
#pragma unroll
        for (int e = 0; e < VC; ++e) store_state(p.final_state, at + e, p.state_bf16, p.initial ? load_state(p.initial, at + e, p.state_bf16) : 0.f);
    }
}

template <typename E, typename G, bool BETA, int VC, int S>
__global__ void __launch_bounds__(kWaves * 64) scan_kernel(ScanParams p, int ncb, int tiles) {
    constexpr int NT = kWaves * 64, TT = kWaves * S;
    __shared__ Sequences<TT> q;
    __shared__ float2 maps[kWaves][VC][64];            // what each wave's tokens do to a state
    __shared__ float2 before[kGroupTiles][VC][64];     // the tiles of the group before this one
    __shared__ float into[VC][64];                     // the state before the group
    __shared__ int cut[kWaves];                        // the last sequence that begins in a wave's tokens, or -1
    __shared__ int ticket;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Handed hand = handed_of(p.ws, tiles, p.D);
    // Tiles are taken in the order of a counter, so that whatever tile a workgroup
    // waits for is with a workgroup that runs already; as each hands its map on
    // before it waits, and the earliest one waits for none, every wait ends.
    if (tiles > 1) {
        if (threadIdx.x == 0) ticket = (int)atomicAdd(hand.counter, 1u);
        __syncthreads();
    }
    const int id = tiles > 1 ? __builtin_amdgcn_readfirstlane(ticket) : blockIdx.x;
    const int tile = id / ncb, cb = id % ncb, t0 = tile * TT;
    const Lane ln = lane_of<VC>(p.D, ncb, cb, lane);
    const int t_end = p.cu_seqlens ? cu_at(p.cu_seqlens, p.N, p.T_tot) : p.T_tot;
    empty_sequences<VC>(p, tile, tiles, ln.c, ln.live);
    if (t0 >= t_end) return;
    const int tw = t0 + w * S, nv = min(max(t_end - tw, 0), S);   // the wave's tokens

    typedef Vector<E, VC> RE;
    typedef Vector<G, VC> RG;
    float a[S][VC], u[S][VC];
    {
        typename RE::T xr[S];
        typename RG::T gr[S], br[S];
        const E *x = (const E *)p.x + (int64_t)tw * p.x_stride;
        const G *g = (const G *)p.g + (int64_t)tw * p.g_stride, *b = (const G *)p.beta + (int64_t)tw * p.beta_stride;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            xr[s] = RE::zero();
            gr[s] = RG::zero();                        // a = 1, u = 0: the state stays
            if (BETA) br[s] = RG::zero();
            if (s < nv && ln.live) {
                xr[s] = RE::load(x + s * p.x_stride + ln.c);
                gr[s] = RG::load(g + s * p.g_stride + ln.c);
                if (BETA) br[s] = RG::load(b + s * p.beta_stride + ln.c);
            }
        }
        find_sequences<TT, NT>(q, p, t0, t_end);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                a[s][e] = decay(RG::get(gr[s], e));
                u[s][e] = RE::get(xr[s], e);
                if (BETA) u[s][e] *= RG::get(br[s], e);
            }
    }
    // sequences that begin at, or end with, the wave's tokens
    const bool is = lane < S && lane < nv;
    const int at = w * S + min(lane, S - 1);
    const uint32_t starts = (uint32_t)__ballot(is && q.start[at] >= 0);
    const uint32_t ends = (uint32_t)__ballot(is && (q.start[at + 1] >= 0 || t0 + at + 1 == t_end));
    // The state that a sequence starts from takes the place of the one that came in:
    // it is read once, before this tile's map is handed on, since its buffer may be
    // the final state's.
    auto initial = [&](int n, float *h) {
        int64_t from = (int64_t)n * p.D + ln.c;
        bool has = p.initial != nullptr && ln.live;
        if (p.indices) {
            const int slot = p.indices[n];
            has = has && slot >= 0 && slot < p.pool_size;
            from = (int64_t)slot * p.D + ln.c;
        }
#pragma unroll
        for (int e = 0; e < VC; ++e) h[e] = has ? load_state(p.initial, from + e, p.state_bf16) : 0.f;
    };
    float A[VC], h[VC];
    int last = -1;                                     // the last sequence that begins here
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        A[e] = 1.f;
        h[e] = 0.f;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (starts >> s & 1) {
            float h0[VC];
            last = __builtin_amdgcn_readfirstlane(q.start[w * S + s]);
            initial(last, h0);
#pragma unroll
            for (int e = 0; e < VC; ++e) h[e] = u[s][e] = fmaf(a[s][e], h0[e], u[s][e]);
        } else {
#pragma unroll
            for (int e = 0; e < VC; ++e) h[e] = fmaf(a[s][e], h[e], u[s][e]);
        }
#pragma unroll
        for (int e = 0; e < VC; ++e) A[e] *= a[s][e];
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) maps[w][e][lane] = float2{A[e], h[e]};
    if (lane == 0) cut[w] = last;
    __syncthreads();
    // the tokens before this wave's in the tile; the last wave hands the tile's map on
    int seq = q.first;                                 // sequence before the wave's first token
    bool own = false;                                  // it began in the tile
    float Ae[VC], he[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        Ae[e] = 1.f;
        he[e] = 0.f;
    }
    for (int k = 0; k < w; ++k) {
        const bool fresh = cut[k] >= 0;
        own = own || fresh;
        seq = max(seq, cut[k]);
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            const float2 m = maps[k][e][lane];
            he[e] = fresh ? m.y : fmaf(m.x, he[e], m.y);
            Ae[e] *= m.x;
        }
    }
    const int base = tile / kGroupTiles * kGroupTiles;
    if (tiles > 1 && w == kWaves - 1 && ln.live) {
#pragma unroll
        for (int e = 0; e < VC; ++e)
            put(hand.maps + (int64_t)tile * p.D + ln.c + e, Ae[e] * A[e], starts ? h[e] : fmaf(A[e], he[e], h[e]));
    }
    // the state that comes into the tile
    const int since = q.first_token / TT;              // tile in which its first sequence begins
    float hin[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) hin[e] = 0.f;
    if (q.first_token < t0) {
        const int from = max(base, since), n = tile - from;
        if (w < n) {
            float m[VC], b[VC];
            if (ln.live) await<VC>(hand.maps + (int64_t)(from + w) * p.D + ln.c, m, b);
#pragma unroll
            for (int e = 0; e < VC; ++e) before[w][e][lane] = float2{m[e], b[e]};
        }
        if (since < base && w == kWaves - 1) {
            float m[VC], b[VC];
            if (ln.live) await<VC>(hand.states + (int64_t)(base / kGroupTiles) * p.D + ln.c, m, b);
#pragma unroll
            for (int e = 0; e < VC; ++e) into[e][lane] = b[e];
        }
        __syncthreads();
        if (since < base)
#pragma unroll
            for (int e = 0; e < VC; ++e) hin[e] = into[e][lane];
        for (int k = 0; k < n; ++k)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const float2 m = before[k][e][lane];
                hin[e] = since == from + k ? m.y : fmaf(m.x, hin[e], m.y);
            }
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) h[e] = own ? he[e] : fmaf(Ae[e], hin[e], he[e]);
    if (tile % kGroupTiles == kGroupTiles - 1 && tile + 1 < tiles && w == kWaves - 1 && ln.live) {
        const float2 *mine = &maps[w][0][lane];
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            const float2 m = mine[e * 64];
            put(hand.states + (int64_t)(tile / kGroupTiles + 1) * p.D + ln.c + e, 0.f, starts ? m.y : fmaf(m.x, h[e], m.y));
        }
    }
    E *y = (E *)p.y + (int64_t)tw * p.D + ln.c;
    seq = __builtin_amdgcn_readfirstlane(seq);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const bool fresh = starts >> s & 1;
        if (fresh) seq = __builtin_amdgcn_readfirstlane(q.start[w * S + s]);
        typename RE::T o = RE::zero();
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            h[e] = fresh ? u[s][e] : fmaf(a[s][e], h[e], u[s][e]);
            RE::set(o, e, h[e]);
        }
        if (s < nv && ln.live) RE::store(y + (int64_t)s * p.D, o);
        if ((ends >> s & 1) && p.final_state && ln.live) {
            int64_t to = (int64_t)seq * p.D + ln.c;
            bool kept = true;
            if (p.indices) {
                const int slot = p.indices[seq];
                kept = slot >= 0 && slot < p.pool_size;
                to = (int64_t)slot * p.D + ln.c;
            }
            if (kept)
#pragma unroll
                for (int e = 0; e < VC; ++e) store_state(p.final_state, to + e, p.state_bf16, h[e]);
        }
    }
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

constexpr int kTokens = 16;                            // of a wave
int tiles_of(int64_t T_tot) { return (int)((T_tot + kWaves * kTokens - 1) / (kWaves * kTokens)); }
// Four channels a lane; rows of fewer have one.
int blocks_of(int D) { return D < 4 ? column_blocks<1>(D) : column_blocks<4>(D); }

enum Pass { kForward, kBackward, kSteps };
template <typename E, typename G, bool BETA, int VC> void launch_tiles(const ScanParams &p, hipStream_t st) {
    const int tiles = std::max(tiles_of(p.T_tot), 1), ncb = column_blocks<VC>(p.D);
    if (tiles > 1) {
        const int64_t n = (handed_words(tiles, p.D) + 1) / 2;
        clear_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0, st>>>((uint4 *)p.ws, n);
    }
    scan_kernel<E, G, BETA, VC, kTokens><<<(unsigned)(tiles * ncb), kWaves * 64, 0, st>>>(p, ncb, tiles);
}
template <typename E, typename G> void launch_e(const ScanParams &p, Pass pass, hipStream_t st) {
    if (pass == kForward) {
        if (p.D < 4)
            p.beta ? launch_tiles<E, G, true, 1>(p, st) : launch_tiles<E, G, false, 1>(p, st);
        else
            p.beta ? launch_tiles<E, G, true, 4>(p, st) : launch_tiles<E, G, false, 4>(p, st);
        return;
    }
    const int cblocks = (p.D + 255) / 256;
    const unsigned grid = (unsigned)((int64_t)p.N * cblocks);
    if (pass == kBackward)
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

size_t scan_workspace_bytes(int64_t T_tot, int D, int, int, bool) {
    const int tiles = tiles_of(T_tot);
    return tiles > 1 ? (size_t)(handed_words(tiles, D) + 1) / 2 * 16 : 0;
}
int64_t scan_grid(int64_t T_tot, int64_t D, int64_t N) {
    return std::max(N * ((D + 255) / 256), (int64_t)tiles_of(T_tot) * blocks_of((int)D));
}

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
