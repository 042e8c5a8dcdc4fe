// Short causal depthwise convolution (width W = 2, 3 or 4) with SiLU for gfx950:
// the operator that mixes each column of the q, k, v projection over the last W
// tokens before the delta rule.  Per sequence, column d and token t
//
//   pre[t, d] = bias[d] + sum_j weight[d, j] x[t - (W-1) + j, d],   y = silu(pre)
//
// with the sequence's history (its W-1 inputs before the first token, oldest
// first, or zeros) before its start; the history after its last token is its
// final state.  The output's columns go to up to three tensors (q, k, v), so that
// the delta rule's kernels read them without a rearranging copy.
//
// Bound by HBM: x is read and y written once.  A lane owns eight columns (16
// bytes in bf16) and walks a strip of tokens with the last W-1 rows in
// registers, so a strip reads W-1 rows more than it writes; a wave covers 512
// columns, the four waves of a workgroup neighbouring strips (a strip's extra
// rows are then in the CU's cache).  Strips ignore the sequences' borders: a
// strip finds its first sequence by a 64-way search over cu_seqlens and
// restarts its window where a sequence begins, so packed batches need no
// schedule.  Arithmetic is fp32, each output rounded once.  64 packed prompts (73,844
// tokens) of 8192 bf16 columns take 435 us, 5.6 TB/s; the gradients of 16,384 tokens
// 175 us, 4.6 TB/s; 256 decode rows 11 us, 3 TB/s (slot, then history).
#include "gdn_layer_device.h"

namespace gdn {
namespace {

using namespace dev;

// The largest n < N with cu[n] <= t (0 if none): every lane probes one entry a
// level.
__device__ __forceinline__ int find_seq(const int32_t *cu, int N, int t, int T_tot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, len = N;
    while (len > 1) {
        const int step = (len + 63) >> 6, i = lane * step;
        const bool le = i < len && (i == 0 || cu_at(cu, lo + i, T_tot) <= t);
        const int k = (int)__popcll(__ballot(le)) - 1;   // cu is non-decreasing: the lanes below
        const int from = max(k, 0) * step;
        lo += from;
        len = min(step, len - from);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// One lane's C columns of one piece of out (or of its gradient).  The last ones of
// a piece whose size is no multiple of C begin inside the neighbour's, so that
// accesses are whole vectors: both lanes compute and store the same values there.
// Where a history is updated in place (INPLACE) that needs the neighbour in the
// same wave, whose loads come before its stores.  Otherwise, and in a piece of
// fewer than C columns, the lane has fewer columns (tails).  A lane behind the last
// column reads what the last one reads and stores nothing, so that a wave without
// tails loads without a condition (32,768 tokens of 4091 columns with the last ones
// by fours, twos and one instead: 267 against 118 us, their gradients 569 against
// 214).
template <typename E, int C, bool INPLACE> struct Lane {
    int d, m, n;         // first column, columns to read, to store
    bool tails;
    E *ptr;              // column d in row 0 of the piece
    int64_t stride;      // between the piece's rows
    typedef typename Raw<E, C>::T V;
    __device__ __forceinline__ Lane(const ConvParams &p, int vec) {
        int v0 = 0, c0 = 0, total = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) total += (p.piece_dim[i] + C - 1) / C;
        const int v = min(vec, total - 1);
        d = m = 0;
        ptr = nullptr;
        stride = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int dim = p.piece_dim[i], nv = (dim + C - 1) / C, c = (v - v0) * C;
            if (v >= v0 && v < v0 + nv) {
                const bool over = dim - c < C && dim >= C && !(INPLACE && (v & 63) == 0);
                const int first = over ? dim - C : c;
                d = c0 + first;
                m = min(dim - first, C);
                ptr = (E *)p.piece[i] + first;
                stride = dim;
            }
            v0 += nv;
            c0 += dim;
        }
        n = vec < total ? m : 0;
        tails = __any(m < C);
    }
    template <bool S = false> __device__ __forceinline__ V read(const E *p) const {
        return tails ? load_n<E, C, S>(p, m, true) : Raw<E, C>::template load<S>(p);
    }
    template <bool S = false> __device__ __forceinline__ void write(E *p, const V &v) const {
        store_n<E, C, S>(p, v, n, tails);
    }
    // row t of the piece; the lane's columns of a row that begins at a uniform address
    __device__ __forceinline__ E *row(int64_t t) const { return ptr + t * stride; }
    __device__ __forceinline__ E *in(const void *r) const { return (E *)((char *)r + (unsigned)(d * (int)sizeof(E))); }
};

// The lane's weights and bias in fp32: w[j][e], b[e].
template <int W, typename E, int C, bool I>
__device__ __forceinline__ void load_weights(const ConvParams &p, const Lane<E, C, I> &ln, float (*w)[C], float *b) {
    // the lane's C W weights are consecutive
    float flat[W * C];
#pragma unroll
    for (int j = 0; j < W; ++j)
        load_w<E, C>(p.weight, (int64_t)ln.d * W + j * C, min(max(ln.m * W - j * C, 0), C), ln.tails, p.w_f32, flat + j * C);
#pragma unroll
    for (int e = 0; e < C; ++e) {
        b[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
    }
    if (p.bias) load_w<E, C>(p.bias, ln.d, ln.m, ln.tails, p.w_f32, b);
}

// A history [D, W-1] at `h`: row j (oldest first) of the lane's columns.
template <int W, typename E, int C, bool I>
__device__ __forceinline__ void load_history(const E *h, const Lane<E, C, I> &ln, float (*win)[C]) {
    float flat[(W - 1) * C];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const auto v = load_n<E, C>(h + (int64_t)ln.d * (W - 1) + j * C, min(max(ln.m * (W - 1) - j * C, 0), C), ln.tails);
#pragma unroll
        for (int e = 0; e < C; ++e) flat[j * C + e] = Raw<E, C>::get(v, e);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < C; ++e) win[j][e] = flat[e * (W - 1) + j];
}
template <int W, typename E, int C, bool I>
__device__ __forceinline__ void store_history(E *h, const Lane<E, C, I> &ln, const float (*win)[C]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        typename Raw<E, C>::T v;
#pragma unroll
        for (int e = 0; e < C; ++e) Raw<E, C>::set(v, e, win[(j * C + e) % (W - 1)][(j * C + e) / (W - 1)]);
        store_n<E, C>(h + (int64_t)ln.d * (W - 1) + j * C, v, min(max(ln.n * (W - 1) - j * C, 0), C), ln.tails);
    }
}

// Start history of sequence n, or null (zeros): the slot of a pool, a row of
// initial, or none.
template <typename E> __device__ __forceinline__ const E *start_of(const ConvParams &p, int n, const void *base) {
    if (!base) return nullptr;
    int64_t s = n;
    if (p.indices) {
        s = p.indices[n];
        if (s < 0 || s >= p.pool_size) return nullptr;
    }
    return (const E *)base + s * p.D * (p.W - 1);
}

// The W-1 rows before token t (as loaded; rows before the first token are not
// meant), and the window they give for a sequence that begins at t0.
template <int W, typename E, int C, bool I>
__device__ __forceinline__ void load_before(const ConvParams &p, const E *x, int t, const Lane<E, C, I> &ln,
                                            typename Raw<E, C>::T *v) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) v[j] = ln.read(ln.in(x + (int64_t)max(t - (W - 1) + j, 0) * p.x_stride));
}
template <int W, typename E, int C, bool I>
__device__ __forceinline__ void window_of(const ConvParams &p, const typename Raw<E, C>::T *v, int t, int t0,
                                          const E *hist, const Lane<E, C, I> &ln, float (*win)[C]) {
    if (t - t0 >= W - 1) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < C; ++e) win[j][e] = Raw<E, C>::get(v[j], e);
        return;
    }
    float old[W - 1][C];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < C; ++e) old[j][e] = 0.f;
    if (hist) load_history<W>(hist, ln, old);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        // position t - t0 - (W-1) + j: a row, or history row t - t0 + j (constant indices keep it in registers)
        const bool in = t - t0 + j >= W - 1;
#pragma unroll
        for (int e = 0; e < C; ++e) win[j][e] = in ? Raw<E, C>::get(v[j], e) : 0.f;
#pragma unroll
        for (int i = j; i < W - 1; ++i)
            if (!in && i == t - t0 + j)
#pragma unroll
                for (int e = 0; e < C; ++e) win[j][e] = old[i][e];
    }
}

// v[i] for a uniform i < U, by selects of values: registers take constant
// indices only.
template <int U, typename V> __device__ __forceinline__ V pick(const V *v, int i) {
    typedef unsigned words __attribute__((ext_vector_type(sizeof(V) / 4)));
    words r = __builtin_bit_cast(words, v[0]);
#pragma unroll
    for (int k = 1; k < U; ++k) {
        const words o = __builtin_bit_cast(words, v[k]);
        r = i == k ? o : r;
    }
    return __builtin_bit_cast(V, r);
}

// Tokens of all sequences: rows behind them are neither read nor written.
__device__ __forceinline__ int tokens_of(const ConvParams &p) {
    return p.cu_seqlens ? cu_at(p.cu_seqlens, p.N, p.T_tot) : p.T_tot;
}

// The sequences as a strip walks them.
struct Walk {
    int seq, t0, t1;     // t0 <= the current token < t1
    // Goes on to the sequence of token r (the strip's first: to the one found for it).
    __device__ __forceinline__ void to(const ConvParams &p, int r, bool first) {
        if (!first && seq + 1 < p.N) ++seq;
        seq_range(p.cu_seqlens, seq, p.T, p.T_tot, t0, t1);
        while (t1 <= r && seq + 1 < p.N) seq_range(p.cu_seqlens, ++seq, p.T, p.T_tot, t0, t1);
        if (t1 <= r) t1 = p.T_tot;                    // tokens behind the last sequence's: its own
        t0 = first ? min(t0, r) : r;
    }
};

template <int W, int C>
__device__ __forceinline__ void shift_in(float (*win)[C], const float *x) {
#pragma unroll
    for (int e = 0; e < C; ++e) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
        win[W - 2][e] = x[e];
    }
}

// pre-activation of one element
template <int W, int C>
__device__ __forceinline__ float pre_of(const float (*w)[C], const float *b, const float (*win)[C], float x, int e) {
    float a = b[e];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], win[j][e], a);
    return fmaf(w[W - 1][e], x, a);
}

// Rows of a load batch: a multiple of W - 1, so that the window's registers are
// back in place after a batch.
constexpr int batch_rows(int W) { return W == 4 ? 3 : 4; }

// Workgroups [0, nmain): four strips of L tokens by 64 lanes' columns.  The ones
// behind them write final states, one wave per sequence and 64 lanes' columns
// (also of empty sequences); they run in a launch of their own where final_state
// is the buffer the strips read histories from.
template <typename E, int W, bool STREAM>
__global__ void __launch_bounds__(256) conv_kernel(ConvParams p, int L, int nstrips, int cblocks, int nmain) {
    constexpr int C = 8, U = batch_rows(W);           // the next batch's loads are in flight
    typedef Raw<E, C> R;
    typedef typename R::T V;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blk = (int)blockIdx.x;
    if (blk >= nmain) {   // final states
        const int64_t u = (int64_t)(blk - nmain) * 4 + wv;
        const int s = (int)(u / cblocks);
        const Lane<E, C, true> ln(p, (int)(u % cblocks) * 64 + lane);
        if (s >= p.N || ln.n == 0) return;
        E *dst = (E *)start_of<E>(p, s, p.final_state);
        if (!dst) return;
        int t0, t1;
        seq_range(p.cu_seqlens, s, p.T, p.T_tot, t0, t1);
        float win[W - 1][C];
        V before[W - 1];
        if (t1 > t0) load_before<W>(p, (const E *)p.x, t1, ln, before);
        window_of<W>(p, before, t1, t0, start_of<E>(p, s, p.initial), ln, win);
        store_history<W>(dst, ln, win);
        return;
    }
    const int strip = (blk / cblocks) * 4 + wv;
    const Lane<E, C, false> ln(p, (blk % cblocks) * 64 + lane);
    const int n = ln.n;
    if (strip >= nstrips) return;
    const int s0 = strip * L, s1 = min(s0 + L, tokens_of(p));
    if (s0 >= s1) return;
    const E *__restrict__ x = (const E *)p.x;
    V xa[U], before[W - 1];
    // rows of one batch, up to the strip's end whatever sequence they belong to
    auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (t + i < s1) xa[i] = ln.read(ln.in(x + (int64_t)(t + i) * p.x_stride));
    };
    load_before<W>(p, x, s0, ln, before);
    load(s0);
    float w[W][C], b[C], win[W - 1][C];
    load_weights<W>(p, ln, w, b);
    Walk at{p.cu_seqlens ? find_seq(p.cu_seqlens, p.N, s0, p.T_tot) : s0 / p.T, 0, 0};
    if (n == 0) return;
    auto begin = [&](int r, bool first) {
        at.to(p, r, first);
        window_of<W>(p, before, r, at.t0, start_of<E>(p, at.seq, p.initial), ln, win);
    };
    auto step = [&](int r, const V &v) {
        float xv[C];
        V o;
#pragma unroll
        for (int e = 0; e < C; ++e) {
            xv[e] = R::get(v, e);
            float a = pre_of<W, C>(w, b, win, xv[e], e);
            if (p.silu) a *= sigmoid_f(a);
            R::set(o, e, a);
        }
        shift_in<W, C>(win, xv);
        ln.template write<STREAM>(ln.row(r), o);
    };
    begin(s0, true);
    for (int t = s0; t < s1; t += U) {
        V xc[U];
#pragma unroll
        for (int i = 0; i < U; ++i) xc[i] = xa[i];
        load(t + U);
        if (t + U <= at.t1 && t + U <= s1) {
#pragma unroll
            for (int i = 0; i < U; ++i) step(t + i, xc[i]);
        } else {   // a sequence or the strip ends in the batch
#pragma unroll 1
            for (int r = t; r < min(t + U, s1); ++r) {
                if (r >= at.t1) begin(r, false);
                step(r, pick<U>(xc, r - t));
            }
        }
    }
}

// A few tokens per sequence with the histories in a pool: one wave per sequence
// and 64 lanes' columns walks the sequence's tokens in order.  It reads the start
// slot before it stores to any (the slots of a row may be the same).  Latency
// counts here, so a lane has four columns: twice the waves of eight at half the
// registers (156 sequences of six tokens, 640 columns: 5.7 against 6.6 us).
constexpr int kFewCols = 4;
template <typename E, int W>
__global__ void __launch_bounds__(256) conv_update_kernel(ConvParams p, int cblocks, int64_t units) {
    constexpr int C = kFewCols, U = 4;
    typedef Raw<E, C> R;
    typedef typename R::T V;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t u = (int64_t)blockIdx.x * 4 + wv;
    if (u >= units) return;
    const int s = (int)(u / cblocks);
    const StepSlots &sl = p.slots;
    const int32_t *idx = sl.indices + (int64_t)s * sl.cols;
    // the first 64 slots of the row in the lanes, looked up while the rows load
    const int slots = idx[min(lane, sl.cols - 1)];
    const int a = sl.accepted ? min(max(sl.accepted[s], 1), sl.cols) : 1;
    const Lane<E, C, true> ln(p, (int)(u % cblocks) * 64 + lane);
    const int n = ln.n;
    int t0, t1;
    seq_range(p.cu_seqlens, s, p.T, p.T_tot, t0, t1);
    if (t0 == t1) return;
    auto slot_of = [&](int col) { return col < 64 ? __builtin_amdgcn_readlane(slots, col) : idx[col]; };
    const E *__restrict__ x = (const E *)p.x;
    V xa[U];
    auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (t + i < t1) xa[i] = ln.read(ln.in(x + (int64_t)(t + i) * p.x_stride));
    };
    load(t0);
    float w[W][C], b[C], win[W - 1][C];
    load_weights<W>(p, ln, w, b);
    const int slot = slot_of(__builtin_amdgcn_readfirstlane(a) - 1);
    if (slot < 0 || slot >= sl.pool_size) {   // padding row
        for (int t = t0; t < t1; ++t) ln.write(ln.row(t), R::zero());
        return;
    }
    E *pool = (E *)sl.data;
    const int64_t hist = (int64_t)p.D * (W - 1);
    load_history<W>(pool + slot * hist, ln, win);
    for (int t = t0; t < t1; t += U) {
        if (t > t0) load(t);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (t + i >= t1) break;
            float xv[C];
            V o;
#pragma unroll
            for (int e = 0; e < C; ++e) {
                xv[e] = R::get(xa[i], e);
                float y = pre_of<W, C>(w, b, win, xv[e], e);
                if (p.silu) y *= sigmoid_f(y);
                R::set(o, e, y);
            }
            shift_in<W, C>(win, xv);
            ln.write(ln.row(t + i), o);
            const int c = min(t + i - t0, sl.cols - 1);
            if (c < sl.cols - 1 || t + i == t1 - 1) {
                const int to = slot_of(c);
                if (to >= 0 && to < sl.pool_size) store_history<W>(pool + to * hist, ln, win);
            }
        }
    }
}

// Backward.  With dpre = dy silu'(pre), silu'(a) = s (1 + a (1 - s)), s = sigmoid(a):
//   dx[t]     = sum_j weight[j] dpre[t + (W-1) - j]          (inside the sequence)
//   dweight[j] = sum_t dpre[t] x[t - (W-1) + j],  dbias = sum_t dpre[t]
// and the same for the history rows.  A strip walks its tokens and the W-1
// behind them, computing pre again; the sums of dx for the last W-1 tokens are
// kept in registers until complete.  The four strips of a workgroup add their
// dweight and dbias through LDS into one row of the workspace.  A lane has four
// columns: windows, weights and sums are 4 W + 1 floats a column, and with eight
// columns one or two waves are left a SIMD to hide the loads behind (16,384
// tokens of 8192 columns 246 us, with four 191 and with the strips and streaming
// below 175; three waves a SIMD instead of two another 8 % where the tokens do not
// fill the card evenly).
constexpr int kBwdCols = 4;

template <typename E, int W, bool STREAM>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3)))
conv_bwd_kernel(ConvParams p, int L, int nstrips, int cblocks, int nmain) {
    constexpr int C = kBwdCols, U = batch_rows(W);
    typedef Raw<E, C> R;
    typedef typename R::T V;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blk = (int)blockIdx.x;
    if (blk >= nmain) {   // gradients of the start histories
        const int64_t u = (int64_t)(blk - nmain) * 4 + wv;
        const int s = (int)(u / cblocks);
        const Lane<E, C, false> ln(p, (int)(u % cblocks) * 64 + lane);
        const int n = ln.n;
        if (s >= p.N || n == 0) return;
        int t0, t1;
        seq_range(p.cu_seqlens, s, p.T, p.T_tot, t0, t1);
        const E *x = (const E *)p.x;
        float w[W][C], b[C], win[W - 1][C], g[W - 1][C];
        load_weights<W>(p, ln, w, b);
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int e = 0; e < C; ++e) g[i][e] = win[i][e] = 0.f;
        if (const E *h = start_of<E>(p, s, p.initial)) load_history<W>(h, ln, win);
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            if (t0 + i < t1) {
                const V xa = ln.read(ln.in(x + (int64_t)(t0 + i) * p.x_stride)), da = ln.read(ln.row(t0 + i));
                float xv[C];
#pragma unroll
                for (int e = 0; e < C; ++e) {
                    xv[e] = R::get(xa, e);
                    const float a = pre_of<W, C>(w, b, win, xv[e], e);
                    const float sg = sigmoid_f(a);
                    const float dp = R::get(da, e) * (p.silu ? sg * fmaf(a, 1.f - sg, 1.f) : 1.f);
                    // token i uses history row r with weight r - i
#pragma unroll
                    for (int r = i; r < W - 1; ++r) g[r][e] = fmaf(w[r - i][e], dp, g[r][e]);
                }
                shift_in<W, C>(win, xv);
            }
        store_history<W>((E *)p.dinitial + (int64_t)s * p.D * (W - 1), ln, g);
        return;
    }
    __shared__ float red[4][W + 1][64 * C];
    const int group = blk / cblocks, strip = group * 4 + wv;
    const Lane<E, C, false> ln(p, (blk % cblocks) * 64 + lane);
    const int n = ln.n;
    float dw[W + 1][C];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < C; ++e) dw[j][e] = 0.f;
    const int end = tokens_of(p);
    if (strip < nstrips && strip * L < end) {
        const int s0 = strip * L, s1 = min(s0 + L, end), se = min(s1 + W - 1, end);
        const E *__restrict__ x = (const E *)p.x;
        E *__restrict__ dx = (E *)p.dx;
        V xa[U], da[U], before[W - 1];
        auto load = [&](int t) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (t + i < se) {
                    xa[i] = ln.template read<STREAM>(ln.in(x + (int64_t)(t + i) * p.x_stride));
                    da[i] = ln.template read<STREAM>(ln.row(t + i));
                }
        };
        load_before<W>(p, x, s0, ln, before);
        load(s0);
        float w[W][C], b[C], win[W - 1][C], acc[W - 1][C];
        load_weights<W>(p, ln, w, b);
        Walk at{p.cu_seqlens ? find_seq(p.cu_seqlens, p.N, s0, p.T_tot) : s0 / p.T, 0, 0};
        int ta = s0;                                   // the sequence's first token in the strip
        auto put = [&](int row, const float *v) {
            V o;
#pragma unroll
            for (int e = 0; e < C; ++e) R::set(o, e, v[e]);
            ln.template write<STREAM>(ln.in(dx + (int64_t)row * p.D), o);
        };
        auto begin = [&](int r, bool first) {
            at.to(p, r, first);
            ta = r;
            window_of<W>(p, before, r, at.t0, start_of<E>(p, at.seq, p.initial), ln, win);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < C; ++e) acc[j][e] = 0.f;
        };
        // own: 0 for a row behind the strip, which counts for another one's dweight
        auto step = [&](int r, const V &xr, const V &dr, float own) {
            float xv[C], whole[C];
#pragma unroll
            for (int e = 0; e < C; ++e) {
                xv[e] = R::get(xr, e);
                const float a = pre_of<W, C>(w, b, win, xv[e], e);
                const float sg = sigmoid_f(a);
                const float dp = R::get(dr, e) * (p.silu ? sg * fmaf(a, 1.f - sg, 1.f) : 1.f), dpo = dp * own;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(dpo, win[j][e], dw[j][e]);
                dw[W - 1][e] = fmaf(dpo, xv[e], dw[W - 1][e]);
                dw[W][e] += dpo;
                // weight j reaches token r - (W-1) + j
                whole[e] = fmaf(w[0][e], dp, acc[0][e]);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) acc[j][e] = fmaf(w[j + 1][e], dp, acc[j + 1][e]);
                acc[W - 2][e] = w[W - 1][e] * dp;
            }
            shift_in<W, C>(win, xv);
            if (r - (W - 1) >= ta) put(r - (W - 1), whole);
        };
        if (n > 0) {
            begin(s0, true);
            for (int t = s0; t < se; t += U) {
                V xc[U], dc[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    xc[i] = xa[i];
                    dc[i] = da[i];
                }
                load(t + U);
                if (t + U < at.t1 && t + U <= s1) {
#pragma unroll
                    for (int i = 0; i < U; ++i) step(t + i, xc[i], dc[i], 1.f);
                    continue;
                }
                // a sequence or the strip ends in the batch
                int r = t;
#pragma unroll 1
                for (; r < min(t + U, se); ++r) {
                    if (r >= at.t1) {
                        if (r >= s1) break;            // nothing of the strip's sequences is left
                        begin(r, false);
                    }
                    step(r, pick<U>(xc, r - t), pick<U>(dc, r - t), r < s1 ? 1.f : 0.f);
                    if (r + 1 == at.t1) {              // the sequence ends: its last tokens' sums are whole
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) {
                            const int row = at.t1 - (W - 1) + j;
                            if (row >= ta && row < s1) put(row, acc[j]);
                        }
                    }
                }
                if (r >= at.t1 && r >= s1) break;
            }
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < C; ++e) red[wv][j][lane * C + e] = dw[j][e];
    __syncthreads();
    for (int j = wv; j <= W; j += 4)
#pragma unroll
        for (int e = 0; e < C; ++e)
            if (e < n) {
                const int c = lane * C + e;
                p.part[((int64_t)group * (W + 1) + j) * p.D + ln.d + e] =
                    (red[0][j][c] + red[1][j][c]) + (red[2][j][c] + red[3][j][c]);
            }
}

int64_t col_blocks(int64_t D, int C) { return (D + 64 * C - 1) / (64 * C); }
// Blocks of 64 lanes over the pieces' vectors (each piece starts a vector).
int lane_blocks(const ConvParams &p, int C) {
    int64_t v = 0;
    for (int i = 0; i < 3; ++i) v += ((int64_t)p.piece_dim[i] + C - 1) / C;
    return (int)((v + 63) / 64);
}
constexpr int kStripWaves = 2048;
// Tokens of a strip: whole load batches; 12 or 16 forward and 48 or 64 backward
// (W = 4: 46,303 packed tokens of 4544 columns forward 159 us, with
// 24 163, with 6 172; the gradients of 16,384 tokens of 8192 columns 173, with 96
// 180, with 24 182: longer ones leave a CU's rows far apart, shorter ones read
// more rows twice and leave more partial sums), fewer where that leaves less than
// 2048 waves (the gradients of 1024 tokens of 4096 columns 18 us, with 4096 waves 24;
// of 2,956 of 1152 fp32 19.5 against 24; of 32,768 of 816 53 against 58).
int strip_len(int64_t T_tot, int64_t D, int C, int lo, int hi) {
    int L = hi;
    while (L > lo && ((T_tot + L - 1) / L) * col_blocks(D, C) < kStripWaves) L >>= 1;
    return L;
}
int fwd_strip(int64_t T_tot, int64_t D, int W) { return strip_len(T_tot, D, 8, batch_rows(W), 4 * batch_rows(W)); }
int bwd_strip(int64_t T_tot, int64_t D, int W) {
    return strip_len(T_tot, D, kBwdCols, batch_rows(W), 16 * batch_rows(W));
}
int bwd_groups(int64_t T_tot, int64_t D, int W) {
    const int64_t L = bwd_strip(T_tot, D, W), strips = (T_tot + L - 1) / L;
    return (int)((strips + 3) / 4);
}

// Passes over more than the 256 MiB of the last cache are streamed past it (the
// forward pass its outputs only: the strips share rows of x): 73,844 packed
// tokens of 8192 columns 437 against 459 us, the gradients of 16,384 tokens 175
// against 182.
bool streams(const ConvParams &p, size_t elem, int tensors) {
    return (size_t)p.T_tot * p.D * elem * tensors > (256u << 20);
}
// The backward pass streams its loads too, which pays only if no two waves share a
// line of a row: rows of whole 64 bytes (16,384 tokens of 8192 columns above; 32,768
// of 4091 236 us streamed, 214 not).
bool whole_lines(const ConvParams &p, size_t elem) {
    const size_t m = 64 / elem;
    bool whole = p.D % m == 0 && p.x_stride % m == 0;
    for (int i = 0; i < 3; ++i) whole = whole && p.piece_dim[i] % m == 0;
    return whole;
}

template <typename E, int W>
void launch_fwd_cfg(const ConvParams &p, hipStream_t st, Profiler *prof) {
    const int L = fwd_strip(p.T_tot, p.D, W), cb = lane_blocks(p, 8);
    const int nstrips = (p.T_tot + L - 1) / L, nmain = (nstrips + 3) / 4 * cb;
    const int nfin = p.final_state ? (int)(((int64_t)p.N * cb + 3) / 4) : 0;
    // final states written over the start histories wait for every strip
    const bool apart = nfin > 0 && p.initial == p.final_state && nmain > 0;
    if (prof) prof->begin(kConvKernel, st);
    if (streams(p, sizeof(E), 2))
        conv_kernel<E, W, true><<<nmain + (apart ? 0 : nfin), 256, 0, st>>>(p, L, nstrips, cb, nmain);
    else
        conv_kernel<E, W, false><<<nmain + (apart ? 0 : nfin), 256, 0, st>>>(p, L, nstrips, cb, nmain);
    if (apart) conv_kernel<E, W, false><<<nfin, 256, 0, st>>>(p, L, nstrips, cb, 0);
    if (prof) prof->end(kConvKernel, st);
}

template <typename E, int W>
void launch_update_cfg(const ConvParams &p, hipStream_t st) {
    const int cb = lane_blocks(p, kFewCols);
    const int64_t units = (int64_t)p.N * cb;
    conv_update_kernel<E, W><<<(unsigned)((units + 3) / 4), 256, 0, st>>>(p, cb, units);
}

template <typename E, int W>
void launch_bwd_cfg(const ConvParams &p, int L, hipStream_t st) {
    const int cb = lane_blocks(p, kBwdCols);
    const int nstrips = (p.T_tot + L - 1) / L, nmain = (nstrips + 3) / 4 * cb;
    const int nfin = p.dinitial ? (int)(((int64_t)p.N * cb + 3) / 4) : 0;
    if (streams(p, sizeof(E), 3) && whole_lines(p, sizeof(E)))
        conv_bwd_kernel<E, W, true><<<nmain + nfin, 256, 0, st>>>(p, L, nstrips, cb, nmain);
    else
        conv_bwd_kernel<E, W, false><<<nmain + nfin, 256, 0, st>>>(p, L, nstrips, cb, nmain);
}

template <typename F> void for_width(int W, F f) {
    if (W == 2) f(std::integral_constant<int, 2>{});
    if (W == 3) f(std::integral_constant<int, 3>{});
    if (W == 4) f(std::integral_constant<int, 4>{});
}

}  // namespace

int64_t conv_grid(int64_t T_tot, int64_t D, int64_t N, int W) {
    const int64_t L = fwd_strip(T_tot, D, W), cb = col_blocks(D + 16, 8);   // three pieces: at most two vectors more
    return ((T_tot + L - 1) / L + 3) / 4 * cb + (N * cb * 2 + 3) / 4;   // lanes of four columns by sequence
}

hipError_t launch_conv(const ConvParams &p, int dtype, hipStream_t stream, Profiler *prof) {
    if (p.T_tot == 0 && (p.N == 0 || !p.final_state)) return hipSuccess;
    for_width(p.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        dtype == 0 ? launch_fwd_cfg<bf16, W>(p, stream, prof) : launch_fwd_cfg<float, W>(p, stream, prof);
    });
    return hipGetLastError();
}

hipError_t launch_conv_update(const ConvParams &p, int dtype, hipStream_t stream, Profiler *prof) {
    if (p.N == 0 || p.T_tot == 0) return hipSuccess;
    if (prof) prof->begin(kConvUpdateKernel, stream);
    for_width(p.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        dtype == 0 ? launch_update_cfg<bf16, W>(p, stream) : launch_update_cfg<float, W>(p, stream);
    });
    const hipError_t err = hipGetLastError();
    if (prof) prof->end(kConvUpdateKernel, stream);
    return err;
}

size_t conv_bwd_workspace_bytes(int64_t T_tot, int D, int W) {
    return (size_t)bwd_groups(T_tot, D, W) * (W + 1) * D * 4;
}

hipError_t launch_conv_bwd(const ConvParams &p, int dtype, hipStream_t stream, Profiler *prof) {
    const int L = bwd_strip(p.T_tot, p.D, p.W);
    if (p.T_tot > 0 || (p.N > 0 && p.dinitial)) {
        if (prof) prof->begin(kConvBwdKernel, stream);
        for_width(p.W, [&](auto w) {
            constexpr int W = decltype(w)::value;
            dtype == 0 ? launch_bwd_cfg<bf16, W>(p, L, stream) : launch_bwd_cfg<float, W>(p, L, stream);
        });
        const hipError_t err = hipGetLastError();
        if (prof) prof->end(kConvBwdKernel, stream);
        if (err != hipSuccess) return err;
    }
    return launch_column_sum(p.part, bwd_groups(p.T_tot, p.D, p.W), (int64_t)(p.W + 1) * p.D, p.dweight, p.D, p.W, p.dbias,
                             stream, prof);
}

}  // namespace gdn
