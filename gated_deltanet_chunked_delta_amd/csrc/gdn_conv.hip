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
// schedule.  Arithmetic is fp32, each output rounded once.
#include "gdn_layer_device.h"

namespace gdn {
namespace {

using namespace dev;

constexpr int kCols = 512;            // columns of a wave

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

// One lane's columns in the pieces of out (or of its gradient).
template <typename E> struct Piece {
    E *ptr;              // column 0 of the lane in row 0
    int64_t stride;      // of its rows
    bool whole;          // the lane's columns lie in one piece
};
template <typename E> __device__ __forceinline__ Piece<E> piece_of(const ConvParams &p, int d, int n) {
    int at = 0;
    Piece<E> r{nullptr, 0, false};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (n > 0 && d >= at && d + n <= at + p.piece_dim[i])
            r = Piece<E>{(E *)p.piece[i] + (d - at), p.piece_dim[i], true};
        at += p.piece_dim[i];
    }
    return r;
}
// Address of one element of the pieces.
template <typename E> __device__ __forceinline__ E *piece_at(const ConvParams &p, int64_t row, int d) {
    if (d < p.piece_dim[0]) return (E *)p.piece[0] + row * p.piece_dim[0] + d;
    d -= p.piece_dim[0];
    if (d < p.piece_dim[1]) return (E *)p.piece[1] + row * p.piece_dim[1] + d;
    d -= p.piece_dim[1];
    return (E *)p.piece[2] + row * p.piece_dim[2] + d;
}
template <typename E>
__device__ __forceinline__ void put_row(const ConvParams &p, const Piece<E> &pc, int64_t row, int d, int n,
                                        const typename Raw8<E>::T &v) {
    if (pc.whole) {
        store_n<E>(pc.ptr + row * pc.stride, v, n);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) *piece_at<E>(p, row, d + e) = to_e<E>(Raw8<E>::get(v, e));
}
template <typename E>
__device__ __forceinline__ typename Raw8<E>::T get_row(const ConvParams &p, const Piece<E> &pc, int64_t row, int d,
                                                       int n) {
    if (pc.whole) return load_n<E>(pc.ptr + row * pc.stride, n);
    typename Raw8<E>::T v = Raw8<E>::zero();
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) Raw8<E>::set(v, e, to_f(*piece_at<E>(p, row, d + e)));
    return v;
}

// The lane's weights and bias in fp32: w[j][e], b[e].
template <typename E, int W>
__device__ __forceinline__ void load_weights(const ConvParams &p, int d, int n, float (*w)[8], float *b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        b[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = 0.f;
    }
    if (n <= 0) return;
    // the lane's 8 W weights are consecutive
    float flat[W * 8];
#pragma unroll
    for (int j = 0; j < W; ++j)
        load_w8<E>(p.weight, (int64_t)d * W + j * 8, min(max(n * W - j * 8, 0), 8), p.w_f32, flat + j * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
    if (p.bias) load_w8<E>(p.bias, d, n, p.w_f32, b);
}

// A history [D, W-1] at `h`: row j (oldest first) of the lane's columns.
template <typename E, int W>
__device__ __forceinline__ void load_history(const E *h, int d, int n, float (*win)[8]) {
    float flat[(W - 1) * 8];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const typename Raw8<E>::T v = load_n<E>(h + (int64_t)d * (W - 1) + j * 8, min(max(n * (W - 1) - j * 8, 0), 8));
#pragma unroll
        for (int e = 0; e < 8; ++e) flat[j * 8 + e] = Raw8<E>::get(v, e);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) win[j][e] = flat[e * (W - 1) + j];
}
template <typename E, int W>
__device__ __forceinline__ void store_history(E *h, int d, int n, const float (*win)[8]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        typename Raw8<E>::T v;
#pragma unroll
        for (int e = 0; e < 8; ++e) Raw8<E>::set(v, e, win[(j * 8 + e) % (W - 1)][(j * 8 + e) / (W - 1)]);
        store_n<E>(h + (int64_t)d * (W - 1) + j * 8, v, min(max(n * (W - 1) - j * 8, 0), 8));
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

// The W-1 rows before token t of a sequence that begins at t0.
template <typename E, int W>
__device__ __forceinline__ void load_window(const ConvParams &p, const E *x, int t, int t0, const E *hist, int d, int n,
                                            float (*win)[8]) {
    float old[W - 1][8];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) old[j][e] = win[j][e] = 0.f;
    if (hist && t - t0 < W - 1) load_history<E, W>(hist, d, n, old);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int s = t - (W - 1) + j;
        if (s >= t0) {
            const typename Raw8<E>::T v = load_n<E>(x + (int64_t)s * p.x_stride, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) win[j][e] = Raw8<E>::get(v, e);
        } else {
            // position s - t0 in [-(W-1), -1]: history row W-1 + s - t0 (constant indices keep it in registers)
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
                if (i == W - 1 + s - t0)
#pragma unroll
                    for (int e = 0; e < 8; ++e) win[j][e] = old[i][e];
        }
    }
}

template <int W>
__device__ __forceinline__ void shift_in(float (*win)[8], const float *x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
        win[W - 2][e] = x[e];
    }
}

// pre-activation of one element
template <int W>
__device__ __forceinline__ float pre_of(const float (*w)[8], const float *b, const float (*win)[8], float x, int e) {
    float a = b[e];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], win[j][e], a);
    return fmaf(w[W - 1][e], x, a);
}

// Workgroups [0, nmain): four strips of L tokens by 512 columns.  The ones
// behind them write final states, one wave per sequence and 512 columns (also
// of empty sequences); they run in a launch of their own where final_state may
// be the buffer the strips read histories from.
template <typename E, int W>
__global__ void __launch_bounds__(256) conv_kernel(ConvParams p, int L, int nstrips, int cblocks, int nmain) {
    typedef Raw8<E> R;
    typedef typename R::T V;
    constexpr int U = sizeof(E) == 2 ? 8 : 4;         // rows in flight
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blk = (int)blockIdx.x;
    if (blk >= nmain) {   // final states
        const int64_t u = (int64_t)(blk - nmain) * 4 + wv;
        const int s = (int)(u / cblocks), d = (int)(u % cblocks) * kCols + lane * 8, n = min(max(p.D - d, 0), 8);
        if (s >= p.N || n == 0) return;
        E *dst = (E *)start_of<E>(p, s, p.final_state);
        if (!dst) return;
        int t0, t1;
        seq_range(p.cu_seqlens, s, p.T, p.T_tot, t0, t1);
        float win[W - 1][8];
        load_window<E, W>(p, (const E *)p.x + d, t1, t0, start_of<E>(p, s, p.initial), d, n, win);
        store_history<E, W>(dst, d, n, win);
        return;
    }
    const int strip = (blk / cblocks) * 4 + wv, d = (blk % cblocks) * kCols + lane * 8, n = min(max(p.D - d, 0), 8);
    if (strip >= nstrips) return;
    const int s0 = strip * L, s1 = min(s0 + L, p.T_tot);
    int seq = p.cu_seqlens ? find_seq(p.cu_seqlens, p.N, s0, p.T_tot) : s0 / p.T;
    if (n == 0) return;
    const E *__restrict__ x = (const E *)p.x + d;
    const Piece<E> pc = piece_of<E>(p, d, n);
    float w[W][8], b[8], win[W - 1][8];
    load_weights<E, W>(p, d, n, w, b);
    for (int t = s0; t < s1;) {
        int t0, t1;
        seq_range(p.cu_seqlens, seq, p.T, p.T_tot, t0, t1);
        while (t1 <= t && seq + 1 < p.N) seq_range(p.cu_seqlens, ++seq, p.T, p.T_tot, t0, t1);
        if (t1 <= t) t1 = p.T_tot;                    // tokens behind the last sequence's: its own
        const int te = min(t1, s1);
        load_window<E, W>(p, x, t, min(t0, t), start_of<E>(p, seq, p.initial), d, n, win);
        while (t < te) {
            V xa[U];
            const int m = min(te - t, U);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (i < m) xa[i] = load_n<E>(x + (int64_t)(t + i) * p.x_stride, n);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (i < m) {
                    float xv[8];
                    V o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        xv[e] = R::get(xa[i], e);
                        float a = pre_of<W>(w, b, win, xv[e], e);
                        if (p.silu) a *= sigmoid_f(a);
                        R::set(o, e, a);
                    }
                    shift_in<W>(win, xv);
                    put_row<E>(p, pc, t + i, d, n, o);
                }
            t += m;
        }
    }
}

// A few tokens per sequence with the histories in a pool: one wave per sequence
// and 512 columns walks the sequence's tokens in order.  It reads the start
// slot before it stores to any (the slots of a row may be the same).
template <typename E, int W>
__global__ void __launch_bounds__(256) conv_update_kernel(ConvParams p, int cblocks, int64_t units) {
    typedef Raw8<E> R;
    typedef typename R::T V;
    constexpr int U = 4;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t u = (int64_t)blockIdx.x * 4 + wv;
    if (u >= units) return;
    const int s = (int)(u / cblocks), d = (int)(u % cblocks) * kCols + lane * 8, n = min(max(p.D - d, 0), 8);
    if (n == 0) return;
    int t0, t1;
    seq_range(p.cu_seqlens, s, p.T, p.T_tot, t0, t1);
    if (t0 == t1) return;
    const StepSlots &sl = p.slots;
    const int32_t *idx = sl.indices + (int64_t)s * sl.cols;
    const int a = sl.accepted ? min(max(sl.accepted[s], 1), sl.cols) : 1;
    const int slot = idx[a - 1];
    const Piece<E> pc = piece_of<E>(p, d, n);
    if (slot < 0 || slot >= sl.pool_size) {   // padding row
        for (int t = t0; t < t1; ++t) put_row<E>(p, pc, t, d, n, R::zero());
        return;
    }
    const E *__restrict__ x = (const E *)p.x + d;
    E *pool = (E *)sl.data;
    const int64_t hist = (int64_t)p.D * (W - 1);
    float w[W][8], b[8], win[W - 1][8];
    load_history<E, W>(pool + slot * hist, d, n, win);
    load_weights<E, W>(p, d, n, w, b);
    for (int t = t0; t < t1;) {
        V xa[U];
        const int m = min(t1 - t, U);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i < m) xa[i] = load_n<E>(x + (int64_t)(t + i) * p.x_stride, n);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i < m) {
                float xv[8];
                V o;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xv[e] = R::get(xa[i], e);
                    float y = pre_of<W>(w, b, win, xv[e], e);
                    if (p.silu) y *= sigmoid_f(y);
                    R::set(o, e, y);
                }
                shift_in<W>(win, xv);
                put_row<E>(p, pc, t + i, d, n, o);
                const int c = min(t + i - t0, sl.cols - 1);
                if (c < sl.cols - 1 || t + i == t1 - 1) {
                    const int to = idx[c];
                    if (to >= 0 && to < sl.pool_size) store_history<E, W>(pool + to * hist, d, n, win);
                }
            }
        t += m;
    }
}

// Backward.  With dpre = dy silu'(pre), silu'(a) = s (1 + a (1 - s)), s = sigmoid(a):
//   dx[t]     = sum_j weight[j] dpre[t + (W-1) - j]          (inside the sequence)
//   dweight[j] = sum_t dpre[t] x[t - (W-1) + j],  dbias = sum_t dpre[t]
// and the same for the history rows.  A strip walks its tokens and the W-1
// behind them, computing pre again; the sums of dx for the last W-1 tokens are
// kept in registers until complete.  The four strips of a workgroup add their
// dweight and dbias through LDS into one row of the workspace.
template <typename E, int W>
__global__ void __launch_bounds__(256) conv_bwd_kernel(ConvParams p, int L, int nstrips, int cblocks, int nmain) {
    typedef Raw8<E> R;
    typedef typename R::T V;
    constexpr int U = sizeof(E) == 2 ? 4 : 2;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blk = (int)blockIdx.x;
    if (blk >= nmain) {   // gradients of the start histories
        const int64_t u = (int64_t)(blk - nmain) * 4 + wv;
        const int s = (int)(u / cblocks), d = (int)(u % cblocks) * kCols + lane * 8, n = min(max(p.D - d, 0), 8);
        if (s >= p.N || n == 0) return;
        int t0, t1;
        seq_range(p.cu_seqlens, s, p.T, p.T_tot, t0, t1);
        const E *x = (const E *)p.x + d;
        const Piece<E> pc = piece_of<E>(p, d, n);
        float w[W][8], b[8], win[W - 1][8], g[W - 1][8];
        load_weights<E, W>(p, d, n, w, b);
        load_window<E, W>(p, x, t0, t0, start_of<E>(p, s, p.initial), d, n, win);
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) g[i][e] = 0.f;
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            if (t0 + i < t1) {
                const V xa = load_n<E>(x + (int64_t)(t0 + i) * p.x_stride, n), da = get_row<E>(p, pc, t0 + i, d, n);
                float xv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xv[e] = R::get(xa, e);
                    const float a = pre_of<W>(w, b, win, xv[e], e);
                    const float sg = sigmoid_f(a);
                    const float dp = R::get(da, e) * (p.silu ? sg * fmaf(a, 1.f - sg, 1.f) : 1.f);
                    // token i uses history row r with weight r - i
#pragma unroll
                    for (int r = i; r < W - 1; ++r) g[r][e] = fmaf(w[r - i][e], dp, g[r][e]);
                }
                shift_in<W>(win, xv);
            }
        store_history<E, W>((E *)p.dinitial + (int64_t)s * p.D * (W - 1), d, n, g);
        return;
    }
    __shared__ float red[4][(W + 1) * kCols];
    const int group = blk / cblocks, c0 = (blk % cblocks) * kCols;
    const int strip = group * 4 + wv, d = c0 + lane * 8, n = min(max(p.D - d, 0), 8);
    float dw[W + 1][8];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.f;
    if (strip < nstrips) {
        const int s0 = strip * L, s1 = min(s0 + L, p.T_tot);
        int seq = p.cu_seqlens ? find_seq(p.cu_seqlens, p.N, s0, p.T_tot) : s0 / p.T;
        const E *__restrict__ x = (const E *)p.x + d;
        E *__restrict__ dx = (E *)p.dx + d;
        const Piece<E> pc = piece_of<E>(p, d, n);
        float w[W][8], b[8], win[W - 1][8], acc[W - 1][8];
        load_weights<E, W>(p, d, n, w, b);
        for (int t = s0; t < s1 && n > 0;) {
            int t0, t1;
            seq_range(p.cu_seqlens, seq, p.T, p.T_tot, t0, t1);
            while (t1 <= t && seq + 1 < p.N) seq_range(p.cu_seqlens, ++seq, p.T, p.T_tot, t0, t1);
            if (t1 <= t) t1 = p.T_tot;
            const int ta = t, tb = min(t1, s1), te = min(t1, tb + W - 1);
            load_window<E, W>(p, x, t, min(t0, t), start_of<E>(p, seq, p.initial), d, n, win);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[j][e] = 0.f;
            auto put = [&](int row, const float *v) {
                V o;
#pragma unroll
                for (int e = 0; e < 8; ++e) R::set(o, e, v[e]);
                store_n<E>(dx + (int64_t)row * p.D, o, n);
            };
            while (t < te) {
                V xa[U], da[U];
                const int m = min(te - t, U);
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (i < m) {
                        xa[i] = load_n<E>(x + (int64_t)(t + i) * p.x_stride, n);
                        da[i] = get_row<E>(p, pc, t + i, d, n);
                    }
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (i < m) {
                        const bool own = t + i < tb;
                        float xv[8], dp[8], done[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            xv[e] = R::get(xa[i], e);
                            const float a = pre_of<W>(w, b, win, xv[e], e);
                            const float sg = sigmoid_f(a);
                            dp[e] = R::get(da[i], e) * (p.silu ? sg * fmaf(a, 1.f - sg, 1.f) : 1.f);
                            if (own) {
#pragma unroll
                                for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(dp[e], win[j][e], dw[j][e]);
                                dw[W - 1][e] = fmaf(dp[e], xv[e], dw[W - 1][e]);
                                dw[W][e] += dp[e];
                            }
                            // weight j reaches token t - (W-1) + j
                            done[e] = fmaf(w[0][e], dp[e], acc[0][e]);
#pragma unroll
                            for (int j = 0; j + 1 < W - 1; ++j) acc[j][e] = fmaf(w[j + 1][e], dp[e], acc[j + 1][e]);
                            acc[W - 2][e] = w[W - 1][e] * dp[e];
                        }
                        shift_in<W>(win, xv);
                        if (t + i - (W - 1) >= ta) put(t + i - (W - 1), done);
                    }
                t += m;
            }
            if (te == t1) {   // the sequence ends: its last tokens' sums are complete
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const int row = t1 - (W - 1) + j;
                    if (row >= ta && row < tb) put(row, acc[j]);
                }
            }
            t = tb;
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) red[wv][j * kCols + lane * 8 + e] = dw[j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * kCols; i += 256) {
        const int j = i / kCols, c = c0 + i % kCols;
        if (c < p.D)
            p.part[((int64_t)group * (W + 1) + j) * p.D + c] = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
    }
}

int64_t col_blocks(int64_t D) { return (D + kCols - 1) / kCols; }
// Tokens of a strip: long enough that the W-1 rows read twice are few, short
// enough for about 8192 waves.
int strip_len(int64_t T_tot, int64_t D, int lo, int hi) {
    int L = hi;
    while (L > lo && ((T_tot + L - 1) / L) * col_blocks(D) < 8192) L >>= 1;
    return L;
}

template <typename E, int W>
void launch_fwd_cfg(const ConvParams &p, hipStream_t st, Profiler *prof) {
    const int L = strip_len(p.T_tot, p.D, 4, 32), cb = (int)col_blocks(p.D);
    const int nstrips = (p.T_tot + L - 1) / L, nmain = (nstrips + 3) / 4 * cb;
    const int nfin = p.final_state ? (int)(((int64_t)p.N * cb + 3) / 4) : 0;
    // final states written over the start histories wait for every strip
    const bool apart = nfin > 0 && p.initial == p.final_state && nmain > 0;
    if (prof) prof->begin(kConvKernel, st);
    conv_kernel<E, W><<<nmain + (apart ? 0 : nfin), 256, 0, st>>>(p, L, nstrips, cb, nmain);
    if (apart) conv_kernel<E, W><<<nfin, 256, 0, st>>>(p, L, nstrips, cb, 0);
    if (prof) prof->end(kConvKernel, st);
}

template <typename E, int W>
void launch_update_cfg(const ConvParams &p, hipStream_t st) {
    const int cb = (int)col_blocks(p.D);
    const int64_t units = (int64_t)p.N * cb;
    conv_update_kernel<E, W><<<(unsigned)((units + 3) / 4), 256, 0, st>>>(p, cb, units);
}

template <typename E, int W>
void launch_bwd_cfg(const ConvParams &p, int L, hipStream_t st) {
    const int cb = (int)col_blocks(p.D);
    const int nstrips = (p.T_tot + L - 1) / L, nmain = (nstrips + 3) / 4 * cb;
    const int nfin = p.dinitial ? (int)(((int64_t)p.N * cb + 3) / 4) : 0;
    conv_bwd_kernel<E, W><<<nmain + nfin, 256, 0, st>>>(p, L, nstrips, cb, nmain);
}

template <typename F> void for_width(int W, F f) {
    if (W == 2) f(std::integral_constant<int, 2>{});
    if (W == 3) f(std::integral_constant<int, 3>{});
    if (W == 4) f(std::integral_constant<int, 4>{});
}

int bwd_strip(int64_t T_tot, int64_t D) { return strip_len(T_tot, D, 8, 64); }
int bwd_groups(int64_t T_tot, int64_t D) {
    const int64_t L = bwd_strip(T_tot, D), strips = (T_tot + L - 1) / L;
    return (int)((strips + 3) / 4);
}

}  // namespace

int64_t conv_grid(int64_t T_tot, int64_t D, int64_t N) {
    const int64_t L = strip_len(T_tot, D, 4, 32);
    return ((T_tot + L - 1) / L + 3) / 4 * col_blocks(D) + (N * col_blocks(D) + 3) / 4;
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
    return (size_t)bwd_groups(T_tot, D) * (W + 1) * D * 4;
}

hipError_t launch_conv_bwd(const ConvParams &p, int dtype, hipStream_t stream, Profiler *prof) {
    const int L = bwd_strip(p.T_tot, p.D);
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
    return launch_column_sum(p.part, bwd_groups(p.T_tot, p.D), (int64_t)(p.W + 1) * p.D, p.dweight, p.D, p.W, p.dbias,
                             stream, prof);
}

}  // namespace gdn
