// Internal interface of the operators around the delta rule in a GDN layer:
// the recurrent steps over several tokens (gdn_steps.hip), the short causal
// convolution (gdn_conv.hip), the RMS norms (gdn_norm.hip, gdn_norm_held.hip), the
// gated linear recurrence (gdn_scan.hip) and values held in 8 and 4 bits
// (gdn_quant.hip).  Not part of the public ABI.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Kernel kinds of the timing hook, after those of gdn_internal.h.
enum LayerKernelKind { kStepsKernel = kNumKernelKinds, kConvKernel, kConvUpdateKernel, kConvBwdKernel, kNormKernel,
                       kNormBwdKernel, kColumnSumKernel, kScanClearKernel, kScanKernel, kScanStepsKernel,
                       kScanBwdKernel, kQuantKernel, kDequantKernel, kNumAllKinds };
const char *layer_kernel_name(int kind);

// Slots of a pool that a few-token step reads and writes: sequence n starts
// from slot indices[n, a - 1], a = accepted[n] clamped to [1, cols] (1 without
// accepted); column c < cols - 1 takes the state after token c + 1 and the last
// column the state after the sequence's last token (if it has cols tokens or
// more).  A start slot outside the pool marks a padding row.
struct StepSlots {
    void *data;
    const int32_t *indices;          // [N, cols]
    const int32_t *accepted;         // [N] or null
    int pool_size, cols;
};

struct StepsParams {
    const void *q, *k, *v;           // [T_tot, H, K], [T_tot, H, K], [T_tot, HV, V]
    const float *g, *beta;           // [T_tot, HV]
    Gates gates;                     // used instead of g, beta when gates.A_log != null
    StepSlots slots;                 // states [pool_size, HV, K, V]
    int state_bf16;
    const int32_t *cu_seqlens;       // [N+1] or null
    void *out;                       // [T_tot, HV, V]
    int T, T_tot, H, HV, K, V, N;
    float scale;
    int use_l2norm;
};
hipError_t launch_steps(const StepsParams &p, int dtype, hipStream_t stream, Profiler *prof);

// The short convolution.  The D columns of the output (of its gradient in the
// backward pass) lie in up to three tensors of piece_dim[i] columns each.
struct ConvParams {
    const void *x;                   // [T_tot, D], rows x_stride elements apart
    int64_t x_stride;
    const void *weight, *bias;       // [D, W], [D] or null
    int w_f32;                       // weight and bias are fp32 (else the element type)
    int silu;
    const void *initial;             // [N, D, W-1], or a pool when indices is set; may be null
    void *final_state;               // same layout, may be null, may be `initial`
    const int32_t *indices;          // [N] slots of initial / final_state (prefill over a pool), or null
    int pool_size;
    StepSlots slots;                 // few-token update
    const int32_t *cu_seqlens;       // [N+1] or null
    void *piece[3];
    int piece_dim[3];
    int T, T_tot, D, W, N;
    // backward
    void *dx;                        // [T_tot, D]
    void *dinitial;                  // [N, D, W-1] or null
    float *dweight, *dbias;          // [D, W], [D] or null
    float *part;                     // workspace: conv_bwd_workspace_bytes
};
hipError_t launch_conv(const ConvParams &p, int dtype, hipStream_t stream, Profiler *prof);
hipError_t launch_conv_update(const ConvParams &p, int dtype, hipStream_t stream, Profiler *prof);
size_t conv_bwd_workspace_bytes(int64_t T_tot, int D, int W);
hipError_t launch_conv_bwd(const ConvParams &p, int dtype, hipStream_t stream, Profiler *prof);
// Workgroups of the largest grid these sizes launch (host check against the grid limit).
int64_t conv_grid(int64_t T_tot, int64_t D, int64_t N, int W);

// The RMS norms.  gated: y = x r w silu(z); else h = residual + alpha x,
// y = h r (w + offset), r = (mean of squares + eps)^-1/2.
struct NormParams {
    const void *x, *z, *residual, *weight;
    void *y, *hidden;
    const void *dy, *dhidden;
    void *dx, *dz, *dresidual;
    float *dweight;
    float *part;                     // workspace: norm_bwd_workspace_bytes
    int64_t rows;
    int64_t z_stride;                // elements between the tokens of z
    int heads, D;                    // rows per token
    float eps, alpha, offset;
    int w_f32;
};
constexpr int kNormMaxD = 16384;     // one row in the registers of one workgroup
constexpr int kGatedMaxD = 1024;     // one row in the registers of one wave
hipError_t launch_norm(const NormParams &p, bool gated, int dtype, hipStream_t stream, Profiler *prof);
size_t norm_bwd_workspace_bytes(int64_t rows, int D);
hipError_t launch_norm_bwd(const NormParams &p, bool gated, int dtype, hipStream_t stream, Profiler *prof);

// Values held in 8 bits: codes [rows, D] and bf16 scales [rows, groups of 32].
struct Held {
    void *codes, *scales;
};
constexpr int kGroup = 32;           // elements of one scale

// The gated norm that also writes its inputs in 8 bits (x8, z8), and its gradients
// from those (x and z of p are not read).
hipError_t launch_norm_held(const NormParams &p, const Held &x8, const Held &z8, int dtype, hipStream_t stream,
                            Profiler *prof);
hipError_t launch_norm_held_bwd(const NormParams &p, const Held &x8, const Held &z8, int dtype, hipStream_t stream,
                                Profiler *prof);

// Rows of D values <-> codes and scales.  Row i of n lies at row src[i] (i without
// src) of its tensor and goes to row dst[i] (i); a row with an index outside
// its tensor is skipped.
struct QuantParams {
    void *values;                    // [value_rows, D], rows stride elements apart
    Held held;                       // [held_rows, D (8 bits) or (D + 1) / 2 bytes (4 bits)], [held_rows, groups]
    const int32_t *value_index, *held_index;   // [n] or null
    int64_t n, D, stride;
    int value_rows, held_rows;
};
hipError_t launch_quant(const QuantParams &p, int dtype, int bits, bool back, hipStream_t stream, Profiler *prof);
int64_t quant_grid(const QuantParams &p, int dtype, int bits, bool back);   // as for scan_grid

// The gated linear recurrence h_t = e^g_t h_(t-1) + beta_t x_t per channel.
struct ScanParams {
    const void *x, *g, *beta;        // [T_tot, D], rows x/g/beta_stride elements apart; beta may be null
    int64_t x_stride, g_stride, beta_stride;
    const void *initial;             // [N, D] fp32, or a pool when indices is set; may be null
    void *final_state;               // the same, may be null, may be `initial`
    const int32_t *indices;          // [N] slots of initial / final_state, or null
    int pool_size;
    int state_bf16;                  // type of a pool's slots
    StepSlots slots;                 // few tokens per sequence
    const int32_t *cu_seqlens;       // [N+1] or null
    void *y;                         // [T_tot, D]; in the backward pass the forward's output (read)
    Held x8, y8;                     // backward: x and y in 8 bits instead (y8.codes non-null)
    const void *dy;                  // [T_tot, D]
    const float *dht;                // [N, D] or null
    void *dx, *dg, *dbeta;           // [T_tot, D]; dbeta null without beta
    float *dinitial;                 // [N, D] or null
    void *ws;                        // scan_workspace_bytes
    int T, T_tot, D, N;
};
// gate_f32: g, beta and their gradients are fp32 (else the element type).
size_t scan_workspace_bytes(int64_t T_tot, int D, int gate_f32, bool backward);
// 256-thread workgroups that a pass over these sizes launches, and a few-token call at
// most (host checks against the grid limit).
int64_t scan_grid(int64_t T_tot, int D, int dtype, int gate_f32, bool beta, bool held, bool backward);
int64_t scan_steps_grid(int64_t N, int D);
hipError_t launch_scan(const ScanParams &p, int dtype, int gate_f32, hipStream_t stream, Profiler *prof);
hipError_t launch_scan_bwd(const ScanParams &p, int dtype, int gate_f32, hipStream_t stream, Profiler *prof);
hipError_t launch_scan_steps(const ScanParams &p, int dtype, int gate_f32, hipStream_t stream, Profiler *prof);

// out[c] = sum over i < n of part[i * cols + c], in a fixed order (gdn_norm.hip).
// With W > 0 the columns are W + 1 planes of D: planes 0 .. W-1 go to
// out[d * W + plane], plane W to out2[d] (if given).
hipError_t launch_column_sum(const float *part, int n, int64_t cols, float *out, int D, int W, float *out2,
                             hipStream_t stream, Profiler *prof);

}  // namespace gdn
