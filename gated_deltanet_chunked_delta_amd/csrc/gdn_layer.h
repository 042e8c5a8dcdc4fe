// Internal interface of the operators around the delta rule in a GDN layer:
// the recurrent steps over several tokens (gdn_steps.hip), the short causal
// convolution (gdn_conv.hip) and the RMS norms (gdn_norm.hip).  Not part of the
// public ABI.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Kernel kinds of the timing hook, after those of gdn_internal.h.
enum LayerKernelKind { kStepsKernel = kNumKernelKinds, kConvKernel, kConvUpdateKernel, kConvBwdKernel, kNormKernel,
                       kNormBwdKernel, kColumnSumKernel, kNumAllKinds };
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

// out[c] = sum over i < n of part[i * cols + c], in a fixed order (gdn_norm.hip).
// With W > 0 the columns are W + 1 planes of D: planes 0 .. W-1 go to
// out[d * W + plane], plane W to out2[d] (if given).
hipError_t launch_column_sum(const float *part, int n, int64_t cols, float *out, int D, int W, float *out2,
                             hipStream_t stream, Profiler *prof);

}  // namespace gdn
