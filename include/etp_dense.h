/* etp_dense.h - C ABI of the dense row operators: linear layers with a fused
 * epilogue and layer norm, forward and backward. They are what a model runs
 * between the edge tensor products of etp.h: channel mixing of each rank, the
 * scalar-track layers on edges, deeper radial networks, norms of node scalars.
 * ("High-performance training and inference for deep equivariant interatomic
 * potentials", section "제안 방법", and "Scaling the leading accuracy of deep
 * equivariant models to biomolecular simulations of realistic size", section
 * "提出的方法": a scalar track of learned layers beside the tensor track. The pages
 * print no formula; the ones below are this library's reading.)
 *
 * Rows. M = groups * per_group rows of channels; row g * per_group + t of an
 * operand starts at data + g * group_stride + t * row_stride (strides in elements;
 * channels are contiguous). So the same call reads plain rows ([M][C]: groups = M,
 * per_group = 1, group_stride = C) and one rank's block of node features x
 * [N][D][C] in place (data = x + l*l*C, groups = N, per_group = 2l + 1,
 * group_stride = D*C, row_stride = C). An input's strides may be zero (a row used
 * many times); an output's rows must not overlap one another. Any alignment of the
 * element type is accepted; rows whose addresses are multiples of 16 bytes (base
 * and strides) are moved in 16-byte units.
 *
 * Types. All operands of a call have one type, ETP_F32 or ETP_BF16; mean and rstd
 * of the layer norm are float32. Sums, statistics and activations are computed in
 * float32 and rounded once when stored. The backward's dz of ETP_BF16 operands with an
 * activation enters the products of grad_x and grad_W as two bfloat16 parts, within 2^-17
 * of it (grad_bias sums it whole); an infinite dz gives NaN there. Products of ETP_F32 operands run on the
 * tensor cores with each operand split into three bfloat16 parts that add up to it
 * exactly (from 2^-110 up in magnitude; below, to within 2^-133); of the nine products
 * of parts the six largest are formed (what is left out is below 2^-22 of a product, of
 * either sign). An infinite ETP_F32 operand of a linear layer therefore
 * gives NaN (not an infinity) in the outputs that it enters.
 *
 * Ownership and execution, errors: as in etp.h. The caller owns every buffer;
 * calls are asynchronous on the given stream, allocate nothing, and overwrite their
 * outputs. Sums over rows are taken in a fixed order: results repeat bit for bit.
 * Outputs must not overlap any other operand, except where a call says so.
 * M = 0 is accepted (weight gradients are then zero). M must stay below 2^31 - 128.
 * First derivatives only: a VJP of the backward calls is not provided. */
#ifndef ETP_DENSE_H_
#define ETP_DENSE_H_

#include "etp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    void* data;           /* device pointer to row 0 (inputs are not written) */
    int64_t group_stride; /* elements between groups; not read when groups = 1 */
    int64_t row_stride;   /* elements between the rows of a group; not read when per_group = 1 */
} etp_rows;

typedef enum { ETP_ACT_NONE = 0, ETP_ACT_SILU = 1 } etp_activation;

/* Largest K and N of a linear layer, and largest C of a layer norm. */
#define ETP_LINEAR_MAX_CHANNELS 65536
#define ETP_NORM_MAX_CHANNELS 8192

/* Bytes of device workspace that etp_linear_forward (backward = 0) or
 * etp_linear_backward (backward = 1, whichever gradients are wanted) needs for these
 * sizes: W rearranged for the tensor cores, partial sums of the weight gradients over
 * ranges of rows. 0 is possible. Host only; it reads the current device's
 * multiprocessor count. */
ETP_API etp_status etp_linear_workspace_size(etp_dtype dtype, int groups, int per_group, int K, int N, int backward,
                                             size_t* bytes);

/* Linear layer: z = x W + bias, out = act(z) + residual.
 * x: rows of K; W [K][N] row-major, contiguous; bias [N] or NULL; residual: rows of
 * N or NULL; z: rows of N, receives the pre-activation (rounded to the type; out is
 * computed from the unrounded value), or NULL; out: rows of N. act: ETP_ACT_NONE or
 * ETP_ACT_SILU (z / (1 + exp(-z))). residual may be out itself (same data and
 * strides): a residual stream updated in place. workspace: etp_linear_workspace_size
 * bytes, 16-byte aligned, owned by the caller (may be NULL when that is 0), free to
 * reuse once the stream has passed the call.
 * Errors: ETP_ERR_INVALID_ARG for a negative size, K or N < 1 or above
 * ETP_LINEAR_MAX_CHANNELS, a NULL x, W or out, a stride that is negative or above 2^31 - 1, overlapping output
 * rows or a pointer misaligned for the type; ETP_ERR_UNSUPPORTED for an unknown
 * dtype or activation; ETP_ERR_TOO_LARGE when M is too large; ETP_ERR_WORKSPACE for a
 * workspace that is too small. */
ETP_API etp_status etp_linear_forward(etp_dtype dtype, int groups, int per_group, int K, int N, const etp_rows* x,
                                      const void* W, const void* bias, etp_activation act, const etp_rows* residual,
                                      const etp_rows* z, const etp_rows* out, void* workspace,
                                      size_t workspace_bytes, etp_stream_t stream);

/* VJP of etp_linear_forward for the cotangent grad_out = dLoss/d(out), rows of N:
 *   dz = grad_out act'(z);  grad_x = dz W^T;  grad_W = x^T dz;  grad_bias = sum of dz over the rows
 * (the residual's gradient is grad_out itself). z: the forward's z, needed for
 * ETP_ACT_SILU, not read for ETP_ACT_NONE (NULL). grad_x (rows of K), grad_W [K][N],
 * grad_bias [N]: each may be NULL (skipped); x may be NULL when grad_W is, W when
 * grad_x is. workspace and errors: as the forward's. */
ETP_API etp_status etp_linear_backward(etp_dtype dtype, int groups, int per_group, int K, int N, const etp_rows* x,
                                       const void* W, etp_activation act, const etp_rows* z,
                                       const etp_rows* grad_out, const etp_rows* grad_x, void* grad_W,
                                       void* grad_bias, void* workspace, size_t workspace_bytes,
                                       etp_stream_t stream);

/* Layer norm over the C channels of each row:
 *   mean = sum(x) / C;  rstd = 1 / sqrt(sum((x - mean)^2) / C + eps);  out = (x - mean) rstd weight + bias
 * weight [C], bias [C]: each may be NULL (ones, zeros). mean, rstd: float32 [M] in
 * row order, each may be NULL. out may be x itself (same data and strides).
 * 1 <= C <= ETP_NORM_MAX_CHANNELS (ETP_ERR_UNSUPPORTED above), eps >= 0 and finite. */
ETP_API etp_status etp_layer_norm_forward(etp_dtype dtype, int groups, int per_group, int C, float eps,
                                          const etp_rows* x, const void* weight, const void* bias,
                                          const etp_rows* out, float* mean, float* rstd, etp_stream_t stream);

/* Bytes of device workspace etp_layer_norm_backward needs (partial sums of the
 * weight and bias gradients). Host only; reads the current device's multiprocessor
 * count. */
ETP_API etp_status etp_layer_norm_workspace_size(etp_dtype dtype, int groups, int per_group, int C, size_t* bytes);

/* VJP of etp_layer_norm_forward for the cotangent grad_out, with the forward's mean
 * and rstd (float32 [M], required):
 *   xh = (x - mean) rstd;  gw = grad_out weight
 *   grad_x = rstd (gw - sum(gw) / C - xh sum(gw xh) / C)
 *   grad_weight = sum over the rows of grad_out xh;  grad_bias = sum over the rows of grad_out
 * xh is formed from the mean as it is given, in float32: in a row whose offset is large beside
 * its spread it is off by half a step of the mean, 2^-24 |mean| rstd, and the gradients with
 * it (offset 1e4, spread 1: 3e-4 of grad_weight). The forward has no such error.
 * weight NULL: ones. Each gradient may be NULL (skipped). grad_x may be grad_out or x
 * itself (same data and strides). workspace: etp_layer_norm_workspace_size bytes,
 * 16-byte aligned (may be NULL when neither grad_weight nor grad_bias is wanted). */
ETP_API etp_status etp_layer_norm_backward(etp_dtype dtype, int groups, int per_group, int C, const etp_rows* x,
                                           const void* weight, const float* mean, const float* rstd,
                                           const etp_rows* grad_out, const etp_rows* grad_x, void* grad_weight,
                                           void* grad_bias, void* workspace, size_t workspace_bytes,
                                           etp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ETP_DENSE_H_ */
