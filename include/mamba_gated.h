/*
 * mamba_gated.h: C ABI of a gated recurrent block's operators beside the
 * selective scan, for AMD Instinct MI355X (gfx950): the gated linear recurrence
 * (whole sequences, gradients, single tokens), the norm behind a block fused
 * with its gate, and the norm before a block fused with the residual sum.
 *
 * As in mamba_scan.h and mamba_layers.h, whose status and dtype codes these
 * calls use: tensors are row-major, and dense but for the inputs that carry a
 * row stride; all pointers are device pointers on the current HIP device,
 * 16-byte aligned, owned by the caller and not kept; no call allocates device
 * memory; work is queued on `stream`; scratch comes from the caller's
 * workspace, which needs no initialisation and may be used again, or by another
 * stream, once the call's work has finished; every check runs on the host
 * before any HIP call but the query of the device's compute-unit count, and a
 * refused call queues nothing. Outputs must not overlap inputs, or each other,
 * unless said otherwise.
 */
#ifndef MAMBA_GATED_H
#define MAMBA_GATED_H

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens between the states that gated_scan_fwd hands to gated_scan_bwd. */
#define MAMBA_GATED_SCAN_BLOCK 64
/* Most channels, and widest row stride, of the gated recurrence. */
#define MAMBA_GATED_SCAN_MAX_DIM (1 << 20)

/*
 * Gated linear recurrence. Per batch row b and channel d:
 *
 *     p_t = sigmoid(decay_gate_t)          a_t = exp(log_decay[d] p_t)
 *     w_t = sqrt(1 - a_t^2) sigmoid(input_gate_t)
 *     h_t = a_t h_{t-1} + w_t x_t          h_{-1} = h0 (or zeros)
 *     y_t = h_t
 *
 * x, decay_gate   (batch, seqlen, dim) I/O dtype   a token's channels are contiguous,
 * input_gate      the same, optional (NULL: 1)     tokens x_stride (decay_stride,
 *                                                  input_stride) >= dim elements
 *                                                  apart, rows seqlen tokens
 * log_decay    (dim) fp32                <= 0 and finite (not checked)
 * lengths      (batch) int32             optional: tokens of each row, taken as 0
 *                                        below 0 and seqlen above it (NULL: seqlen)
 * h0           (batch, dim) fp32         optional (NULL: zeros)
 * y            (batch, seqlen, dim)      written; zeros behind a row's length
 * hL           (batch, dim) fp32         optional: the state after each row's last
 *                                        token (h0 for an empty row); may alias h0
 * block_states (batch, ceil(seqlen / MAMBA_GATED_SCAN_BLOCK), dim) fp32
 *                                        optional: the state entering each block of
 *                                        tokens, which gated_scan_bwd takes; blocks
 *                                        that start behind a row's length are left
 *                                        as they were
 *
 * dim and the strides are at most MAMBA_GATED_SCAN_MAX_DIM, batch * seqlen at
 * most 2^28 and batch * ceil(dim / 64) below 2^23 (else
 * MAMBA_ERR_UNSUPPORTED). batch == 0 or dim == 0 is a no-op; seqlen == 0 writes hL =
 * h0 (or zeros) and reads nothing else, whose pointers may be NULL. What stands
 * behind a row's length is never read. A NaN or infinite value stays in its channel
 * and reaches no earlier output; where the definition has an infinity, NaN may come
 * out. Sums and states are fp32, and the decay over many tokens is carried by its
 * logarithm, so that slow channels keep fp32's accuracy over long sequences. Decays
 * and sigmoids below 2^-126, the least normal fp32 number, may count as zero, here and
 * in the gradients.
 */
int gated_scan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                                  size_t* bytes);

int gated_scan_fwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x,
                   int64_t x_stride, const void* decay_gate, int64_t decay_stride,
                   const float* log_decay, const void* input_gate, int64_t input_stride,
                   const int32_t* lengths, const float* h0, void* y, float* hL,
                   float* block_states, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

/*
 * Gradients of sum(dy * y) + sum(dhL * hL) for the gated_scan_fwd call with the
 * same inputs.
 *
 * block_states    as gated_scan_fwd wrote them (h0 is their first block)
 * dy              (batch, seqlen, dim)  I/O dtype, dense
 * dhL             (batch, dim) fp32     optional (NULL: zeros)
 * dx, ddecay_gate (batch, seqlen, dim)  I/O dtype, dense; written; zeros behind a
 *                                       row's length
 * dinput_gate     the same; required with input_gate, else not written
 * dlog_decay      (dim) fp32            optional, summed over rows and tokens; without
 *                                       it sequences of fewer than 512 tokens need no
 *                                       workspace
 * dh0             (batch, dim) fp32     optional; may alias dhL
 * Sums are taken in a fixed order: results are reproducible bit for bit on one
 * kind of device. batch == 0 or seqlen == 0 writes zero dlog_decay and dh0 = dhL,
 * and reads nothing else. Where nothing enters the state (a_t = 1) the derivative of
 * w_t by log_decay counts as zero.
 */
int gated_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                                  size_t* bytes);

int gated_scan_bwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x,
                   int64_t x_stride, const void* decay_gate, int64_t decay_stride,
                   const float* log_decay, const void* input_gate, int64_t input_stride,
                   const int32_t* lengths, const float* block_states, const void* dy,
                   const float* dhL, void* dx, void* ddecay_gate, void* dinput_gate,
                   float* dlog_decay, float* dh0, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

/*
 * One token of the recurrence: equivalent to gated_scan_fwd with seqlen 1 and
 * h0 = hL = h.
 *
 * h                         (batch, dim) fp32  read and updated in place
 * x, decay_gate, input_gate (batch, dim)       rows x_stride, decay_stride,
 *                                              input_stride elements apart
 * y                         (batch, dim)       written
 * batch * ceil(dim / 64) is below 2^23 (else MAMBA_ERR_UNSUPPORTED).
 */
int gated_scan_update(int64_t batch, int64_t dim, int dtype, float* h, const void* x,
                      int64_t x_stride, const void* decay_gate, int64_t decay_stride,
                      const float* log_decay, const void* input_gate, int64_t input_stride,
                      void* y, hipStream_t stream);

/* Widest part (dim / groups) of the norms. */
#define MAMBA_GATED_NORM_MAX_DIM 16384

typedef enum mamba_norm_gate {
    MAMBA_GATE_NONE = 0,     /* z is not looked at */
    MAMBA_GATE_FIRST = 1,    /* the norm of the gated values */
    MAMBA_GATE_BEHIND = 2    /* the gate on the normed values */
} mamba_norm_gate;

/*
 * The norm behind a block, fused with the block's gate: over each of the
 * `groups` equal parts of a row, with silu(z) = z / (1 + exp(-z)),
 *
 *     MAMBA_GATE_FIRST    v = x silu(z)    y = v rstd weight
 *     MAMBA_GATE_BEHIND   v = x            y = v rstd weight silu(z)
 *     MAMBA_GATE_NONE     v = x            y = v rstd weight
 *     rstd = 1 / sqrt(mean(v^2) + eps)
 *
 * the mean taken over a part's dim / groups values. Sums are fp32 (where squares of v
 * add up past its range rstd is 0); sigmoids of z below 2^-126, the least normal fp32
 * number, may count as zero, here and in the gradients.
 *
 * x, z     (rows, dim) I/O dtype       a row's channels are contiguous, rows
 *                                      x_stride (z_stride) >= dim elements apart
 * weight   (dim) fp32                  optional (NULL: ones)
 * eps      >= 0 and finite
 * y        (rows, dim) I/O dtype       dense; may be x, or z, where that is dense
 * rstd     (rows, groups) fp32         optional: what the backward pass reads
 * dim is a multiple of groups (else MAMBA_ERR_INVALID_ARG) and dim / groups at
 * most MAMBA_GATED_NORM_MAX_DIM, dim and the strides at most 2^27, groups 2^22
 * and rows * groups 2^30 (else MAMBA_ERR_UNSUPPORTED). rows == 0 or dim == 0 is
 * a no-op.
 */
int gated_norm_fwd(int64_t rows, int64_t dim, int64_t groups, int dtype, int gate, const void* x,
                   int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                   float eps, void* y, float* rstd, hipStream_t stream);

/*
 * Gradients of sum(dy * y) for the gated_norm_fwd call with the same x, z and
 * weight.
 *
 * rstd      (rows, groups) fp32        as gated_norm_fwd wrote it
 * dy        (rows, dim) I/O dtype      dense
 * dx        (rows, dim) I/O dtype      dense; written; may be dy
 * dz        (rows, dim) I/O dtype      dense; written where there is a gate
 * dweight   (dim) fp32                 optional: summed over rows
 * The sums over rows are taken in a fixed order (reproducible bit for bit on one
 * kind of device). rows == 0 writes a zero dweight.
 */
int gated_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups, int dtype,
                                  size_t* bytes);

int gated_norm_bwd(int64_t rows, int64_t dim, int64_t groups, int dtype, int gate, const void* x,
                   int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                   const float* rstd, const void* dy, void* dx, void* dz, float* dweight,
                   void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The norm before a block, fused with the sum of the residual stream and the
 * scaled output of the block before:
 *
 *     total = residual + scale x
 *     y = total rstd weight,   rstd = 1 / sqrt(mean(total^2) + eps)
 *
 * x, y             (rows, dim) I/O dtype    y may be x
 * residual, total  (rows, dim)              of total_dtype: the I/O dtype or fp32;
 *                                           total may be residual. The norm is taken
 *                                           of the sum before its rounding to that type
 * scale, weight    (dim) fp32               optional (NULL: ones)
 * eps              >= 0 and finite
 * rstd             (rows) fp32              optional: what the backward pass reads
 * dim is at most MAMBA_GATED_NORM_MAX_DIM, rows 2^30 (else
 * MAMBA_ERR_UNSUPPORTED). rows == 0 or dim == 0 is a no-op.
 */
int residual_norm_fwd(int64_t rows, int64_t dim, int dtype, int total_dtype, const void* x,
                      const void* residual, const float* scale, const float* weight, float eps,
                      void* y, void* total, float* rstd, hipStream_t stream);

/*
 * Gradients of sum(dy * y) + sum(dtotal * total) for the residual_norm_fwd call
 * that wrote total and rstd.
 *
 * x          (rows, dim) I/O dtype     needed for dscale only
 * dy         (rows, dim) I/O dtype
 * dtotal     (rows, dim) total_dtype   optional (NULL: zeros)
 * dresidual  (rows, dim) total_dtype   written; may be dtotal
 * dx         (rows, dim) I/O dtype     optional: scale times the same gradient;
 *                                      may be dy
 * dscale     (dim) fp32                optional, with scale only: summed over rows
 * dweight    (dim) fp32                optional: summed over rows
 * The sums over rows are taken in a fixed order (reproducible bit for bit on one
 * kind of device). rows == 0 writes zero dscale and dweight.
 */
int residual_norm_bwd_workspace_size(int64_t rows, int64_t dim, int dtype, int total_dtype,
                                     size_t* bytes);

int residual_norm_bwd(int64_t rows, int64_t dim, int dtype, int total_dtype, const void* total,
                      const float* weight, const float* rstd, const void* x, const float* scale,
                      const void* dy, const void* dtotal, void* dx, void* dresidual,
                      float* dscale, float* dweight, void* workspace, size_t workspace_bytes,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_GATED_H */
