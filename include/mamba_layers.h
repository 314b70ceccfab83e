/*
 * mamba_layers.h: C ABI of the layer operators beside the selective scan, for
 * AMD Instinct MI355X (gfx950): linear attention with a decay for each head
 * (whole sequences, gradients, single tokens) and layer norm (forward and
 * gradients).
 *
 * As in mamba_scan.h, whose status and dtype codes these calls use: tensors
 * are dense and row-major; all pointers are device pointers on the current
 * HIP device, 16-byte aligned, owned by the caller and not kept; no call
 * allocates device memory; work is queued on `stream`; scratch comes from
 * the caller's workspace, which needs no initialisation and may be used
 * again, or by another stream, once the call's work has finished; every
 * check runs on the host before any HIP call but the automatic plans' query
 * of the device's compute-unit count, and a refused call queues nothing.
 * Outputs must not overlap inputs, or each other, unless said otherwise.
 */
#ifndef MAMBA_LAYERS_H
#define MAMBA_LAYERS_H

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest head (dk, dv) of linear attention, and their unit. */
#define MAMBA_LINATTN_MAX_DIM 256
#define MAMBA_LINATTN_DIM_UNIT 8
/* Most heads of a call. */
#define MAMBA_LINATTN_MAX_HEADS 4096

/*
 * Linear attention with a decay for each head. Per batch row b and head h,
 * with lam = exp(log_decay[h]) and a state S of dk x dv values:
 *
 *     S_t = lam S_{t-1} + k_t^T v_t          S_{-1} = h0 (or zeros)
 *     o_t = scale q_t S_t
 *
 * that is, o_t = scale sum_{j <= t} lam^(t-j) (q_t . k_j) v_j without h0.
 *
 * q           (batch, seqlen, heads, dk)     I/O dtype
 * k           (batch, seqlen, kv_heads, dk)  heads is a multiple of kv_heads;
 * v           (batch, seqlen, kv_heads, dv)  head h reads k and v of head
 *                                            h / (heads / kv_heads)
 * log_decay   (heads) fp32                   <= 0, -inf allowed (not checked)
 * lengths     (batch) int32                  optional: tokens of each row, taken
 *                                            as 0 below 0 and seqlen above it
 *                                            (NULL: seqlen)
 * h0          (batch, heads, dk, dv) fp32    optional (NULL: zeros)
 * o           (batch, seqlen, heads, dv)     written; zeros behind a row's length
 * hL          (batch, heads, dk, dv) fp32    optional: the state after each row's
 *                                            last token (h0 for an empty row);
 *                                            may alias h0
 * segment_len tokens per parallel segment, 0: automatic, else a multiple of
 *             64. A cut sequence takes a pass over k and v that gives each
 *             segment's share of the state, a join, and the pass that writes
 *             the outputs; the result is the same up to rounding. A forced
 *             segment_len below seqlen takes at most 65536 segments and 65535
 *             rows times heads (else MAMBA_ERR_UNSUPPORTED).
 *
 * dk and dv are multiples of MAMBA_LINATTN_DIM_UNIT up to
 * MAMBA_LINATTN_MAX_DIM, heads at most MAMBA_LINATTN_MAX_HEADS, and a launch,
 * of 256 threads (512 for heads wider than 128) per row, head, segment and 64
 * columns, three times that for gradients, counts fewer than 2^32 (else
 * MAMBA_ERR_UNSUPPORTED). What stands behind a row's length is never read.
 * Inside it a NaN or infinite value may, since the chunk products multiply the
 * causal mask's zeros by it, reach the earlier outputs of its own chunk of 64
 * tokens, in its own row and head, and gradients the later tokens' as well; and
 * where the definition has an infinity, from infinite values or a state that
 * overflows, NaN may come out. A row without tokens keeps an infinite h0 or dhL,
 * and linear_attn_update an infinite h. Sums and states are fp32; with bf16 I/O the
 * products' operands are bf16; what reaches a state or a decay gradient that
 * the caller gets is carried as three bf16 terms, with fp32's accuracy. Powers of
 * the decay below 2^-126, the least normal fp32 number, may count as zero.
 */
int linear_attn_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                                   int64_t dk, int64_t dv, int dtype, int64_t segment_len,
                                   size_t* bytes);

int linear_attn_fwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads, int64_t dk,
                    int64_t dv, int dtype, const void* q, const void* k, const void* v,
                    const float* log_decay, const int32_t* lengths, const float* h0, float scale,
                    void* o, float* hL, int64_t segment_len, void* workspace,
                    size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of sum(d_o * o) + sum(dhL * hL) for the linear_attn_fwd call with
 * the same inputs.
 *
 * d_o          (batch, seqlen, heads, dv)      I/O dtype
 * dhL          (batch, heads, dk, dv) fp32     optional (NULL: zeros)
 * dq, d_k, d_v as q, k, v, I/O dtype           written; zeros behind a row's
 *                                              length; d_k and d_v are summed
 *                                              over the heads that share them
 * dlog_decay   (heads) fp32                    optional, summed over rows
 * dh0          (batch, heads, dk, dv) fp32     optional
 * Sums are taken in a fixed order: results are reproducible bit for bit for a
 * given segment_len. batch == 0 or seqlen == 0 writes zero dlog_decay and
 * dh0 = dhL.
 */
int linear_attn_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                                   int64_t dk, int64_t dv, int dtype, int64_t segment_len,
                                   size_t* bytes);

int linear_attn_bwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads, int64_t dk,
                    int64_t dv, int dtype, const void* q, const void* k, const void* v,
                    const float* log_decay, const int32_t* lengths, const float* h0, float scale,
                    const void* d_o, const float* dhL, void* dq, void* d_k, void* d_v,
                    float* dlog_decay, float* dh0, int64_t segment_len, void* workspace,
                    size_t workspace_bytes, hipStream_t stream);

/*
 * One token of linear attention: equivalent to linear_attn_fwd with seqlen 1
 * and h0 = hL = h.
 *
 * h   (batch, heads, dk, dv) fp32   read and updated in place
 * q   (batch, heads, dk), k (batch, kv_heads, dk), v (batch, kv_heads, dv)
 * o   (batch, heads, dv)            written
 * batch * heads * ceil(dv / 64) * 256 is below 2^32 (else
 * MAMBA_ERR_UNSUPPORTED).
 */
int linear_attn_update(int64_t batch, int64_t heads, int64_t kv_heads, int64_t dk, int64_t dv,
                       int dtype, float* h, const void* q, const void* k, const void* v,
                       const float* log_decay, float scale, void* o, hipStream_t stream);

/* Widest part (dim / groups) of layer norm. */
#define MAMBA_NORM_MAX_DIM 16384

/*
 * Layer norm over each of the `groups` equal parts of a row:
 *
 *     y = (x - mean) rstd weight + bias,   rstd = 1 / sqrt(var + eps)
 *
 * mean and var (the mean square of the centred values) are taken over a
 * part's dim / groups values. groups = 1 is the norm of whole rows; groups =
 * heads that of each head's output.
 *
 * x, y         (rows, dim) I/O dtype      y may be x
 * weight, bias (dim) fp32                 optional (NULL: ones, zeros)
 * eps          >= 0 and finite
 * mean, rstd   (rows, groups) fp32        optional: what the backward pass reads
 * dim is a multiple of groups (else MAMBA_ERR_INVALID_ARG) and dim / groups at
 * most MAMBA_NORM_MAX_DIM, dim at most 2^27, groups 2^22 and rows * groups 2^30
 * (else MAMBA_ERR_UNSUPPORTED). rows == 0 or dim == 0 is a no-op.
 */
int layer_norm_fwd(int64_t rows, int64_t dim, int64_t groups, int dtype, const void* x,
                   const float* weight, const float* bias, float eps, void* y, float* mean,
                   float* rstd, hipStream_t stream);

/*
 * Gradients of sum(dy * y) for the layer_norm_fwd call with the same x and
 * weight.
 *
 * mean, rstd   (rows, groups) fp32        as layer_norm_fwd wrote them
 * dy           (rows, dim) I/O dtype
 * dx           (rows, dim) I/O dtype      written; may be dy
 * dweight      (dim) fp32                 optional: sum over rows of dy (x - mean) rstd
 * dbias        (dim) fp32                 optional: sum over rows of dy
 * The sums over rows are taken in a fixed order (reproducible bit for bit on
 * one kind of device). rows == 0 writes zero dweight and dbias.
 */
int layer_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups, int dtype,
                                  size_t* bytes);

int layer_norm_bwd(int64_t rows, int64_t dim, int64_t groups, int dtype, const void* x,
                   const float* weight, const float* mean, const float* rstd, const void* dy,
                   void* dx, float* dweight, float* dbias, void* workspace,
                   size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_LAYERS_H */
