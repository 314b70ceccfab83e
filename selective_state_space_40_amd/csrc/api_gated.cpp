// C ABI of the gated recurrent block's operators (mamba_gated.h): argument
// checks and error mapping around gated_scan.hip and gated_norm.hip. Every check
// runs on the host before any launch.
#include <hip/hip_runtime_api.h>

#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "mamba_gated.h"

namespace {

static_assert(mamba::kGatedBlock == MAMBA_GATED_SCAN_BLOCK, "tokens between kept states");
static_assert(mamba::kGatedNormMaxDim == MAMBA_GATED_NORM_MAX_DIM, "widest part of a norm");
static_assert(mamba::kGateNone == MAMBA_GATE_NONE && mamba::kGateFirst == MAMBA_GATE_FIRST &&
                  mamba::kGateBehind == MAMBA_GATE_BEHIND, "places of the gate");

bool known_dtype(int dtype) { return dtype == MAMBA_DTYPE_F32 || dtype == MAMBA_DTYPE_BF16; }

int io_of(int dtype) { return dtype == MAMBA_DTYPE_F32 ? mamba::kIoF32 : mamba::kIoBF16; }

template <int N>
int check_aligned(const void* const (&ptrs)[N]) {
    for (const void* p : ptrs)
        if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return MAMBA_ERR_MISALIGNED;
    return MAMBA_OK;
}

// Threads that a launch counts (32 bits), and elements of a tensor.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
constexpr int64_t kMaxElems = int64_t(1) << 48;
// Channels and most threads of a workgroup of the recurrence.
constexpr int64_t kGroupChannels = 64, kGroupThreads = 512;

int check_scan(int64_t batch, int64_t seqlen, int64_t dim, int dtype) {
    if (batch < 0 || seqlen < 0 || dim < 0 || !known_dtype(dtype)) return MAMBA_ERR_INVALID_ARG;
    if (dim > MAMBA_GATED_SCAN_MAX_DIM) return MAMBA_ERR_UNSUPPORTED;
    const int64_t groups = (dim + kGroupChannels - 1) / kGroupChannels;
    if (groups > 0 && batch > kMaxThreads / kGroupThreads / groups) return MAMBA_ERR_UNSUPPORTED;
    if (seqlen > kMaxElems / MAMBA_GATED_SCAN_MAX_DIM ||
        (seqlen > 0 && batch > kMaxElems / MAMBA_GATED_SCAN_MAX_DIM / seqlen))
        return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

// A stride that is not used (a gate that is not there) is not looked at.
int check_stride(const void* p, int64_t stride, int64_t dim) {
    if (p == nullptr) return MAMBA_OK;
    if (stride < dim) return MAMBA_ERR_INVALID_ARG;
    return stride > MAMBA_GATED_SCAN_MAX_DIM ? MAMBA_ERR_UNSUPPORTED : MAMBA_OK;
}

int check_inputs(int64_t dim, const void* x, int64_t x_stride, const void* decay_gate, int64_t decay_stride,
                 const float* log_decay, const void* input_gate, int64_t input_stride) {
    if (x == nullptr || decay_gate == nullptr || log_decay == nullptr) return MAMBA_ERR_INVALID_ARG;
    int st = check_stride(x, x_stride, dim);
    if (st == MAMBA_OK) st = check_stride(decay_gate, decay_stride, dim);
    if (st == MAMBA_OK) st = check_stride(input_gate, input_stride, dim);
    return st;
}

mamba::GatedScanArgs scan_args(int64_t batch, int64_t seqlen, int64_t dim, int dtype) {
    mamba::GatedScanArgs a = {};
    a.batch = batch;
    a.seqlen = seqlen;
    a.dim = dim;
    a.io = io_of(dtype);
    return a;
}

void set_inputs(mamba::GatedScanArgs* a, const void* x, int64_t x_stride, const void* decay_gate,
                int64_t decay_stride, const float* log_decay, const void* input_gate, int64_t input_stride) {
    a->x = x;
    a->x_stride = x_stride;
    a->decay_gate = decay_gate;
    a->decay_stride = decay_stride;
    a->log_decay = log_decay;
    a->input_gate = input_gate;
    a->input_stride = input_gate != nullptr ? input_stride : 0;
}

int scan_workspace(int64_t batch, int64_t seqlen, int64_t dim, int dtype, bool bwd, size_t* bytes) {
    if (bytes == nullptr) return MAMBA_ERR_INVALID_ARG;
    const int st = check_scan(batch, seqlen, dim, dtype);
    if (st != MAMBA_OK) return st;
    *bytes = 0;
    if (batch == 0 || seqlen == 0 || dim == 0) return MAMBA_OK;
    const mamba::GatedScanArgs a = scan_args(batch, seqlen, dim, dtype);
    int cu = 0;
    const int got = mamba::current_cu_count(&cu);
    if (got != MAMBA_OK) return got;
    *bytes = bwd ? mamba::gated_scan_bwd_workspace_bytes(a, cu) : mamba::gated_scan_fwd_workspace_bytes(a, cu);
    return MAMBA_OK;
}

// Rows times groups, channels and row stride of a norm.
constexpr int64_t kMaxParts = int64_t(1) << 30;
constexpr int64_t kMaxChannels = int64_t(1) << 27;

int check_norm(int64_t rows, int64_t dim, int64_t groups, int dtype) {
    if (rows < 0 || dim < 0 || groups < 1 || !known_dtype(dtype) || dim % groups != 0)
        return MAMBA_ERR_INVALID_ARG;
    if (dim / groups > MAMBA_GATED_NORM_MAX_DIM || dim > kMaxChannels || groups > kMaxChannels / 32 ||
        rows > kMaxParts / groups)
        return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

bool known_gate(int gate) { return gate >= MAMBA_GATE_NONE && gate <= MAMBA_GATE_BEHIND; }

// The rows of an input of a gated norm.
int check_rows(const void* p, int64_t stride, int64_t rows, int64_t dim) {
    if (p == nullptr || stride < dim) return MAMBA_ERR_INVALID_ARG;
    return stride > kMaxChannels || rows > kMaxElems / stride ? MAMBA_ERR_UNSUPPORTED : MAMBA_OK;
}

int check_total(int dtype, int total_dtype) {
    if (!known_dtype(total_dtype)) return MAMBA_ERR_INVALID_ARG;
    return total_dtype == dtype || total_dtype == MAMBA_DTYPE_F32 ? MAMBA_OK : MAMBA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int gated_scan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                                  size_t* bytes) {
    return scan_workspace(batch, seqlen, dim, dtype, false, bytes);
}

int gated_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                                  size_t* bytes) {
    return scan_workspace(batch, seqlen, dim, dtype, true, bytes);
}

int gated_scan_fwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x,
                   int64_t x_stride, const void* decay_gate, int64_t decay_stride,
                   const float* log_decay, const void* input_gate, int64_t input_stride,
                   const int32_t* lengths, const float* h0, void* y, float* hL,
                   float* block_states, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
    int st = check_scan(batch, seqlen, dim, dtype);
    if (st != MAMBA_OK) return st;
    if (batch == 0 || dim == 0) return MAMBA_OK;
    mamba::GatedScanArgs a = scan_args(batch, seqlen, dim, dtype);
    if (seqlen > 0) {
        st = check_inputs(dim, x, x_stride, decay_gate, decay_stride, log_decay, input_gate, input_stride);
        if (st != MAMBA_OK) return st;
        if (y == nullptr) return MAMBA_ERR_INVALID_ARG;
    }
    const void* const ptrs[] = {x, decay_gate, log_decay, input_gate, lengths, h0, y, hL, block_states, workspace};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    int cu = 1;
    if (seqlen > 0) {
        st = mamba::current_cu_count(&cu);
        if (st != MAMBA_OK) return st;
        const size_t need = mamba::gated_scan_fwd_workspace_bytes(a, cu);
        if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    } else if (hL == nullptr) {
        return MAMBA_OK;
    }
    set_inputs(&a, x, x_stride, decay_gate, decay_stride, log_decay, input_gate, input_stride);
    a.lengths = lengths;
    a.h0 = h0;
    a.y = y;
    a.hL = hL;
    a.states = block_states;
    return mamba::launch_gated_scan_fwd(a, cu, workspace, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int gated_scan_bwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x,
                   int64_t x_stride, const void* decay_gate, int64_t decay_stride,
                   const float* log_decay, const void* input_gate, int64_t input_stride,
                   const int32_t* lengths, const float* block_states, const void* dy,
                   const float* dhL, void* dx, void* ddecay_gate, void* dinput_gate,
                   float* dlog_decay, float* dh0, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
    int st = check_scan(batch, seqlen, dim, dtype);
    if (st != MAMBA_OK) return st;
    if (dim == 0) return MAMBA_OK;
    mamba::GatedScanArgs a = scan_args(batch, seqlen, dim, dtype);
    const bool tokens = batch > 0 && seqlen > 0;
    if (tokens) {
        st = check_inputs(dim, x, x_stride, decay_gate, decay_stride, log_decay, input_gate, input_stride);
        if (st != MAMBA_OK) return st;
        if (block_states == nullptr || dy == nullptr || dx == nullptr || ddecay_gate == nullptr ||
            (input_gate != nullptr && dinput_gate == nullptr))
            return MAMBA_ERR_INVALID_ARG;
    }
    const void* const ptrs[] = {x,  decay_gate,  log_decay,   input_gate, lengths, block_states, dy,
                                dhL, dx,          ddecay_gate, dinput_gate, dlog_decay, dh0,      workspace};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    a.lengths = lengths;
    a.dlog_decay = dlog_decay;
    int cu = 1;
    if (tokens) {
        st = mamba::current_cu_count(&cu);
        if (st != MAMBA_OK) return st;
        const size_t need = mamba::gated_scan_bwd_needed_bytes(a, cu);
        if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    } else if (dlog_decay == nullptr && dh0 == nullptr) {
        return MAMBA_OK;
    }
    set_inputs(&a, x, x_stride, decay_gate, decay_stride, log_decay, input_gate, input_stride);
    a.states = const_cast<float*>(block_states);
    a.dy = dy;
    a.dhL = dhL;
    a.dx = dx;
    a.ddecay = ddecay_gate;
    a.dinput = dinput_gate;
    a.dh0 = dh0;
    return mamba::launch_gated_scan_bwd(a, cu, workspace, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int gated_scan_update(int64_t batch, int64_t dim, int dtype, float* h, const void* x,
                      int64_t x_stride, const void* decay_gate, int64_t decay_stride,
                      const float* log_decay, const void* input_gate, int64_t input_stride,
                      void* y, hipStream_t stream) {
    int st = check_scan(batch, 1, dim, dtype);
    if (st != MAMBA_OK) return st;
    if (batch == 0 || dim == 0) return MAMBA_OK;
    st = check_inputs(dim, x, x_stride, decay_gate, decay_stride, log_decay, input_gate, input_stride);
    if (st != MAMBA_OK) return st;
    if (h == nullptr || y == nullptr) return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {h, x, decay_gate, log_decay, input_gate, y};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    mamba::GatedScanArgs a = scan_args(batch, 1, dim, dtype);
    set_inputs(&a, x, x_stride, decay_gate, decay_stride, log_decay, input_gate, input_stride);
    a.h = h;
    a.y = y;
    return mamba::launch_gated_scan_update(a, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int gated_norm_fwd(int64_t rows, int64_t dim, int64_t groups, int dtype, int gate, const void* x,
                   int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                   float eps, void* y, float* rstd, hipStream_t stream) {
    int st = check_norm(rows, dim, groups, dtype);
    if (st != MAMBA_OK) return st;
    if (!known_gate(gate) || !(eps >= 0.0f) || !isfinite(eps)) return MAMBA_ERR_INVALID_ARG;
    if (rows == 0 || dim == 0) return MAMBA_OK;
    if (gate == MAMBA_GATE_NONE) z = nullptr;
    st = check_rows(x, x_stride, rows, dim);
    if (st == MAMBA_OK && gate != MAMBA_GATE_NONE) st = check_rows(z, z_stride, rows, dim);
    if (st != MAMBA_OK) return st;
    if (y == nullptr) return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {x, z, weight, y, rstd};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    int cu = 0;
    st = mamba::current_cu_count(&cu);
    if (st != MAMBA_OK) return st;
    mamba::GatedNormArgs a = {};
    a.rows = rows;
    a.dim = dim;
    a.groups = groups;
    a.io = io_of(dtype);
    a.gate = gate;
    a.x_stride = x_stride;
    a.z_stride = z_stride;
    a.eps = eps;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.y = y;
    a.rstd = rstd;
    return mamba::launch_gated_norm_fwd(a, cu, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int gated_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups, int dtype,
                                  size_t* bytes) {
    if (bytes == nullptr) return MAMBA_ERR_INVALID_ARG;
    int st = check_norm(rows, dim, groups, dtype);
    if (st != MAMBA_OK) return st;
    *bytes = 0;
    if (rows == 0 || dim == 0) return MAMBA_OK;
    int cu = 0;
    st = mamba::current_cu_count(&cu);
    if (st != MAMBA_OK) return st;
    *bytes = mamba::gated_norm_bwd_workspace_bytes(rows, dim, groups, cu);
    return MAMBA_OK;
}

int gated_norm_bwd(int64_t rows, int64_t dim, int64_t groups, int dtype, int gate, const void* x,
                   int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                   const float* rstd, const void* dy, void* dx, void* dz, float* dweight,
                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_norm(rows, dim, groups, dtype);
    if (st != MAMBA_OK) return st;
    if (!known_gate(gate)) return MAMBA_ERR_INVALID_ARG;
    if (dim == 0) return MAMBA_OK;
    if (gate == MAMBA_GATE_NONE) z = dz = nullptr;
    if (rows > 0) {
        st = check_rows(x, x_stride, rows, dim);
        if (st == MAMBA_OK && gate != MAMBA_GATE_NONE) st = check_rows(z, z_stride, rows, dim);
        if (st != MAMBA_OK) return st;
        if (rstd == nullptr || dy == nullptr || dx == nullptr || (gate != MAMBA_GATE_NONE && dz == nullptr))
            return MAMBA_ERR_INVALID_ARG;
    }
    const void* const ptrs[] = {x, z, weight, rstd, dy, dx, dz, dweight, workspace};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    int cu = 1;
    if (rows > 0) {
        st = mamba::current_cu_count(&cu);
        if (st != MAMBA_OK) return st;
        const size_t need = mamba::gated_norm_bwd_workspace_bytes(rows, dim, groups, cu);
        if (dweight != nullptr && need > 0 && (workspace == nullptr || workspace_bytes < need))
            return MAMBA_ERR_WORKSPACE;
    } else if (dweight == nullptr) {
        return MAMBA_OK;
    }
    mamba::GatedNormArgs a = {};
    a.rows = rows;
    a.dim = dim;
    a.groups = groups;
    a.io = io_of(dtype);
    a.gate = gate;
    a.x_stride = x_stride;
    a.z_stride = z_stride;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dx = dx;
    a.dz = dz;
    a.dweight = dweight;
    return mamba::launch_gated_norm_bwd(a, cu, workspace, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int residual_norm_fwd(int64_t rows, int64_t dim, int dtype, int total_dtype, const void* x,
                      const void* residual, const float* scale, const float* weight, float eps,
                      void* y, void* total, float* rstd, hipStream_t stream) {
    int st = check_norm(rows, dim, 1, dtype);
    if (st == MAMBA_OK) st = check_total(dtype, total_dtype);
    if (st != MAMBA_OK) return st;
    if (!(eps >= 0.0f) || !isfinite(eps)) return MAMBA_ERR_INVALID_ARG;
    if (rows == 0 || dim == 0) return MAMBA_OK;
    if (x == nullptr || residual == nullptr || y == nullptr || total == nullptr) return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {x, residual, scale, weight, y, total, rstd};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    int cu = 0;
    st = mamba::current_cu_count(&cu);
    if (st != MAMBA_OK) return st;
    mamba::ResidualNormArgs a = {};
    a.rows = rows;
    a.dim = dim;
    a.io = io_of(dtype);
    a.total_io = io_of(total_dtype);
    a.eps = eps;
    a.x = x;
    a.residual = residual;
    a.scale = scale;
    a.weight = weight;
    a.y = y;
    a.total = total;
    a.rstd = rstd;
    return mamba::launch_residual_norm_fwd(a, cu, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int residual_norm_bwd_workspace_size(int64_t rows, int64_t dim, int dtype, int total_dtype,
                                     size_t* bytes) {
    if (bytes == nullptr) return MAMBA_ERR_INVALID_ARG;
    int st = check_norm(rows, dim, 1, dtype);
    if (st == MAMBA_OK) st = check_total(dtype, total_dtype);
    if (st != MAMBA_OK) return st;
    *bytes = 0;
    if (rows == 0 || dim == 0) return MAMBA_OK;
    int cu = 0;
    st = mamba::current_cu_count(&cu);
    if (st != MAMBA_OK) return st;
    *bytes = mamba::residual_norm_bwd_workspace_bytes(rows, dim, cu);
    return MAMBA_OK;
}

int residual_norm_bwd(int64_t rows, int64_t dim, int dtype, int total_dtype, const void* total,
                      const float* weight, const float* rstd, const void* x, const float* scale,
                      const void* dy, const void* dtotal, void* dx, void* dresidual,
                      float* dscale, float* dweight, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    int st = check_norm(rows, dim, 1, dtype);
    if (st == MAMBA_OK) st = check_total(dtype, total_dtype);
    if (st != MAMBA_OK) return st;
    if (dim == 0) return MAMBA_OK;
    if (dscale != nullptr && scale == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (rows > 0 && (total == nullptr || rstd == nullptr || dy == nullptr || dresidual == nullptr ||
                     (dscale != nullptr && x == nullptr)))
        return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {total, weight, rstd, x, scale, dy, dtotal, dx, dresidual, dscale, dweight, workspace};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    int cu = 1;
    if (rows > 0) {
        st = mamba::current_cu_count(&cu);
        if (st != MAMBA_OK) return st;
        const size_t need = mamba::residual_norm_bwd_workspace_bytes(rows, dim, cu);
        if ((dscale != nullptr || dweight != nullptr) && need > 0 && (workspace == nullptr || workspace_bytes < need))
            return MAMBA_ERR_WORKSPACE;
    } else if (dscale == nullptr && dweight == nullptr) {
        return MAMBA_OK;
    }
    mamba::ResidualNormArgs a = {};
    a.rows = rows;
    a.dim = dim;
    a.io = io_of(dtype);
    a.total_io = io_of(total_dtype);
    a.x = x;
    a.scale = scale;
    a.weight = weight;
    a.total = const_cast<void*>(total);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dtotal = dtotal;
    a.dx = dx;
    a.dresidual = dresidual;
    a.dscale = dscale;
    a.dweight = dweight;
    return mamba::launch_residual_norm_bwd(a, cu, workspace, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
