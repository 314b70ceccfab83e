// Linear attention kernels of one (I/O dtype, mode) pair, given by
// MAMBA_VARIANT_IO and MAMBA_VARIANT_MODE, for every head width.
#include "linear_attn_kernel.h"

namespace mamba {

template <int IO, int MODE>
hipError_t launch_linear_attn_variant(const LinArgs& a, int dc_pad, int block_cols, hipStream_t s) {
    const int64_t segs = MODE == kLinState ? a.nseg - 1 : a.nseg;
    const dim3 grid(static_cast<unsigned>(a.batch * a.heads * segs * a.npass * a.nblk));
    const dim3 block(static_cast<unsigned>(block_cols / kLinCols * kWave));
    if (dc_pad == 64 && block_cols == 64) hipLaunchKernelGGL((linear_attn_kernel<IO, 64, 4, MODE>), grid, block, 0, s, a);
    else if (dc_pad == 64) hipLaunchKernelGGL((linear_attn_kernel<IO, 64, 8, MODE>), grid, block, 0, s, a);
    else if (dc_pad == 128 && block_cols == 64) hipLaunchKernelGGL((linear_attn_kernel<IO, 128, 4, MODE>), grid, block, 0, s, a);
    else if (dc_pad == 128) hipLaunchKernelGGL((linear_attn_kernel<IO, 128, 8, MODE>), grid, block, 0, s, a);
    else if (block_cols == 64) hipLaunchKernelGGL((linear_attn_kernel<IO, 256, 4, MODE>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((linear_attn_kernel<IO, 256, 8, MODE>), grid, block, 0, s, a);
    return hipGetLastError();
}

template hipError_t launch_linear_attn_variant<MAMBA_VARIANT_IO, MAMBA_VARIANT_MODE>(
    const LinArgs&, int, int, hipStream_t);

}  // namespace mamba
