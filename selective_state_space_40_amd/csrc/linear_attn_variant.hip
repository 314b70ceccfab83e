// Linear attention kernels of one (I/O dtype, mode) pair, given by
// MAMBA_VARIANT_IO and MAMBA_VARIANT_MODE, for every head width.
#include "linear_attn_kernel.h"

namespace mamba {

template <int IO, int MODE, int DC>
hipError_t launch_width(const LinArgs& a, unsigned blocks, hipStream_t s) {
    hipLaunchKernelGGL((linear_attn_kernel<IO, DC, MODE>), dim3(blocks), dim3(lin_waves(DC) * kWave), 0, s, a);
    return hipGetLastError();
}

template <int IO, int MODE>
hipError_t launch_linear_attn_variant(const LinArgs& a, int dc_pad, hipStream_t s) {
    const int64_t segs = MODE == kLinState ? a.nseg - 1 : a.nseg;
    const unsigned blocks = static_cast<unsigned>(a.batch * a.heads * segs * a.npass * a.nblk);
    if (dc_pad == 64) return launch_width<IO, MODE, 64>(a, blocks, s);
    if (dc_pad == 128) return launch_width<IO, MODE, 128>(a, blocks, s);
    return launch_width<IO, MODE, 256>(a, blocks, s);
}

template hipError_t launch_linear_attn_variant<MAMBA_VARIANT_IO, MAMBA_VARIANT_MODE>(
    const LinArgs&, int, hipStream_t);

}  // namespace mamba
