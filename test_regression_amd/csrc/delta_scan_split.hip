// delta_scan_split.hip -- launches of the gated delta rule's pass over the chunks
// (delta_scan_split.h): the forward's, and the segments' ends.
#include "delta_scan_split.h"

namespace mesa {

template <int DKP, typename In, bool OUT>
__global__ __launch_bounds__(768) void delta_scan_split_kernel(DeltaArgs a, int waves) {
    __shared__ ScanSplitLds<DKP, In, OUT> L;
    scan_split<DKP, In, OUT, false>(L, a, waves, blockIdx.x);
}

template <int DKP, typename In, bool OUT>
hipError_t scan_split_go(const DeltaArgs& a, hipStream_t s) {
    const long heads = a.BH * (OUT ? a.nseg : a.nseg - 1);
    const int cols = OUT ? a.dv : a.dv + a.dk, waves = scan_waves(heads, cols);
    hipLaunchKernelGGL((delta_scan_split_kernel<DKP, In, OUT>), dim3(scan_blocks(heads, cols, waves)), dim3(768), 0, s, a, waves);
    return hipGetLastError();
}
template <bool OUT>
hipError_t scan_split_dk(const DeltaArgs& a, hipStream_t s) {
    if (!a.bf16) return a.dk <= 32 ? scan_split_go<32, float, OUT>(a, s) : scan_split_go<64, float, OUT>(a, s);
    return a.dk <= 32 ? scan_split_go<32, bf16_t, OUT>(a, s)
                      : a.dk == 64 ? scan_split_go<64, bf16_t, OUT>(a, s) : scan_split_go<128, bf16_t, OUT>(a, s);
}

hipError_t launch_delta_scan_split(const DeltaArgs& a, hipStream_t s) { return scan_split_dk<true>(a, s); }
hipError_t launch_delta_ends_split(const DeltaArgs& a, hipStream_t s) { return scan_split_dk<false>(a, s); }

}  // namespace mesa
