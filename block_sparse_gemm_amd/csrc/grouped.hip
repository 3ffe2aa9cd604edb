// Dispatch of the ragged grouped products, and their weight gradient.
#include "grouped.hpp"

namespace bsg {

template <int DT, int OUT, int H, int W>
static hipError_t wgrad_tile(const GroupedParams& p, hipStream_t s) {
    const int64_t grid = (int64_t)p.E * ((p.K + H - 1) / H) * ((p.N + W - 1) / W);
    hipLaunchKernelGGL((grouped_wgrad_kernel<DT, OUT, H, W>), dim3((unsigned)grid), dim3(kGemmThreads),
                       0, s, p);
    return hipGetLastError();
}

template <int DT, int OUT>
static hipError_t wgrad_go(const GroupedParams& p, hipStream_t s) {
    if (p.tile_cols == 128) return wgrad_tile<DT, OUT, 128, 128>(p, s);
    return p.tile_rows == 128 ? wgrad_tile<DT, OUT, 128, 256>(p, s) : wgrad_tile<DT, OUT, 256, 256>(p, s);
}

hipError_t launch_grouped_wgrad(const GroupedParams& p, int c_dtype, int dtype, hipStream_t s) {
    if (dtype == kF32) return wgrad_go<kF32, kF32>(p, s);
    return c_dtype == kF32 ? wgrad_go<kBf16, kF32>(p, s) : wgrad_go<kBf16, kBf16>(p, s);
}

hipError_t launch_grouped_gemm(const GroupedParams& p, int trans_b, int epi, int c_dtype, int dtype,
                               hipStream_t s) {
    if (dtype == kE4m3) return launch_grouped_e4m3(p, epi, s);
    if (dtype == kF32) return launch_grouped_f32(p, trans_b, epi, s);
    return launch_grouped_bf16(p, trans_b, epi, c_dtype, s);
}

}  // namespace bsg
