// Dispatch of the ragged grouped products, and their weight gradient.
#include "grouped.hpp"

namespace bsg {

template <int DT, int OUT, int H>
static hipError_t wgrad_h(const GroupedParams& p, hipStream_t s) {
    const int64_t grid = (int64_t)p.E * ((p.K + H - 1) / H) * ((p.N + 255) / 256);
    hipLaunchKernelGGL((grouped_wgrad_kernel<DT, OUT, H>), dim3((unsigned)grid), dim3(kGemmThreads), 0,
                       s, p);
    return hipGetLastError();
}

template <int DT, int OUT>
static hipError_t wgrad_go(const GroupedParams& p, hipStream_t s) {
    // Short sums (few rows an expert) run two workgroups a compute unit.
    // Measured, 128 / 256 rows a tile: 64 experts of 256 rows 53 / 62 us, of
    // 2048 rows 1099 / 1071 us.
    return p.M / p.E <= 512 ? wgrad_h<DT, OUT, 128>(p, s) : wgrad_h<DT, OUT, 256>(p, s);
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
