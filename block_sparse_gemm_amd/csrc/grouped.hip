// Dispatch of the ragged grouped products, and their weight gradient.
#include "grouped.hpp"

namespace bsg {

template <int DT, int OUT, int H, int W, bool SPLIT>
static hipError_t wgrad_tile(const GroupedParams& p, hipStream_t s) {
    const int64_t grid = (int64_t)p.E * ((p.K + H - 1) / H) * ((p.N + W - 1) / W) * (SPLIT ? p.nseg : 1);
    hipLaunchKernelGGL((grouped_wgrad_kernel<DT, OUT, H, W, SPLIT>), dim3((unsigned)grid), dim3(kGemmThreads),
                       0, s, p);
    return hipGetLastError();
}

template <int DT, int OUT>
static hipError_t wgrad_go(const GroupedParams& p, hipStream_t s) {
    if (p.nseg > 1) {
        const hipError_t e = wgrad_tile<DT, kF32, 128, 128, true>(p, s);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(grouped_wgrad_join_kernel<OUT>,
                           dim3((unsigned)(p.E * p.K), (unsigned)((p.N + 4 * kGemmThreads - 1) / (4 * kGemmThreads))),
                           dim3(kGemmThreads), 0, s, p);
        return hipGetLastError();
    }
    if (p.tile_cols == 128) return wgrad_tile<DT, OUT, 128, 128, false>(p, s);
    return p.tile_rows == 128 ? wgrad_tile<DT, OUT, 128, 256, false>(p, s)
                              : wgrad_tile<DT, OUT, 256, 256, false>(p, s);
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
