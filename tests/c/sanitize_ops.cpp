// The norm's, the grouped products' and clipping's C entry points (api_ops.cpp)
// and the products' host rules under the sanitizers: ordinary, degenerate and
// extreme arguments; the kernel launchers are host stand-ins that record the call.
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "../../block_sparse_gemm_amd/csrc/kernels.hpp"
#include "../../include/bsg.h"

static int g_launches = 0, g_failed = 0;
static bsg::GroupedParams g_last;

namespace bsg {
int rms_norm_backward_rows(int64_t, int, int) { return 1; }
hipError_t launch_rms_norm(const NormParams&, int, int, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_rms_norm_backward(const NormParams&, int, float*, hipStream_t) {
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_grouped_gemm(const GroupedParams& p, int, int, int, int, hipStream_t) {
    ++g_launches;
    g_last = p;
    return hipSuccess;
}
hipError_t launch_grouped_wgrad(const GroupedParams&, int, int, hipStream_t) {
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_grad_norm(const void* const*, const int64_t*, const int*, int, float*, double*,
                            hipStream_t) {
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_grad_clip(const void* const*, void* const*, const int64_t*, const int*, int,
                            const float*, float, hipStream_t) {
    ++g_launches;
    return hipErrorInvalidValue;  // a failed launch is reported
}
}  // namespace bsg

#define EXPECT(cond)                                                       \
    do {                                                                   \
        if (!(cond)) {                                                     \
            ++g_failed;                                                    \
            printf("line %d: %s (%s)\n", __LINE__, #cond, bsg_last_error()); \
        }                                                                  \
    } while (0)

int main() {
    char* const base = (char*)0x100000;
    void* P = base;
    float* fp = (float*)base;
    int32_t* ip = (int32_t*)base;

    // ---- norm
    EXPECT(bsg_rms_norm(P, 64, P, 64, P, 1e-5f, 3, 64, BSG_BF16, P, 64, P, 64, BSG_BF16, nullptr, fp,
                        nullptr) == BSG_OK);
    EXPECT(bsg_rms_norm(P, 64, nullptr, 0, P, 0.0f, INT_MAX, 64, BSG_F32, nullptr, 0, P, 64, BSG_E4M3, fp,
                        nullptr, nullptr) == BSG_OK);
    const int launched = g_launches;
    EXPECT(bsg_rms_norm(P, INT64_MAX, P, 64, P, 1e-5f, 3, 64, BSG_BF16, P, 64, P, 64, BSG_BF16, nullptr,
                        fp, nullptr) == BSG_EINVAL);
    EXPECT(bsg_rms_norm(P, 64, P, INT64_MIN, P, 1e-5f, 3, 64, BSG_BF16, P, 64, P, 64, BSG_BF16, nullptr,
                        fp, nullptr) == BSG_EINVAL);
    EXPECT(bsg_rms_norm(P, 64, P, 64, P, 1e-5f, INT64_MAX, 64, BSG_BF16, P, 64, P, 64, BSG_BF16, nullptr,
                        fp, nullptr) == BSG_EINVAL);
    EXPECT(bsg_rms_norm(P, 64, P, 64, P, 1e-5f, 3, INT_MAX, BSG_F32, P, 64, P, 64, BSG_F32, nullptr, fp,
                        nullptr) == BSG_EINVAL);
    EXPECT(bsg_rms_norm(P, 64, P, 64, P, 1e-5f, 3, INT_MIN, BSG_F32, P, 64, P, 64, BSG_F32, nullptr, fp,
                        nullptr) == BSG_EINVAL);
    EXPECT(g_launches == launched);
    EXPECT(bsg_rms_norm_backward_workspace_bytes(INT64_MAX, INT_MAX) == 0);
    EXPECT(bsg_rms_norm_backward_workspace_bytes(INT_MAX, 1 << 24) == (size_t)512 * (1 << 24) * 4);
    EXPECT(bsg_rms_norm_backward(P, 64, P, 64, P, 64, P, fp, 3, 64, BSG_BF16, P, 64, fp, P, SIZE_MAX,
                                 nullptr) == BSG_OK);
    EXPECT(bsg_rms_norm_backward(P, 64, P, 64, P, 64, P, fp, 3, 64, BSG_BF16, P, 64, fp, P, 0, nullptr) ==
           BSG_EINVAL);

    // ---- grouped products: every rule at the extremes of its sizes
    const int64_t Ms[] = {1, 2, 17, 96, 97, 4096, 1 << 20, INT_MAX};
    const int widths[] = {16, 128, 4096, 1 << 24};
    const int Es[] = {1, 3, 64, 1024};
    for (int64_t M : Ms)
        for (int K : widths)
            for (int N : widths)
                for (int E : Es)
                    for (int epi = BSG_EPI_NONE; epi <= BSG_EPI_SILU_MUL_BWD; ++epi) {
                        const size_t ws = bsg_grouped_gemm_workspace_bytes(M, K, N, E, epi);
                        for (int dt : {BSG_F32, BSG_BF16, BSG_E4M3}) {
                            const bsg::GroupedPlan p =
                                bsg::grouped_plan(M, K, N, E, epi, dt, 256, bsg::kMaxSegments);
                            const int seg = p.segments;
                            EXPECT(seg >= 1 && seg <= bsg::kMaxSegments);
                            EXPECT(p.rows == 128 || p.rows == 256);
                            EXPECT(p.cols == 256 || (p.cols == 128 && p.rows == 128 && seg == 1));
                            EXPECT(bsg::grouped_plan(M, K, N, E, epi, dt, 256, 1).segments == 1);
                            const bsg::GroupedPlan w = bsg::grouped_wgrad_plan(M, K, N, E, dt, 256, bsg::kMaxSegments);
                            EXPECT((w.rows == 128 || w.rows == 256) && (w.cols == 256 || w.rows == 128));
                            EXPECT(w.segments >= 1 && w.segments <= bsg::kMaxSegments);
                            if (w.segments > 1 && dt != BSG_E4M3)
                                EXPECT(bsg_grouped_wgrad_workspace_bytes(M, K, N, E) / ((size_t)K * N * 4) / E >=
                                       (size_t)w.segments);
                            EXPECT(bsg::grouped_wgrad_plan(M, K, N, E, dt, 256, 1).segments == 1);
                            // the size query allows every plan
                            if (seg > 1) EXPECT(ws / ((size_t)M * N * 4) >= (size_t)seg);
                        }
                        const bool dual = epi == BSG_EPI_SILU_MUL;
                        const bool bwd = epi == BSG_EPI_GELU_BWD || epi == BSG_EPI_SILU_MUL_BWD;
                        for (size_t bytes : {(size_t)0, (size_t)16, ws, SIZE_MAX}) {
                            const bsg_status s = bsg_grouped_gemm(
                                P, nullptr, K, nullptr, P, dual ? P : nullptr, N,
                                std::min((int64_t)K * N, (int64_t)1 << 40), nullptr, 0,
                                ip, E, M, K, N, epi, bwd ? P : nullptr, P, N, BSG_BF16, nullptr, BSG_BF16, P,
                                bytes, nullptr);
                            EXPECT(s == BSG_OK || s == BSG_EUNSUPPORTED);
                            if (s == BSG_OK && g_last.nseg > 1)
                                EXPECT((size_t)g_last.nseg * M * N * 4 * (dual ? 2 : 1) <= bytes);
                        }
                    }
    EXPECT(bsg_grouped_gemm_workspace_bytes(INT64_MAX, 64, 64, 1, 0) == 0);
    EXPECT(bsg_grouped_gemm_workspace_bytes(1, INT_MAX, 64, 1, 0) == 0);
    EXPECT(bsg_grouped_gemm_workspace_bytes(1, 64, INT_MIN, 1, 0) == 0);
    EXPECT(bsg_grouped_gemm_workspace_bytes(1, 64, 64, 0, 0) == 0);
    EXPECT(bsg_grouped_gemm_workspace_bytes(1, 64, 64, 1, 99) == 0);
    for (int64_t bad : {INT64_MAX, INT64_MIN, (int64_t)-8, ((int64_t)1 << 40) + 8}) {
        EXPECT(bsg_grouped_gemm(P, nullptr, bad, nullptr, P, nullptr, 128, 8192, nullptr, 0, ip, 4, 10, 64, 128,
                                0, nullptr, P, 128, BSG_BF16, nullptr, BSG_BF16, nullptr, 0, nullptr) == BSG_EINVAL);
        EXPECT(bsg_grouped_gemm(P, nullptr, 64, nullptr, P, nullptr, bad, 8192, nullptr, 0, ip, 4, 10, 64, 128, 0,
                                nullptr, P, 128, BSG_BF16, nullptr, BSG_BF16, nullptr, 0, nullptr) == BSG_EINVAL);
        EXPECT(bsg_grouped_gemm(P, nullptr, 64, nullptr, P, nullptr, 128, bad, nullptr, 0, ip, 4, 10, 64, 128, 0,
                                nullptr, P, 128, BSG_BF16, nullptr, BSG_BF16, nullptr, 0, nullptr) == BSG_EINVAL);
        EXPECT(bsg_grouped_wgrad(P, 64, P, 128, ip, 4, 10, 64, 128, P, bad, 8192, BSG_BF16, BSG_BF16, P, 64,
                                 nullptr) == BSG_EINVAL);
        EXPECT(bsg_grouped_wgrad(P, 64, P, 128, ip, 4, bad, 64, 128, P, 128, 8192, BSG_BF16, BSG_BF16, P, 64,
                                 nullptr) == BSG_EINVAL);
    }
    EXPECT(bsg_grouped_wgrad(P, 64, P, 128, ip, 1024, INT_MAX, 64, 128, P, 128, 8192, BSG_F32, BSG_BF16,
                             P, SIZE_MAX, nullptr) == BSG_OK);

    // ---- clipping: lists of every length, and the overlap check
    for (int n : {0, 1, 2, 97, 5000}) {
        std::vector<void*> in(n + 1), out(n + 1);
        std::vector<int64_t> count(n + 1);
        std::vector<int> dt(n + 1);
        for (int i = 0; i < n; ++i) {
            count[i] = i % 7;
            dt[i] = i & 1;
            in[i] = base + 64 * (n - i);
            out[i] = base + (1 << 20) + 64 * i;
        }
        EXPECT(bsg_grad_norm(in.data(), count.data(), dt.data(), n, fp, P, 1 << 20, nullptr) == BSG_OK);
        EXPECT(bsg_grad_clip(in.data(), nullptr, count.data(), dt.data(), n, fp, 1.0f, nullptr) == BSG_EHIP);
        EXPECT(bsg_grad_clip(in.data(), out.data(), count.data(), dt.data(), n, fp, INFINITY, nullptr) == BSG_EHIP);
        if (n > 20) {
            out[n - 1] = (char*)in[2] + 4;  // tensor 2 has 2 values of 4 bytes
            dt[n - 1] = BSG_F32;
            count[n - 1] = 1;
            EXPECT(bsg_grad_clip(in.data(), out.data(), count.data(), dt.data(), n, fp, 1.0f, nullptr) ==
                   BSG_EINVAL);
        }
    }
    EXPECT(bsg_grad_norm(nullptr, nullptr, nullptr, INT_MAX, fp, P, 1 << 20, nullptr) == BSG_EINVAL);
    EXPECT(bsg_grad_clip(nullptr, nullptr, nullptr, nullptr, 3, fp, 1.0f, nullptr) == BSG_EINVAL);

    if (g_failed) return 1;
    printf("sanitized operator checks passed (%d launches)\n", g_launches);
    return 0;
}
