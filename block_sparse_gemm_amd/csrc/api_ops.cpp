// C ABI of what stands around the padded expert products: the norm, the
// ragged grouped products and gradient clipping.  Every check runs before any
// HIP call, as in api.cpp.
#include <float.h>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>

#include "api.hpp"
#include "kernels.hpp"

using namespace bsg;

static_assert(bsg::kE4m3 == BSG_E4M3, "one code");

extern "C" {

// ------------------------------------------------------------------- norm

static bsg_status check_norm(int64_t T, int d, int dtype) {
    REQUIRE(dtype_ok(dtype), "unknown dtype %d", dtype);
    REQUIRE(T >= 0 && T <= INT32_MAX, "T out of range");
    REQUIRE(d >= 1 && d <= kMaxWidth && (d * elt_bytes(dtype)) % 16 == 0,
            "d must keep rows 16-byte aligned");
    if (d * elt_bytes(dtype) > bsg::kNormRowBytes)
        return fail(BSG_EUNSUPPORTED, "rows above %d bytes are not implemented", bsg::kNormRowBytes);
    return BSG_OK;
}

#define REQUIRE_ROWS(p, ld, width, es)                                                      \
    do {                                                                                    \
        REQUIRE_VEC_PTR(p);                                                                 \
        REQUIRE((ld) >= (width) && (ld) <= kMaxLd && ((ld) * (es)) % 16 == 0,               \
                #ld " must be >= the row's width with 16-byte aligned rows");               \
    } while (0)

bsg_status bsg_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                        const void* weight, float eps, int64_t T, int d, int dtype, void* h,
                        int64_t ldh, void* y, int64_t ldy, int y_dtype, float* y_scale,
                        float* rstd, bsg_stream_t stream) {
    const bsg_status s = check_norm(T, d, dtype);
    if (s != BSG_OK) return s;
    REQUIRE(y_dtype == dtype || y_dtype == BSG_E4M3, "y_dtype must be dtype or e4m3");
    REQUIRE(eps >= 0.0f && eps <= FLT_MAX, "eps must be finite and >= 0");
    const int es = elt_bytes(dtype);
    REQUIRE(h == nullptr || residual != nullptr, "h is only written with a residual");
    REQUIRE((y_scale != nullptr) == (y_dtype == BSG_E4M3), "y_scale goes with an e4m3 y");
    if (T == 0) return ok();
    REQUIRE_ROWS(x, ldx, d, es);
    if (residual) REQUIRE_ROWS(residual, ldr, d, es);
    if (h) REQUIRE_ROWS(h, ldh, d, es);
    REQUIRE_VEC_PTR(weight);
    if (y_dtype == BSG_E4M3) {
        const int vec = 16 / es;  // the bytes that one 16-byte vector of x becomes
        REQUIRE(y != nullptr && aligned(y, vec), "y must be a non-null aligned device pointer");
        REQUIRE(ldy >= d && ldy <= kMaxLd && ldy % vec == 0,
                "ldy must be >= d with %d-byte aligned rows", vec);
        REQUIRE_PTR(y_scale);
    } else {
        REQUIRE_ROWS(y, ldy, d, es);
    }
    REQUIRE(rstd == nullptr || aligned(rstd, 4), "rstd must be 4-byte aligned");
    bsg::NormParams p{};
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.h = h;
    p.y = y;
    p.y_scale = y_scale;
    p.rstd = rstd;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldh = ldh;
    p.ldy = ldy;
    p.T = T;
    p.d = d;
    p.eps = eps;
    return hip_status(bsg::launch_rms_norm(p, dtype, y_dtype == BSG_E4M3, (hipStream_t)stream),
                      "rms_norm");
}

size_t bsg_rms_norm_backward_workspace_bytes(int64_t T, int d) {
    if (T < 0 || T > INT32_MAX || d < 1 || d > kMaxWidth) return 0;
    return (size_t)std::min<int64_t>(std::max<int64_t>(T, 1), bsg::kNormPartials) * d * sizeof(float);
}

bsg_status bsg_rms_norm_backward(const void* dy, int64_t lddy, const void* dh, int64_t lddh,
                                 const void* h, int64_t ldh, const void* weight,
                                 const float* rstd, int64_t T, int d, int dtype, void* dx,
                                 int64_t lddx, float* dweight, void* workspace,
                                 size_t workspace_bytes, bsg_stream_t stream) {
    const bsg_status s = check_norm(T, d, dtype);
    if (s != BSG_OK) return s;
    const int es = elt_bytes(dtype);
    REQUIRE_PTR(dweight);
    REQUIRE(workspace != nullptr && aligned(workspace, 16),
            "workspace must be a non-null 16-byte aligned device pointer");
    REQUIRE(workspace_bytes >= bsg_rms_norm_backward_workspace_bytes(T, d),
            "workspace too small (%zu < %zu)", workspace_bytes,
            bsg_rms_norm_backward_workspace_bytes(T, d));
    if (T > 0) {
        REQUIRE_ROWS(dy, lddy, d, es);
        if (dh) REQUIRE_ROWS(dh, lddh, d, es);
        REQUIRE_ROWS(h, ldh, d, es);
        REQUIRE_VEC_PTR(weight);
        REQUIRE_PTR(rstd);
        REQUIRE_ROWS(dx, lddx, d, es);
    }
    bsg::NormParams p{};
    p.x = h;
    p.residual = dh;
    p.dy = dy;
    p.weight = weight;
    p.y = dx;
    p.rstd = const_cast<float*>(rstd);
    p.partial = (float*)workspace;
    p.ldx = ldh;
    p.ldr = lddh;
    p.ldh = lddx;
    p.ldy = lddy;
    p.T = T;
    p.d = d;
    return hip_status(bsg::launch_rms_norm_backward(p, dtype, dweight, (hipStream_t)stream),
                      "rms_norm_backward");
}

// ------------------------------------------------------- grouped products

// The grouped products' lane offsets inside an operand's 256 rows (K
// contiguous) or K-tile stay below 2^31, which leaves the bit that puts a
// lane out of its operand's range; so does a row, the scalar offset's range.
static bool grouped_ld_fits(int64_t ld, int es, bool k_contiguous) {
    const int64_t last_row = k_contiguous ? 255 : (es == 2 ? 31 : 15);
    const int64_t row_bytes = k_contiguous ? 64 + (int64_t)kMaxWidth * es : 512 * es;
    return last_row * ld * es + row_bytes <= (int64_t)INT32_MAX;
}

#define REQUIRE_GROUPED_LD(ld, es, kc)                                                     \
    do {                                                                                   \
        if (!grouped_ld_fits((ld), (es), (kc)))                                            \
            return fail(BSG_EUNSUPPORTED, #ld " = %lld is too large for the products' "    \
                        "31-bit offsets", (long long)(ld));                          \
    } while (0)

static int grouped_elt_bytes(int dtype) { return dtype == BSG_E4M3 ? 1 : elt_bytes(dtype); }

// Compute units that tiles and segments are planned for (an MI355X's: the size
// query has no stream to ask).
constexpr int kPlanCus = 256;

// Workgroups of 256 threads that one launch may have (2^32 threads).
constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

size_t bsg_grouped_gemm_workspace_bytes(int64_t M, int K, int N, int E, int epilogue) {
    if (M < 0 || M > INT32_MAX || K < 1 || K > kMaxWidth || N < 1 || N > kMaxWidth || E < 1 ||
        E > BSG_MAX_EXPERTS || epilogue < BSG_EPI_NONE || epilogue > BSG_EPI_SILU_MUL_BWD)
        return 0;
    if (M == 0) return 0;
    // the most segments that any type has on a device of this many compute units
    int n = 1;
    for (const int dtype : {BSG_F32, BSG_BF16, BSG_E4M3})
        n = std::max(n, bsg::grouped_plan(M, K, N, E, epilogue, dtype, kPlanCus, bsg::kMaxSegments).segments);
    return n == 1 ? 0 : (size_t)n * M * N * (epilogue == BSG_EPI_SILU_MUL ? 2 : 1) * sizeof(float);
}

bsg_status bsg_grouped_gemm(const void* a, const void* a2, int64_t lda, const float* a_scale,
                            const void* b, const void* b2, int64_t ldb, int64_t stride_b,
                            const float* b_scale, int trans_b, const int32_t* row_offsets, int E,
                            int64_t M, int K, int N, int epilogue, const void* aux_in, void* c,
                            int64_t ldc, int c_dtype, void* aux_out, int dtype, void* workspace,
                            size_t workspace_bytes, bsg_stream_t stream) {
    REQUIRE(dtype_ok(dtype) || dtype == BSG_E4M3, "unknown dtype %d", dtype);
    REQUIRE(dtype_ok(c_dtype), "unknown c_dtype %d", c_dtype);
    REQUIRE(epilogue >= BSG_EPI_NONE && epilogue <= BSG_EPI_SILU_MUL_BWD, "unknown epilogue %d",
            epilogue);
    REQUIRE(trans_b == 0 || trans_b == 1, "trans_b must be 0 or 1");
    REQUIRE(E >= 1 && E <= BSG_MAX_EXPERTS, "E must be in [1, %d]", BSG_MAX_EXPERTS);
    REQUIRE(M >= 0 && M <= INT32_MAX, "M out of range");
    const bool f8 = dtype == BSG_E4M3;
    if (dtype == BSG_F32 && c_dtype != BSG_F32)
        return fail(BSG_EUNSUPPORTED, "fp32 operands need an fp32 output");
    if (f8 && c_dtype != BSG_BF16) return fail(BSG_EUNSUPPORTED, "e4m3 operands need a bf16 output");
    if (dtype != BSG_F32 && c_dtype == BSG_F32 && epilogue != BSG_EPI_NONE)
        return fail(BSG_EUNSUPPORTED, "an fp32 output of narrower operands needs BSG_EPI_NONE");
    if (f8) {
        if (!trans_b) return fail(BSG_EUNSUPPORTED, "e4m3 weights need trans_b = 1");
        if (a2 || aux_out || epilogue == BSG_EPI_GELU_BWD || epilogue == BSG_EPI_SILU_MUL_BWD)
            return fail(BSG_EUNSUPPORTED, "e4m3 operands: forward products only");
    }
    const int es = grouped_elt_bytes(dtype), ces = elt_bytes(c_dtype);
    const int kq = 16 / es, nq = dtype == BSG_F32 ? 4 : 8;
    REQUIRE(K >= kq && K <= kMaxWidth && K % kq == 0, "K must be a positive multiple of %d", kq);
    REQUIRE(N >= nq && N <= kMaxWidth && N % nq == 0, "N must be a positive multiple of %d", nq);
    REQUIRE(lda >= K && lda <= kMaxLd && (lda * es) % 16 == 0,
            "lda must be >= K with 16-byte aligned rows");
    REQUIRE(ldb >= (trans_b ? K : N) && ldb <= kMaxLd && (ldb * es) % 16 == 0,
            "ldb too small or rows not 16-byte aligned");
    REQUIRE(stride_b >= 0 && stride_b <= kMaxLd && (stride_b * es) % 16 == 0,
            "stride_b must be >= 0 and keep matrices 16-byte aligned");
    REQUIRE(ldc >= N && ldc <= kMaxLd && (ldc * ces) % 16 == 0,
            "ldc must be >= N with 16-byte aligned rows");
    REQUIRE_GROUPED_LD(lda, es, true);
    REQUIRE_GROUPED_LD(ldb, es, trans_b == 1);
    if (epilogue == BSG_EPI_SILU_MUL) {
        REQUIRE(a2 == nullptr, "a2 is only used by BSG_EPI_NONE");
        REQUIRE_VEC_PTR(b2);
    } else if (epilogue == BSG_EPI_NONE) {
        REQUIRE((a2 == nullptr) == (b2 == nullptr), "a2 and b2 go together");
        if (M > 0) REQUIRE(aligned(a2, 16) && aligned(b2, 16), "a2 and b2 must be 16-byte aligned");
    } else {
        REQUIRE(a2 == nullptr && b2 == nullptr, "a2 and b2 are not used by this epilogue");
    }
    if (epilogue == BSG_EPI_GELU_BWD || epilogue == BSG_EPI_SILU_MUL_BWD) {
        if (M > 0) REQUIRE_VEC_PTR(aux_in);
    } else {
        REQUIRE(aux_in == nullptr, "aux_in is only used by the backward epilogues");
    }
    if (epilogue != BSG_EPI_GELU && epilogue != BSG_EPI_SILU_MUL)
        REQUIRE(aux_out == nullptr, "aux_out is only used by BSG_EPI_GELU and BSG_EPI_SILU_MUL");
    REQUIRE(aux_out == nullptr || aligned(aux_out, 16), "aux_out must be 16-byte aligned");
    if (f8) {
        if (M > 0) REQUIRE_PTR(a_scale);
        REQUIRE_VEC_PTR(b_scale);
    } else {
        REQUIRE(a_scale == nullptr && b_scale == nullptr, "scales are only used by e4m3 operands");
    }
    REQUIRE(workspace == nullptr || aligned(workspace, 16), "workspace must be 16-byte aligned");
    REQUIRE_VEC_PTR(b);
    REQUIRE_PTR(row_offsets);
    if (M == 0) return ok();
    REQUIRE_VEC_PTR(a);
    REQUIRE_VEC_PTR(c);
    bsg::GroupedParams p{};
    p.a = a;
    p.a2 = a2;
    p.b = b;
    p.b2 = b2;
    p.aux_in = aux_in;
    p.a_scale = a_scale;
    p.b_scale = b_scale;
    p.row_offsets = row_offsets;
    p.c = c;
    p.aux_out = aux_out;
    // segments as many as planned, or as the workspace holds
    const int64_t share = M * N * (epilogue == BSG_EPI_SILU_MUL ? 2 : 1) * (int64_t)sizeof(float);
    const int64_t fit = workspace ? (int64_t)std::min<size_t>(workspace_bytes, INT64_MAX) / share : 1;
    const bsg::GroupedPlan plan = bsg::grouped_plan(M, K, N, E, epilogue, dtype, kPlanCus, fit);
    const int64_t ne = std::min<int64_t>(E, M), w = epilogue == BSG_EPI_SILU_MUL ? 128 : plan.cols;
    if ((M + (plan.rows - 1) * ne) / plan.rows * ((N + w - 1) / w) * plan.segments > kMaxGrid)
        return fail(BSG_EUNSUPPORTED, "too many tiles for one launch");
    p.ws = (float*)workspace;
    p.nseg = plan.segments;
    p.tile_rows = plan.rows;
    p.tile_cols = plan.cols;
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = ldc;
    p.stride_b = stride_b;
    p.M = M;
    p.K = K;
    p.N = N;
    p.E = E;
    return hip_status(bsg::launch_grouped_gemm(p, trans_b, epilogue, c_dtype, dtype,
                                               (hipStream_t)stream),
                      "grouped_gemm");
}

size_t bsg_grouped_wgrad_workspace_bytes(int64_t M, int K, int N, int E) {
    if (M < 0 || M > INT32_MAX || K < 1 || K > kMaxWidth || N < 1 || N > kMaxWidth || E < 1 ||
        E > BSG_MAX_EXPERTS)
        return 0;
    int n = 1;
    for (const int dtype : {BSG_F32, BSG_BF16})
        n = std::max(n, bsg::grouped_wgrad_plan(M, K, N, E, dtype, kPlanCus, bsg::kMaxSegments).segments);
    return n == 1 ? 0 : (size_t)n * E * K * N * sizeof(float);
}

bsg_status bsg_grouped_wgrad(const void* a, int64_t lda, const void* dmat, int64_t ldd,
                             const int32_t* row_offsets, int E, int64_t M, int K, int N, void* c,
                             int64_t ldc, int64_t stride_c, int c_dtype, int dtype,
                             void* workspace, size_t workspace_bytes, bsg_stream_t stream) {
    REQUIRE(dtype_ok(dtype), "unknown dtype %d", dtype);
    REQUIRE(dtype_ok(c_dtype), "unknown c_dtype %d", c_dtype);
    if (dtype == BSG_F32 && c_dtype != BSG_F32)
        return fail(BSG_EUNSUPPORTED, "fp32 operands need an fp32 output");
    REQUIRE(E >= 1 && E <= BSG_MAX_EXPERTS, "E must be in [1, %d]", BSG_MAX_EXPERTS);
    REQUIRE(M >= 0 && M <= INT32_MAX, "M out of range");
    const int es = elt_bytes(dtype), ces = elt_bytes(c_dtype), q = 16 / es;
    REQUIRE(K >= q && K <= kMaxWidth && K % q == 0, "K must be a positive multiple of %d", q);
    REQUIRE(N >= q && N <= kMaxWidth && N % q == 0, "N must be a positive multiple of %d", q);
    REQUIRE(lda >= K && lda <= kMaxLd && (lda * es) % 16 == 0,
            "lda must be >= K with 16-byte aligned rows");
    REQUIRE(ldd >= N && ldd <= kMaxLd && (ldd * es) % 16 == 0,
            "ldd must be >= N with 16-byte aligned rows");
    REQUIRE(ldc >= N && ldc <= kMaxLd && (ldc * ces) % 16 == 0,
            "ldc must be >= N with 16-byte aligned rows");
    REQUIRE(stride_c >= 1 && stride_c <= kMaxLd && (stride_c * ces) % 16 == 0,
            "stride_c must be positive and keep matrices 16-byte aligned");
    REQUIRE_GROUPED_LD(lda, es, false);
    REQUIRE_GROUPED_LD(ldd, es, false);
    REQUIRE_VEC_PTR(c);
    REQUIRE_PTR(row_offsets);
    if (M > 0) {
        REQUIRE_VEC_PTR(a);
        REQUIRE_VEC_PTR(dmat);
    }
    REQUIRE(workspace == nullptr || aligned(workspace, 16), "workspace must be 16-byte aligned");
    // segments as many as planned, or as the workspace holds (a share's bytes
    // may pass 2^63: compared as a quotient)
    const int64_t fit = workspace ? (int64_t)std::min<size_t>(workspace_bytes, INT64_MAX) / 4 /
                                        ((int64_t)K * N) / E
                                  : 1;
    const bsg::GroupedPlan plan = bsg::grouped_wgrad_plan(M, K, N, E, dtype, kPlanCus, fit);
    if ((int64_t)E * ((K + plan.rows - 1) / plan.rows) * ((N + plan.cols - 1) / plan.cols) *
            plan.segments > kMaxGrid)
        return fail(BSG_EUNSUPPORTED, "too many tiles for one launch");
    bsg::GroupedParams p{};
    p.ws = (float*)workspace;
    p.nseg = plan.segments;
    p.a = a;
    p.b = dmat;
    p.row_offsets = row_offsets;
    p.c = c;
    p.lda = lda;
    p.ldb = ldd;
    p.ldc = ldc;
    p.stride_b = stride_c;
    p.M = M;
    p.K = K;
    p.N = N;
    p.E = E;
    p.tile_rows = plan.rows;
    p.tile_cols = plan.cols;
    return hip_status(bsg::launch_grouped_wgrad(p, c_dtype, dtype, (hipStream_t)stream),
                      "grouped_wgrad");
}

// --------------------------------------------------------------- clipping

size_t bsg_grad_norm_workspace_bytes(void) { return bsg::kClipBlocks * sizeof(double); }

static bsg_status check_grads(const void* const* grads, const int64_t* counts, const int* dtypes,
                              int n, const char* what) {
    REQUIRE(n >= 0 && n <= (1 << 20), "n must be in [0, 2^20]");
    REQUIRE(n == 0 || (grads && counts && dtypes), "%s, counts and dtypes must not be NULL", what);
    for (int i = 0; i < n; ++i) {
        REQUIRE(dtype_ok(dtypes[i]), "tensor %d: unknown dtype %d", i, dtypes[i]);
        REQUIRE(counts[i] >= 0 && counts[i] <= kMaxLd, "tensor %d: bad size", i);
        REQUIRE(counts[i] == 0 || (grads[i] && aligned(grads[i], elt_bytes(dtypes[i]))),
                "%s[%d] must be a non-null device pointer aligned to its values", what, i);
    }
    return BSG_OK;
}

bsg_status bsg_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes,
                         int n, float* norm, void* workspace, size_t workspace_bytes,
                         bsg_stream_t stream) {
    const bsg_status s = check_grads(grads, counts, dtypes, n, "grads");
    if (s != BSG_OK) return s;
    REQUIRE_PTR(norm);
    REQUIRE_VEC_PTR(workspace);
    REQUIRE(workspace_bytes >= bsg_grad_norm_workspace_bytes(), "workspace too small (%zu < %zu)",
            workspace_bytes, bsg_grad_norm_workspace_bytes());
    return hip_status(bsg::launch_grad_norm(grads, counts, dtypes, n, norm, (double*)workspace,
                                            (hipStream_t)stream),
                      "grad_norm");
}

bsg_status bsg_grad_clip(void* const* grads, void* const* out, const int64_t* counts,
                         const int* dtypes, int n, const float* norm, float max_norm,
                         bsg_stream_t stream) {
    bsg_status s = check_grads(grads, counts, dtypes, n, "grads");
    if (s == BSG_OK && out) s = check_grads(out, counts, dtypes, n, "out");
    if (s != BSG_OK) return s;
    REQUIRE_PTR(norm);
    REQUIRE(max_norm >= 0.0f, "max_norm must be >= 0");
    // what is written overlaps nothing else, the norm included, which every
    // workgroup reads: ranges sorted by address, an input that is its own
    // output counted once
    struct Range {
        uintptr_t lo, hi;
        bool written;
    };
    Range* r = new (std::nothrow) Range[2 * (size_t)n + 1];
    REQUIRE(r != nullptr, "out of host memory");
    size_t m = 0;
    r[m++] = Range{(uintptr_t)norm, (uintptr_t)norm + sizeof(float), false};
    for (int i = 0; i < n; ++i) {
        if (counts[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)counts[i] * elt_bytes(dtypes[i]);
        const uintptr_t in = (uintptr_t)grads[i], to = out ? (uintptr_t)out[i] : in;
        r[m++] = Range{to, to + bytes, true};
        if (to != in) r[m++] = Range{in, in + bytes, false};
    }
    std::sort(r, r + m, [](const Range& x, const Range& y) { return x.lo < y.lo; });
    bool apart = true;
    uintptr_t end = 0, written_end = 0;  // furthest end of any range, of any written one
    for (size_t i = 0; i < m && apart; ++i) {
        apart = r[i].lo >= (r[i].written ? end : written_end);
        end = std::max(end, r[i].hi);
        if (r[i].written) written_end = std::max(written_end, r[i].hi);
    }
    delete[] r;
    REQUIRE(apart, "a tensor that is written overlaps the norm or another one of the call");
    return hip_status(bsg::launch_grad_clip(grads, out, counts, dtypes, n, norm, max_norm,
                                            (hipStream_t)stream),
                      "grad_clip");
}

}  // extern "C"
