// Root-mean-square norm in front of the experts, with the residual stream's
// addition, its output in the storage type or in e4m3 with one scale a row;
// and its gradient.
//
// Forward, row by row:  h = rd(x + r) (h = x without a residual),
//   rstd = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j rstd w_j.
// The norm is taken of h as it is stored, not of the sum before rounding,
// so that the backward, which has only the stored h, differentiates what
// the forward computed.  8 bits: s = max_j |y_j| / 448 and q_j = rne(y_j / s)
// from the unrounded fp32 y, one rounding in all.
// Backward, n_j = h_j rstd:
//   dx_j = rstd (w_j dy_j - n_j mean_i(w_i dy_i n_i)) + dh_j,
//   dw_j = sum over rows of dy_j n_j.
//
// Both are HBM-bound (at most 10 flop a value).  A row stays in registers
// between its reductions, so everything is read once and written once: a
// wave owns a row where it holds it in few registers, several waves a wider
// one.  The weight row is loaded once per wave and kept over its rows, and the
// next rows' loads are in flight while a row is worked on.  Measured
// (rotating inputs larger than the caches): forward with the residual, 8192 x
// 4096 bf16 49 us (5.4 TB/s; a large copy reaches 5.7), to e4m3 46 us, 65536 x
// 1024 103 us, four rows of 4096 3.4 us; backward with the residual's
// gradient, 65536 x 1024 102 us (5.3 TB/s), 8192 x 4096 55 us.
#include "common.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace bsg {

namespace {

template <int DT>
struct Vec;  // 16 bytes of a row: 8 bf16 or 4 fp32
template <>
struct Vec<kBf16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void to_f32(u32x4 v, float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ u32x4 of_f32(const float* f) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        return v;
    }
};
template <>
struct Vec<kF32> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void to_f32(u32x4 v, float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
    }
    static __device__ __forceinline__ u32x4 of_f32(const float* f) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
        return v;
    }
};

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, off, kWave);
        v = o > v ? o : v;
    }
    return v;
}

// Sum (or maximum) over the TPR threads of a row.  Rows of several waves
// meet in LDS: `red` holds one slot per wave of the workgroup.  Every thread
// of the workgroup takes part, whether its row exists or not.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = wave_sum(v);
    if constexpr (TPR > kWave) {
        const int wave = threadIdx.x / kWave, first = wave / (TPR / kWave) * (TPR / kWave);
        __syncthreads();  // the slots' last readers are done
        red[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / kWave; ++i) v += red[first + i];
    }
    return v;
}

// The largest |y| as a bit pattern: as integers the patterns of magnitudes
// order like the magnitudes, with infinity and then every NaN on top, so a
// NaN is kept where a floating maximum would drop it.
template <int TPR>
__device__ __forceinline__ uint32_t row_umax(uint32_t v, float* red) {
    v = wave_umax(v);
    if constexpr (TPR > kWave) {
        const int wave = threadIdx.x / kWave, first = wave / (TPR / kWave) * (TPR / kWave);
        __syncthreads();
        red[wave] = __uint_as_float(v);
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < TPR / kWave; ++i) {
            const uint32_t o = __float_as_uint(red[first + i]);
            v = o > v ? o : v;
        }
    }
    return v;
}

// Four fp32 to four e4m3 (round to nearest even; the callers' values are at
// most 448 apart from infinities and NaN, which become NaN).
__device__ __forceinline__ uint32_t pack_e4m3x4(const float* f) {
    int v = 0;
    v = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], v, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], v, true);
    return (uint32_t)v;
}

// Rows whose largest |y| is below this are all zeros in 8 bits under scale 1
// (448 / s would overflow on the way to them).
constexpr float kTinyRow = 0x1p-100f;

// TPR threads a row, NV 16-byte vectors a thread, WG threads a workgroup.
template <int DT, bool Q8, int TPR, int NV, int WG>
__global__ __launch_bounds__(WG) void rms_norm_kernel(NormParams p) {
    constexpr int VN = Vec<DT>::kN;
    constexpr int ROWS = WG / TPR;  // rows a workgroup has in hand
    __shared__ float red[WG / kWave];
    const int tr = threadIdx.x % TPR;
    const int vecs = p.d / VN;
    const int64_t esz = DT == kBf16 ? 2 : 4;
    u32x4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tr + i * TPR;
        w[i] = c < vecs ? ((const u32x4*)p.weight)[c] : u32x4{0, 0, 0, 0};
    }
    const float inv_d = 1.0f / (float)p.d;
    auto load = [&](u32x4* v, u32x4* r, int64_t base) {
        const int64_t t = base + threadIdx.x / TPR;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tr + i * TPR;
            const bool on = t < p.T && c < vecs;
            v[i] = on ? *(const u32x4*)((const char*)p.x + t * p.ldx * esz + (int64_t)c * 16)
                      : u32x4{0, 0, 0, 0};
            if (p.residual)
                r[i] = on ? *(const u32x4*)((const char*)p.residual + t * p.ldr * esz + (int64_t)c * 16)
                          : u32x4{0, 0, 0, 0};
        }
    };
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    u32x4 v[NV], r[NV], vn[NV], rn[NV];
    load(v, r, (int64_t)blockIdx.x * ROWS);
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < p.T; base += stride) {
        load(vn, rn, base + stride);  // the next rows' loads, in flight beside this row's work
        const int64_t t = base + threadIdx.x / TPR;
        const bool here = t < p.T;
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float a[VN], b[VN];
                Vec<DT>::to_f32(v[i], a);
                Vec<DT>::to_f32(r[i], b);
#pragma unroll
                for (int j = 0; j < VN; ++j) a[j] += b[j];
                v[i] = Vec<DT>::of_f32(a);
                const int c = tr + i * TPR;
                if (p.h && here && c < vecs)
                    *(u32x4*)((char*)p.h + t * p.ldh * esz + (int64_t)c * 16) = v[i];
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float a[VN];
            Vec<DT>::to_f32(v[i], a);
#pragma unroll
            for (int j = 0; j < VN; ++j) ss = fmaf(a[j], a[j], ss);
        }
        ss = row_sum<TPR>(ss, red);
        const float rstd = 1.0f / sqrtf(fmaf(ss, inv_d, p.eps));
        if (here && tr == 0 && p.rstd) p.rstd[t] = rstd;
        if constexpr (!Q8) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tr + i * TPR;
                float a[VN], g[VN];
                Vec<DT>::to_f32(v[i], a);
                Vec<DT>::to_f32(w[i], g);
#pragma unroll
                for (int j = 0; j < VN; ++j) a[j] = a[j] * rstd * g[j];
                if (here && c < vecs)
                    *(u32x4*)((char*)p.y + t * p.ldy * esz + (int64_t)c * 16) = Vec<DT>::of_f32(a);
            }
        } else {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float a[VN], g[VN];
                Vec<DT>::to_f32(v[i], a);
                Vec<DT>::to_f32(w[i], g);
                const bool on = tr + i * TPR < vecs;  // infinite rows: 0 * inf past the end
#pragma unroll
                for (int j = 0; j < VN; ++j) {
                    const uint32_t u = on ? __float_as_uint(fabsf(a[j] * rstd * g[j])) : 0u;
                    most = u > most ? u : most;
                }
            }
            const float top = __uint_as_float(row_umax<TPR>(most, red));
            const float scale = top < kTinyRow ? 1.0f : top / 448.0f;
            const float inv = 1.0f / scale;
            if (here && tr == 0) p.y_scale[t] = scale;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tr + i * TPR;
                float a[VN], g[VN];
                Vec<DT>::to_f32(v[i], a);
                Vec<DT>::to_f32(w[i], g);
#pragma unroll
                for (int j = 0; j < VN; ++j) a[j] = a[j] * rstd * g[j] * inv;
                if (here && c < vecs) {
                    char* dst = (char*)p.y + t * p.ldy + (int64_t)c * VN;
                    if constexpr (VN == 8)
                        *(u32x2*)dst = u32x2{pack_e4m3x4(a), pack_e4m3x4(a + 4)};
                    else
                        *(uint32_t*)dst = pack_e4m3x4(a);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = vn[i], r[i] = rn[i];
    }
}

// The gradient: 512 threads a workgroup, 512 / TPR rows in hand, the next
// rows' loads in flight while these are worked on.  Each thread sums its
// columns' dw over all its rows; at the end the workgroup's rows join in LDS in
// a fixed order and the partial row goes to the workspace, which a second
// launch sums over the workgroups: no atomics, so the sums are the same on
// every run.
constexpr int kBwdThreads = 512;

template <int DT, int TPR, int NV>
__global__ __launch_bounds__(kBwdThreads) void rms_norm_backward_kernel(NormParams p) {
    constexpr int VN = Vec<DT>::kN;
    constexpr int ROWS = kBwdThreads / TPR;
    __shared__ float red[kBwdThreads / kWave];
    __shared__ float acc[TPR * NV * VN];
    const int tr = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int vecs = p.d / VN;
    const int64_t esz = DT == kBf16 ? 2 : 4;
    u32x4 w[NV];
    float dw[NV][VN];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tr + i * TPR;
        w[i] = c < vecs ? ((const u32x4*)p.weight)[c] : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < VN; ++j) dw[i][j] = 0.0f;
    }
    const float inv_d = 1.0f / (float)p.d;
    struct Row {
        u32x4 g[NV], h[NV], e[NV];
        float rstd;
    };
    auto load = [&](Row& r, int64_t base) {
        const int64_t t = base + slot;
        const bool here = t < p.T;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tr + i * TPR;
            const bool on = here && c < vecs;
            const u32x4 zero{0, 0, 0, 0};
            r.g[i] = on ? *(const u32x4*)((const char*)p.dy + t * p.ldy * esz + (int64_t)c * 16) : zero;
            r.h[i] = on ? *(const u32x4*)((const char*)p.x + t * p.ldx * esz + (int64_t)c * 16) : zero;
            r.e[i] = zero;
            if (p.residual)
                r.e[i] = on ? *(const u32x4*)((const char*)p.residual + t * p.ldr * esz + (int64_t)c * 16)
                            : zero;
        }
        r.rstd = here ? p.rstd[t] : 0.0f;
    };
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    Row cur, nxt;
    load(cur, (int64_t)blockIdx.x * ROWS);
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < p.T; base += stride) {
        load(nxt, base + stride);  // (no row there: nothing is read)
        const int64_t t = base + slot;
        const bool here = t < p.T;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float a[VN], b[VN], k[VN];
            Vec<DT>::to_f32(cur.g[i], a);
            Vec<DT>::to_f32(cur.h[i], b);
            Vec<DT>::to_f32(w[i], k);
#pragma unroll
            for (int j = 0; j < VN; ++j) {
                const float n = b[j] * cur.rstd;
                dot = fmaf(a[j] * k[j], n, dot);
                dw[i][j] = fmaf(a[j], n, dw[i][j]);
            }
        }
        const float c1 = row_sum<TPR>(dot, red) * inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tr + i * TPR;
            float a[VN], b[VN], k[VN], x[VN];
            Vec<DT>::to_f32(cur.g[i], a);
            Vec<DT>::to_f32(cur.h[i], b);
            Vec<DT>::to_f32(w[i], k);
            Vec<DT>::to_f32(cur.e[i], x);
#pragma unroll
            for (int j = 0; j < VN; ++j)
                x[j] = fmaf(cur.rstd, fmaf(-(b[j] * cur.rstd), c1, a[j] * k[j]), x[j]);
            if (here && c < vecs)
                *(u32x4*)((char*)p.y + t * p.ldh * esz + (int64_t)c * 16) = Vec<DT>::of_f32(x);
        }
        cur = nxt;
    }
    // the workgroup's rows, slot by slot
    for (int s = 0; s < ROWS; ++s) {
        if (slot == s) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VN; ++j) {
                    float* a = &acc[(i * VN + j) * TPR + tr];
                    *a = s == 0 ? dw[i][j] : *a + dw[i][j];
                }
        }
        __syncthreads();
    }
    float* out = p.partial + (int64_t)blockIdx.x * p.d;
    for (int c = threadIdx.x; c < p.d; c += kBwdThreads) {
        const int vec = c / VN, j = c % VN;
        out[c] = acc[((vec / TPR) * VN + j) * TPR + vec % TPR];
    }
}

// dw[c] = the sum of the workgroups' partial rows: 16 columns a workgroup, its
// 64 groups of 16 lanes every 64th row, joined in LDS in group order.
__global__ __launch_bounds__(1024) void rms_norm_dw_kernel(const float* __restrict__ partial,
                                                           int rows, int d,
                                                           float* __restrict__ dw) {
    __shared__ float part[64][17];
    const int lane = threadIdx.x % 16, group = threadIdx.x / 16;
    const int c = blockIdx.x * 16 + lane;
    float s = 0.0f;
    if (c < d) {
#pragma unroll 8
        for (int r = group; r < rows; r += 64) s += partial[(int64_t)r * d + c];
    }
    part[group][lane] = s;
    __syncthreads();
    if (group == 0 && c < d) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) s += part[i][lane];
        dw[c] = s;
    }
}

template <int DT, bool Q8, int TPR, int NV, int WG>
hipError_t norm_go(const NormParams& p, hipStream_t s) {
    constexpr int ROWS = WG / TPR;
    // rows beyond 8 workgroups a compute unit are looped over
    const int64_t grid = std::min<int64_t>((p.T + ROWS - 1) / ROWS, 2048);
    hipLaunchKernelGGL((rms_norm_kernel<DT, Q8, TPR, NV, WG>), dim3((unsigned)grid), dim3(WG), 0, s, p);
    return hipGetLastError();
}

template <int DT, bool Q8>
hipError_t norm_pick(const NormParams& p, hipStream_t s) {
    const int vecs = p.d / Vec<DT>::kN;
    // a wave a row while it takes at most 4 vectors a lane (no barriers), then
    // four waves, whose loads are in flight together; 2 vectors a thread where
    // the row allows, so that 4 or more waves a SIMD stay resident
    if (vecs <= 64) return norm_go<DT, Q8, 64, 1, 256>(p, s);
    if (vecs <= 128) return norm_go<DT, Q8, 64, 2, 256>(p, s);
    if (vecs <= 256) return norm_go<DT, Q8, 64, 4, 256>(p, s);
    if (vecs <= 512) return norm_go<DT, Q8, 256, 2, 256>(p, s);
    if (vecs <= 1024) return norm_go<DT, Q8, 256, 4, 256>(p, s);
    return norm_go<DT, Q8, 1024, 2, 1024>(p, s);
}

template <int DT, int TPR, int NV>
hipError_t bwd_go(const NormParams& p, int grid, hipStream_t s) {
    hipLaunchKernelGGL((rms_norm_backward_kernel<DT, TPR, NV>), dim3((unsigned)grid),
                       dim3(kBwdThreads), 0, s, p);
    return hipGetLastError();
}

template <int DT>
hipError_t bwd_pick(const NormParams& p, int grid, hipStream_t s) {
    const int vecs = p.d / Vec<DT>::kN;
    // three rows of values and the next three stay in registers, so a wave
    // holds at most 2 vectors a lane of each (4 in the widest rows only) and wider
    // rows take more threads; 2 vectors a thread from 4 waves on: 8192 x 4096 bf16, 256 threads of 2 / 512
    // of 1, 55.3 / 57.9 us.  Loads ahead / not: 65536 x 1024 102 / 107 us, 16384 x
    // 512 15.7 / 19.4.
    if (vecs <= 64) return bwd_go<DT, 64, 1>(p, grid, s);
    if (vecs <= 128) return bwd_go<DT, 64, 2>(p, grid, s);
    if (vecs <= 256) return bwd_go<DT, 256, 1>(p, grid, s);
    if (vecs <= 512) return bwd_go<DT, 256, 2>(p, grid, s);
    if (vecs <= 1024) return bwd_go<DT, 512, 2>(p, grid, s);
    return bwd_go<DT, 512, 4>(p, grid, s);
}

// Threads that share a row in the backward, as bwd_pick chooses them.
int bwd_tpr(int dtype, int d) {
    const int vecs = d / (dtype == kBf16 ? 8 : 4);
    return vecs <= 128 ? 64 : vecs <= 512 ? 256 : 512;
}

}  // namespace

int rms_norm_backward_rows(int64_t T, int d, int dtype) {
    const int rows = kBwdThreads / bwd_tpr(dtype, d);
    return (int)std::min<int64_t>((T + rows - 1) / rows, kNormPartials);
}

hipError_t launch_rms_norm(const NormParams& p, int dtype, int q8, hipStream_t s) {
    if (dtype == kBf16) return q8 ? norm_pick<kBf16, true>(p, s) : norm_pick<kBf16, false>(p, s);
    return q8 ? norm_pick<kF32, true>(p, s) : norm_pick<kF32, false>(p, s);
}

hipError_t launch_rms_norm_backward(const NormParams& p, int dtype, float* dweight, hipStream_t s) {
    const int grid = rms_norm_backward_rows(p.T, p.d, dtype);
    if (grid > 0) {  // no rows: dw = 0
        const hipError_t e = dtype == kBf16 ? bwd_pick<kBf16>(p, grid, s) : bwd_pick<kF32>(p, grid, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(rms_norm_dw_kernel, dim3((unsigned)((p.d + 15) / 16)), dim3(1024), 0,
                       s, p.partial, grid, p.d, dweight);
    return hipGetLastError();
}

}  // namespace bsg
