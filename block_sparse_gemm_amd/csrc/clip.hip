// The 2-norm over a list of gradients, and their scaling down to a limit:
//   norm = sqrt(sum over tensors and values of g^2),
//   g' = rd(g * (norm <= max_norm ? 1 : max_norm / norm)).
//
// Both passes are HBM-bound: one read for the norm, one read and one write
// for the scaling.  The tensors' addresses and sizes travel in the launch's
// arguments (kList tensors a launch), so nothing is copied to the device
// and a captured graph holds its own list.  The list is cut into chunks of
// kChunkVecs 16-byte vectors (16 KB, the block of the library's large copy);
// workgroup b takes the chunks b, b + grid, ...  Measured for 537M bf16
// gradients: norm 181 us (5.95 TB/s), scaling 373 us (5.76 TB/s; 408 us in
// blocks of 32 KB under 2048 workgroups).
//
// The squares are summed in fp64: a sum over 10^9 values in fp32 would lose
// digits with every order of magnitude, and a bf16 or fp32 gradient's square
// overflows fp32 from 1.8e19 on.  Each workgroup writes one partial sum, a
// second launch adds them in a fixed order: no atomics, the same bits on
// every run.
#include "common.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace bsg {

namespace {

constexpr int kClipThreads = 256;
constexpr int kList = 96;             // tensors a launch
constexpr int kUnroll = 4;            // 16-byte vectors a thread and chunk
constexpr int kChunkVecs = kClipThreads * kUnroll;

struct List {
    const void* in[kList];
    void* out[kList];
    int64_t count[kList];
    int64_t first[kList + 1];  // first chunk of each tensor
    uint8_t bf16[kList];
    int n;
};

// A tensor's vectors: `head` values before the first 16-byte boundary, then
// whole vectors, then `tail` values.  A chunk covers vectors
// [at, at + kChunkVecs) of it; the first chunk takes the head and the last
// one the tail.
struct Piece {
    const char* in;
    char* out;
    int64_t vecs;  // whole vectors of the tensor
    int64_t at;    // first vector of the chunk
    int head, tail, es;
    bool apart;  // in and out lie differently to the 16-byte boundaries
    int64_t count;
};

__host__ __device__ inline int head_of(const void* p, int64_t count, int es) {
    const int64_t h = ((16 - (int64_t)((uintptr_t)p & 15)) & 15) / es;
    return (int)(h < count ? h : count);
}

__host__ __device__ inline int64_t chunks_of(const void* p, int64_t count, int es) {
    const int64_t vecs = (count - head_of(p, count, es)) * es / 16;
    const int64_t c = (vecs + kChunkVecs - 1) / kChunkVecs;
    return c > 0 ? c : 1;  // head and tail alone make a chunk too
}

__device__ __forceinline__ Piece piece_of(const List& l, int64_t chunk) {
    int lo = 0, hi = l.n - 1;  // the last tensor whose first chunk is at or before this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (l.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    Piece p;
    p.es = l.bf16[lo] ? 2 : 4;
    p.in = (const char*)l.in[lo];
    p.out = (char*)l.out[lo];
    p.count = l.count[lo];
    p.head = head_of(p.in, p.count, p.es);
    p.vecs = (p.count - p.head) * p.es / 16;
    p.tail = (int)(p.count - p.head - p.vecs * 16 / p.es);
    p.at = (chunk - l.first[lo]) * kChunkVecs;
    p.apart = (((uintptr_t)p.in ^ (uintptr_t)p.out) & 15) != 0;
    return p;
}

__device__ __forceinline__ float value(const char* p, int es) {
    return es == 2 ? bf16_to_f32(*(const uint16_t*)p) : *(const float*)p;
}

__device__ __forceinline__ double square(uint32_t u, int es) {
    if (es == 4) {
        const double d = (double)__uint_as_float(u);
        return d * d;
    }
    // a bf16's square has 16 significant bits; its exponent may leave fp32's range
    const double a = (double)__uint_as_float(u << 16), b = (double)__uint_as_float(u & 0xffff0000u);
    return fma(a, a, b * b);
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// `add`: a further launch of the same list adds to what the earlier ones left.
__global__ __launch_bounds__(kClipThreads) void grad_squares_kernel(List l, int64_t chunks, int add,
                                                                    double* __restrict__ partial) {
    __shared__ double red[kClipThreads / kWave];
    double s = 0.0;
    for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const Piece p = piece_of(l, chunk);
        const u32x4* v = (const u32x4*)(p.in + (int64_t)p.head * p.es);
        u32x4 x[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t c = p.at + i * kClipThreads + threadIdx.x;
            x[i] = c < p.vecs ? v[c] : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s += square(x[i][j], p.es);
        if (p.at == 0 && (int)threadIdx.x < p.head) {
            const double a = value(p.in + (int64_t)threadIdx.x * p.es, p.es);
            s += a * a;
        }
        if (p.at + kChunkVecs >= p.vecs && (int)threadIdx.x < p.tail) {
            const double a = value(p.in + (p.count - p.tail + threadIdx.x) * p.es, p.es);
            s += a * a;
        }
    }
    s = wave_sum64(s);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = add ? partial[blockIdx.x] : 0.0;
#pragma unroll
        for (int i = 0; i < kClipThreads / kWave; ++i) t += red[i];
        partial[blockIdx.x] = t;
    }
}

__global__ __launch_bounds__(kClipThreads) void grad_norm_kernel(const double* __restrict__ partial,
                                                                 int n, float* __restrict__ norm) {
    __shared__ double red[kClipThreads / kWave];
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kClipBlocks / kClipThreads; ++i) {
        const int c = i * kClipThreads + threadIdx.x;
        if (c < n) s += partial[c];
    }
    s = wave_sum64(s);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
#pragma unroll
        for (int i = 0; i < kClipThreads / kWave; ++i) s += red[i];
        *norm = (float)sqrt(s);
    }
}

__global__ __launch_bounds__(kClipThreads) void grad_clip_kernel(List l, int64_t chunks,
                                                                 const float* __restrict__ norm,
                                                                 float max_norm) {
    const float nm = *norm;
    const bool keep = nm <= max_norm;  // false for NaN: the gradients become NaN with it
    const float scale = keep ? 1.0f : max_norm / nm;
    for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const Piece p = piece_of(l, chunk);
        if (keep && p.in == p.out) continue;
        // one value at a time
        auto one = [&](int64_t i) {
            const float a = value(p.in + i * p.es, p.es) * scale;
            if (p.es == 2) *(uint16_t*)(p.out + i * 2) = (uint16_t)f32_to_bf16(a);
            else *(float*)(p.out + i * 4) = a;
        };
        const int64_t off = (int64_t)p.head * p.es;
        if (p.apart) {
            const int per = 16 / p.es;
            const int64_t end = std::min<int64_t>(p.vecs, p.at + kChunkVecs) * per;
            for (int64_t i = p.at * per + threadIdx.x; i < end; i += kClipThreads) one(p.head + i);
        } else {
            const u32x4* v = (const u32x4*)(p.in + off);
            u32x4* o = (u32x4*)(p.out + off);
            u32x4 x[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int64_t c = p.at + i * kClipThreads + threadIdx.x;
                if (c < p.vecs) x[i] = v[c];
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int64_t c = p.at + i * kClipThreads + threadIdx.x;
                if (c >= p.vecs) continue;
                u32x4 y;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (p.es == 2)
                        y[j] = pack_bf16x2(__uint_as_float(x[i][j] << 16) * scale,
                                           __uint_as_float(x[i][j] & 0xffff0000u) * scale);
                    else
                        y[j] = __float_as_uint(__uint_as_float(x[i][j]) * scale);
                }
                o[c] = y;
            }
        }
        if (p.at == 0 && (int)threadIdx.x < p.head) one(threadIdx.x);
        if (p.at + kChunkVecs >= p.vecs && (int)threadIdx.x < p.tail)
            one(p.count - p.tail + threadIdx.x);
    }
}

// The next at most kList non-empty tensors of the list from `at` on.
int64_t fill(List& l, const void* const* in, void* const* out, const int64_t* counts,
             const int* dtypes, int n, int& at) {
    l.n = 0;
    int64_t chunks = 0;
    for (; at < n && l.n < kList; ++at) {
        if (counts[at] == 0) continue;
        const int es = dtypes[at] == kBf16 ? 2 : 4;
        l.in[l.n] = in[at];
        l.out[l.n] = out ? out[at] : const_cast<void*>(in[at]);
        l.count[l.n] = counts[at];
        l.bf16[l.n] = dtypes[at] == kBf16;
        l.first[l.n] = chunks;
        chunks += chunks_of(in[at], counts[at], es);
        ++l.n;
    }
    l.first[l.n] = chunks;
    return chunks;
}

}  // namespace

hipError_t launch_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes,
                            int n, float* norm, double* partial, hipStream_t stream) {
    int at = 0, used = 0, launches = 0;
    while (at < n) {
        List l;
        const int64_t chunks = fill(l, grads, nullptr, counts, dtypes, n, at);
        if (l.n == 0) break;
        // later launches add to the partial sums of the first, so they all
        // run its number of workgroups or fewer, and it the most it may use
        const int grid = launches == 0 && at < n ? kClipBlocks
                                                 : (int)std::min<int64_t>(chunks, launches ? used : kClipBlocks);
        if (launches == 0) used = grid;
        hipLaunchKernelGGL(grad_squares_kernel, dim3((unsigned)grid), dim3(kClipThreads), 0, stream,
                           l, chunks, launches > 0, partial);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ++launches;
    }
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kClipThreads), 0, stream, partial, used, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const void* const* grads, void* const* out, const int64_t* counts,
                            const int* dtypes, int n, const float* norm, float max_norm,
                            hipStream_t stream) {
    int at = 0;
    while (at < n) {
        List l;
        const int64_t chunks = fill(l, grads, out, counts, dtypes, n, at);
        if (l.n == 0) break;
        const int grid = (int)std::min<int64_t>(chunks, 65536);
        hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)grid), dim3(kClipThreads), 0, stream, l,
                           chunks, norm, max_norm);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bsg
