// What the C ABI's sources share: the calling thread's error text, argument
// checks and the compute units of a stream's device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/bsg.h"

namespace bsg {

inline thread_local char g_err[512] = "";

inline bsg_status fail(bsg_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

inline bsg_status ok() {
    g_err[0] = '\0';
    return BSG_OK;
}

inline bsg_status hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(BSG_EHIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Bounds checked before any size is multiplied, so that validation itself
// never overflows: tokens and block rows fit int32 ids, leading dimensions
// and widths stay far below the point where a byte count would wrap.
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr int kMaxWidth = 1 << 24;

inline int elt_bytes(int dtype) { return dtype == BSG_BF16 ? 2 : 4; }

inline bool dtype_ok(int dtype) { return dtype == BSG_F32 || dtype == BSG_BF16; }

#define REQUIRE(cond, ...)                                 \
    do {                                                   \
        if (!(cond)) return fail(BSG_EINVAL, __VA_ARGS__); \
    } while (0)

// A device array read or written with 16-byte vectors.
#define REQUIRE_VEC_PTR(p) REQUIRE((p) != nullptr && aligned((p), 16), #p " must be a non-null 16-byte aligned device pointer")
// A device array of 4-byte elements.
#define REQUIRE_PTR(p) REQUIRE((p) != nullptr && aligned((p), 4), #p " must be a non-null 4-byte aligned device pointer")

// Compute units of the stream's device, looked up once per device.
hipError_t device_cus(hipStream_t stream, int* ncu);

}  // namespace bsg
