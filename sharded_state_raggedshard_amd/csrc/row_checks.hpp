// Host checks shared by the entry points over rows of logits (objectives,
// router balance).
#pragma once
#include <hip/hip_runtime_api.h>

#include <initializer_list>
#include <string>

#include "plan.hpp"
#include "raggedshard.h"

namespace rs {
namespace rowcheck {

inline rs_status fail(rs_status st, std::string msg) { return rs::set_error(st, std::move(msg)); }

inline rs_status hip_fail(hipError_t e, const char* what) {
    return fail(RS_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t kMaxElems = int64_t(1) << 50;
// What every call over rows of logits takes (width: values of a row).
inline rs_status check_logits(const void* z, int32_t dtype, int64_t rows, int64_t width, int64_t ld,
                       const void* work) {
    if (dtype != RS_F32 && dtype != RS_BF16) return fail(RS_EINVAL, "unknown dtype");
    if (rows < 0) return fail(RS_EINVAL, "negative number of rows");
    if (ld < width) return fail(RS_EINVAL, "row stride below the row's length");
    if (rows > kMaxElems / ld) return fail(RS_EOVERFLOW, "rows * ld beyond 2^50 elements");
    if (rows > 0 && !z) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(z, dtype == RS_F32 ? 4 : 2)) return fail(RS_EINVAL, "misaligned pointer");
    if (!work) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(work, 16)) return fail(RS_EINVAL, "workspace not 16-byte aligned");
    return RS_OK;
}

// d must be z with the same stride, or share no element with it.
inline rs_status check_gradient(const void* z, const void* d, int32_t dtype, int64_t rows, int64_t width,
                         int64_t ld, int64_t ldd) {
    if (!d) return RS_OK;
    const int64_t size = dtype == RS_F32 ? 4 : 2;
    if (!aligned(d, size_t(size))) return fail(RS_EINVAL, "misaligned pointer");
    if (ldd < width) return fail(RS_EINVAL, "row stride below the row's length");
    if (rows > kMaxElems / ldd) return fail(RS_EOVERFLOW, "rows * ldd beyond 2^50 elements");
    if (rows == 0) return RS_OK;
    const uintptr_t z0 = reinterpret_cast<uintptr_t>(z), d0 = reinterpret_cast<uintptr_t>(d);
    const uintptr_t z1 = z0 + uintptr_t(((rows - 1) * ld + width) * size);
    const uintptr_t d1 = d0 + uintptr_t(((rows - 1) * ldd + width) * size);
    if (d1 <= z0 || z1 <= d0) return RS_OK;
    if (ld == ldd && d0 == z0) return RS_OK;
    if (ld == ldd) {  // columns of one array, side by side
        const uintptr_t step = uintptr_t(ld * size), row = uintptr_t(width * size);
        const uintptr_t off = d0 >= z0 ? (d0 - z0) % step : (step - (z0 - d0) % step) % step;
        if (off >= row && off + row <= step) return RS_OK;
    }
    return fail(RS_EINVAL, "the gradient overlaps the logits without being them");
}

// An array of n binary32 values; NULL takes no room.
struct Floats {
    const float* p;
    int64_t n;
};

// out must share no value with any of the others: a workgroup may write it
// while another still reads them.
inline rs_status check_apart(Floats out, std::initializer_list<Floats> others) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p), a1 = a + uintptr_t(out.n) * 4;
    for (const Floats& o : others) {
        const uintptr_t b = reinterpret_cast<uintptr_t>(o.p), b1 = b + uintptr_t(o.n) * 4;
        if (out.p && o.p && a < b1 && b < a1)
            return fail(RS_EINVAL, "an output overlaps another array");
    }
    return RS_OK;
}

}  // namespace rowcheck
}  // namespace rs
