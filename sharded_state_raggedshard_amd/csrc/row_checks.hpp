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

// Bytes of an array: `rows` pieces of `bytes`, `step` apart.  A NULL pointer
// takes no room.
struct Extent {
    const void* p;
    int64_t bytes;
    int64_t rows = 1, step = 0;
};
inline Extent floats(const float* p, int64_t n) { return {p, n * 4}; }
inline Extent longs(const int64_t* p, int64_t n) { return {p, n * 8}; }
inline Extent matrix(const void* p, int64_t rows, int64_t width, int64_t ld, int64_t size) {
    return {p, width * size, rows, rows > 1 && p ? ld * size : 0};
}

// Whether two arrays share no byte; pieces of different steps, both with
// gaps, count as sharing one where their ranges meet.
inline bool apart(const Extent& x, const Extent& y) {
    if (!x.p || !y.p || x.bytes == 0 || y.bytes == 0 || x.rows == 0 || y.rows == 0) return true;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    const uintptr_t a1 = a + uintptr_t((x.rows - 1) * x.step + x.bytes);
    const uintptr_t b1 = b + uintptr_t((y.rows - 1) * y.step + y.bytes);
    if (a1 <= b || b1 <= a) return true;
    if (x.rows == 1 && y.rows == 1) return false;
    if (x.rows == 1) return apart(y, x);
    const uintptr_t step = uintptr_t(x.step);
    if (y.rows == 1 && b < a) return false;  // y reaches into x's first piece
    if (y.rows != 1 && y.step != x.step) return false;
    // y between two pieces of x, or each piece of y between two of x
    const uintptr_t off = b >= a ? (b - a) % step : (step - (a - b) % step) % step;
    return off >= uintptr_t(x.bytes) && off + uintptr_t(y.bytes) <= step;
}

// d must be z with the same stride, or share no element with it.
inline rs_status check_gradient(const void* z, const void* d, int32_t dtype, int64_t rows, int64_t width,
                         int64_t ld, int64_t ldd) {
    if (!d) return RS_OK;
    const int64_t size = dtype == RS_F32 ? 4 : 2;
    if (!aligned(d, size_t(size))) return fail(RS_EINVAL, "misaligned pointer");
    if (ldd < width) return fail(RS_EINVAL, "row stride below the row's length");
    if (rows > kMaxElems / ldd) return fail(RS_EOVERFLOW, "rows * ldd beyond 2^50 elements");
    if (d == z && ld == ldd) return RS_OK;
    if (apart(matrix(z, rows, width, ld, size), matrix(d, rows, width, ldd, size))) return RS_OK;
    return fail(RS_EINVAL, "the gradient overlaps the logits without being them");
}

// No output shares a byte with an input or another output: a workgroup may
// write it while another still reads the others.
inline rs_status check_apart(std::initializer_list<Extent> outputs, std::initializer_list<Extent> inputs) {
    for (const Extent* out = outputs.begin(); out != outputs.end(); ++out) {
        for (const Extent* other = out + 1; other != outputs.end(); ++other)
            if (!apart(*out, *other)) return fail(RS_EINVAL, "an output overlaps another array");
        for (const Extent& in : inputs)
            if (!apart(*out, in)) return fail(RS_EINVAL, "an output overlaps another array");
    }
    return RS_OK;
}

}  // namespace rowcheck
}  // namespace rs
