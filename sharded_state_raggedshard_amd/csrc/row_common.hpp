// Device helpers shared by the kernels over rows of logits (objectives,
// router balance): 16-byte pieces of bf16 or binary32 rows, the fast
// exponential, fixed-order workgroup sums and the search for a row's sequence.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

namespace rs {
namespace rows {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any element's address (global accesses need no alignment on
// gfx950; an odd row length leaves rows at any element)
typedef u32x4 u32x4_any __attribute__((aligned(2), may_alias));

constexpr float kNegInf = -__builtin_inff();

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void open(const u32x4& v, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ u32x4 close(const float (&x)[8]) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 p = {x[2 * i], x[2 * i + 1]};
            v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
        }
        return v;
    }
    static __device__ __forceinline__ u32x4 lowest() {  // -inf
        return u32x4{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
    }
    static __device__ __forceinline__ float one(uint16_t h) {
        return __uint_as_float((uint32_t)h << 16);
    }
    static __device__ __forceinline__ uint16_t pack(float x) {
        const f32x2 p = {x, 0.0f};
        return (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
    }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void open(const u32x4& v, float (&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
    }
    static __device__ __forceinline__ u32x4 close(const float (&x)[4]) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(x[i]);
        return v;
    }
    static __device__ __forceinline__ u32x4 lowest() {  // -inf
        return u32x4{0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u};
    }
    static __device__ __forceinline__ float one(float x) { return x; }
    static __device__ __forceinline__ float pack(float x) { return x; }
};

// Data read once or written for a later kernel goes past the caches
// (non-temporal): reading 8192 x 128256 bf16 logits 373 -> 321 us.
template <typename T>
__device__ __forceinline__ u32x4 load16(const T* p) {
    return *reinterpret_cast<const u32x4_any*>(p);
}
template <typename T>
__device__ __forceinline__ u32x4 load16_once(const T* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}
template <typename T>
__device__ __forceinline__ void store16(T* p, const u32x4& v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
}

// v_exp_f32 (one ulp; results below 2^-126 count as 0)
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Sum of v over the workgroup in a fixed order; valid in thread 0.
template <int NT>
__device__ __forceinline__ double wg_sum(double v, double* lds) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < NT / 64; ++i) s += lds[i];
    __syncthreads();
    return s;
}

// Number of the entries start[1 .. n] that are <= row: the wave's 64 probes
// narrow the range [lo, hi] of the count by a factor 64 a round.
// One 64-bit min a round, and no more: with a second one the compiler took the
// first one's condition for both (s_cselect without its own compare, in a
// uniform loop), and the search returned a wrong sequence.  A change here
// needs a look at the generated loop and the tests of many short sequences.
__device__ __forceinline__ int64_t sequence_of(const int64_t* start, int64_t n, int64_t row) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t at = lo + (lane + 1) * step;
        const bool below = at <= hi && start[at] <= row;
        lo += __popcll(__ballot(below)) * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// A grid of at most this many workgroups strides over the rest (a launch
// holds fewer than 2^32 threads).
constexpr int64_t kMaxGrid = int64_t(1) << 22;

inline unsigned grid_of(int64_t items) { return (unsigned)std::min(items, kMaxGrid); }

}  // namespace rows
}  // namespace rs
