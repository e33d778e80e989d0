// Device helpers over the lanes of a wave, without LDS: a shuffle through it
// takes about 100 cycles, a move inside the vector unit a few.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace rs {
namespace lanes {

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// f over groups of L neighbouring lanes (f commutes and associates), in every
// lane and in a fixed order.
template <int L, typename F>
__device__ __forceinline__ float reduce(float v, F f) {
    if (L > 1) v = f(v, dpp<0xB1>(v));   // quad_perm: lane ^ 1
    if (L > 2) v = f(v, dpp<0x4E>(v));   // quad_perm: lane ^ 2
    if (L > 4) v = f(v, dpp<0x141>(v));  // mirrored halves of 8 (quads are even by now)
    if (L > 8) v = f(v, dpp<0x140>(v));  // mirrored rows of 16
    if (L > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if (L > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

template <int L>
__device__ __forceinline__ float sum(float v) {
    return reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float max(float v) {
    return reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// The same sum of binary64 values.
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}
__device__ __forceinline__ double sum64(double v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    const auto swap = [](double x, bool far) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
        const auto a = far ? __builtin_amdgcn_permlane32_swap(lo, lo, false, false)
                           : __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
        const auto b = far ? __builtin_amdgcn_permlane32_swap(hi, hi, false, false)
                           : __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        return __builtin_bit_cast(double, ((uint64_t)b[0] << 32) | a[0]) +
               __builtin_bit_cast(double, ((uint64_t)b[1] << 32) | a[1]);
    };
    v = swap(v, false);
    return swap(v, true);
}

// Sum of the lanes up to and with this one: within rows of 16, then the last
// lane of a row to the next one, and lane 31 to the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_rows(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, ROWS == 0xf);
}
__device__ __forceinline__ uint32_t sum_upto(uint32_t v) {
    v += dpp_rows<0x111, 0xf>(v);  // row_shr: 1, 2, 4, 8, zeros coming in
    v += dpp_rows<0x112, 0xf>(v);
    v += dpp_rows<0x114, 0xf>(v);
    v += dpp_rows<0x118, 0xf>(v);
    v += dpp_rows<0x142, 0xa>(v);  // row_bcast: 15, to rows 1 and 3
    v += dpp_rows<0x143, 0xc>(v);  // row_bcast: 31, to rows 2 and 3
    return v;
}

// Index of the wave in its workgroup, known to be the same in all lanes.
__device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }
__device__ __forceinline__ int lane() { return (int)(threadIdx.x & 63); }

}  // namespace lanes
}  // namespace rs
