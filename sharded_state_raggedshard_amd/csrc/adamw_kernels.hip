// AdamW over many tensors in one launch, for gfx950: binary32 moments, or the
// 8-bit ones of the blockwise-int8 step (one binary32 absmax per block, m as
// int8 over 127 levels, v as uint8 over 255 levels) or those with the root of v
// in its place, master parameters in binary32 (with a bf16 copy beside them
// where asked) or bf16 parameters.
//
// One workgroup takes a chunk of 4096 elements of one tensor from a work
// table.  A lane owns 16 elements: wave w covers [1024 w, 1024 (w + 1)) of the
// chunk as four slices of 256, and lane l elements 4 l .. 4 l + 3 of each, so
// every wave instruction moves one contiguous span.  Chunks of one tensor are
// independent: a quantisation block is a power of two up to the chunk, so its
// absmax never leaves the workgroup.  Every byte is read once and written
// once, past the caches; what bounds the step is HBM: 218M bf16 weights with
// binary32 moments 787 us (22 bytes each, 6.1 TB/s), 51.4M binary32 ones with a
// bf16 copy 220 us behind the norm (28 bytes, 6.5 TB/s), 14.3M with 8-bit
// moments 36 us (14 bytes, 5.5 TB/s), 51.4M of them 119 us (6.1 TB/s) and with
// the root of v in their codes 125.  Small tensors are bound by the launch and
// three loads that wait for each other (chunk, tensor, data): 65 vectors of 2048
// 4.8 us.
//
// Arithmetic: the moments follow the blockwise-int8 step's fixed binary32
// order with no FMA contraction, and the codes come from correctly rounded
// quotients, so 8-bit states equal that step's bit for bit.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "adamw.hpp"
#include "kernel_common.hpp"
#include "lanes.hpp"
#include "raggedshard.h"

namespace rs {
namespace aw {
namespace {

constexpr int NT = 256, KG = 4;  // KG slices of 4 elements a lane
static_assert(4 * KG * NT == kChunk, "a chunk is one workgroup's");

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// at the alignment of the elements: tensors are views that start anywhere
typedef u32x4 u32x4_f32 __attribute__((aligned(4), may_alias));
typedef u32x2 u32x2_bf16 __attribute__((aligned(2), may_alias));
typedef uint32_t u32_code __attribute__((aligned(1), may_alias));

// A pointer read from a table, as one to global memory (the compiler cannot
// know, and flat accesses also wait for LDS).
template <typename T>
using Global = __attribute__((address_space(1))) T*;
template <typename T, typename U>
__device__ __forceinline__ Global<T> global(U* p) {
    return (Global<T>)p;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const f32x2 p = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}

// Four elements as loaded (past the caches, or kept in them), and their values.
struct F32 {
    typedef float type;
    typedef u32x4 raw;
    static __device__ __forceinline__ raw load(const float* p) {
        return __builtin_nontemporal_load(global<const u32x4_f32>(p));
    }
    static __device__ __forceinline__ raw kept(const float* p) { return *global<const u32x4_f32>(p); }
    static __device__ __forceinline__ raw one(const float* p, int n) {
        raw r = {0u, 0u, 0u, 0u};
        for (int j = 0; j < n; ++j) r[j] = __float_as_uint(global<const float>(p)[j]);
        return r;
    }
    static __device__ __forceinline__ float get(const raw& r, int j) { return __uint_as_float(r[j]); }
    static __device__ __forceinline__ raw close(const float (&x)[4]) {
        return raw{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    }
    static __device__ __forceinline__ void store(float* p, const raw& r) {
        __builtin_nontemporal_store(r, global<u32x4_f32>(p));
    }
    static __device__ __forceinline__ void put(float* p, const raw& r, int n) {
        for (int j = 0; j < n; ++j) global<float>(p)[j] = __uint_as_float(r[j]);
    }
};
struct BF16 {
    typedef uint16_t type;
    typedef u32x2 raw;
    static __device__ __forceinline__ raw load(const uint16_t* p) {
        return __builtin_nontemporal_load(global<const u32x2_bf16>(p));
    }
    static __device__ __forceinline__ raw kept(const uint16_t* p) { return *global<const u32x2_bf16>(p); }
    static __device__ __forceinline__ raw one(const uint16_t* p, int n) {
        raw r = {0u, 0u};
        for (int j = 0; j < n; ++j) r[j >> 1] |= (uint32_t)global<const uint16_t>(p)[j] << (16 * (j & 1));
        return r;
    }
    static __device__ __forceinline__ float get(const raw& r, int j) {
        return __uint_as_float(j & 1 ? r[j >> 1] & 0xffff0000u : r[j >> 1] << 16);
    }
    static __device__ __forceinline__ raw close(const float (&x)[4]) {
        return raw{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
    }
    static __device__ __forceinline__ void store(uint16_t* p, const raw& r) {
        __builtin_nontemporal_store(r, global<u32x2_bf16>(p));
    }
    static __device__ __forceinline__ void put(uint16_t* p, const raw& r, int n) {
        for (int j = 0; j < n; ++j) global<uint16_t>(p)[j] = (uint16_t)(r[j >> 1] >> (16 * (j & 1)));
    }
};
struct Code {
    typedef uint8_t type;
    typedef uint32_t raw;
    static __device__ __forceinline__ raw load(const uint8_t* p) {
        return __builtin_nontemporal_load(global<const u32_code>(p));
    }
    static __device__ __forceinline__ raw one(const uint8_t* p, int n) {
        raw r = 0u;
        for (int j = 0; j < n; ++j) r |= (uint32_t)global<const uint8_t>(p)[j] << (8 * j);
        return r;
    }
    static __device__ __forceinline__ void store(uint8_t* p, raw r) {
        __builtin_nontemporal_store(r, global<u32_code>(p));
    }
    static __device__ __forceinline__ void put(uint8_t* p, raw r, int n) {
        for (int j = 0; j < n; ++j) global<uint8_t>(p)[j] = (uint8_t)(r >> (8 * j));
    }
};

// Elements of this lane's slice k that the chunk has: 4, fewer at its end, 0.
__device__ __forceinline__ int slice_at(int k) {
    return (threadIdx.x >> 6) * (256 * KG) + 256 * k + 4 * (threadIdx.x & 63);
}
__device__ __forceinline__ int slice_count(int k, int n) {
    const int left = n - slice_at(k);
    return left >= 4 ? 4 : left > 0 ? left : 0;
}

template <typename A>
__device__ __forceinline__ typename A::raw take(const typename A::type* p, int at, int count) {
    if (__builtin_expect(count == 4, 1)) return A::load(p + at);
    return A::one(p + at, count);
}
template <typename A>
__device__ __forceinline__ void give(typename A::type* p, int at, int count, const typename A::raw& r) {
    if (__builtin_expect(count == 4, 1))
        A::store(p + at, r);
    else
        A::put(p + at, r, count);
}

// q / 127 and q / 255, correctly rounded (every code checked).
__device__ __forceinline__ float level_m(uint32_t code) {
    return kc::ratio_fast((float)(int8_t)(uint8_t)code, 127.0f, 1.0f / 127.0f);
}
// The second moment's codes are of v / absmax, or of its square root: then an
// element is kept down to 1 / 260,000 of its block's largest instead of 1 / 510.
__device__ __forceinline__ float level_v(uint32_t code, bool root) {
    const float x = kc::ratio_fast((float)code, 255.0f, 1.0f / 255.0f);
    return root ? x * x : x;
}

// New parameters of four elements from their new moments: the hardware square
// root and reciprocal (one ulp each, the update then within 8 ulp), or
// correctly rounded operations where an update beyond 0.02, infinite or NaN
// could leave 1e-8 + 1e-6 |theta| with them, or an unusual eps asks for them.
__device__ __forceinline__ void new_params(const StepScalars& sc, const float (&th)[4], const float* m,
                                           const float* v, float (&t)[4]) {
    bool exact = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float den = (__builtin_amdgcn_sqrtf(v[j]) * sc.kappa) + sc.eps;
        const float u = sc.step_size * (m[j] * __builtin_amdgcn_rcpf(den));
        exact = exact || !(fabsf(u) <= sc.limit);
        t[j] = (th[j] * sc.c_decay) - u;
    }
    if (__builtin_expect(exact, 0)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            t[j] = (th[j] * sc.c_decay) - (sc.step_size * (m[j] / ((sqrtf(v[j]) * sc.kappa) + sc.eps)));
    }
}

// Codes of four elements of one block.  |m| <= absmax bounds them; int8 by a
// +128 offset.  A code of a square root is 0 only for 0.
template <bool ROOT>
__device__ __forceinline__ void quantise(const float* m, const float* v, float am, float av, uint32_t& qm,
                                         uint32_t& qv) {
    const float ym = kc::quant_recip(am), yv = kc::quant_recip(av);
    const bool slow_m = kc::quant_slow(am), slow_v = kc::quant_slow(av);
    qm = qv = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float rm = kc::ratio_fast(m[j], am, ym), rv = kc::ratio_fast(v[j], av, yv);
        if (__builtin_expect(slow_m, 0)) rm = m[j] / am;
        if (__builtin_expect(slow_v, 0)) rv = v[j] / av;
        qm = __builtin_amdgcn_cvt_pk_u8_f32(rintf(rm * 127.0f) + 128.0f, j, qm);
        float cv = rintf((ROOT ? sqrtf(rv) : rv) * 255.0f);
        if (ROOT && v[j] > 0.0f) cv = fmaxf(cv, 1.0f);
        qv = __builtin_amdgcn_cvt_pk_u8_f32(cv, j, qv);
    }
    qm ^= 0x80808080u;
}

// Absmax of the blocks that this lane's slices lie in, from the slices' own.
__device__ __forceinline__ void block_max(float (&am)[KG], float (&av)[KG], int log2, float (*red)[2]) {
    if (log2 > 8) {  // a block spans 2 or more slices of a wave
#pragma unroll
        for (int k = 0; k < KG; k += 2) {
            am[k] = am[k + 1] = fmaxf(am[k], am[k + 1]);
            av[k] = av[k + 1] = fmaxf(av[k], av[k + 1]);
        }
    }
    if (log2 > 9) {
        am[0] = am[2] = fmaxf(am[0], am[2]);
        av[0] = av[2] = fmaxf(av[0], av[2]);
        am[1] = am[3] = am[0];
        av[1] = av[3] = av[0];
    }
    const int lanes = log2 > 8 ? 64 : 1 << (log2 - 2);
    for (int off = 1; off < lanes; off <<= 1) {
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            am[k] = fmaxf(am[k], __shfl_xor(am[k], off, 64));
            av[k] = fmaxf(av[k], __shfl_xor(av[k], off, 64));
        }
    }
    if (log2 > 10) {  // 2 or all 4 waves of the workgroup
        const int wave = threadIdx.x >> 6, waves = 1 << (log2 - 10);
        if ((threadIdx.x & 63) == 0) {
            red[wave][0] = am[0];
            red[wave][1] = av[0];
        }
        __syncthreads();
        float x = 0.0f, y = 0.0f;
        for (int w = wave & -waves; w < (wave & -waves) + waves; ++w) {
            x = fmaxf(x, red[w][0]);
            y = fmaxf(y, red[w][1]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            am[k] = x;
            av[k] = y;
        }
    }
}

// How the moments are kept.
enum { STATE_F32, STATE_INT8, STATE_ROOT };

template <typename P, typename G, int STATE>
__device__ __forceinline__ void step_chunk(const Tensor& t, const StepScalars& sc, float s, int64_t pos, int n,
                                           float (*red)[2]) {
    constexpr bool INT8 = STATE != STATE_F32, ROOT = STATE == STATE_ROOT;
    using S = typename std::conditional<INT8, Code, F32>::type;
    typename P::type* param = static_cast<typename P::type*>(t.param) + pos;
    const typename G::type* grad = static_cast<const typename G::type*>(t.grad) + pos;
    typename S::type* m = static_cast<typename S::type*>(t.m) + pos;
    typename S::type* v = static_cast<typename S::type*>(t.v) + pos;
    typename P::raw rp[KG];
    typename G::raw rg[KG];
    typename S::raw rm[KG], rv[KG];
    float am[KG], av[KG];
#pragma unroll
    for (int k = 0; k < KG; ++k) {
        const int at = slice_at(k), count = slice_count(k, n);
        if (INT8) {
            const int64_t blk = (pos + at) >> t.block_log2;
            am[k] = count ? global<const float>(t.amax_m)[blk] : 0.0f;
            av[k] = count ? global<const float>(t.amax_v)[blk] : 0.0f;
        }
        rg[k] = take<G>(grad, at, count);
        rm[k] = take<S>(m, at, count);
        rv[k] = take<S>(v, at, count);
        rp[k] = take<P>(param, at, count);
    }
    float M[4 * KG], V[4 * KG];
#pragma unroll
    for (int k = 0; k < KG; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float mh, vh;
            if constexpr (INT8) {
                mh = level_m((rm[k] >> (8 * j)) & 0xffu) * am[k];
                vh = level_v((rv[k] >> (8 * j)) & 0xffu, ROOT) * av[k];
            } else {
                mh = F32::get(rm[k], j);
                vh = F32::get(rv[k], j);
            }
            const float g = G::get(rg[k], j) * s;
            M[4 * k + j] = (sc.beta1 * mh) + (sc.omega1 * g);
            V[4 * k + j] = (sc.beta2 * vh) + (sc.omega2 * (g * g));
        }
        if (INT8) {
            am[k] = fmaxf(fmaxf(fabsf(M[4 * k]), fabsf(M[4 * k + 1])), fmaxf(fabsf(M[4 * k + 2]), fabsf(M[4 * k + 3])));
            av[k] = fmaxf(fmaxf(V[4 * k], V[4 * k + 1]), fmaxf(V[4 * k + 2], V[4 * k + 3]));
        }
    }
#pragma unroll
    for (int k = 0; k < KG; ++k) {
        const int at = slice_at(k), count = slice_count(k, n);
        float th[4], x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) th[j] = P::get(rp[k], j);
        new_params(sc, th, M + 4 * k, V + 4 * k, x);
        give<P>(param, at, count, P::close(x));
        if (std::is_same<P, F32>::value && t.out) give<BF16>(t.out + pos, at, count, BF16::close(x));
        if constexpr (!INT8) {
            const float mk[4] = {M[4 * k], M[4 * k + 1], M[4 * k + 2], M[4 * k + 3]};
            const float vk[4] = {V[4 * k], V[4 * k + 1], V[4 * k + 2], V[4 * k + 3]};
            give<F32>(m, at, count, F32::close(mk));
            give<F32>(v, at, count, F32::close(vk));
        }
    }
    if constexpr (INT8) {
        block_max(am, av, t.block_log2, red);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            const int at = slice_at(k), count = slice_count(k, n);
            uint32_t qm, qv;
            quantise<ROOT>(M + 4 * k, V + 4 * k, am[k], av[k], qm, qv);
            give<Code>(m, at, count, qm);
            give<Code>(v, at, count, qv);
            if (count && (at & ((1 << t.block_log2) - 1)) == 0) {
                const int64_t blk = (pos + at) >> t.block_log2;
                global<float>(t.amax_m)[blk] = am[k];
                global<float>(t.amax_v)[blk] = av[k];
            }
        }
    }
}

template <int STATE>
__device__ __forceinline__ void step_types(const Tensor& t, const StepScalars& g, float s, int64_t pos, int n,
                                           float (*red)[2]) {
    switch (t.kind & (KIND_PARAM_F32 | KIND_GRAD_F32)) {
    case 0: step_chunk<BF16, BF16, STATE>(t, g, s, pos, n, red); break;
    case KIND_PARAM_F32: step_chunk<F32, BF16, STATE>(t, g, s, pos, n, red); break;
    case KIND_GRAD_F32: step_chunk<BF16, F32, STATE>(t, g, s, pos, n, red); break;
    default: step_chunk<F32, F32, STATE>(t, g, s, pos, n, red); break;
    }
}

__global__ __launch_bounds__(NT) void step_kernel(const Tensor* __restrict__ tensors,
                                                const Chunk* __restrict__ chunks, int64_t n_chunks,
                                                Scalars sc, const float* gscale) {
    __shared__ float red[NT / 64][2];
    const float s = gscale ? *gscale : 1.0f;
    for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        const Chunk ch = chunks[c];
        const Tensor t = tensors[ch.tensor];
        const int64_t pos = (int64_t)ch.index * kChunk;
        const int n = (int)(t.n - pos < kChunk ? t.n - pos : kChunk);
        const StepScalars& g = sc.group[t.group];
        if (!(t.kind & KIND_INT8))
            step_types<STATE_F32>(t, g, s, pos, n, red);
        else if (!(t.kind & KIND_ROOT))
            step_types<STATE_INT8>(t, g, s, pos, n, red);
        else
            step_types<STATE_ROOT>(t, g, s, pos, n, red);
    }
}

// ------------------------------------------------------------ global norm

// Sum over the workgroup in a fixed order; valid in thread 0.
template <int THREADS>
__device__ __forceinline__ double wg_sum(double v, double* lds) {
    v = lanes::sum64(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < THREADS / 64; ++i) s += lds[i];
    return s;
}

template <typename G>
__device__ __forceinline__ double sumsq_chunk(const Tensor& t, int64_t pos, int n) {
    const typename G::type* grad = static_cast<const typename G::type*>(t.grad) + pos;
    typename G::raw r[KG];
#pragma unroll
    for (int k = 0; k < KG; ++k) {
        const int at = slice_at(k), count = slice_count(k, n);
        r[k] = count == 4 ? G::kept(grad + at) : G::one(grad + at, count);
    }
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < KG; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double x = (double)G::get(r[k], j);
            sum = __builtin_fma(x, x, sum);
        }
    }
    return sum;
}

// Workgroup b sums the squares of chunks b, b + gridDim.x, ... in binary64 and
// leaves its sum in slot b; the grid's last workgroup adds the slots up in a
// fixed order.  (With a second launch for that, norm and step of 64 tensors of
// 4096 took 13.8 us instead of 10.9, of 100M elements the same 423.)  A slot is the sum's two halves, each in a
// 64-bit word beside the call's number, one more than the last call's, which
// every workgroup reads at its start and the last one writes back at its end:
// so a slot counts only once both words are this call's, and nothing is
// cleared in between.  Relaxed device-scope accesses pass the XCDs' L2 caches
// by; an ordered one would write them back.  The wait is for workgroups that
// wait for nobody, and bounded all the same: a call that gives up, as only
// overlapping calls on one workspace could, returns NaN and leaves a mark
// beside the number.  A workgroup of it that starts after its end takes the
// number that it left for the last call's, and its slot would pass for the next
// call's: so behind a mark every call returns NaN, until the next upload clears
// both.  (One load brings both: a second one cost 1.3 us.)
//
// What the memory-side cache keeps of the gradients is there for the step that
// follows: norm and step of 51.4M parameters 241 us instead of 254.
constexpr uint32_t kSpinLimit = 1u << 22;
__device__ __forceinline__ uint64_t slot_load(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void slot_store(uint64_t* p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void half_store(uint32_t* p, uint32_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(NT) void sumsq_kernel(const Tensor* __restrict__ tensors,
                                                 const Chunk* __restrict__ chunks, int64_t n_chunks,
                                                 uint64_t* slots, double* sumsq, double max_norm, float* scale) {
    __shared__ double lds[NT / 64];
    __shared__ uint32_t call;
    const int tid = threadIdx.x;
    uint64_t* last = slots + 2 * kSumBlocks;
    uint32_t *number = reinterpret_cast<uint32_t*>(last), *mark = number + 1;
    bool marked = false;
    if (tid == 0) {
        const uint64_t both = slot_load(last);
        call = (uint32_t)both + 1u;
        marked = both >> 32 != 0;
    }
    double sum = 0.0;
    for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        const Chunk ch = chunks[c];
        const Tensor t = tensors[ch.tensor];
        const int64_t pos = (int64_t)ch.index * kChunk;
        const int n = (int)(t.n - pos < kChunk ? t.n - pos : kChunk);
        sum += t.kind & KIND_GRAD_F32 ? sumsq_chunk<F32>(t, pos, n) : sumsq_chunk<BF16>(t, pos, n);
    }
    sum = wg_sum<NT>(sum, lds);  // its barrier also publishes `call`
    const uint64_t tag = (uint64_t)call << 32;
    if (tid == 0) {
        const uint64_t bits = __builtin_bit_cast(uint64_t, sum);
        slot_store(&slots[2 * blockIdx.x], tag | (uint32_t)bits);
        slot_store(&slots[2 * blockIdx.x + 1], tag | (bits >> 32));
    }
    if (blockIdx.x != gridDim.x - 1) return;
    __syncthreads();  // lds is free again
    double total = 0.0;
    uint32_t spins = 0;
    bool lost = false;
    for (int i = tid; i < (int)gridDim.x; i += NT) {
        uint64_t lo, hi;
        for (;;) {
            lo = slot_load(&slots[2 * i]);
            hi = slot_load(&slots[2 * i + 1]);
            if (lo >> 32 == call && hi >> 32 == call) break;
            if (++spins > kSpinLimit) {
                lost = true;
                half_store(mark, 1);
                break;
            }
            __builtin_amdgcn_s_sleep(1);
        }
        total += __builtin_bit_cast(double, (hi << 32) | (uint32_t)lo);
    }
    total = wg_sum<NT>(lost || marked ? __builtin_nan("") : total, lds);
    if (tid != 0) return;
    *sumsq = total;
    if (scale) {
        const double c = max_norm / (sqrt(total) + 1e-6);
        *scale = (float)(c < 1.0 ? c : total == total ? 1.0 : total);
    }
    half_store(number, call);
}

// ----------------------------------------------------- moments as values

// (8 elements a lane, stored as two 8-byte halves past the caches, took twice
// the time: each store then touches every other 8 bytes of its lines.)
template <typename O>
__device__ __forceinline__ void moments_chunk(const Tensor& t, int64_t pos, int n, typename O::type* out, bool second) {
    out += t.first + pos;
    const int log2 = t.block_log2;
#pragma unroll
    for (int k = 0; k < KG; ++k) {
        const int at = slice_at(k), count = slice_count(k, n);
        if (count == 0) continue;
        float x[4];
        if (t.kind & KIND_INT8) {
            const uint32_t r = take<Code>(static_cast<const uint8_t*>(second ? t.v : t.m) + pos, at, count);
            const float a = global<const float>(second ? t.amax_v : t.amax_m)[(pos + at) >> log2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t c = (r >> (8 * j)) & 0xffu;
                x[j] = (second ? level_v(c, t.kind & KIND_ROOT) : level_m(c)) * a;
            }
        } else {
            const u32x4 r = take<F32>(static_cast<const float*>(second ? t.v : t.m) + pos, at, count);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = F32::get(r, j);
        }
        give<O>(out, at, count, O::close(x));
    }
}

template <typename O>
__global__ __launch_bounds__(NT) void moments_kernel(const Tensor* __restrict__ tensors,
                                                   const Chunk* __restrict__ chunks, int64_t n_chunks,
                                                   typename O::type* m, typename O::type* v) {
    for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        const Chunk ch = chunks[c];
        const Tensor t = tensors[ch.tensor];
        const int64_t pos = (int64_t)ch.index * kChunk;
        const int n = (int)(t.n - pos < kChunk ? t.n - pos : kChunk);
        if (m) moments_chunk<O>(t, pos, n, m, false);
        if (v) moments_chunk<O>(t, pos, n, v, true);
    }
}

// A grid of at most this many workgroups strides over the rest (a launch
// holds fewer than 2^32 threads).
constexpr int64_t kMaxGrid = int64_t(1) << 22;

}  // namespace

hipError_t launch_step(const Work& w, const Scalars& sc, const float* gscale, hipStream_t s) {
    if (w.n_chunks == 0) return hipSuccess;
    hipLaunchKernelGGL(step_kernel, dim3((unsigned)std::min(w.n_chunks, kMaxGrid)), dim3(NT), 0, s, w.tensors,
                       w.chunks, w.n_chunks, sc, gscale);
    return hipGetLastError();
}

hipError_t launch_l2norm(const Work& w, uint64_t* slots, double* sumsq, double max_norm, float* scale,
                         hipStream_t s) {
    const unsigned g = (unsigned)std::max<int64_t>(1, std::min<int64_t>(w.n_chunks, kSumBlocks));
    hipLaunchKernelGGL(sumsq_kernel, dim3(g), dim3(NT), 0, s, w.tensors, w.chunks, w.n_chunks, slots, sumsq, max_norm,
                       scale);
    return hipGetLastError();
}

hipError_t launch_moments(const Work& w, void* m, void* v, bool f32, hipStream_t s) {
    if (w.n_chunks == 0 || (!m && !v)) return hipSuccess;
    const unsigned g = (unsigned)std::min(w.n_chunks, kMaxGrid);
    if (f32)
        hipLaunchKernelGGL(moments_kernel<F32>, dim3(g), dim3(NT), 0, s, w.tensors, w.chunks, w.n_chunks,
                           static_cast<float*>(m), static_cast<float*>(v));
    else
        hipLaunchKernelGGL(moments_kernel<BF16>, dim3(g), dim3(NT), 0, s, w.tensors, w.chunks, w.n_chunks,
                           static_cast<uint16_t*>(m), static_cast<uint16_t*>(v));
    return hipGetLastError();
}

}  // namespace aw
}  // namespace rs
