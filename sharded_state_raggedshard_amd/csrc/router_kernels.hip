// Router balance loss for gfx950: per-expert counts, mean probabilities, the
// balance and z losses of packed sequences and the router logits' gradient.
//
// The gradient of a row needs its sequence's counts but not its mean
// probabilities, so the counts come first (from the expert ids alone) and
// the logits are read once.  A workgroup takes a chunk of consecutive rows;
// L lanes share a row (16 bytes a lane), keep their columns' probability
// sums in registers, and the workgroup writes them once per sequence its
// chunk touches, into slot chunk + sequence (both only grow along the rows,
// so no two workgroups share a slot); a last kernel adds the slots in order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "raggedshard.h"
#include "router.hpp"
#include "row_common.hpp"

namespace rs {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ int64_t seq_begin(const RouterBalance& a, int64_t s) {
    return a.start ? a.start[s] : 0;
}
__device__ __forceinline__ int64_t seq_end(const RouterBalance& a, int64_t s) {
    return a.start ? a.start[s + 1] : a.rows;
}
__device__ __forceinline__ int64_t seq_of(const RouterBalance& a, int64_t row) {
    return a.start ? sequence_of(a.start, a.n_seq, row) : 0;
}
// Row bounds [lo, hi) of sequence s inside [r0, r1).
__device__ __forceinline__ void clip_rows(const RouterBalance& a, int64_t s, int64_t r0, int64_t r1,
                                          int64_t& lo, int64_t& hi) {
    const int64_t b = seq_begin(a, s), e = seq_end(a, s);
    lo = b > r0 ? b : r0;
    hi = e < r1 ? e : r1;
}

__global__ __launch_bounds__(kThreads) void router_zero_kernel(int32_t* counts, int64_t n,
                                                               int32_t* tokens, int64_t m) {
    const int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    if (i < n) counts[i] = 0;
    if (i < m) tokens[i] = 0;
}

// Counts of a chunk of rows: a histogram in LDS per sequence, added to the
// outputs with integer atomics (whole numbers: their order does not matter).
__global__ __launch_bounds__(kThreads) void router_count_kernel(RouterBalance a, int64_t per) {
    __shared__ int32_t hist[kMaxExperts];
    __shared__ int32_t live;
    const int tid = threadIdx.x;
    const int64_t r0 = blockIdx.x * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
    for (int64_t s = seq_of(a, r0); s < a.n_seq; ++s) {
        int64_t lo, hi;
        clip_rows(a, s, r0, r1, lo, hi);
        if (seq_begin(a, s) >= r1) break;
        if (lo >= hi) continue;
        for (int e = tid; e < a.experts; e += kThreads) hist[e] = 0;
        if (tid == 0) live = 0;
        __syncthreads();
        int n = 0;
        for (int64_t row = lo + tid; row < hi; row += kThreads) n += !a.mask || a.mask[row];
        if (n) atomicAdd(&live, n);
        const int64_t items = (hi - lo) * a.k;
        for (int64_t i = tid; i < items; i += kThreads) {
            const int64_t row = lo + i / a.k;
            if (a.mask && !a.mask[row]) continue;
            const int64_t e = a.topk[row * a.ldk + i % a.k];
            if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
        }
        __syncthreads();
        for (int e = tid; e < a.experts; e += kThreads)
            if (hist[e]) atomicAdd(&a.counts[s * a.experts + e], hist[e]);
        if (tid == 0 && live) atomicAdd(&a.tokens[s], live);
        __syncthreads();
    }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) v += __shfl_xor(v, off, 64);
    return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

template <typename T, int L, int NV, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void router_main_kernel(RouterBalance a, int64_t per) {
    constexpr int N = Vec<T>::n, C = N * NV, GROUPS = kThreads / L;
    __shared__ float sums[kThreads / 64][L * C];
    __shared__ double red[kThreads / 64];
    const int tid = threadIdx.x, lane = tid % L, group = tid / L;
    const int64_t r0 = blockIdx.x * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
    double balance = 0.0, zl = 0.0;
    for (int64_t s = seq_of(a, r0); s < a.n_seq; ++s) {
        int64_t lo, hi;
        clip_rows(a, s, r0, r1, lo, hi);
        if (seq_begin(a, s) >= r1) break;
        if (lo >= hi) continue;
        const double n = (double)max(a.tokens[s], 1);
        const float share = (float)(a.experts / (a.k * n));
        const float c1 = (float)(a.balance_coef / n), c2 = (float)(2.0 * a.z_coef / n);
        float f[C], acc[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = ((i / N) * L + lane) * N + i % N;
            f[i] = e < a.experts ? share * (float)a.counts[s * a.experts + e] : 0.0f;
            acc[i] = 0.0f;
        }
        double dots = 0.0, squares = 0.0;
        for (int64_t row = lo + group; row < hi; row += GROUPS) {
            const T* z = static_cast<const T*>(a.z) + row * a.ld;
            T* d = static_cast<T*>(a.d) + row * a.ldd;
            float x[C], p[C];
            const bool live = !a.mask || a.mask[row];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e0 = (v * L + lane) * N;
                float y[N];
                if (e0 + N <= a.experts) {
                    Vec<T>::open(load16(z + e0), y);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        y[i] = e0 + i < a.experts ? Vec<T>::one(z[e0 + i]) : kNegInf;
                }
#pragma unroll
                for (int i = 0; i < N; ++i) x[v * N + i] = y[i];
            }
            // without a shift first: a sum in (2^-10, 2^20) keeps the values
            // that matter within +-14 of 0, where x log2(e) is rounded by
            // less than 2^-20; any other row again around its maximum
            float w[C];  // sigmoid: 1 - s(x)
            float sum = 0.0f, fs = 0.0f, shift = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (SIGMOID) {
                    const float u = exp2_fast(-fabsf(x[i]) * kLog2e);
                    const float r = __builtin_amdgcn_rcpf(1.0f + u);
                    const bool pos = x[i] >= 0.0f;
                    p[i] = x[i] == x[i] ? (pos ? r : u * r) : x[i];
                    w[i] = pos ? u * r : r;
                } else {
                    p[i] = exp2_fast(x[i] * kLog2e);
                }
                sum += p[i];
                fs += f[i] * p[i];
            }
            sum = group_sum<L>(sum);
            fs = group_sum<L>(fs);
            if (!(sum > 0x1p-10f && sum < 0x1p20f)) {
                float m = x[0];
#pragma unroll
                for (int i = 1; i < C; ++i) m = fmaxf(m, x[i]);
                m = group_max<L>(m);
                shift = m == kNegInf ? 0.0f : m;
                sum = fs = 0.0f;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    p[i] = exp2_fast((x[i] - shift) * kLog2e);
                    sum += p[i];
                    fs += f[i] * p[i];
                }
                sum = group_sum<L>(sum);
                fs = group_sum<L>(fs);
            }
            const bool part = live && sum != 0.0f;  // 0: nothing but -inf
            const float inv = part ? 1.0f / sum : 0.0f;
            const float dot = part ? fs * inv : 0.0f;
            float zc = 0.0f;
            if (!SIGMOID && c2 != 0.0f && part) {
                const float lse = shift + logf(sum);
                squares += (double)lse * (double)lse;
                zc = c2 * lse;
            }
            dots += (double)dot;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float q = part ? p[i] * inv : 0.0f;
                acc[i] += q;
                const float slope = SIGMOID ? q * w[i] : q;
                x[i] = part ? slope * (c1 * (f[i] - dot)) + zc * q : 0.0f;
            }
            if (!a.d) continue;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e0 = (v * L + lane) * N;
                if (e0 + N <= a.experts) {
                    float y[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) y[i] = x[v * N + i];
                    store16(d + e0, Vec<T>::close(y));
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (e0 + i < a.experts) d[e0 + i] = Vec<T>::pack(x[v * N + i]);
                }
            }
        }
        // probability sums: the wave's groups, then the waves
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int off = L; off < 64; off <<= 1) acc[i] += __shfl_xor(acc[i], off, 64);
            if ((tid & 63) < L) sums[tid >> 6][((i / N) * L + lane) * N + i % N] = acc[i];
        }
        __syncthreads();
        float* slot = a.part + (blockIdx.x + s) * a.experts;
        for (int e = tid; e < a.experts; e += kThreads) {
            float q = 0.0f;
#pragma unroll
            for (int v = 0; v < kThreads / 64; ++v) q += sums[v][e];
            slot[e] = q;
        }
        __syncthreads();
        if (lane == 0) {
            balance += a.balance_coef * dots / n;
            zl += a.z_coef * squares / n;
        }
    }
    balance = wg_sum<kThreads>(balance, red);
    zl = wg_sum<kThreads>(zl, red);
    if (tid == 0) {
        a.loss[2 * blockIdx.x] = balance;
        a.loss[2 * blockIdx.x + 1] = zl;
    }
}

// Workgroup (s, b): mean probabilities of 32 columns of a sequence; the last
// workgroup: the losses.
constexpr int kColumns = 32;
__global__ __launch_bounds__(1024) void router_finish_kernel(RouterBalance a, int64_t chunks,
                                                             int64_t per, int64_t blocks) {
    __shared__ double lds[1024];
    const int tid = threadIdx.x;
    if (blockIdx.x == a.n_seq * blocks) {
        for (int i = 0; i < 2; ++i) {
            double v = 0.0;
            for (int64_t c = tid; c < chunks; c += 1024) v += a.loss[2 * c + i];
            v = wg_sum<1024>(v, lds);
            if (tid == 0) a.stats[i] = (float)v;
        }
        return;
    }
    const int64_t s = blockIdx.x / blocks;
    const int e = (int)(blockIdx.x - s * blocks) * kColumns + tid % kColumns;
    int64_t lo, hi;
    clip_rows(a, s, 0, a.rows, lo, hi);
    double v = 0.0;
    if (lo < hi && e < a.experts) {
        const int64_t c1 = (hi - 1) / per;
        for (int64_t c = lo / per + tid / kColumns; c <= c1; c += 1024 / kColumns)
            v += (double)a.part[(c + s) * a.experts + e];
    }
    lds[tid] = v;
    __syncthreads();
    if (tid < kColumns && e < a.experts) {
        double t = 0.0;
        for (int i = 0; i < 1024 / kColumns; ++i) t += lds[i * kColumns + tid];
        a.mean_prob[s * a.experts + e] = (float)(t / (double)max(a.tokens[s], 1));
    }
}

template <typename T, int L, int NV>
hipError_t launch_main(const RouterBalance& a, const RouterChunks& c, hipStream_t s) {
    if (a.sigmoid)
        hipLaunchKernelGGL((router_main_kernel<T, L, NV, true>), dim3((unsigned)c.n), dim3(kThreads), 0,
                           s, a, c.rows);
    else
        hipLaunchKernelGGL((router_main_kernel<T, L, NV, false>), dim3((unsigned)c.n), dim3(kThreads),
                           0, s, a, c.rows);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_main(const RouterBalance& a, const RouterChunks& c, hipStream_t s) {
    const int pieces = (a.experts + Vec<T>::n - 1) / Vec<T>::n;
    if (pieces <= 4) return launch_main<T, 4, 1>(a, c, s);
    if (pieces <= 8) return launch_main<T, 8, 1>(a, c, s);
    if (pieces <= 16) return launch_main<T, 16, 1>(a, c, s);
    if (pieces <= 32) return launch_main<T, 32, 1>(a, c, s);
    if (pieces <= 64) return launch_main<T, 64, 1>(a, c, s);
    if (pieces <= 128) return launch_main<T, 64, 2>(a, c, s);
    return launch_main<T, 64, 4>(a, c, s);
}

}  // namespace

RouterChunks router_chunks(int64_t rows, int32_t experts) {
    (void)experts;
    RouterChunks c;
    c.rows = std::max<int64_t>(64, (rows + 2047) / 2048);
    c.n = (rows + c.rows - 1) / c.rows;
    return c;
}

hipError_t launch_router_balance(const RouterBalance& a, hipStream_t s) {
    const RouterChunks c = router_chunks(a.rows, a.experts);
    const int64_t cells = a.n_seq * a.experts;
    const int64_t zero = (std::max<int64_t>(cells, a.n_seq) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(router_zero_kernel, dim3((unsigned)zero), dim3(kThreads), 0, s, a.counts,
                       cells, a.tokens, a.n_seq);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (c.n > 0) {
        hipLaunchKernelGGL(router_count_kernel, dim3((unsigned)c.n), dim3(kThreads), 0, s, a, c.rows);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        e = a.f32 ? launch_main<float>(a, c, s) : launch_main<uint16_t>(a, c, s);
        if (e != hipSuccess) return e;
    }
    const int64_t blocks = (a.experts + kColumns - 1) / kColumns;
    hipLaunchKernelGGL(router_finish_kernel, dim3((unsigned)(a.n_seq * blocks + 1)), dim3(1024), 0, s,
                       a, c.n, c.rows, blocks);
    return hipGetLastError();
}

}  // namespace rs
