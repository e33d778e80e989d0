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

// Adds rows [lo, hi) to hist (experts words) and *live, both in LDS; a thread
// a row.
template <int NT>
__device__ __forceinline__ void count_rows(const RouterBalance& a, int64_t lo, int64_t hi,
                                           int32_t* hist, int32_t* live) {
    int n = 0;
    for (int64_t row = lo + threadIdx.x; row < hi; row += NT) {
        if (a.mask && !a.mask[row]) continue;
        ++n;
        const int64_t* ids = a.topk + row * a.ldk;
        for (int j = 0; j < a.k; j += 8) {  // eight loads in flight
            int64_t e[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) e[u] = j + u < a.k ? ids[j + u] : -1;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (e[u] >= 0 && e[u] < a.experts) atomicAdd(&hist[e[u]], 1);
        }
    }
    if (n) atomicAdd(live, n);
}

// Counts of a chunk of rows: a histogram in LDS per sequence, added to the
// outputs with integer atomics (whole numbers: their order does not matter).
constexpr int kCountThreads = 512;
__global__ __launch_bounds__(kCountThreads) void router_count_kernel(RouterBalance a, int64_t per) {
    __shared__ int32_t hist[kMaxExperts];
    __shared__ int32_t live;
    const int tid = threadIdx.x;
    const int64_t r0 = blockIdx.x * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
    for (int64_t s = seq_of(a, r0); s < a.n_seq; ++s) {
        int64_t lo, hi;
        clip_rows(a, s, r0, r1, lo, hi);
        if (seq_begin(a, s) >= r1) break;
        if (lo >= hi) continue;
        for (int e = tid; e < a.experts; e += kCountThreads) hist[e] = 0;
        if (tid == 0) live = 0;
        __syncthreads();
        count_rows<kCountThreads>(a, lo, hi, hist, &live);
        __syncthreads();
        for (int e = tid; e < a.experts; e += kCountThreads)
            if (hist[e]) atomicAdd(&a.counts[s * a.experts + e], hist[e]);
        if (tid == 0 && live) atomicAdd(&a.tokens[s], live);
        __syncthreads();
    }
}

// The same for short sequences, straight to the outputs: a thread a row.
// Needs a.start.
__global__ __launch_bounds__(kThreads) void router_count_short_kernel(RouterBalance a) {
    const int64_t row = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    if (row >= a.rows || (a.mask && !a.mask[row])) return;
    int64_t s = 0;  // number of entries start[1 .. n_seq] that are <= row
    for (int64_t n = a.n_seq; n > 0;) {
        const int64_t half = (n + 1) / 2;
        if (a.start[s + half] <= row) {
            s += half;
            n -= half;
        } else {
            n = half - 1;
        }
    }
    if (s >= a.n_seq || a.start[0] > row) return;
    atomicAdd(&a.tokens[s], 1);
    for (int j = 0; j < a.k; ++j) {
        const int64_t e = a.topk[row * a.ldk + j];
        if (e >= 0 && e < a.experts) atomicAdd(&a.counts[s * a.experts + e], 1);
    }
}

// Sum over groups of L neighbouring lanes, in every lane: cross-lane moves
// inside the vector unit (a shuffle through LDS takes about 100 cycles).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    if (L > 1) v += dpp<0xB1>(v);   // quad_perm: lane ^ 1
    if (L > 2) v += dpp<0x4E>(v);   // quad_perm: lane ^ 2
    if (L > 4) v += dpp<0x141>(v);  // mirrored halves of 8 (quads are even by now)
    if (L > 8) v += dpp<0x140>(v);  // mirrored rows of 16
    if (L > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (L > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

// A lane's columns of a row: C values, 16-byte pieces L lanes apart.  FULL:
// the experts fill whole pieces.
template <typename T, int L, int NV, bool FULL>
struct Lane {
    static constexpr int N = Vec<T>::n, C = N * NV, GROUPS = kThreads / L;

    static __device__ __forceinline__ int column(int lane, int i) {
        return ((i / N) * L + lane) * N + i % N;
    }

    // z: the lane's first column
    static __device__ __forceinline__ void load(const T* z, int lane, int experts, u32x4 (&w)[NV]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int e0 = (v * L + lane) * N;
            w[v] = Vec<T>::lowest();
            if (e0 + N <= experts) {
                w[v] = load16_once(z + v * L * N);
            } else if (!FULL && e0 < experts) {  // the last columns, one by one
                float y[N];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    y[i] = e0 + i < experts ? Vec<T>::one(z[v * L * N + i]) : kNegInf;
                w[v] = Vec<T>::close(y);
            }
        }
    }

    static __device__ __forceinline__ void store(T* d, int lane, int experts, const float (&x)[C]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int e0 = (v * L + lane) * N;
            float y[N];
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = x[v * N + i];
            if (e0 + N <= experts) {
                store16(d + v * L * N, Vec<T>::close(y));
            } else if (!FULL) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (e0 + i < experts) d[v * L * N + i] = Vec<T>::pack(y[i]);
            }
        }
    }
};

// What a sequence's rows share.
struct Shared {
    double n;        // tokens
    double pull;     // balance_coef f_e / n of one count of e
    float c2;        // 2 z_coef / n
    __device__ __forceinline__ Shared(const RouterBalance& a, int32_t tokens) {
        n = (double)max(tokens, 1);
        pull = a.balance_coef / n * (a.experts / (a.k * n));
        c2 = (float)(2.0 * a.z_coef / n);
    }
};

struct Losses {
    double balance = 0.0, squares = 0.0;
};

// One row by a group of lanes: its values x become its gradient's and its
// shares are added to acc.  g = balance_coef f / n, so that sum g p is the
// row's part of the loss and a gradient value slope (g - sum g p).
//
// The exponentials take no shift first: a sum in (2^-10, 2^20) keeps the
// values that matter within +-14 of 0, where x log2(e) is rounded by less
// than 2^-20 (giving that back as a factor 1 + r costs 1 to 3 % of ordinary
// softmax batches and 14 % of 2^24 x 8: dropped).  If a row of the wave is
// out of that, or masked, the wave takes its rows again, with selects, and
// those out of it around their maximum.  (A sum of sigmoids is out of it
// below 2^-10 only, where every x < -6.9.)
template <int L, int C, bool SIGMOID>
__device__ __forceinline__ void balance_row(float (&x)[C], const float (&g)[C], float (&acc)[C],
                                            bool live, float c2, Losses& loss) {
    float p[C], u[C];
    float sum = 0.0f, gs = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (SIGMOID) {
            u[i] = exp2_fast(x[i] * -kLog2e);
            p[i] = __builtin_amdgcn_rcpf(1.0f + u[i]);
        } else {
            p[i] = exp2_fast(x[i] * kLog2e);
        }
        sum += p[i];
        gs = __builtin_fmaf(g[i], p[i], gs);
    }
    sum = group_sum<L>(sum);
    gs = group_sum<L>(gs);
    if (!__any(!live || !(sum > 0x1p-10f && sum < 0x1p20f))) {
        const float inv = __builtin_amdgcn_rcpf(sum), dot = gs * inv;
        float zc = 0.0f;
        if (!SIGMOID && c2 != 0.0f) {
            const float lse = logf(sum);
            loss.squares += (double)lse * (double)lse;
            zc = c2 * lse;
        }
        loss.balance += (double)dot;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float q = p[i] * inv;
            acc[i] += q;
            // 1 - s(x) = u s(x); u held finite where s(x) is 0 (a NaN is in q)
            x[i] = SIGMOID ? q * (fminf(u[i], 0x1p126f) * p[i] * (g[i] - dot))
                           : q * (g[i] - dot + zc);
        }
        return;
    }
    float m = x[0], shift = 0.0f, w[C];
#pragma unroll
    for (int i = 1; i < C; ++i) m = fmaxf(m, x[i]);
    m = group_max<L>(m);
    const bool ordinary = sum > 0x1p-10f && sum < 0x1p20f;  // the same bits as above
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (SIGMOID)
            w[i] = ordinary ? fminf(u[i], 0x1p126f) * p[i]
                   : x[i] > 0.0f ? u[i] * p[i] : 1.0f - p[i];
    if (!ordinary) {
        shift = m == kNegInf ? 0.0f : m;
        sum = gs = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            p[i] = exp2_fast((x[i] - shift) * kLog2e);
            // s(x) = e^x (1 - s(x)): a softmax's share alone would be off by
            // s(x) of itself, up to 2^-10 here
            if (SIGMOID) p[i] *= w[i];
            sum += p[i];
            gs = __builtin_fmaf(g[i], p[i], gs);
        }
        sum = group_sum<L>(sum);
        gs = group_sum<L>(gs);
    }
    const bool part = live && sum != 0.0f;  // 0: nothing but -inf
    const float inv = part ? __builtin_amdgcn_rcpf(sum) : 0.0f, dot = part ? gs * inv : 0.0f;
    float zc = 0.0f;
    if (!SIGMOID && c2 != 0.0f && part) {
        const float lse = shift + logf(sum);
        loss.squares += (double)lse * (double)lse;
        zc = c2 * lse;
    }
    loss.balance += (double)dot;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const float q = part ? p[i] * inv : 0.0f;
        acc[i] += q;
        const float slope = SIGMOID ? q * (w[i] * (g[i] - dot)) : q * (g[i] - dot + zc);
        x[i] = part ? slope : 0.0f;
    }
}

// A group's rows of [lo, hi): each group keeps the loads of its next rows in
// flight.
template <typename T, int L, int NV, bool FULL>
struct RowsAhead {
    using Ln = Lane<T, L, NV, FULL>;
    static constexpr int DEPTH = NV == 1 ? 2 : 1;
    u32x4 w[DEPTH][NV];
    uint32_t live[DEPTH];
    int64_t row, hi;
    const T* z;  // DEPTH rows ahead

    __device__ __forceinline__ void load(const RouterBalance& a, int lane, int u, int64_t r) {
        live[u] = 1;
        if (r >= hi) return;
        Ln::load(z, lane, a.experts, w[u]);
        if (a.mask) live[u] = a.mask[r];
    }
    __device__ __forceinline__ RowsAhead(const RouterBalance& a, int64_t lo, int64_t hi) : hi(hi) {
        const int lane = threadIdx.x % L;
        row = lo + threadIdx.x / L;
        z = static_cast<const T*>(a.z) + row * a.ld + lane * Ln::N;
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            load(a, lane, u, row + u * Ln::GROUPS);
            z += Ln::GROUPS * a.ld;
        }
    }
};

// The rows of one sequence by one workgroup: gradients, and the sums of
// their shares in sums[wave][column] (a barrier follows).  Bound by the
// vector unit: a sigmoid value costs two transcendental and 13 other
// instructions, 67% of the issue slots of 262144 x 256 (66 us, 4.1 TB/s).
template <typename T, int L, int NV, bool SIGMOID, bool FULL>
__device__ __forceinline__ void balance_rows(const RouterBalance& a, RowsAhead<T, L, NV, FULL>& rows,
                                             const int32_t* counts, const Shared& sh,
                                             float (*sums)[L * Vec<T>::n * NV], Losses& loss) {
    using Ln = Lane<T, L, NV, FULL>;
    constexpr int N = Ln::N, C = Ln::C, GROUPS = Ln::GROUPS, DEPTH = RowsAhead<T, L, NV, FULL>::DEPTH;
    const int tid = threadIdx.x, lane = tid % L;
    float g[C], acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = Ln::column(lane, i);
        g[i] = e < a.experts ? (float)(sh.pull * counts[e]) : 0.0f;
        acc[i] = 0.0f;
    }
    T* d = static_cast<T*>(a.d) + rows.row * a.ldd + lane * N;
    while (rows.row < rows.hi) {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            if (rows.row >= rows.hi) break;
            float x[C];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float y[N];
                Vec<T>::open(rows.w[u][v], y);
#pragma unroll
                for (int i = 0; i < N; ++i) x[v * N + i] = y[i];
            }
            const bool on = rows.live[u] != 0;
            rows.load(a, lane, u, rows.row + DEPTH * GROUPS);
            balance_row<L, C, SIGMOID>(x, g, acc, on, sh.c2, loss);
            if (a.d) Ln::store(d, lane, a.experts, x);
            rows.row += GROUPS;
            rows.z += GROUPS * a.ld;
            d += GROUPS * a.ldd;
        }
    }
    // the wave's groups
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
        for (int off = L; off < 64; off <<= 1) acc[i] += __shfl_xor(acc[i], off, 64);
        if ((tid & 63) < L) sums[tid >> 6][Ln::column(lane, i)] = acc[i];
    }
    __syncthreads();
}

template <int W>
__device__ __forceinline__ float column_sum(const float (*sums)[W], int e) {
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < kThreads / 64; ++v) q += sums[v][e];
    return q;
}

template <typename T, int L, int NV, bool SIGMOID, bool FULL>
__global__ __launch_bounds__(kThreads, NV == 1 ? 4 : 1) void router_main_kernel(RouterBalance a, int64_t per) {
    constexpr int W = L * Vec<T>::n * NV;
    __shared__ float sums[kThreads / 64][W];
    __shared__ double red[kThreads / 64];
    const int tid = threadIdx.x;
    const int64_t r0 = blockIdx.x * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
    double balance = 0.0, zl = 0.0;
    for (int64_t s = seq_of(a, r0); s < a.n_seq; ++s) {
        int64_t lo, hi;
        clip_rows(a, s, r0, r1, lo, hi);
        if (seq_begin(a, s) >= r1) break;
        if (lo >= hi) continue;
        RowsAhead<T, L, NV, FULL> rows(a, lo, hi);
        const Shared sh(a, a.tokens[s]);
        Losses part;
        balance_rows<T, L, NV, SIGMOID, FULL>(a, rows, a.counts + s * a.experts, sh, sums, part);
        float* slot = a.part + (blockIdx.x + s) * a.experts;
        for (int e = tid; e < a.experts; e += kThreads) slot[e] = column_sum(sums, e);
        __syncthreads();
        if (tid % L == 0) {
            balance += part.balance;
            zl += a.z_coef * part.squares / sh.n;
        }
    }
    balance = wg_sum<kThreads>(balance, red);
    zl = wg_sum<kThreads>(zl, red);
    if (tid == 0) {
        a.loss[2 * blockIdx.x] = balance;
        a.loss[2 * blockIdx.x + 1] = zl;
    }
}

// Average rows of a sequence below which rows are counted without LDS.
constexpr int64_t kShort = 256;

// Everything by one workgroup, for batches where the launches would take
// longer than the work.
template <typename T, int L, int NV, bool SIGMOID, bool FULL>
__global__ __launch_bounds__(kThreads) void router_small_kernel(RouterBalance a) {
    constexpr int W = L * Vec<T>::n * NV;
    __shared__ float sums[kThreads / 64][W];
    __shared__ double red[kThreads / 64];
    __shared__ int32_t hist[kMaxExperts];
    __shared__ int32_t live;
    const int tid = threadIdx.x;
    double balance = 0.0, zl = 0.0;
    for (int64_t s = 0; s < a.n_seq; ++s) {
        int64_t lo, hi;
        clip_rows(a, s, 0, a.rows, lo, hi);
        RowsAhead<T, L, NV, FULL> rows(a, lo, hi);
        for (int e = tid; e < a.experts; e += kThreads) hist[e] = 0;
        if (tid == 0) live = 0;
        __syncthreads();
        count_rows<kThreads>(a, lo, hi, hist, &live);
        __syncthreads();
        const Shared sh(a, live);
        Losses part;
        balance_rows<T, L, NV, SIGMOID, FULL>(a, rows, hist, sh, sums, part);
        for (int e = tid; e < a.experts; e += kThreads) {
            a.counts[s * a.experts + e] = hist[e];
            a.mean_prob[s * a.experts + e] = (float)((double)column_sum(sums, e) / sh.n);
        }
        __syncthreads();
        if (tid % L == 0) {
            balance += part.balance;
            zl += a.z_coef * part.squares / sh.n;
        }
    }
    balance = wg_sum<kThreads>(balance, red);
    zl = wg_sum<kThreads>(zl, red);
    if (tid == 0) {
        a.stats[0] = (float)balance;
        a.stats[1] = (float)zl;
    }
}

// Workgroup (s, b): mean probabilities of `columns` (a power of two) columns
// of a sequence; the last workgroup: the losses.
template <int NT>
__global__ __launch_bounds__(NT) void router_finish_kernel(RouterBalance a, int64_t chunks,
                                                             int64_t per, int64_t blocks,
                                                             int columns) {
    __shared__ double lds[NT];
    const int tid = threadIdx.x;
    if (blockIdx.x == a.n_seq * blocks) {
        for (int i = 0; i < 2; ++i) {
            double v = 0.0;
            for (int64_t c = tid; c < chunks; c += NT) v += a.loss[2 * c + i];
            v = wg_sum<NT>(v, lds);
            if (tid == 0) a.stats[i] = (float)v;
        }
        return;
    }
    const int64_t s = blockIdx.x / blocks;
    const int lanes = NT / columns;
    const int e = (int)(blockIdx.x - s * blocks) * columns + tid % columns;
    int64_t lo, hi;
    clip_rows(a, s, 0, a.rows, lo, hi);
    double v = 0.0;
    if (lo < hi && e < a.experts) {
        const int64_t c1 = (hi - 1) / per;
        for (int64_t c = lo / per + tid / columns; c <= c1; c += 8 * lanes) {
            float q[8];  // eight loads in flight
#pragma unroll
            for (int u = 0; u < 8; ++u)
                q[u] = c + u * lanes <= c1 ? a.part[(c + u * lanes + s) * a.experts + e] : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += (double)q[u];
        }
    }
    lds[tid] = v;
    __syncthreads();
    if (tid < columns && e < a.experts) {
        double t = 0.0;
        for (int i = 0; i < lanes; ++i) t += lds[i * columns + tid];
        a.mean_prob[s * a.experts + e] = (float)(t / (double)max(a.tokens[s], 1));
    }
}

// Lanes that share a row (16 bytes each, up to 4 times for the widest rows).
int lanes_of(int pieces) {
    int l = 4;
    while (l < pieces) l *= 2;
    return l;
}

// Rows of a chunk: a group of lanes adds up at most 64 rows' shares in
// binary32 (the lanes of binary32 rows; bf16 rows take half as many), so that
// a mean's error does not grow with the rows: in chunks of one round, 2^26
// rows of two experts were off by 240 half steps.  More chunks cost little (us,
// one round / so): 2^20 x 256 bf16 244.2 / 244.5, 2^24 x 8 bf16 366 / 367,
// 2^20 x 128 binary32 in one sequence 231 / 241 (the last kernel's sums).
constexpr int kChain = 64;
int64_t most_chunk_rows(int32_t experts) {
    return kChain * (kThreads / std::min(64, lanes_of((experts + 3) / 4)));
}

// One workgroup does everything up to 16 passes over its rows (us, against
// four launches, in a graph): 96 x 32 binary32 7.3 / 13.9, 256 x 64 13.2 /
// 14.7, 128 x 128 13.4 / 15.7, 128 x 256 bf16 14.3 / 16.8; 32 passes 21 / 15.
bool small_batch(const RouterBalance& a) {
    const int n = a.f32 ? 4 : 8;
    return a.rows * lanes_of((a.experts + n - 1) / n) <= 16 * kThreads && a.n_seq <= 8;
}

template <typename T, int L, int NV, bool SIGMOID, bool FULL>
hipError_t launch_main(const RouterBalance& a, const RouterChunks& c, hipStream_t s) {
    if (small_batch(a))
        hipLaunchKernelGGL((router_small_kernel<T, L, NV, SIGMOID, FULL>), dim3(1), dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((router_main_kernel<T, L, NV, SIGMOID, FULL>), dim3((unsigned)c.n), dim3(kThreads),
                           0, s, a, c.rows);
    return hipGetLastError();
}

template <typename T, int L, int NV>
hipError_t launch_main(const RouterBalance& a, const RouterChunks& c, hipStream_t s) {
    if (a.experts % Vec<T>::n == 0)
        return a.sigmoid ? launch_main<T, L, NV, true, true>(a, c, s)
                         : launch_main<T, L, NV, false, true>(a, c, s);
    return a.sigmoid ? launch_main<T, L, NV, true, false>(a, c, s)
                     : launch_main<T, L, NV, false, false>(a, c, s);
}

template <typename T>
hipError_t launch_main(const RouterBalance& a, const RouterChunks& c, hipStream_t s) {
    switch (lanes_of((a.experts + Vec<T>::n - 1) / Vec<T>::n)) {
        case 4: return launch_main<T, 4, 1>(a, c, s);
        case 8: return launch_main<T, 8, 1>(a, c, s);
        case 16: return launch_main<T, 16, 1>(a, c, s);
        case 32: return launch_main<T, 32, 1>(a, c, s);
        case 64: return launch_main<T, 64, 1>(a, c, s);
        case 128: return launch_main<T, 64, 2>(a, c, s);
        default: break;
    }
    if constexpr (sizeof(T) == 4) return launch_main<T, 64, 4>(a, c, s);  // above 512 experts
    return hipErrorInvalidValue;  // (1024 bf16 experts are 128 pieces)
}

hipError_t launch_main(const RouterBalance& a, const RouterChunks& c, hipStream_t s) {
    return a.f32 ? launch_main<float>(a, c, s) : launch_main<uint16_t>(a, c, s);
}

}  // namespace

RouterChunks router_chunks(int64_t rows, int32_t experts, int64_t n_seq) {
    // one round of the 1024 workgroups the device holds, not below 32 rows
    // each (with 16, the last kernel's sums take longer than is won), but no
    // more than a sequence: a workgroup takes its sequences one after another
    // (40 rows in 60 sequences: 114 us in two chunks)
    RouterChunks c;
    const int64_t least = std::min<int64_t>(32, std::max<int64_t>(1, rows / n_seq));
    c.rows = std::max<int64_t>(least, (rows + kRoundChunks - 1) / kRoundChunks);
    c.rows = std::min(c.rows, most_chunk_rows(experts));
    c.n = (rows + c.rows - 1) / c.rows;
    return c;
}

int64_t router_chunk_room(int64_t rows, int32_t experts) {
    const int64_t most = most_chunk_rows(experts);
    return std::max(std::min(rows, kRoundChunks), (rows + most - 1) / most);
}

hipError_t launch_router_balance(const RouterBalance& a, hipStream_t s) {
    const RouterChunks c = router_chunks(a.rows, a.experts, a.n_seq);
    if (small_batch(a)) return launch_main(a, c, s);
    const int64_t cells = a.n_seq * a.experts;
    const int64_t zero = (std::max<int64_t>(cells, a.n_seq) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(router_zero_kernel, dim3((unsigned)zero), dim3(kThreads), 0, s, a.counts,
                       cells, a.tokens, a.n_seq);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (c.n > 0) {
        if (a.start && a.rows / a.n_seq < kShort) {
            hipLaunchKernelGGL(router_count_short_kernel,
                               dim3((unsigned)((a.rows + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                               s, a);
        } else {
            const int64_t per = std::max<int64_t>(kCountThreads, (a.rows + 255) / 256);
            hipLaunchKernelGGL(router_count_kernel, dim3((unsigned)((a.rows + per - 1) / per)),
                               dim3(kCountThreads), 0, s, a, per);
        }
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        e = launch_main(a, c, s);
        if (e != hipSuccess) return e;
    }
    // few sequences: more workgroups of fewer columns (16383 x 128, one
    // sequence: 7.1 -> 5.6 us; 61 sequences of 256 experts: 4.6 -> 6.2)
    const int columns = a.n_seq < 8 ? 16 : 32;
    const int64_t blocks = (a.experts + columns - 1) / columns;
    const dim3 g((unsigned)(a.n_seq * blocks + 1));
    if (c.n >= 16 * a.n_seq)
        hipLaunchKernelGGL(router_finish_kernel<1024>, g, dim3(1024), 0, s, a, c.n, c.rows, blocks,
                           columns);
    else
        hipLaunchKernelGGL(router_finish_kernel<256>, g, dim3(256), 0, s, a, c.n, c.rows, blocks,
                           columns);
    return hipGetLastError();
}

}  // namespace rs
