// Training objectives over rows of logits for gfx950: the token
// log-probability, the clipped policy loss and the preference loss with
// their logits' gradients.
//
// A row's softmax needs its maximum m and s = sum exp((z - m) / T).  A term
// is exp2((z - m) k), k = log2(e) / T in two binary32 pieces: one alone
// would shift every term the same way (up to 2^-24 |z - m| / T, so the
// row's logarithm with them), where the product's own rounding averages out.
// (Folding m into one fused multiply-add, z k - m k, saves an instruction
// but overflows on masks of the type's lowest value.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "objectives.hpp"
#include "row_common.hpp"
#include "raggedshard.h"

namespace rs {
namespace {

using namespace rows;

// What is subtracted for maximum m; 0 while nothing but -inf was seen, so
// that -inf values give exp2(-inf) = 0.
__device__ __forceinline__ float reference(float m) { return m == kNegInf ? 0.0f : m; }

__device__ __forceinline__ float term(float x, float r, ExpScale k) {
    const float d = x - r;
    return exp2_fast(__builtin_fmaf(d, k.hi, d * k.lo));
}

// Running maximum and sum.  The sum is binary64: where one term is nearly
// the whole row, as a trained model's are, a binary32 sum would round away
// the rest that 1 - p is made of.  It takes N terms at a time, added up in
// binary32.
struct Running {
    float m = kNegInf;
    double s = 0.0;

    template <int N>
    __device__ __forceinline__ void take(const float (&x)[N], ExpScale k) {
        float v = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) v = fmaxf(v, x[i]);
        const float M = fmaxf(m, v), r = reference(M);
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            a += term(x[i], r, k);
            if (i + 1 < N) b += term(x[i + 1], r, k);
        }
        s = __builtin_fma(s, (double)term(m, r, k), (double)(a + b));
        m = M;
    }

    __device__ __forceinline__ void join(float m2, double s2, ExpScale k) {
        const float M = fmaxf(m, m2), r = reference(M);
        s = s * (double)term(m, r, k) + s2 * (double)term(m2, r, k);
        m = M;
    }
};

// The Running of a whole workgroup, in a fixed order; valid in every thread.
// lds: 2 doubles per wave.
template <int NT>
__device__ __forceinline__ void wg_join(Running& x, ExpScale k, double* lds) {
    float M = x.m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    x.s *= (double)term(x.m, reference(M), k);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x.s += __shfl_xor(x.s, off, 64);
    x.m = M;
    if (NT == 64) return;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        lds[2 * wave] = x.s;
        lds[2 * wave + 1] = (double)x.m;
    }
    __syncthreads();
    M = kNegInf;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) M = fmaxf(M, (float)lds[2 * w + 1]);
    double S = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w)
        S += lds[2 * w] * (double)term((float)lds[2 * w + 1], reference(M), k);
    __syncthreads();
    x.m = M;
    x.s = S;
}

// What the statistics of a row come to.
struct RowEnd {
    float m, r;    // maximum; what the exponentials subtract
    float inv;     // 1 / sum
    double s;
    double lse_m;  // log sum exp((z - m) / T)
    bool empty;    // nothing but -inf
};

__device__ __forceinline__ RowEnd row_end(const Running& x) {
    RowEnd e;
    e.m = x.m;
    e.s = x.s;
    e.empty = x.m == kNegInf && x.s == 0.0;
    e.r = reference(x.m);
    e.inv = (float)(1.0 / x.s);
    e.lse_m = e.empty ? 0.0 : log(x.s);
    return e;
}

__device__ __forceinline__ RowEnd row_of(const LogitRows& a, int64_t row, ExpScale k) {
    const RowStat* p = a.stat + row * a.parts;
    Running x;
    x.m = p[0].m;
    x.s = p[0].s;
    for (int i = 1; i < a.parts; ++i) x.join(p[i].m, p[i].s, k);
    return row_end(x);
}

__device__ __forceinline__ double logp_of(const RowEnd& e, float token, double scale) {
    return ((double)token - (double)e.m) * scale - e.lse_m;
}

__device__ __forceinline__ bool has_token(const LogitRows& a, int64_t row) {
    const int64_t y = a.target[row];
    return y >= 0 && y < a.vocab && (!a.weight || a.weight[row] != 0.0f);
}

// --------------------------------------------------------- row statistics

enum { MARK_OUTSIDE = 0, MARK_ZERO = 1, MARK_TOKEN = 2 };

// One workgroup per part of a row: its maximum and sum in one pass, four
// 16-byte loads a thread in flight.  For the preference loss it also marks
// the rows (outside every sequence, without a token, with one).
template <typename T, int NT, bool PREF>
__global__ __launch_bounds__(NT) void row_stats_kernel(LogitRows a, PreferenceTerms t) {
    constexpr int N = Vec<T>::n, U = 4;
    __shared__ double lds[2 * (NT / 64)];
    const int tid = threadIdx.x;
    const ExpScale k = a.k;
    const int64_t items = a.rows * a.parts;
    const int64_t nv = a.vocab / N;
    const int64_t per = (nv + a.parts - 1) / a.parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / a.parts;
        const int part = (int)(item - row * a.parts);
        bool live = has_token(a, row);
        if (PREF) {
            const int64_t seq = sequence_of(t.start, 2 * t.pairs, row);
            const bool inside = seq < 2 * t.pairs && row >= t.start[0];
            if (inside && t.weight)
                live = live && t.weight[seq < t.pairs ? seq : seq - t.pairs] != 0.0f;
            live = live && inside;
            if (part == 0 && tid == 0)
                t.mark[row] = !inside ? MARK_OUTSIDE : live ? MARK_TOKEN : MARK_ZERO;
        }
        if (!live) continue;
        const T* z = static_cast<const T*>(a.z) + row * a.ld;
        Running run;
        const int64_t v0 = part * per, v1 = min(nv, v0 + per);
        int64_t v = v0 + tid;
        for (; v + (U - 1) * NT < v1; v += U * NT) {
            u32x4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = load16(z + (v + u * NT) * N);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[N];
                Vec<T>::open(w[u], x);
                run.take(x, k);
            }
        }
        for (; v < v1; v += NT) {
            float x[N];
            Vec<T>::open(load16(z + v * N), x);
            run.take(x, k);
        }
        if (part == a.parts - 1 && nv * N + tid < a.vocab) {
            const float x[1] = {Vec<T>::one(z[nv * N + tid])};
            run.take(x, k);
        }
        wg_join<NT>(run, k, lds);
        if (tid == 0) {
            a.stat[item] = RowStat{run.s, run.m, 0.0f};
            if (part == 0) a.token[row] = Vec<T>::one(z[a.target[row]]);
        }
    }
}

// --------------------------------------------------------------- token logp

__global__ __launch_bounds__(256) void logp_kernel(LogitRows a, float* logp, float* lse) {
    const ExpScale k = a.k;
    for (int64_t row = blockIdx.x * 256ll + threadIdx.x; row < a.rows; row += gridDim.x * 256ll) {
        double l = 0.0, all = 0.0;
        if (has_token(a, row)) {
            const RowEnd e = row_of(a, row, k);
            if (!e.empty) {
                l = logp_of(e, a.token[row], a.scale);
                all = (double)e.m * a.scale + e.lse_m;
            }
        }
        logp[row] = (float)l;
        if (lse) lse[row] = (float)all;
    }
}

// -------------------------------------------------------------- policy loss

struct PolicyRow {
    double logp = 0.0, coef = 0.0;  // coef: dloss / dlogp
    double pg = 0.0, kl = 0.0, clipped = 0.0;  // weighted
};

__device__ __forceinline__ PolicyRow policy_row(const LogitRows& a, const PolicyTerms& t,
                                                int64_t row, const RowEnd& e, float token) {
    PolicyRow p;
    if (e.empty) return p;
    p.logp = logp_of(e, token, a.scale);
    const double w = a.weight[row], A = t.advantage[row];
    const double r = exp(p.logp - (double)t.old_logp[row]);
    const double open = -A * r, held = -A * fmin(fmax(r, t.lo), t.hi);
    const bool clipped = open < held;
    p.pg = w * (clipped ? held : open);
    p.clipped = clipped ? w : 0.0;
    double slope = clipped ? 0.0 : open;
    if (t.ref_logp) {
        const double away = (double)t.ref_logp[row] - p.logp, q = exp(away);
        p.kl = w * (q - away - 1.0);
        slope += t.kl_coef * (1.0 - q);
    }
    p.coef = w * slope;
    return p;
}

// Per-row outputs and the loss sums, by one workgroup in a fixed order.
template <int NT>
__device__ void policy_summary(const LogitRows& a, const PolicyTerms& t, float* logp,
                               float* stats, double* lds) {
    const ExpScale k = a.k;
    double pg = 0.0, kl = 0.0, cl = 0.0;
    for (int64_t row = threadIdx.x; row < a.rows; row += NT) {
        PolicyRow p;
        if (has_token(a, row)) p = policy_row(a, t, row, row_of(a, row, k), a.token[row]);
        pg += p.pg;
        kl += p.kl;
        cl += p.clipped;
        if (logp) logp[row] = (float)p.logp;
    }
    pg = wg_sum<NT>(pg, lds);
    kl = wg_sum<NT>(kl, lds);
    cl = wg_sum<NT>(cl, lds);
    if (threadIdx.x == 0) {
        stats[0] = (float)(pg + (t.ref_logp ? t.kl_coef * kl : 0.0));
        stats[1] = (float)pg;
        stats[2] = (float)kl;
        stats[3] = (float)cl;
    }
}

// ----------------------------------------------------------- logits gradient

// Elements of a row that one workgroup of the gradient kernels writes.
constexpr int64_t kGradSpan = 16384;

// d[i] = cs ([i = token] - p_i) for the vectors [v0, v1) of a row and, with
// `tail`, the values behind the last vector.
template <typename T, int NT>
__device__ __forceinline__ void grad_span(const T* z, T* d, int64_t vocab, int64_t v0, int64_t v1,
                                          bool tail, ExpScale k, const RowEnd& e, float cs, int64_t y,
                                          float token) {
    constexpr int N = Vec<T>::n, U = 4;
    const int tid = threadIdx.x;
    const float f = -cs * e.inv;
    int64_t v = v0 + tid;
    for (; v + (U - 1) * NT < v1; v += U * NT) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = load16(z + (v + u * NT) * N);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[N];
            Vec<T>::open(w[u], x);
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = f * term(x[i], e.r, k);
            store16(d + (v + u * NT) * N, Vec<T>::close(x));
        }
    }
    for (; v < v1; v += NT) {
        float x[N];
        Vec<T>::open(load16(z + v * N), x);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = f * term(x[i], e.r, k);
        store16(d + v * N, Vec<T>::close(x));
    }
    const int64_t nv = vocab / N, last = nv * N + tid;
    if (tail && last < vocab)
        d[last] = Vec<T>::pack(f * term(Vec<T>::one(z[last]), e.r, k));
    // the token's own value, by the thread that has just written its place
    const int64_t yv = y / N;
    const bool mine = yv < nv ? yv >= v0 && yv < v1 && (yv - v0) % NT == tid
                              : tail && y - nv * N == tid;
    // (1 - p from the binary64 sum: next to p = 1 it is all that is left)
    if (mine)
        d[y] = Vec<T>::pack(cs * (float)((e.s - (double)term(token, e.r, k)) / e.s));
}

template <typename T, int NT>
__device__ __forceinline__ void zero_span(T* d, int64_t vocab, int64_t v0, int64_t v1, bool tail) {
    constexpr int N = Vec<T>::n;
    const u32x4 z = {0u, 0u, 0u, 0u};
    for (int64_t v = v0 + threadIdx.x; v < v1; v += NT) store16(d + v * N, z);
    const int64_t last = vocab / N * N + threadIdx.x;
    if (tail && last < vocab) d[last] = T(0);
}

// Workgroup 0 sums the losses; the others each write a span of a row.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void policy_grad_kernel(LogitRows a, PolicyTerms t, T* d,
                                                         int64_t ldd, int64_t spans, float* logp,
                                                         float* stats) {
    __shared__ double lds[NT / 64];
    __shared__ float coef;
    if (blockIdx.x == 0) {
        policy_summary<NT>(a, t, logp, stats, lds);
        return;
    }
    const ExpScale k = a.k;
    constexpr int N = Vec<T>::n;
    const int64_t nv = a.vocab / N, per = (nv + spans - 1) / spans;
    for (int64_t item = blockIdx.x - 1; item < a.rows * spans; item += gridDim.x - 1) {
        const int64_t row = item / spans, part = item - row * spans;
        const int64_t v0 = part * per, v1 = min(nv, v0 + per);
        T* to = d + row * ldd;
        RowEnd e;
        bool live = has_token(a, row);
        if (live) {
            e = row_of(a, row, k);
            live = !e.empty;
        }
        if (!live) {
            zero_span<T, NT>(to, a.vocab, v0, v1, part == spans - 1);
            continue;
        }
        const float token = a.token[row];
        __syncthreads();
        if (threadIdx.x == 0) coef = (float)(policy_row(a, t, row, e, token).coef * a.scale);
        __syncthreads();
        grad_span<T, NT>(static_cast<const T*>(a.z) + row * a.ld, to, a.vocab, v0, v1,
                         part == spans - 1, k, e, coef, a.target[row], token);
    }
}

// ---------------------------------------------------------- preference loss

// One workgroup per pair: its sequences' log-probabilities, its loss and
// the coefficient dloss / dlogp / T of its rows.
template <int NT>
__global__ __launch_bounds__(NT) void pair_kernel(LogitRows a, PreferenceTerms t, float* seq_logp) {
    __shared__ double lds[NT / 64];
    __shared__ double sum[2], count[2], slope;
    const ExpScale k = a.k;
    const int tid = threadIdx.x;
    const int64_t p = blockIdx.x;
    const double w = t.weight ? (double)t.weight[p] : 1.0 / (double)t.pairs;
    for (int side = 0; side < 2; ++side) {
        const int64_t q = p + side * t.pairs;
        const int64_t r0 = min(max(t.start[q], int64_t(0)), a.rows);
        const int64_t r1 = min(max(t.start[q + 1], r0), a.rows);
        double l = 0.0, n = 0.0;
        for (int64_t row = r0 + tid; row < r1; row += NT) {
            if (t.mark[row] != MARK_TOKEN) continue;
            const RowEnd e = row_of(a, row, k);
            if (e.empty) {
                t.mark[row] = MARK_ZERO;
                continue;
            }
            l += logp_of(e, a.token[row], a.scale);
            n += 1.0;
        }
        l = wg_sum<NT>(l, lds);
        n = wg_sum<NT>(n, lds);
        if (tid == 0) {
            count[side] = t.average ? fmax(n, 1.0) : 1.0;
            sum[side] = l / count[side];
            if (seq_logp) seq_logp[q] = (float)sum[side];
        }
    }
    if (tid == 0) {
        double D = sum[0] - sum[1];
        if (t.ref_logp && w != 0.0) D -= (double)t.ref_logp[p] - (double)t.ref_logp[p + t.pairs];
        const double h = t.beta * D - t.margin;
        double loss, g;  // g: dloss / dD
        if (t.kind == RS_PREF_IPO) {
            const double x = D - 0.5 / t.beta;
            loss = x * x;
            g = 2.0 * x;
        } else if (t.kind == RS_PREF_HINGE) {
            loss = h >= 1.0 ? 0.0 : 1.0 - h;  // a NaN stays one
            g = h >= 1.0 ? 0.0 : -t.beta;
        } else {
            // -log s(h) = log(1 + e^-h), stable on either side of 0
            const double soft = log1p(exp(-fabs(h)));
            const double up = soft + fmax(-h, 0.0), down = soft + fmax(h, 0.0);
            loss = t.smoothing == 0.0 ? up : (1.0 - t.smoothing) * up + t.smoothing * down;
            const double miss = h >= 0.0 ? exp(-h) / (1.0 + exp(-h)) : 1.0 / (1.0 + exp(h));
            g = t.beta * (t.smoothing - miss);
        }
        const bool out = w == 0.0;
        t.terms[3 * p] = out ? 0.0 : w * loss;
        t.terms[3 * p + 1] = out ? 0.0 : w * h;
        t.terms[3 * p + 2] = out || !(h > 0.0) ? 0.0 : w;
        slope = out ? 0.0 : w * g * a.scale;
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        const int64_t q = p + side * t.pairs;
        const int64_t r0 = min(max(t.start[q], int64_t(0)), a.rows);
        const int64_t r1 = min(max(t.start[q + 1], r0), a.rows);
        const float c = (float)((side ? -slope : slope) / count[side]);
        for (int64_t row = r0 + tid; row < r1; row += NT) t.coef[row] = c;
    }
}

template <int NT>
__device__ void preference_summary(const PreferenceTerms& t, float* stats, double* lds) {
    for (int i = 0; i < 3; ++i) {
        double x = 0.0;
        for (int64_t p = threadIdx.x; p < t.pairs; p += NT) x += t.terms[3 * p + i];
        x = wg_sum<NT>(x, lds);
        if (threadIdx.x == 0) stats[i] = (float)x;
    }
}

template <typename T, int NT>
__global__ __launch_bounds__(NT) void preference_grad_kernel(LogitRows a, PreferenceTerms t, T* d,
                                                             int64_t ldd, int64_t spans,
                                                             float* stats) {
    __shared__ double lds[NT / 64];
    if (blockIdx.x == 0) {
        preference_summary<NT>(t, stats, lds);
        return;
    }
    const ExpScale k = a.k;
    constexpr int N = Vec<T>::n;
    const int64_t nv = a.vocab / N, per = (nv + spans - 1) / spans;
    for (int64_t item = blockIdx.x - 1; item < a.rows * spans; item += gridDim.x - 1) {
        const int64_t row = item / spans, part = item - row * spans;
        const int64_t v0 = part * per, v1 = min(nv, v0 + per);
        const int mark = t.mark[row];
        if (mark == MARK_OUTSIDE) continue;
        T* to = d + row * ldd;
        if (mark == MARK_ZERO) {
            zero_span<T, NT>(to, a.vocab, v0, v1, part == spans - 1);
            continue;
        }
        const RowEnd e = row_of(a, row, k);
        grad_span<T, NT>(static_cast<const T*>(a.z) + row * a.ld, to, a.vocab, v0, v1,
                         part == spans - 1, k, e, t.coef[row], a.target[row], a.token[row]);
    }
}

// Rows up to this many values take one wave each.
constexpr int64_t kWaveRow = 2048;

template <bool PREF>
hipError_t launch_stats(const LogitRows& a, const PreferenceTerms& t, hipStream_t s) {
    const unsigned g = grid_of(a.rows * a.parts);
    if (a.vocab <= kWaveRow) {
        if (a.f32)
            hipLaunchKernelGGL((row_stats_kernel<float, 64, PREF>), dim3(g), dim3(64), 0, s, a, t);
        else
            hipLaunchKernelGGL((row_stats_kernel<uint16_t, 64, PREF>), dim3(g), dim3(64), 0, s, a, t);
    } else {
        if (a.f32)
            hipLaunchKernelGGL((row_stats_kernel<float, 256, PREF>), dim3(g), dim3(256), 0, s, a, t);
        else
            hipLaunchKernelGGL((row_stats_kernel<uint16_t, 256, PREF>), dim3(g), dim3(256), 0, s, a, t);
    }
    return hipGetLastError();
}

int64_t grad_spans(int64_t vocab) { return (vocab + kGradSpan - 1) / kGradSpan; }

}  // namespace

int32_t stat_parts(int64_t rows, int64_t vocab) {
    if (rows < 1) return 1;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(32, vocab / 4096));
    return (int32_t)std::min(most, std::max<int64_t>(1, 1024 / rows));
}

hipError_t launch_token_logp(const LogitRows& a, float* logp, float* lse, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    hipError_t e = launch_stats<false>(a, PreferenceTerms{}, s);
    if (e != hipSuccess) return e;
    const int64_t wgs = (a.rows + 255) / 256;
    hipLaunchKernelGGL(logp_kernel, dim3(grid_of(wgs)), dim3(256), 0, s, a, logp, lse);
    return hipGetLastError();
}

hipError_t launch_policy(const LogitRows& a, const PolicyTerms& t, void* d, int64_t ldd,
                         float* logp, float* stats, hipStream_t s) {
    if (a.rows > 0) {
        hipError_t e = launch_stats<false>(a, PreferenceTerms{}, s);
        if (e != hipSuccess) return e;
    }
    const int64_t spans = grad_spans(a.vocab);
    const unsigned g = 1 + (d ? grid_of(a.rows * spans) : 0);
    if (a.f32)
        hipLaunchKernelGGL((policy_grad_kernel<float, 256>), dim3(g), dim3(256), 0, s, a, t,
                           (float*)d, ldd, spans, logp, stats);
    else
        hipLaunchKernelGGL((policy_grad_kernel<uint16_t, 256>), dim3(g), dim3(256), 0, s, a, t,
                           (uint16_t*)d, ldd, spans, logp, stats);
    return hipGetLastError();
}

hipError_t launch_preference(const LogitRows& a, const PreferenceTerms& t, void* d, int64_t ldd,
                             float* seq_logp, float* stats, hipStream_t s) {
    hipError_t e;
    if (a.rows > 0) {
        e = launch_stats<true>(a, t, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((pair_kernel<256>), dim3((unsigned)t.pairs), dim3(256), 0, s, a, t, seq_logp);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t spans = grad_spans(a.vocab);
    const unsigned g = 1 + (d ? grid_of(a.rows * spans) : 0);
    if (a.f32)
        hipLaunchKernelGGL((preference_grad_kernel<float, 256>), dim3(g), dim3(256), 0, s, a, t,
                           (float*)d, ldd, spans, stats);
    else
        hipLaunchKernelGGL((preference_grad_kernel<uint16_t, 256>), dim3(g), dim3(256), 0, s, a, t,
                           (uint16_t*)d, ldd, spans, stats);
    return hipGetLastError();
}

}  // namespace rs
