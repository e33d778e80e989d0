// Token statistics over rows of logits for gfx950: log-probability of the
// row's token, entropy and the most probable alternatives in one pass, and
// the logits' gradient from the gradients of both.
//
// With m the row's maximum, d_i = (z_i - m) k, k = log2(e) / T in binary32,
// e_i = 2^d_i, S = sum e and W = sum e d:
//   log p_i = ln 2 d_i - ln S,   H = -sum p log p = ln S - ln 2 W / S.
// Every quantity takes the same rounded k, a temperature off by up to 2^-24 of
// itself, which moves a log-probability by 2^-24 (|log p| + H); so one
// product gives an exponent.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lanes.hpp"
#include "row_common.hpp"
#include "token_stats.hpp"

namespace rs {
namespace {

using namespace rows;

constexpr double kLn2 = 0.69314718055994530942;
// Exponents from here on count as this: 2^kLeast is 0, and 0 times it too
// (a value of -inf has d = -inf).
constexpr float kLeast = -200.0f;

__device__ __forceinline__ float exponent(float x, float m, float k) { return (x - m) * k; }

// Maximum and sums of a thread's share of a row, a part of it or a row, the
// row's token in the maximum from the start but not in the sums (it joins
// last: where it is nearly the whole row, any sum with it would round away
// the rest that 1 - p and the entropy are made of).  `best` is the share's own
// largest value.  Sums are binary64; the C values of a call are added up in
// binary32 in four chains.
struct Sums {
    float m, best;
    double s, w;

    __device__ __forceinline__ void rescale(float M, float r, float k) {
        const float d = fmaxf(exponent(m, r, k), kLeast);
        const double f = (double)exp2_fast(d);
        w = f * __builtin_fma((double)d, s, w);
        s *= f;
        m = M;
    }

    template <int C>
    __device__ __forceinline__ void take(const float (&x)[C], float k) {
        float v = x[0];
#pragma unroll
        for (int i = 1; i < C; ++i) v = fmaxf(v, x[i]);
        best = fmaxf(best, v);
        const float M = fmaxf(m, v);
        const float r = M == kNegInf ? 0.0f : M;  // -inf - 0 gives 2^-inf = 0
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float d = exponent(x[i], r, k), e = exp2_fast(d);
            a[i % 4] += e;
            b[i % 4] = __builtin_fmaf(e, fmaxf(d, kLeast), b[i % 4]);
        }
        rescale(M, r, k);
        s += (double)((a[0] + a[1]) + (a[2] + a[3]));
        w += (double)((b[0] + b[1]) + (b[2] + b[3]));
    }

    __device__ __forceinline__ void join(float m2, double s2, double w2, float k) {
        Sums o{m2, kNegInf, s2, w2};
        const float M = fmaxf(m, m2), r = M == kNegInf ? 0.0f : M;
        rescale(M, r, k);
        o.rescale(M, r, k);
        s += o.s;
        w += o.w;
    }
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// What the statistics of a row come to, its token among the values.
struct RowEnd {
    float m, token;
    bool empty;         // nothing but -inf
    double rest, S;     // sums of e, `rest` without the token's
    double ln_s, down;  // ln S; E[(m - z) / T]
};

__device__ __forceinline__ RowEnd row_end(const Sums& x, float token, bool has, float k) {
    RowEnd e;
    const float r = x.m == kNegInf ? 0.0f : x.m, d = exponent(token, r, k);
    const float own = has ? exp2_fast(d) : 0.0f;
    e.m = r;
    e.token = token;
    e.rest = x.s;
    e.S = x.s + (double)own;
    e.empty = x.m == kNegInf && e.S == 0.0;
    const double w = x.w + (has ? (double)own * (double)fmaxf(d, kLeast) : 0.0);
    // ln(1 + rest) of a small rest: 1 + rest has rounded its digits away
    const bool sure = own == 1.0f && e.rest < 0x1p-20;
    e.ln_s = e.empty ? 0.0 : sure ? e.rest - 0.5 * e.rest * e.rest : log(e.S);
    e.down = e.empty ? 0.0 : -kLn2 * w / e.S;
    return e;
}

// log p of value v
__device__ __forceinline__ double log_p(const RowEnd& e, float v, float k) {
    return ((double)v - (double)e.m) * ((double)k * kLn2) - e.ln_s;
}

__device__ __forceinline__ bool takes_part(const TokenStats& a, int64_t row) {
    if (!a.target) return true;
    const int64_t y = a.target[row];
    return y >= 0 && y < a.vocab;
}

// The outputs of a row but its alternatives, by one thread.
__device__ __forceinline__ void write_row(const TokenStats& a, int64_t row, bool live, const RowEnd& e) {
    const bool none = !live || e.empty;
    if (a.logp) a.logp[row] = none ? 0.0f : (float)log_p(e, e.token, a.k);
    if (a.entropy) a.entropy[row] = none ? 0.0f : (float)(e.ln_s + e.down);
    if (a.saved) {
        float* to = a.saved + 4 * row;
        to[0] = none ? 0.0f : e.m;
        to[1] = none ? 0.0f : (float)(1.0 / e.S);
        to[2] = none ? 0.0f : (float)e.down;
        to[3] = none ? 0.0f : (float)(e.rest / e.S);
    }
}

// Alternative `rank` of a row: value v of index id, or none (id < 0).  A row
// with a NaN or +inf has no order: NaN for all of them.
__device__ __forceinline__ void write_top(const TokenStats& a, int64_t row, int rank, float v, int id, const RowEnd& e) {
    const bool bad = e.S != e.S;
    a.top_id[row * a.top + rank] = bad || id < 0 ? -1 : id;
    a.top_logp[row * a.top + rank] = bad ? __builtin_nanf("") : id < 0 ? kNegInf : (float)log_p(e, v, a.k);
}

// Candidates for the alternatives of a part of a row: the best n of them come
// out, by value and then by index.
constexpr int kRoom = 256;
struct Candidates {
    float v[kRoom];
    int32_t id[kRoom];
    int32_t n;  // found, may pass kRoom

    __device__ __forceinline__ void add(float x, int i) {
        const int at = atomicAdd(&n, 1);
        if (at < kRoom) {
            v[at] = x;
            id[at] = i;
        }
    }
};

__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// The n-th largest of the wave's 64 values (n <= 64), ties counted by lane.
__device__ __forceinline__ float nth_of_wave(float v, int n) {
    const int lane = lanes::lane();
    int rank = 0;
#pragma unroll 8
    for (int l = 0; l < 64; ++l) {
        const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
        rank += before(o, l, v, lane) ? 1 : 0;
    }
    const uint64_t at = __ballot(rank == n - 1);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), __builtin_ctzll(at)));
}

// The values of a part of a row that are taken one by one, a thread each: the
// edges, and the piece of token y (from the 33rd thread on), if that is one of
// the part's; index -1 for a thread without one.
template <typename T>
struct Single {
    int at;
    T raw;
    __device__ __forceinline__ Single(const T* z, const Pieces<T>& ps, const Part& part, int y) : at(-1) {
        constexpr int N = Vec<T>::n;
        const int tid = threadIdx.x, yv = ps.piece(y);
        if (part.ends && tid < ps.edges) at = ps.edge(tid);
        if (yv >= part.v0 && yv < part.v1 && tid >= 32 && tid < 32 + N) at = ps.head + yv * N + tid - 32;
        raw = z[at < 0 ? 0 : at];
    }
    __device__ __forceinline__ float value() const { return at < 0 ? kNegInf : Vec<T>::one(raw); }
};

template <int NT>
struct StatsLds {
    double s[NT / 64], w[NT / 64];
    float m[NT / 64];
    float group[64];
    float least;
    int32_t hot[NT];
    int32_t n_hot;
    Candidates c;
};

// Sums of the whole workgroup, in a fixed order; valid in every thread.  Ends
// with a barrier.
template <int NT>
__device__ __forceinline__ Sums wg_join(Sums x, float k, StatsLds<NT>& lds) {
    float M = x.m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    x.rescale(M, M == kNegInf ? 0.0f : M, k);
    x.s = wave_sum(x.s);
    x.w = wave_sum(x.w);
    if (NT == 64) return x;
    if (lanes::lane() == 0) {
        lds.s[threadIdx.x >> 6] = x.s;
        lds.w[threadIdx.x >> 6] = x.w;
        lds.m[threadIdx.x >> 6] = M;
    }
    __syncthreads();
    Sums all{lds.m[0], kNegInf, lds.s[0], lds.w[0]};
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) all.join(lds.m[i], lds.s[i], lds.w[i], k);
    __syncthreads();
    return all;
}

// The part's best a.top values into lds.c, unordered, from the threads' own
// largest values.  64 groups of neighbouring threads: the n-th largest of the
// groups' largest values is reached by n values at least, so the n best are
// among what reaches it: about n to 2 n values, in the shares of as many
// threads, which the workgroup reads again.  lds.c.n passes kRoom where that
// many tie with it or a few shares hold them.
template <typename T, int NT>
__device__ __forceinline__ void gather_best(const T* z, const Pieces<T>& ps, const Part& part, int y, float best,
                                            const Single<T>& one, int n, StatsLds<NT>& lds) {
    constexpr int N = Vec<T>::n, L = NT / 64;
    const int tid = threadIdx.x;
    const float group = lanes::max<L>(best);
    if (tid % L == 0) lds.group[tid / L] = group;
    if (tid == 0) lds.n_hot = lds.c.n = 0;
    __syncthreads();
    if (tid < 64) {
        const float least = nth_of_wave(lds.group[tid], n);
        if (tid == 0) lds.least = least;
    }
    __syncthreads();
    const float least = lds.least;
    const auto fits = [&](float x) { return x >= least && x > kNegInf; };
    if (fits(best)) lds.hot[atomicAdd(&lds.n_hot, 1)] = tid;
    if (one.at >= 0 && fits(one.value())) lds.c.add(one.value(), one.at);
    __syncthreads();
    const int hot = lds.n_hot, per = (part.v1 - part.v0 + NT - 1) / NT, yv = ps.piece(y);
    const T* base = z + ps.head;
    for (int q = tid; q < hot * per; q += NT) {
        const int h = q / per, v = part.v0 + lds.hot[h] + (q - h * per) * NT;
        if (v >= part.v1 || v == yv) continue;
        float x[N];
        Vec<T>::open(load16(base + v * N), x);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (fits(x[i])) lds.c.add(x[i], ps.head + v * N + i);
    }
    __syncthreads();
}

// The same for a part whose candidates did not fit: rounds over the part, each
// taking the next smaller value and how often it is there, until n are found;
// then what lies above the last one, and of its equals the first by index.
template <typename T, int NT>
__device__ void gather_slow(const T* z, const Pieces<T>& ps, const Part& part, int n, StatsLds<NT>& lds) {
    constexpr int N = Vec<T>::n;
    const int tid = threadIdx.x;
    const T* base = z + ps.head;
    const int edges = part.ends ? ps.edges : 0;
    float last = -kNegInf;
    int above = 0;
    for (int found = 0; found < n;) {
        float top = kNegInf;
        int count = 0;
        const auto see = [&](float x) {
            if (!(x < last) || x < top || x == kNegInf) return;
            count = x > top ? 1 : count + 1;
            top = x;
        };
        for (int v = part.v0 + tid; v < part.v1; v += NT) {
            float x[N];
            Vec<T>::open(load16(base + v * N), x);
            for (int i = 0; i < N; ++i) see(x[i]);
        }
        if (tid < edges) see(Vec<T>::one(z[ps.edge(tid)]));
        const float most = lanes::max<64>(top);
        if (lanes::lane() == 0) lds.m[tid >> 6] = most;
        if (tid == 0) lds.n_hot = 0;
        __syncthreads();
        last = lds.m[0];
        for (int i = 1; i < NT / 64; ++i) last = fmaxf(last, lds.m[i]);
        if (top == last && count > 0) atomicAdd(&lds.n_hot, count);
        __syncthreads();
        above = found;
        found += lds.n_hot;
        if (last == kNegInf) break;  // fewer than n values
        __syncthreads();
    }
    if (tid == 0) {
        lds.c.n = 0;
        lds.n_hot = 0;
    }
    __syncthreads();
    for (int v = part.v0 + tid; v < part.v1; v += NT) {
        float x[N];
        Vec<T>::open(load16(base + v * N), x);
        for (int i = 0; i < N; ++i)
            if (x[i] > last) lds.c.add(x[i], ps.head + v * N + i);
    }
    if (tid < edges) {
        const float x = Vec<T>::one(z[ps.edge(tid)]);
        if (x > last) lds.c.add(x, ps.edge(tid));
    }
    if (last == kNegInf) {
        __syncthreads();
        return;
    }
    // equals in the order of their indexes: the head's edges, pieces, the tail's
    const int need = n - above;
    int have = 0;  // the same in every thread
    const auto edges_of = [&](int i0, int i1) {
        for (int i = i0; i < i1 && have < need; ++i) {
            if (Vec<T>::one(z[ps.edge(i)]) != last) continue;
            if (tid == 0) lds.c.add(last, ps.edge(i));
            ++have;
        }
    };
    const int head = ps.head < edges ? ps.head : edges;
    edges_of(0, head);
    for (int v0 = part.v0; v0 < part.v1 && have < need; v0 += NT) {
        const int v = v0 + tid;
        float x[N];
        int mine = 0;
        if (v < part.v1) {
            Vec<T>::open(load16(base + v * N), x);
            for (int i = 0; i < N; ++i) mine += x[i] == last ? 1 : 0;
        }
        int upto = mine;
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(upto, off, 64);
            if (lanes::lane() >= off) upto += o;
        }
        __syncthreads();
        if (lanes::lane() == 63) lds.hot[tid >> 6] = upto;
        __syncthreads();
        int at = have + upto - mine;
        for (int i = 0; i < NT / 64; ++i) {
            if (i < (tid >> 6)) at += lds.hot[i];
            have += lds.hot[i];
        }
        if (mine)
            for (int i = 0; i < N; ++i)
                if (x[i] == last && at++ < need) lds.c.add(last, ps.head + v * N + i);
    }
    edges_of(head, edges);
    __syncthreads();
}

// One workgroup per part of a row.
template <typename T, int NT, bool TOP>
__global__ __launch_bounds__(NT) void stats_kernel(TokenStats a) {
    constexpr int N = Vec<T>::n, U = 4;
    __shared__ StatsLds<NT> lds;
    const int tid = threadIdx.x;
    const float k = a.k;
    const int64_t items = a.rows * a.parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = a.parts == 1 ? item : item / a.parts;
        const int index = (int)(item - row * a.parts);
        const bool live = takes_part(a, row);
        if (!live) {
            if (a.parts == 1) {
                if (tid == 0) write_row(a, row, false, RowEnd{});
                if (TOP && tid < a.top) write_top(a, row, tid, 0.0f, -1, RowEnd{});
            }
            continue;
        }
        const T* z = static_cast<const T*>(a.z) + row * a.ld;
        const int y = a.target ? (int)a.target[row] : -1;
        const float token = y >= 0 ? Vec<T>::one(z[y]) : kNegInf;
        const Pieces<T> ps(z, a.vocab);
        const Part part = part_of(z, ps, index, a.parts);
        const Single<T> one(z, ps, part, y);
        const T* base = z + ps.head;
        const int yv = ps.piece(y);
        Sums run{token, kNegInf, 0.0, 0.0};
        for (int v = part.v0 + tid; v < part.v1; v += U * NT) {
            u32x4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u] = Vec<T>::lowest();
                const int at = v + u * NT;
                if (at < part.v1 && at != yv) raw[u] = TOP ? load16(base + at * N) : load16_once(base + at * N);
            }
            float x[U * N];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[N];
                Vec<T>::open(raw[u], f);
#pragma unroll
                for (int i = 0; i < N; ++i) x[u * N + i] = f[i];
            }
            run.take(x, k);
        }
        const float best = run.best;
        if (tid < 64) run.take({one.at == y ? kNegInf : one.value()}, k);
        const Sums all = wg_join<NT>(run, k, lds);
        const RowEnd e = row_end(all, token, y >= 0, k);
        if (tid == 0) {
            if (a.parts == 1)
                write_row(a, row, true, e);
            else
                a.stat[item] = PartStat{all.s, all.w, all.m, 0.0f};
        }
        if (!TOP) continue;
        gather_best<T, NT>(z, ps, part, y, best, one, a.top, lds);
        if (lds.c.n > kRoom) gather_slow<T, NT>(z, ps, part, a.top, lds);
        const int n = lds.c.n;
        for (int i = tid; i < n; i += NT) {
            const float v = lds.c.v[i];
            const int id = lds.c.id[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += before(lds.c.v[j], lds.c.id[j], v, id) ? 1 : 0;
            if (rank >= a.top) continue;
            if (a.parts == 1) {
                write_top(a, row, rank, v, id, e);
            } else {
                a.best[item * a.top + rank] = v;
                a.best_id[item * a.top + rank] = id;
            }
        }
        for (int r = n + tid; r < a.top; r += NT) {
            if (a.parts == 1) {
                write_top(a, row, r, kNegInf, -1, e);
            } else {
                a.best[item * a.top + r] = kNegInf;
                a.best_id[item * a.top + r] = -1;
            }
        }
        __syncthreads();
    }
}

// Rows in several parts: a wave joins a row's statistics, a lane a part, and
// picks the best of its parts' best, at most 16 a lane.
constexpr int kMostBest = kMaxParts * kMaxTop;
template <typename T>
__global__ __launch_bounds__(64) void stats_join_kernel(TokenStats a) {
    __shared__ float lv[kMostBest];
    __shared__ int32_t li[kMostBest];
    __shared__ int32_t kept;
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    const bool live = takes_part(a, row);
    RowEnd e{};
    if (live) {
        const T* z = static_cast<const T*>(a.z) + row * a.ld;
        const int64_t y = a.target ? a.target[row] : -1;
        const float token = y >= 0 ? Vec<T>::one(z[y]) : kNegInf;
        const PartStat p = a.stat[row * a.parts + lane % a.parts];
        Sums x{p.m, kNegInf, p.s, p.w};
        for (int off = 1; off < a.parts; off <<= 1)
            x.join(__shfl_xor(x.m, off, 64), __shfl_xor(x.s, off, 64), __shfl_xor(x.w, off, 64), a.k);
        e = row_end(x, token, y >= 0, a.k);
    }
    if (lane == 0) write_row(a, row, live, e);
    if (a.top == 0) return;
    if (!live) {
        if (lane < a.top) write_top(a, row, lane, 0.0f, -1, e);
        return;
    }
    const int n = a.parts * a.top;
    const float* v = a.best + row * n;
    const int32_t* id = a.best_id + row * n;
    float best = kNegInf;
    for (int i = lane; i < n; i += 64) best = fmaxf(best, v[i]);
    const float least = nth_of_wave(best, a.top);
    if (lane == 0) kept = 0;
    __syncthreads();
    for (int i = lane; i < n; i += 64) {
        if (!(v[i] >= least) || v[i] == kNegInf) continue;
        const int at = atomicAdd(&kept, 1);
        lv[at] = v[i];
        li[at] = id[i];
    }
    __syncthreads();
    for (int i = lane; i < kept; i += 64) {
        int rank = 0;
        for (int j = 0; j < kept; ++j) rank += before(lv[j], li[j], lv[i], li[i]) ? 1 : 0;
        if (rank < a.top) write_top(a, row, rank, lv[i], li[i], e);
    }
    for (int r = kept + lane; r < a.top; r += 64) write_top(a, row, r, kNegInf, -1, e);
}

// ---------------------------------------------------------------- gradient

// dz_i = (c ([i = y] - p_i) - b p_i (log p_i + H)) / T for c = dlogp and b =
// dentropy.  With q = E[(m - z) / T], log p_i + H = ln 2 d_i + q, so a value
// takes p_i (slope d_i + level), and the token's own value c (1 - p) from the
// sum of the others.
struct GradRow {
    float m, level, slope, own;
};

// One workgroup per span of a row, as the values lie in memory.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void stats_grad_kernel(TokenStatsGrad a, int spans) {
    constexpr int N = Vec<T>::n, U = 4;
    const int tid = threadIdx.x;
    const float k = a.k;
    const int64_t items = a.rows * spans;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / spans;
        const T* z = static_cast<const T*>(a.z) + row * a.ld;
        T* to = static_cast<T*>(a.d) + row * a.ldd;
        const Pieces<T> ps(z, a.vocab);
        const Part part = part_of(z, ps, (int)(item - row * spans), spans);
        const float* saved = a.saved + 4 * row;
        const float m = saved[0], f = saved[1], q = saved[2];
        const double c = a.dlogp ? (double)a.dlogp[row] : 0.0, b = a.dentropy ? (double)a.dentropy[row] : 0.0;
        const bool none = f == 0.0f || (c == 0.0 && b == 0.0);
        const double cf = -a.scale * (double)f;
        const float level = (float)(cf * (c + b * (double)q)), slope = (float)(cf * (b * kLn2));
        const auto grad = [&](float x) {
            const float d = exponent(x, m, k);
            return exp2_fast(d) * __builtin_fmaf(slope, fmaxf(d, kLeast), level);
        };
        // the thread that writes the token's place: nobody else does, so that
        // it may read it before, in place or not
        const int y = a.target ? (int)a.target[row] : -1, yv = none ? -1 : ps.piece(y);
        bool mine = yv >= part.v0 && yv < part.v1 && (yv - part.v0) % NT == tid;
        if (!none && y >= 0 && yv < 0) mine = part.ends && tid < ps.edges && ps.edge(tid) == y;
        float own = 0.0f;
        if (mine) {
            const float d = exponent(Vec<T>::one(z[y]), m, k);
            const double p = (double)exp2_fast(d) * (double)f;
            own = (float)(a.scale * (c * (double)saved[3] - b * p * (kLn2 * (double)fmaxf(d, kLeast) + (double)q)));
        }
        for (int v = part.v0 + tid; v < part.v1; v += U * NT) {
            u32x4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (!none && v + u * NT < part.v1) raw[u] = load16_once(z + ps.head + (v + u * NT) * N);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (v + u * NT >= part.v1) continue;
                u32x4 out = {0u, 0u, 0u, 0u};
                if (!none) {
                    float x[N];
                    Vec<T>::open(raw[u], x);
#pragma unroll
                    for (int i = 0; i < N; ++i) x[i] = grad(x[i]);
                    out = Vec<T>::close(x);
                }
                store16(to + ps.head + (v + u * NT) * N, out);
            }
        }
        if (part.ends && tid < ps.edges) {
            const int at = ps.edge(tid);
            to[at] = none ? T(0) : Vec<T>::pack(grad(Vec<T>::one(z[at])));
        }
        if (mine) to[y] = Vec<T>::pack(own);
    }
}

int64_t row_bytes(int64_t vocab, int32_t f32) { return vocab * (f32 ? 4 : 2); }

template <int NT>
hipError_t launch_stats_nt(const TokenStats& a, hipStream_t s) {
    const unsigned g = grid_of(a.rows * a.parts);
    if (a.f32) {
        if (a.top)
            hipLaunchKernelGGL((stats_kernel<float, NT, true>), dim3(g), dim3(NT), 0, s, a);
        else
            hipLaunchKernelGGL((stats_kernel<float, NT, false>), dim3(g), dim3(NT), 0, s, a);
    } else {
        if (a.top)
            hipLaunchKernelGGL((stats_kernel<uint16_t, NT, true>), dim3(g), dim3(NT), 0, s, a);
        else
            hipLaunchKernelGGL((stats_kernel<uint16_t, NT, false>), dim3(g), dim3(NT), 0, s, a);
    }
    return hipGetLastError();
}

// Rows of up to this many bytes take one wave each.
constexpr int64_t kWaveRow = 16 << 10;
// Values of a row that one workgroup of the gradient writes.
constexpr int64_t kGradSpan = 4096;

}  // namespace

hipError_t launch_token_stats(const TokenStats& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    hipError_t e = row_bytes(a.vocab, a.f32) <= kWaveRow ? launch_stats_nt<64>(a, s) : launch_stats_nt<256>(a, s);
    if (e != hipSuccess || a.parts == 1) return e;
    if (a.f32)
        hipLaunchKernelGGL(stats_join_kernel<float>, dim3((unsigned)a.rows), dim3(64), 0, s, a);
    else
        hipLaunchKernelGGL(stats_join_kernel<uint16_t>, dim3((unsigned)a.rows), dim3(64), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_token_stats_grad(const TokenStatsGrad& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const int spans = (int)((a.vocab + kGradSpan - 1) / kGradSpan);
    const unsigned g = grid_of(a.rows * spans);
    if (a.f32)
        hipLaunchKernelGGL((stats_grad_kernel<float, 256>), dim3(g), dim3(256), 0, s, a, spans);
    else
        hipLaunchKernelGGL((stats_grad_kernel<uint16_t, 256>), dim3(g), dim3(256), 0, s, a, spans);
    return hipGetLastError();
}

}  // namespace rs
