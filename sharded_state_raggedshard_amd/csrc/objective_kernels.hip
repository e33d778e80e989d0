// Training objectives over rows of logits for gfx950: the token
// log-probability, the clipped policy loss and the preference loss with
// their logits' gradients.
//
// A row's softmax needs its maximum m and s = sum exp((z - m) / T).  A term
// is exp2((z - m) k), k = log2(e) / T in two binary32 pieces: one alone
// would shift every term the same way (up to 2^-24 |z - m| / T, so the
// row's logarithm with them), where the product's own rounding averages out.
// (Folding m into one fused multiply-add, z k - m k, saves two instructions
// of eleven a value, measured no faster, as memory bounds these kernels; it
// rounds at the size of m k and overflows on masks of the type's lowest
// value.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "objectives.hpp"
#include "row_common.hpp"
#include "raggedshard.h"

namespace rs {
namespace {

using namespace rows;

// exp((x - m) / T)
__device__ __forceinline__ float term(float x, float m, ExpScale k) {
    const float d = x - m;
    return exp2_fast(__builtin_fmaf(d, k.hi, d * k.lo));
}

// Maximum and sum of a thread's share of a row, a part of it or a row; the
// row's token is in the maximum from the start, but not in the sum.  Its term
// joins last (row_end()): where it is nearly the whole row, as a trained
// model's are, any sum with it would round away the rest that 1 - p is made
// of (a runner-up 17 below, among the values that binary32 adds up with the
// token, left a gradient of 0).  The sum is binary64; the C values of a call
// are added up in binary32 in four chains.
struct MaxSum {
    float m;  // the token's value at first
    double s;

    template <int C>
    __device__ __forceinline__ void take(const float (&x)[C], ExpScale k) {
        float v = x[0];
#pragma unroll
        for (int i = 1; i < C; ++i) v = fmaxf(v, x[i]);
        const float M = fmaxf(m, v);
        const float r = M == kNegInf ? 0.0f : M;  // -inf - 0 gives exp2(-inf) = 0
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) a[i % 4] += term(x[i], r, k);
        s = __builtin_fma(s, (double)term(m, r, k), (double)((a[0] + a[1]) + (a[2] + a[3])));
        m = M;
    }

    __device__ __forceinline__ void join(float m2, double s2, ExpScale k) {
        const float M = fmaxf(m, m2);
        const float r = M == kNegInf ? 0.0f : M;
        s = s * (double)term(m, r, k) + s2 * (double)term(m2, r, k);
        m = M;
    }
};

// LDS of wg_join.
template <int NT>
struct JoinLds {
    double s[NT / 64];
    float m[NT / 64];
};

// The MaxSum of the whole workgroup, in a fixed order; valid in every
// thread.  Ends with a barrier.
template <int NT>
__device__ __forceinline__ MaxSum wg_join(MaxSum x, ExpScale k, JoinLds<NT>& lds) {
    float M = x.m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    x.s *= (double)term(x.m, M == kNegInf ? 0.0f : M, k);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x.s += __shfl_xor(x.s, off, 64);
    x.m = M;
    if (NT == 64) return x;
    if ((threadIdx.x & 63) == 0) {
        lds.s[threadIdx.x >> 6] = x.s;
        lds.m[threadIdx.x >> 6] = M;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) M = fmaxf(M, lds.m[w]);
    x.m = M;
    x.s = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w)
        x.s += lds.s[w] * (double)term(lds.m[w], M == kNegInf ? 0.0f : M, k);
    __syncthreads();
    return x;
}

// What the statistics of a row come to, its token among the values.
struct RowEnd {
    float m;
    double s, rest;  // sums of exp((z - m) / T), `rest` without the token's
    double lse_m;    // log s
    bool empty;      // nothing but -inf
};

__device__ __forceinline__ RowEnd row_end(const MaxSum& x, float token, ExpScale k) {
    RowEnd e;
    const float own = term(token, x.m == kNegInf ? 0.0f : x.m, k);
    e.m = x.m;
    e.rest = x.s;
    e.s = x.s + (double)own;
    e.empty = e.m == kNegInf && e.s == 0.0;
    // log(1 + rest) of a small rest: 1 + rest has rounded its digits away
    const bool sure = own == 1.0f && e.rest < 0x1p-20;
    e.lse_m = e.empty ? 0.0 : sure ? e.rest - 0.5 * e.rest * e.rest : log(e.s);
    return e;
}

__device__ __forceinline__ RowEnd row_of(const LogitRows& a, int64_t row, ExpScale k) {
    const RowStat* p = a.stat + row * a.parts;
    MaxSum x{p[0].m, p[0].s};
    for (int i = 1; i < a.parts; ++i) {
        const RowStat q = p[i];
        x.join(q.m, q.s, k);
    }
    return row_end(x, a.token[row], k);
}

__device__ __forceinline__ double logp_of(const RowEnd& e, float token, double scale) {
    return ((double)token - (double)e.m) * scale - e.lse_m;
}

__device__ __forceinline__ bool has_token(const LogitRows& a, int64_t row) {
    const int64_t y = a.target[row];
    return y >= 0 && y < a.vocab && (!a.weight || a.weight[row] != 0.0f);
}

// --------------------------------------------------------- row statistics

// A row of `vocab` values in 16-byte pieces at 16-byte addresses: rows of an
// odd length start anywhere, and pieces across 16-byte lines cost a quarter
// of the bandwidth (6001 x 32003 bf16: 85 us, x 32000: 66 us).  `head` values
// lie in front of the pieces; `edges` values, fewer than 2 N, in front of and
// behind them, one each for the first threads.
template <typename T>
struct Pieces {
    static constexpr int N = Vec<T>::n;
    int head, n, edges;
    __device__ __forceinline__ Pieces(const T* row, int64_t vocab) {
        const int to_line = (int)((16u - (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / (int)sizeof(T);
        head = to_line < (int)vocab ? to_line : (int)vocab;
        n = ((int)vocab - head) / N;
        edges = (int)vocab - n * N;
    }
    __device__ __forceinline__ int edge(int i) const { return i < head ? i : n * N + i; }
    // piece of value y, -1 for an edge
    __device__ __forceinline__ int piece(int y) const {
        return y >= head && (y - head) / N < n ? (y - head) / N : -1;
    }
};

// A part of a row: pieces [v0, v1) and, if `ends`, the edges.  Parts meet at
// 128-byte lines: a line that two workgroups write, on two L2 caches, costs
// a read and a merge (gradients of 4470 of 6697 rows x 128256 bf16 in parts
// of 32 to 50 KB: 540 to 560 us with lines shared, 505 us without).
struct Part {
    int v0, v1;
    bool ends;
};

template <typename T>
__device__ __forceinline__ Part part_of(const T* row, const Pieces<T>& ps, int part, int parts) {
    if (parts == 1) return Part{0, ps.n, true};
    const int shift = (int)(reinterpret_cast<uintptr_t>(row + ps.head) >> 4) & 7;
    const int per = ((ps.n + shift + parts - 1) / parts + 7) / 8 * 8;
    const int a = part * per - shift, b = a + per;
    return Part{a < 0 ? 0 : a < ps.n ? a : ps.n, b < ps.n ? b : ps.n, part == parts - 1};
}

// The values of a part of a row that are taken one by one, a thread each: the
// edges, and the values beside token y in its piece (from the 33rd thread
// on), if that is one of [v0, part.v1).  Every thread loads one, the token
// where it has none, and opens it in value(), after the pieces' loads have
// begun: waiting for it first took 0.7 us a row.
template <typename T>
struct Single {
    int at, y;
    T raw;
    __device__ __forceinline__ Single(const T* z, const Pieces<T>& ps, Part part, int v0, int y) : at(y), y(y) {
        constexpr int N = Vec<T>::n;
        const int tid = threadIdx.x, yv = ps.piece(y);
        if (part.ends && tid < ps.edges) at = ps.edge(tid);
        if (yv >= v0 && yv < part.v1 && tid >= 32 && tid < 32 + N) at = ps.head + yv * N + tid - 32;
        raw = z[at];
    }
    __device__ __forceinline__ float value() const { return at != y ? Vec<T>::one(raw) : kNegInf; }
};

// Statistics of a part of a row without the piece of token y and the values
// that Single takes, by the whole workgroup: U loads a thread in flight
// (the last ones padded with -inf).  ONCE: not read again soon.
template <typename T, int NT, bool ONCE>
__device__ __forceinline__ void take_part(MaxSum& run, const T* z, const Pieces<T>& ps, Part part,
                                          int y, ExpScale k) {
    constexpr int N = Vec<T>::n, U = 4;
    const T* base = z + ps.head;
    const int yv = ps.piece(y);
    for (int v = part.v0 + threadIdx.x; v < part.v1; v += U * NT) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            w[u] = Vec<T>::lowest();
            const int at = v + u * NT;
            if (at < part.v1 && at != yv) w[u] = ONCE ? load16_once(base + at * N) : load16(base + at * N);
        }
        float x[U * N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[N];
            Vec<T>::open(w[u], f);
#pragma unroll
            for (int i = 0; i < N; ++i) x[u * N + i] = f[i];
        }
        run.take(x, k);
    }
}

enum { MARK_OUTSIDE = 0, MARK_ZERO = 1, MARK_TOKEN = 2 };

// What row_stats_kernel does beside the statistics: nothing; writes logp (and
// lse) of whole rows; marks rows for the preference loss (outside every
// sequence, without a token, with one); nothing, but leaves the logits in the
// caches for the gradient.
enum { STATS_ONLY = 0, STATS_LOGP = 1, STATS_MARK = 2, STATS_KEEP = 3 };

__device__ __forceinline__ void write_logp(const LogitRows& a, int64_t row, const RowEnd& e,
                                           float token, float* logp, float* lse) {
    logp[row] = e.empty ? 0.0f : (float)logp_of(e, token, a.scale);
    if (lse) lse[row] = e.empty ? 0.0f : (float)((double)e.m * a.scale + e.lse_m);
}

// One workgroup per part of a row: its maximum and sum in one pass over the
// logits.  Bound by HBM: 6.5 TB/s on 8192 x 128256 bf16 (322 us).
template <typename T, int NT, int MODE>
__global__ __launch_bounds__(NT) void row_stats_kernel(LogitRows a, PreferenceTerms t, float* logp,
                                                       float* lse) {
    __shared__ JoinLds<NT> lds;
    const int tid = threadIdx.x;
    const ExpScale k = a.k;
    const int64_t items = a.rows * a.parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = a.parts == 1 ? item : item / a.parts;
        const int part = (int)(item - row * a.parts);
        bool live = has_token(a, row);
        if (MODE == STATS_MARK) {
            const int64_t seq = sequence_of(t.start, 2 * t.pairs, row);
            const bool inside = seq < 2 * t.pairs && row >= t.start[0];
            if (inside && t.weight)
                live = live && t.weight[seq < t.pairs ? seq : seq - t.pairs] != 0.0f;
            live = live && inside;
            if (part == 0 && tid == 0)
                t.mark[row] = !inside ? MARK_OUTSIDE : live ? MARK_TOKEN : MARK_ZERO;
        }
        if (!live) {
            if (MODE == STATS_LOGP && tid == 0) {
                logp[row] = 0.0f;
                if (lse) lse[row] = 0.0f;
            }
            continue;
        }
        const T* z = static_cast<const T*>(a.z) + row * a.ld;
        const int y = (int)a.target[row];
        const float token = Vec<T>::one(z[y]);
        const Pieces<T> ps(z, a.vocab);
        const Part p = part_of(z, ps, part, a.parts);
        const Single<T> one(z, ps, p, p.v0, y);
        MaxSum run{token, 0.0};
        if (MODE == STATS_KEEP || (MODE == STATS_MARK && row >= t.kept_from))
            take_part<T, NT, false>(run, z, ps, p, y, k);
        else
            take_part<T, NT, true>(run, z, ps, p, y, k);
        if (tid < 64) run.take({one.value()}, k);
        run = wg_join<NT>(run, k, lds);
        if (tid != 0) continue;
        if (MODE == STATS_LOGP) {
            write_logp(a, row, row_end(run, token, k), token, logp, lse);
        } else {
            a.stat[item] = RowStat{run.s, run.m, 0.0f};
            if (part == 0) a.token[row] = token;
        }
    }
}

// --------------------------------------------------------------- token logp

// Joins the parts of split rows (parts: a power of two up to 32), a lane a
// part.
__device__ __forceinline__ MaxSum join_parts(const LogitRows& a, int64_t row, int part) {
    const RowStat p = a.stat[row * a.parts + part];
    MaxSum x{p.m, p.s};
    for (int off = 1; off < a.parts; off <<= 1)
        x.join(__shfl_xor(x.m, off, 64), __shfl_xor(x.s, off, 64), a.k);
    return x;
}

__global__ __launch_bounds__(256) void logp_kernel(LogitRows a, float* logp, float* lse) {
    const int64_t at = blockIdx.x * 256ll + threadIdx.x, row = at / a.parts;
    const int part = (int)(at - row * a.parts);
    if (row >= a.rows) return;
    RowEnd e;
    e.empty = true;
    float token = 0.0f;
    if (has_token(a, row)) {
        token = a.token[row];
        e = row_end(join_parts(a, row, part), token, a.k);
    }
    if (part == 0) write_logp(a, row, e, token, logp, lse);
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
        if (t.kl_coef != 0.0) slope += t.kl_coef * (1.0 - q);
    }
    p.coef = w * slope;
    return p;
}

// Sums of n triples, by one workgroup in a fixed order; valid in thread 0.
template <int NT>
__device__ __forceinline__ void sum_terms(const double* terms, int64_t n, double (&sum)[3],
                                          double* lds) {
    double x[3] = {0.0, 0.0, 0.0};
    for (int64_t i = threadIdx.x; i < n; i += NT)
        for (int j = 0; j < 3; ++j) x[j] += terms[3 * i + j];
    for (int j = 0; j < 3; ++j) sum[j] = wg_sum<NT>(x[j], lds);
}

__device__ __forceinline__ void policy_stats(const PolicyTerms& t, const double (&sum)[3],
                                             float* stats) {
    stats[0] = (float)(sum[0] + (t.kl_coef != 0.0 ? t.kl_coef * sum[1] : 0.0));
    for (int j = 0; j < 3; ++j) stats[1 + j] = (float)sum[j];
}

// ----------------------------------------------------------- logits gradient

// What the gradient of a row, cs ([i = y] - p_i), takes: f = -cs / s and the
// token's own value cs (1 - p), where 1 - p is the sum of the others over all.
__device__ __forceinline__ GradRow grad_row(const RowEnd& e, double cs, int64_t y) {
    GradRow g;
    g.m = e.m;
    g.f = (float)(-cs / e.s);
    g.own = (float)(cs * (e.rest / e.s));
    g.y = (int32_t)y;
    return g;
}

__device__ __forceinline__ float grad_one(const GradRow& g, float x, ExpScale k) {
    return g.f * term(x, g.m, k);
}

// 16 bytes of a row's gradient.
template <typename T>
__device__ __forceinline__ u32x4 grad16(const GradRow& g, const u32x4& w, ExpScale k) {
    constexpr int N = Vec<T>::n;
    float x[N];
    Vec<T>::open(w, x);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = grad_one(g, x[i], k);
    return Vec<T>::close(x);
}

// The gradient of a part of a row; get() gives the row's GradRow to every
// thread, after the first loads are under way.
template <typename T, int NT, typename F>
__device__ __forceinline__ void grad_part(const T* z, T* d, const Pieces<T>& ps, Part part,
                                          ExpScale k, F get) {
    constexpr int N = Vec<T>::n, U = 4;
    const int tid = threadIdx.x;
    const T* from = z + ps.head;
    T* to = d + ps.head;
    u32x4 w[U];
    const auto load = [&](int v) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * NT < part.v1) w[u] = load16_once(from + (v + u * NT) * N);
    };
    int v = part.v0 + tid;
    load(v);
    const GradRow g = get();
    while (v < part.v1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * NT < part.v1) store16(to + (v + u * NT) * N, grad16<T>(g, w[u], k));
        v += U * NT;
        load(v);
    }
    if (part.ends && tid < ps.edges)
        d[ps.edge(tid)] = Vec<T>::pack(grad_one(g, Vec<T>::one(z[ps.edge(tid)]), k));
    // the token's own value, by the thread that has just written its place
    const int yv = ps.piece(g.y);
    const bool mine = yv >= 0 ? yv >= part.v0 && yv < part.v1 && (yv - part.v0) % NT == tid
                              : part.ends && tid < ps.edges && ps.edge(tid) == g.y;
    if (mine) d[g.y] = Vec<T>::pack(g.own);
}

template <typename T, int NT>
__device__ __forceinline__ void zero_part(T* d, const Pieces<T>& ps, Part part) {
    const u32x4 z = {0u, 0u, 0u, 0u};
    for (int v = part.v0 + threadIdx.x; v < part.v1; v += NT)
        store16(d + ps.head + v * Vec<T>::n, z);
    if (part.ends && (int)threadIdx.x < ps.edges) d[ps.edge(threadIdx.x)] = T(0);
}

// ------------------------------------------------------- policy loss, split

// Up to this many rows of the policy loss are split over workgroups, more
// take one each (us, split against the best of one each): 16 x 129280
// binary32 12 / 27, 64 x 23 / 28, 128 x 39 / 32; 64 x 128256 bf16 18 / 26,
// 128 x 27 / 26; 64 x 8192 8.9 / 8.8.
constexpr int64_t kSplitRows = 64;

// Few long rows: row_stats_kernel over parts, then this kernel, in which
// workgroup 0 computes the rows' outputs and the loss sums and every other
// one writes a part of a row's gradient.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void policy_grad_kernel(LogitRows a, PolicyTerms t, T* d,
                                                         int64_t ldd, int spans, float* logp,
                                                         float* stats) {
    __shared__ double lds[NT / 64];
    __shared__ GradRow g;
    const int tid = threadIdx.x;
    const ExpScale k = a.k;
    if (blockIdx.x == 0) {
        // four lanes a row (all rows at once: this workgroup is the one that
        // the launch waits for)
        static_assert(NT == 4 * kSplitRows, "four lanes a row");
        const int64_t row = tid / 4;
        const int sub = tid % 4, per = a.parts < 4 ? 1 : a.parts / 4;
        PolicyRow p;
        if (row < a.rows) {
            const float token = a.token[row];
            MaxSum x{token, 0.0};
            if (sub * per < a.parts) {
                const RowStat* q = a.stat + row * a.parts + sub * per;
                x = MaxSum{q[0].m, q[0].s};
                for (int i = 1; i < per; ++i) x.join(q[i].m, q[i].s, k);
            }
            x.join(__shfl_xor(x.m, 1, 64), __shfl_xor(x.s, 1, 64), k);
            x.join(__shfl_xor(x.m, 2, 64), __shfl_xor(x.s, 2, 64), k);
            if (sub == 0 && has_token(a, row)) p = policy_row(a, t, row, row_end(x, token, k), token);
            if (sub == 0 && logp) logp[row] = (float)p.logp;
        }
        const double pg = p.pg, kl = p.kl, cl = p.clipped;
        const double sum[3] = {wg_sum<NT>(pg, lds), wg_sum<NT>(kl, lds), wg_sum<NT>(cl, lds)};
        if (tid == 0) policy_stats(t, sum, stats);
        return;
    }
    const int64_t item = blockIdx.x - 1, row = item / spans;
    const int span = (int)(item - row * spans);
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    T* to = d + row * ldd;
    const Pieces<T> ps(z, a.vocab);
    const Part part = part_of(z, ps, span, spans);
    if (!has_token(a, row)) {
        zero_part<T, NT>(to, ps, part);
        return;
    }
    grad_part<T, NT>(z, to, ps, part, k, [&] {
        const float token = a.token[row];
        const RowEnd e = row_end(join_parts(a, row, tid % a.parts), token, k);
        if (tid == 0) {
            g = GradRow{0.0f, 0.0f, 0.0f, -1};  // a row of nothing but -inf: zeros, no token
            if (!e.empty) g = grad_row(e, policy_row(a, t, row, e, token).coef * a.scale, a.target[row]);
        }
        __syncthreads();
        return g;
    });
}

// ------------------------------------------------------ policy loss, by row

// One workgroup per row: statistics, coefficient and gradient.  The first
// kHeld pieces of every thread stay in its registers in between; the rest is
// read again, out of the cache that holds it if few enough rows are under
// way.  Four waves a SIMD (128 registers) is what 12 held pieces leave: 2
// workgroups of 512 a unit, so that one reads while the other writes.
//
// 6144 of 8192 rows x 128256 bf16, in us: two kernels over all rows 981;
// nothing held 793 (512 threads); 12 held 743; with the gradient stored past
// the caches 710, and held pieces read past them 698 (5.3 TB/s of the
// 3.68 GB it cannot do without); the token apart from the sums, for its
// 1 - p, takes 1.5 % more.  16 held (spills) 747, 8 held 750.  Holding
// all of a row in 1024 threads and loading the next row while storing took
// 920: four waves a SIMD in step leave the memory idle while they sum.
// Neither 9 more pieces a thread in LDS (685, but 64000-value rows 186 ->
// 204) nor a quarter fewer instructions (694) change it: what bounds it is
// how the memory takes 512 rows read and written side by side (one linear
// sweep, as the preference gradient's, reaches 6.2 TB/s).
constexpr int kHeld = 12;

template <typename T, int NT>
__global__ __launch_bounds__(NT, 4) void policy_row_kernel(LogitRows a, PolicyTerms t, int64_t row0,
                                                           T* d, int64_t ldd, float* logp) {
    constexpr int N = Vec<T>::n;
    __shared__ JoinLds<NT> lds;
    __shared__ GradRow g;
    const ExpScale k = a.k;
    const int tid = threadIdx.x;
    const int64_t row = row0 + blockIdx.x;
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    T* to = d + row * ldd;
    const Pieces<T> ps(z, a.vocab);
    RowEnd e;
    e.empty = true;
    u32x4 w[kHeld];
    if (has_token(a, row)) {
        const int y = (int)a.target[row];
        const float token = Vec<T>::one(z[y]);
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j * NT + tid < ps.n) w[j] = load16_once(z + ps.head + (j * NT + tid) * N);
        const Part rest{kHeld * NT, ps.n, true};
        const Single<T> one(z, ps, rest, 0, y);
        const int yv = ps.piece(y);
        MaxSum run{token, 0.0};
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            if (j * NT + tid < ps.n && j * NT + tid != yv) {
                float x[N];
                Vec<T>::open(w[j], x);
                run.take(x, k);
            }
        }
        take_part<T, NT, false>(run, z, ps, rest, y, k);
        if (tid < 64) run.take({one.value()}, k);
        e = row_end(wg_join<NT>(run, k, lds), token, k);
        if (tid == 0 && !e.empty) {
            const PolicyRow p = policy_row(a, t, row, e, token);
            g = grad_row(e, p.coef * a.scale, y);
            t.terms[3 * row] = p.pg;
            t.terms[3 * row + 1] = p.kl;
            t.terms[3 * row + 2] = p.clipped;
            if (logp) logp[row] = (float)p.logp;
        }
        __syncthreads();
    }
    if (e.empty) {
        if (tid == 0) {
            for (int i = 0; i < 3; ++i) t.terms[3 * row + i] = 0.0;
            if (logp) logp[row] = 0.0f;
        }
        if (d) zero_part<T, NT>(to, ps, Part{0, ps.n, true});
        return;
    }
    if (!d) return;
    const GradRow gr = g;
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
        if (j * NT + tid < ps.n) store16(to + ps.head + (j * NT + tid) * N, grad16<T>(gr, w[j], k));
    const int yv = ps.piece(gr.y);
    if (yv >= 0 && yv < kHeld * NT && yv % NT == tid) to[gr.y] = Vec<T>::pack(gr.own);
    grad_part<T, NT>(z, to, ps, Part{kHeld * NT, ps.n, true}, k, [&] { return gr; });
}

__global__ __launch_bounds__(1024) void policy_sum_kernel(PolicyTerms t, const double* terms,
                                                          int64_t n, float* stats) {
    __shared__ double lds[16];
    double sum[3];
    sum_terms<1024>(terms, n, sum, lds);
    if (threadIdx.x == 0) policy_stats(t, sum, stats);
}

// Many rows: workgroup b first sums their b-th slice.
__global__ __launch_bounds__(256) void policy_slice_kernel(PolicyTerms t, int64_t rows, int64_t per) {
    __shared__ double lds[4];
    const int64_t r0 = blockIdx.x * per, left = rows - r0;
    double sum[3];
    sum_terms<256>(t.terms + 3 * r0, left < per ? left : per, sum, lds);
    if (threadIdx.x == 0)
        for (int j = 0; j < 3; ++j) t.slices[3 * blockIdx.x + j] = sum[j];
}

// ---------------------------------------------------------- preference loss

// One workgroup per pair, half of it per sequence: the sequences'
// log-probabilities, the loss and what the rows' gradients take.
template <int NT>
__global__ __launch_bounds__(NT) void pair_kernel(LogitRows a, PreferenceTerms t, float* seq_logp) {
    constexpr int HALF = NT / 2, WAVES = HALF / 64;
    __shared__ double logp_lds[2 * WAVES], tokens_lds[2 * WAVES];
    __shared__ double factor[2];  // dloss / dlogp / T of a side's rows
    const ExpScale k = a.k;
    const int tid = threadIdx.x, side = tid / HALF, at = tid % HALF;
    const int64_t p = blockIdx.x, q = p + side * t.pairs;
    const double w = t.weight ? (double)t.weight[p] : 1.0 / (double)t.pairs;
    int64_t r0 = t.start[q], r1 = t.start[q + 1];
    if (r0 < 0) r0 = 0;
    if (r1 > a.rows) r1 = a.rows;
    double l = 0.0, n = 0.0;
    RowEnd first;  // of the thread's first row
    first.empty = true;
    for (int64_t row = r0 + at; row < r1; row += HALF) {
        if (t.mark[row] != MARK_TOKEN) continue;
        const RowEnd e = row_of(a, row, k);
        if (row == r0 + at) first = e;
        if (e.empty) {
            t.mark[row] = MARK_ZERO;
            continue;
        }
        l += logp_of(e, a.token[row], a.scale);
        n += 1.0;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        l += __shfl_xor(l, off, 64);
        n += __shfl_xor(n, off, 64);
    }
    if ((tid & 63) == 0) {
        logp_lds[tid >> 6] = l;
        tokens_lds[tid >> 6] = n;
    }
    __syncthreads();
    if (tid == 0) {
        double sum[2], count[2];
        for (int i = 0; i < 2; ++i) {
            sum[i] = 0.0;
            count[i] = 0.0;
            for (int v = 0; v < WAVES; ++v) {
                sum[i] += logp_lds[i * WAVES + v];
                count[i] += tokens_lds[i * WAVES + v];
            }
            count[i] = t.average ? fmax(count[i], 1.0) : 1.0;
            sum[i] /= count[i];
            if (seq_logp) seq_logp[p + i * t.pairs] = (float)sum[i];
        }
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
        const double slope = out ? 0.0 : w * g * a.scale;
        factor[0] = slope / count[0];
        factor[1] = -slope / count[1];
    }
    __syncthreads();
    const double cs = factor[side];
    for (int64_t row = r0 + at; row < r1; row += HALF) {
        if (t.mark[row] != MARK_TOKEN) continue;
        const RowEnd e = row == r0 + at ? first : row_of(a, row, k);
        t.grad[row] = grad_row(e, cs, a.target[row]);
    }
}

template <int NT>
__device__ void preference_summary(const PreferenceTerms& t, float* stats, double* lds) {
    double sum[3];
    sum_terms<NT>(t.terms, t.pairs, sum, lds);
    if (threadIdx.x == 0)
        for (int i = 0; i < 3; ++i) stats[i] = (float)sum[i];
}

// Workgroup 0 sums the losses; the others each write a part of a row, the
// last rows first: the statistics have left those in the memory-side cache.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void preference_grad_kernel(LogitRows a, PreferenceTerms t, T* d,
                                                             int64_t ldd, int spans, float* stats) {
    __shared__ double lds[NT / 64];
    if (blockIdx.x == 0) {
        preference_summary<NT>(t, stats, lds);
        return;
    }
    const int64_t items = a.rows * spans;
    for (int64_t i = blockIdx.x - 1; i < items; i += gridDim.x - 1) {
        const int64_t item = items - 1 - i, row = item / spans;
        const int mark = t.mark[row];
        if (mark == MARK_OUTSIDE) continue;
        const T* z = static_cast<const T*>(a.z) + row * a.ld;
        T* to = d + row * ldd;
        const Pieces<T> ps(z, a.vocab);
        const Part part = part_of(z, ps, (int)(item - row * spans), spans);
        if (mark == MARK_ZERO)
            zero_part<T, NT>(to, ps, part);
        else
            grad_part<T, NT>(z, to, ps, part, a.k, [&] { return t.grad[row]; });
    }
}

// Rows of up to this many bytes take one wave each in the statistics.
constexpr int64_t kWaveRow = 16 << 10;

int64_t row_bytes(const LogitRows& a) { return a.vocab * (a.f32 ? 4 : 2); }

template <int NT, int MODE>
hipError_t launch_stats_nt(const LogitRows& a, const PreferenceTerms& t, float* logp, float* lse,
                           hipStream_t s) {
    const unsigned g = grid_of(a.rows * a.parts);
    if (a.f32)
        hipLaunchKernelGGL((row_stats_kernel<float, NT, MODE>), dim3(g), dim3(NT), 0, s, a, t, logp, lse);
    else
        hipLaunchKernelGGL((row_stats_kernel<uint16_t, NT, MODE>), dim3(g), dim3(NT), 0, s, a, t, logp,
                           lse);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_stats(const LogitRows& a, const PreferenceTerms& t, float* logp, float* lse,
                        hipStream_t s) {
    return row_bytes(a) <= kWaveRow ? launch_stats_nt<64, MODE>(a, t, logp, lse, s)
                                    : launch_stats_nt<256, MODE>(a, t, logp, lse, s);
}

// Values of a row that one workgroup of the preference gradient writes: 4470
// of 6697 rows x 128256 bf16 take 464 us in spans of 4096 (6.2 TB/s), 611 of
// 2048, 515 of 8192, 505 to 520 of more.
constexpr int64_t kGradSpan = 4096;
int grad_spans(int64_t vocab) { return (int)((vocab + kGradSpan - 1) / kGradSpan); }

// Threads of a row's workgroup.  Long rows want many, as held pieces are
// what is not read twice; many short rows want small workgroups, as a row's
// start and end take a few us (us at 64 / 256 / 512 / 1024 threads, bf16):
// 4000 x 1000 13 / 23 / 37 / 80, 4000 x 8192 31 / 37 / 52 / 91, 512 x 8192
// 15 / 11 / 11 / 16, 4000 x 32000 119 / 97 / 100 / 150, 512 x 32000 37 / 21 /
// 19 / 25, 4000 x 64000 254 / 202 / 186 / 238, 4000 x 128256 543 / 437 / 394 /
// 441, 256 x 128256 113 / 42 / 34 / 32; binary32: 1500 x 129280 407 / 361 /
// 326 / 300, 1500 x 60000 179 / 159 / 141 / 143.
int policy_row_threads(int64_t rows, int64_t bytes) {
    if (bytes > (256 << 10)) return 1024;
    if (rows <= 256) return bytes > (128 << 10) ? 1024 : 512;
    if (bytes > (64 << 10)) return 512;
    if (rows <= 512) return bytes > (16 << 10) ? 512 : 256;
    return rows >= 2048 && bytes <= (16 << 10) ? 64 : 256;
}

// Rows whose sums one workgroup adds up in the time of another launch.
constexpr int64_t kSumRows = 16384;

template <int NT>
hipError_t launch_policy_rows(const LogitRows& a, const PolicyTerms& t, void* d, int64_t ldd,
                              float* logp, hipStream_t s) {
    constexpr int64_t kMost = int64_t(1) << 21;  // fewer than 2^32 threads a launch
    for (int64_t row0 = 0; row0 < a.rows; row0 += kMost) {
        const unsigned g = (unsigned)std::min(a.rows - row0, kMost);
        if (a.f32)
            hipLaunchKernelGGL((policy_row_kernel<float, NT>), dim3(g), dim3(NT), 0, s, a, t, row0,
                               (float*)d, ldd, logp);
        else
            hipLaunchKernelGGL((policy_row_kernel<uint16_t, NT>), dim3(g), dim3(NT), 0, s, a, t, row0,
                               (uint16_t*)d, ldd, logp);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int32_t stat_parts(int64_t rows, int64_t vocab) {
    int32_t parts = 1;
    while (rows > 0 && parts < kMaxParts && rows * 2 * parts <= kSplitItems && vocab >= 2 * parts * 4096)
        parts *= 2;
    return parts;
}

hipError_t launch_token_logp(const LogitRows& a, float* logp, float* lse, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    if (a.parts == 1) return launch_stats<STATS_LOGP>(a, PreferenceTerms{}, logp, lse, s);
    hipError_t e = launch_stats<STATS_ONLY>(a, PreferenceTerms{}, nullptr, nullptr, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(logp_kernel, dim3((unsigned)((a.rows * a.parts + 255) / 256)), dim3(256), 0, s, a,
                       logp, lse);
    return hipGetLastError();
}

hipError_t launch_policy(const LogitRows& a, const PolicyTerms& t, void* d, int64_t ldd,
                         float* logp, float* stats, hipStream_t s) {
    if (a.rows <= kSplitRows) {
        hipError_t e;
        if (a.rows > 0) {
            e = launch_stats<STATS_KEEP>(a, PreferenceTerms{}, nullptr, nullptr, s);
            if (e != hipSuccess) return e;
        }
        // 16 KB a workgroup, one round of loads: more cost more starts than
        // they win (61 x 201088 bf16 19 us, of 8 KB 21; 16 x 129280 binary32
        // 11 us, of 32 KB 12)
        const int spans = (int)((row_bytes(a) + (16 << 10) - 1) / (16 << 10));
        const unsigned g = 1 + (d ? (unsigned)(a.rows * spans) : 0);
        if (a.f32)
            hipLaunchKernelGGL((policy_grad_kernel<float, 256>), dim3(g), dim3(256), 0, s, a, t,
                               (float*)d, ldd, spans, logp, stats);
        else
            hipLaunchKernelGGL((policy_grad_kernel<uint16_t, 256>), dim3(g), dim3(256), 0, s, a, t,
                               (uint16_t*)d, ldd, spans, logp, stats);
        return hipGetLastError();
    }
    const int nt = policy_row_threads(a.rows, row_bytes(a));
    hipError_t e = nt == 64    ? launch_policy_rows<64>(a, t, d, ldd, logp, s)
                   : nt == 256 ? launch_policy_rows<256>(a, t, d, ldd, logp, s)
                   : nt == 512 ? launch_policy_rows<512>(a, t, d, ldd, logp, s)
                               : launch_policy_rows<1024>(a, t, d, ldd, logp, s);
    if (e != hipSuccess) return e;
    const double* terms = t.terms;
    int64_t n = a.rows;
    if (n > kSumRows) {
        const int64_t per = (n + kTermSlices - 1) / kTermSlices;
        n = (n + per - 1) / per;
        hipLaunchKernelGGL(policy_slice_kernel, dim3((unsigned)n), dim3(256), 0, s, t, a.rows, per);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        terms = t.slices;
    }
    hipLaunchKernelGGL(policy_sum_kernel, dim3(1), dim3(1024), 0, s, t, terms, n, stats);
    return hipGetLastError();
}

hipError_t launch_preference(const LogitRows& a, const PreferenceTerms& t0, void* d, int64_t ldd,
                             float* seq_logp, float* stats, hipStream_t s) {
    hipError_t e;
    // The statistics keep the last rows in the 256 MB memory-side cache for
    // the gradient (2003 x 50000 binary32, 400 MB: 52 + 147 us all past the
    // cache, 54 + 120 so; with everything through it the statistics of 1.7
    // GB take 203 us instead of 178).
    constexpr int64_t kCache = int64_t(256) << 20;
    PreferenceTerms t = t0;
    t.kept_from = d ? std::max<int64_t>(0, a.rows - kCache / row_bytes(a)) : a.rows;
    if (a.rows > 0) {
        e = launch_stats<STATS_MARK>(a, t, nullptr, nullptr, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((pair_kernel<1024>), dim3((unsigned)t.pairs), dim3(1024), 0, s, a, t, seq_logp);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int spans = grad_spans(a.vocab);
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
