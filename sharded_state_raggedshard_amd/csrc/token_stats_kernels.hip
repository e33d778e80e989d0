// Token statistics over rows of logits for gfx950: log-probability of the
// row's token, entropy and the most probable alternatives in one pass, and
// the logits' gradient from the gradients of both.
//
// With m the row's maximum, d_i = (z_i - m) k, k = log2(e) / T in binary32,
// e_i = 2^d_i, S = sum e and W = sum e d:
//   log p_i = ln 2 d_i - ln S,   H = -sum p log p = ln S - ln 2 W / S.
// One product gives an exponent, with the rounded k: a temperature off by s = up
// to 2^-24 of itself.  What that does to ln S is known at the row's end to first
// order, s E[(z - m) / T] (the second is s^2 / 2 of the exponents' variance), and
// the value's own (z - m) / T is taken in binary64: so log-probabilities are
// free of it.  The entropy keeps it, 2^-24 of that variance, and the gradient,
// whose p_i are then off by 2^-24 (|log p_i| + H) of themselves, like a rounding
// of their exponents.
//
// Both kernels are bound by HBM where rows are many: 4096 x 128256 bf16 (1.05
// GB) take 160 us (6.6 TB/s), with 8 alternatives 169 and with 32 182, and
// their gradient 346 us (6.1 TB/s of 2.1 GB); 6001 x 32003 binary32 116 us and
// 127 with 8.  Few rows are split over workgroups and joined by a second
// launch: 16 x 128256 8.1 us, with 20 alternatives 13.2.
//
// A row's first loads go out before its token is known, so a row that takes no
// part still costs them, 16 KB a workgroup: 4096 x 128256 of which half take
// part 99 us, none 12.5.
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
constexpr float kNear = 1024.0f;
// A value whose exponent lies this far above the others' may be nearly the whole
// row: 2^-10 of it and less is known to its own last digits, more to 2^-22 as all
// sums of 32 values are.
constexpr float kFar = 10.0f;

__device__ __forceinline__ float exponent(float x, float m, float k) { return (x - m) * k; }

// A value that is the same in all lanes, as one that the compiler knows to be.
__device__ __forceinline__ float wave_uniform(float v) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}

// Sums of a thread's share of a row, a part of it or a row around a reference
// that the wave's threads share: the row's token at first (it is in no sum, but
// joins last: where it is nearly the whole row, any sum with it would round
// away the rest that 1 - p and the entropy are made of), then any value seen
// that lies more than a factor 2 above.  A thread's own maximum as a reference
// cost a rescaling of binary64 sums for every 32 values.  `best` is the share's
// own largest value.  Sums are binary64; the C values of a call are added up in
// binary32 in four chains.
struct Sums {
    float best;
    double s, w;

    __device__ __forceinline__ void rescale(float from, float to, float k) {
        const float d = fmaxf(exponent(from, to, k), kLeast);
        const double f = (double)exp2_fast(d);
        w = f * __builtin_fma((double)d, s, w);
        s *= f;
    }

    // While values are taken, e and d are of the exponent x k - c, one FMA, for c
    // = r k rounded, of a reference r with |c| <= kNear: a shift of all of them by
    // gap = r k - c, which plain() takes out again (2^gap by its series: |gap| <=
    // 2^-15, the first term left out below 2^-64).  For bf16 the vector unit
    // would bound rows that HBM brings at its rate: a subtraction and a product
    // are 64 of some 250 instructions for 32 values.
    static __device__ __forceinline__ double gap(float r, float k) {
        const float c = r * k;
        return fabsf(c) <= kNear ? (double)r * (double)k - (double)c : 0.0;
    }
    __device__ __forceinline__ void move(double by) {  // exponents by `by` higher
        const double l = kLn2 * by, f = 1.0 + l * (1.0 + l * (0.5 + l * (1.0 / 6.0)));
        w = f * __builtin_fma(by, s, w);
        s *= f;
    }
    __device__ __forceinline__ void plain(float ref, float k) {
        if (ref != kNegInf) move(-gap(ref, k));
    }

    template <int C, typename F>
    __device__ __forceinline__ void add(const float (&x)[C], F exponent_of) {
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float d = exponent_of(x[i]), e = exp2_fast(d);
            a[i % 4] += e;
            b[i % 4] = __builtin_fmaf(e, fmaxf(d, kLeast), b[i % 4]);
        }
        s += (double)((a[0] + a[1]) + (a[2] + a[3]));
        w += (double)((b[0] + b[1]) + (b[2] + b[3]));
    }

    // A new reference is itself one of the values.  Where it is nearly the whole
    // row, a binary32 sum with it would round away the rest that the entropy and
    // its own log-probability are made of: then the wave's values of its size join
    // s here, exactly 1 each as their exponent is 0, and x goes on without them.
    // It can be only if no other lane's largest value comes near it; doing so for
    // every new reference cost rows of one take 11%.
    template <int C>
    __device__ __forceinline__ void apart(float (&x)[C], float ref) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const bool is = x[i] == ref;
            n += __popcll(__ballot(is));
            x[i] = is ? kNegInf : x[i];
        }
        s += (double)(lanes::lane() == 0 ? n : 0);
    }

    // FAST: by one FMA where it can be; some: values have been taken before.
    template <bool FAST, int C>
    __device__ __forceinline__ void take(float (&x)[C], float& ref, float k, bool some) {
        float v = x[0];
#pragma unroll
        for (int i = 1; i < C; ++i) v = fmaxf(v, x[i]);
        best = fmaxf(best, v);
        if (__any(exponent(v, ref, k) > 1.0f)) {
            const float to = wave_uniform(lanes::max<64>(fmaxf(ref, v)));
            if (some) {
                if (FAST) plain(ref, k);
                rescale(ref, to, k);
            }
            ref = to;
            // (of +inf none does: its difference is a NaN, and shall be the sum's)
            if (__popcll(__ballot(exponent(v, to, k) > -kFar)) == 1) apart(x, to);
            if (FAST) move(gap(to, k));
        }
        const float r = ref == kNegInf ? 0.0f : ref;  // -inf - 0 gives 2^-inf = 0
        const float c = wave_uniform(r * k);
        if (FAST && fabsf(c) <= kNear)
            add(x, [=](float v) { return __builtin_fmaf(v, k, -c); });
        else
            add(x, [=](float v) { return exponent(v, r, k); });
    }
};

// What the statistics of a row come to, its token among the values.
struct RowEnd {
    float m, token;     // m: the reference
    bool empty;         // nothing but -inf
    double rest, S;     // sums of e, `rest` without the token's
    double ln_s, down;  // ln S; E[(m - z) / T]
};

__device__ __forceinline__ RowEnd row_end(const Sums& x, float ref, float token, bool has, float k) {
    RowEnd e;
    const float r = ref == kNegInf ? 0.0f : ref, d = exponent(token, r, k);
    const float own = has ? exp2_fast(d) : 0.0f;
    e.m = r;
    e.token = token;
    e.rest = x.s;
    e.S = x.s + (double)own;
    e.empty = ref == kNegInf && e.S == 0.0;
    const double w = x.w + (has ? (double)own * (double)fmaxf(d, kLeast) : 0.0);
    // ln(1 + rest) of a small rest: 1 + rest has rounded its digits away
    const bool sure = own == 1.0f && e.rest < 0x1p-20;
    e.ln_s = e.empty ? 0.0 : sure ? e.rest - 0.5 * e.rest * e.rest : log(e.S);
    e.down = e.empty ? 0.0 : -kLn2 * w / e.S;
    return e;
}

// log p of value v.  (Neither it nor an entropy passes 0 by a rounding.)
__device__ __forceinline__ double log_p(const TokenStats& a, const RowEnd& e, float v) {
    const double l = ((double)v - (double)e.m) * a.scale - (e.ln_s - a.skew * e.down);
    return l > 0.0 ? 0.0 : l;
}
__device__ __forceinline__ double entropy(const RowEnd& e) {
    const double h = e.ln_s + e.down;
    return h < 0.0 ? 0.0 : h;
}

// The outputs of a row but its alternatives, by one thread.
__device__ __forceinline__ void write_row(const TokenStats& a, int64_t row, bool live, const RowEnd& e) {
    const bool none = !live || e.empty;
    if (a.logp) a.logp[row] = none ? 0.0f : (float)log_p(a, e, e.token);
    if (a.entropy) a.entropy[row] = none ? 0.0f : (float)entropy(e);
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
    a.top_logp[row * a.top + rank] = bad ? __builtin_nanf("") : id < 0 ? kNegInf : (float)log_p(a, e, v);
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
    // The same, but of more than kRoom of them a fair choice is left (each takes a
    // place of those before it at random, and keeps it if there is one), in which
    // v and id need not match.
    __device__ __forceinline__ void sample(float x, int i) {
        const uint32_t before = (uint32_t)atomicAdd(&n, 1);
        const uint32_t at = before < kRoom ? before : __umulhi((uint32_t)i * 2654435761u, before + 1);
        if (at < kRoom) {
            v[at] = x;
            id[at] = i;
        }
    }
    __device__ __forceinline__ bool full() const {
        return __hip_atomic_load(&n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) > kRoom;
    }
};

__device__ __forceinline__ float lane_value(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

// By value and then by index, as one comparison: v in i comes before w in j if
// order(v, i) > order(w, j).  (-0 counts as 0.  Two comparisons in a row, of the
// value and then of the index, wait for each other's loads: 160 us for a row of
// ties in 16 parts, 49 so.)
__device__ __forceinline__ uint64_t order(float v, int i) {
    const uint32_t bits = __float_as_uint(v + 0.0f);
    const uint32_t up = bits ^ (bits & 0x80000000u ? 0xffffffffu : 0x80000000u);
    return (uint64_t)up << 32 | (uint32_t)~i;
}
__device__ __forceinline__ uint64_t lane_key(uint64_t key, int l) {
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(key >> 32), l);
    return (uint64_t)hi << 32 | (uint32_t)__builtin_amdgcn_readlane((uint32_t)key, l);
}

// The n-th largest of the wave's 64 values (n <= 64): the least of those that
// fewer than n are above.
__device__ __forceinline__ float nth_of_wave(float v, int n) {
    int above = 0;
#pragma unroll
    for (int l = 0; l < 64; ++l) above += lane_value(v, l) > v ? 1 : 0;
    return wave_uniform(-lanes::max<64>(above < n ? -v : kNegInf));
}

// Ranks of n candidates, and write(rank, value, index) for the best `top` of
// them, by one wave; write(rank, -inf, -1) for what is missing.
template <typename F>
__device__ __forceinline__ void write_best(const float* v, const int32_t* id, int n, int top, F write) {
    const int lane = lanes::lane();
    if (n <= 64) {
        const float mine = lane < n ? v[lane] : kNegInf;
        const int i = lane < n ? id[lane] : 0x7fffffff;
        const uint64_t key = order(mine, i);
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += lane_key(key, j) > key ? 1 : 0;
        if (lane < n && rank < top) write(rank, mine, i);
    } else {
        for (int i = lane; i < n; i += 64) {
            const float mine = v[i];
            const int at = id[i];
            const uint64_t key = order(mine, at);
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) rank += order(v[j], id[j]) > key ? 1 : 0;
            if (rank < top) write(rank, mine, at);
        }
    }
    for (int r = n + lane; r < top; r += 64) write(r, kNegInf, -1);
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

// A thread's largest value is kept for up to kSegments stretches of its share.
constexpr int kSegments = 8, kTake = 4;  // kTake pieces a thread in flight

template <int NT>
struct StatsLds {
    // of the waves; two rows' worth, as a row's end is written by the first
    // wave while the others go on
    double s[2][NT / 64], w[2][NT / 64];
    float ref[2][NT / 64];
    float group[64];
    float least;
    float best[kSegments][NT];
    int32_t hot[kSegments * NT];
    int32_t n_hot;
    float red[NT / 64];
    Candidates c;
};

// The stretches of a part: takes of kTake NT pieces, `per` of them each.
template <int NT>
struct Segments {
    int takes, per, n;
    __device__ __forceinline__ explicit Segments(const Part& part) {
        takes = part.v1 > part.v0 ? (part.v1 - part.v0 + kTake * NT - 1) / (kTake * NT) : 0;
        per = takes > kSegments ? (takes + kSegments - 1) / kSegments : 1;
        n = (takes + per - 1) / per;
    }
};

// The part's best a.top values into lds.c, unordered, from the threads' own
// largest values.  64 groups of neighbouring threads: the n-th largest of the
// groups' largest values is reached by n values at least, so the n best are
// among what reaches it: about n to 2 n values, in as many threads' stretches,
// which the workgroup reads again (from a cache, if the first read went
// through it).  lds.c.n passes kRoom where that many tie with it or a few
// stretches hold them; then the rest is not looked at.  Begins behind the
// barrier that lds.group is written before; ends with one.
// HELD: a part is one take, still in registers.
template <typename T, int NT, bool HELD>
__device__ __forceinline__ void gather_best(const T* z, const Pieces<T>& ps, const Part& part, const Segments<NT>& seg,
                                            int y, const Single<T>& one, const u32x4 (&held)[kTake], float best,
                                            int n, StatsLds<NT>& lds) {
    constexpr int N = Vec<T>::n, B = 4;
    const int tid = threadIdx.x;
    if (tid < 64) {
        if (tid == 0) lds.n_hot = lds.c.n = 0;
        const float least = nth_of_wave(lds.group[tid], n);
        if (tid == 0) lds.least = least;
    }
    __syncthreads();
    const float least = lds.least;
    const auto fits = [&](float x) { return x >= least && x > kNegInf; };
    if (one.at >= 0 && fits(one.value())) lds.c.add(one.value(), one.at);
    if (HELD) {
        if (fits(best)) {
#pragma unroll
            for (int u = 0; u < kTake; ++u) {
                float x[N];
                Vec<T>::open(held[u], x);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (fits(x[i])) lds.c.add(x[i], ps.head + (part.v0 + tid + u * NT) * N + i);
            }
        }
        __syncthreads();
        return;
    }
    for (int i = 0; i < seg.n; ++i)
        if (fits(lds.best[i][tid])) lds.hot[atomicAdd(&lds.n_hot, 1)] = i * NT + tid;
    __syncthreads();
    // piece j of stretch i of thread h is part.v0 + h + (i length + j) NT;
    // places are dealt out by a power of two that holds a stretch
    const int length = seg.per * kTake, shift = length > 1 ? 32 - __builtin_clz((unsigned)(length - 1)) : 0;
    const int all = lds.n_hot << shift, yv = ps.piece(y);
    const T* base = z + ps.head;
#pragma unroll 1
    for (int q0 = tid; q0 < all && !lds.c.full(); q0 += B * NT) {
        u32x4 raw[B];
        int at[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int q = q0 + b * NT;
            at[b] = -1;
            if (q >= all) continue;
            const int unit = lds.hot[q >> shift], j = q & ((1 << shift) - 1);
            const int v = part.v0 + unit % NT + ((unit / NT) * length + j) * NT;
            if (j < length && v < part.v1 && v != yv) at[b] = v;
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (at[b] >= 0) raw[b] = load16(base + at[b] * N);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (at[b] < 0) continue;
            float x[N];
            Vec<T>::open(raw[b], x);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (fits(x[i])) lds.c.add(x[i], ps.head + at[b] * N + i);
        }
    }
    __syncthreads();
}

// The same for a part whose candidates did not fit: what lies above the bound
// alone, and as far as n are missing then, its equals by index.  That is little
// in a row masked with the type's lowest value.  Where it does not fit either,
// the n-th largest of a sample is a higher bound that n values reach, and about
// n / kRoom of them lie above it: rows of 128256 with 7 values beside the lowest
// and 8 alternatives 383 us for 4096 of them (170 with -inf in their place; the
// next smaller value found pass by pass took 2284).
template <typename T, int NT>
__device__ void gather_slow(const T* z, const Pieces<T>& ps, const Part& part, int n, StatsLds<NT>& lds) {
    constexpr int N = Vec<T>::n;
    const int tid = threadIdx.x;
    const T* base = z + ps.head;
    const int edges = part.ends ? ps.edges : 0;
    float last = lds.least;
    int above;
    for (;;) {
        __syncthreads();  // every thread has seen what is overwritten now
        if (tid == 0) lds.c.n = 0;
        __syncthreads();
        for (int v = part.v0 + tid; v < part.v1; v += NT) {
            float x[N];
            Vec<T>::open(load16(base + v * N), x);
            for (int i = 0; i < N; ++i)
                if (x[i] > last) lds.c.sample(x[i], ps.head + v * N + i);
        }
        if (tid < edges) {
            const float x = Vec<T>::one(z[ps.edge(tid)]);
            if (x > last) lds.c.sample(x, ps.edge(tid));
        }
        __syncthreads();
        above = lds.c.n;
        __syncthreads();
        if (above <= kRoom) break;
        float least = -kNegInf;
        for (int i = tid; i < kRoom; i += NT) {
            const float x = lds.c.v[i];
            int higher = 0;
#pragma unroll 8
            for (int j = 0; j < kRoom; ++j) higher += lds.c.v[j] > x ? 1 : 0;
            if (higher < n) least = fminf(least, x);
        }
        const float of_wave = -lanes::max<64>(-least);
        if (lanes::lane() == 0) lds.red[tid >> 6] = of_wave;
        __syncthreads();
        last = lds.red[0];
        for (int i = 1; i < NT / 64; ++i) last = fminf(last, lds.red[i]);
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

// What stats_kernel does beside the sums: nothing; finds the alternatives; does
// so in parts of one take.
enum { TOP_NONE = 0, TOP_LONG = 1, TOP_HELD = 2 };

// One workgroup per part of a row; its first wave ends the row while the
// others go on to the next.  256 threads: with 1024 a row's end is too large a
// share of it.  Four waves a SIMD is what the registers of 32 values and 32 more
// under way leave without spills (five without alternatives spill: 4096 x 128256
// bf16 163 us, 200); binary32 with alternatives is held to five (5000 x 9382 45
// us, 52 with four).  What the alternatives cost (8 us of 170 with 8) is the
// row's end: five barriers, and the stretches read again.
template <typename T, int NT, int MODE>
__global__ __launch_bounds__(NT, sizeof(T) == 4 && MODE == TOP_LONG ? 5 : 4) void stats_kernel(TokenStats a) {
    constexpr bool TOP = MODE != TOP_NONE;
    // The next take is under way while one is computed, and bf16 exponents are
    // one FMA each (4096 x 128256 bf16 with 8 alternatives 184 us without both,
    // 177 with the FMA alone, 188 with the loads alone).  Binary32 has half the
    // values to compute for a byte, and with alternatives no registers for it
    // (5000 x 9382 49 us, 57); a part of one take has latency for its bound (16
    // x 128256 bf16 12.2 us, 12.9).
    constexpr bool FAST = sizeof(T) == 2 && MODE != TOP_HELD;
    constexpr bool AHEAD = MODE == TOP_NONE || (MODE == TOP_LONG && sizeof(T) == 2);
    constexpr int N = Vec<T>::n, U = kTake, WAVES = NT / 64;
    __shared__ StatsLds<NT> lds;
    const int tid = threadIdx.x, lane = lanes::lane();
    const float k = a.k;
    const int64_t items = a.rows * a.parts;
    int turn = 0;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = a.parts == 1 ? item : item / a.parts;
        const int index = (int)(item - row * a.parts);
        // the first loads need nothing but the row's place: they are under way
        // while the token's index and value are fetched
        const T* z = static_cast<const T*>(a.z) + row * a.ld;
        const Pieces<T> ps(z, a.vocab);
        const Part part = part_of(z, ps, index, a.parts);
        const Segments<NT> seg(part);
        const T* base = z + ps.head;
        u32x4 raw[U];
        const auto load = [&](int t) {
            const int v = part.v0 + tid + t * U * NT;
            if (AHEAD && part.v0 + (t + 1) * U * NT <= part.v1) {  // all of them, in every thread
#pragma unroll
                for (int u = 0; u < U; ++u) raw[u] = load16_once(base + (v + u * NT) * N);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    raw[u] = Vec<T>::lowest();
                    if (v + u * NT < part.v1) raw[u] = load16_once(base + (v + u * NT) * N);
                }
            }
        };
        load(0);
        const int64_t target = a.target ? a.target[row] : -1;
        if (a.target && (target < 0 || target >= a.vocab)) {
            if (a.parts == 1 && tid < 64) {
                if (tid == 0) write_row(a, row, false, RowEnd{});
                if (TOP && tid < a.top) write_top(a, row, tid, 0.0f, -1, RowEnd{});
            }
            continue;
        }
        const int y = (int)target;
        const float token = y >= 0 ? Vec<T>::one(z[y]) : kNegInf;
        const Single<T> one(z, ps, part, y);
        const int yv = ps.piece(y);
        Sums run{kNegInf, 0.0, 0.0};
        float ref = wave_uniform(token), best = kNegInf;
        for (int t = 0, next = seg.per, i = 0; t < seg.takes; ++t) {
            if (!AHEAD && t > 0) load(t);
            const int there = yv - part.v0 - t * U * NT;
            if (!AHEAD || (there >= 0 && there < U * NT)) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (tid + u * NT == there) raw[u] = Vec<T>::lowest();
            }
            float x[U * N];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[N];
                Vec<T>::open(raw[u], f);
#pragma unroll
                for (int i = 0; i < N; ++i) x[u * N + i] = f[i];
            }
            if (AHEAD && t + 1 < seg.takes) load(t + 1);
            run.template take<FAST>(x, ref, k, t > 0);
            if (TOP && (t + 1 == next || t + 1 == seg.takes)) {
                lds.best[i++][tid] = run.best;
                best = fmaxf(best, run.best);
                run.best = kNegInf;
                next += seg.per;
            }
        }
        if (tid < 64) {
            float x[1] = {one.at == y ? kNegInf : one.value()};
            run.template take<FAST>(x, ref, k, true);
        }
        if (FAST) run.plain(ref, k);
        const double s = lanes::sum64(run.s), w = lanes::sum64(run.w);
        const int wave = tid >> 6;
        turn ^= 1;
        if (lane == 0) {
            lds.s[turn][wave] = s;
            lds.w[turn][wave] = w;
            lds.ref[turn][wave] = ref;
        }
        if (TOP) {
            const float group = lanes::max<WAVES>(best);
            if (tid % WAVES == 0) lds.group[tid / WAVES] = group;
        }
        __syncthreads();
        if (TOP) {
            gather_best<T, NT, MODE == TOP_HELD>(z, ps, part, seg, y, one, raw, best, a.top, lds);
            // (out of the row's way, or rows without need of it take 2% longer)
            if (__builtin_expect(lds.c.n > kRoom, 0)) gather_slow<T, NT>(z, ps, part, a.top, lds);
        }
        if (tid >= 64) continue;
        // the waves' sums, a lane each and all of them in every lane
        const int from = lane % WAVES;
        Sums all{kNegInf, lds.s[turn][from], lds.w[turn][from]};
        const float mine = lds.ref[turn][from], top = wave_uniform(lanes::max<64>(mine));
        all.rescale(mine, top == kNegInf ? 0.0f : top, k);
#pragma unroll
        for (int off = 1; off < WAVES; off <<= 1) {
            all.s += __shfl_xor(all.s, off, 64);
            all.w += __shfl_xor(all.w, off, 64);
        }
        RowEnd e{};
        if (a.parts == 1) {
            e = row_end(all, top, token, y >= 0, k);
            if (tid == 0) write_row(a, row, true, e);
        } else if (tid == 0) {
            a.stat[item] = PartStat{all.s, all.w, top, token};
        }
        if (!TOP) continue;
        const int n = lds.c.n;
        const auto write = [&](int rank, float v, int id) {
            if (a.parts == 1) {
                write_top(a, row, rank, v, id, e);
            } else {
                a.best[item * a.top + rank] = v;
                a.best_id[item * a.top + rank] = id;
            }
        };
        write_best(lds.c.v, lds.c.id, n, a.top, write);
    }
}

// Rows in several parts: a wave joins a row's statistics, a lane a part, and
// picks the best of its parts' best.
constexpr int kMostBest = kMaxParts * kMaxTop;
__global__ __launch_bounds__(64) void stats_join_kernel(TokenStats a) {
    __shared__ float lv[kMostBest];
    __shared__ int32_t li[kMostBest];
    __shared__ int32_t kept;
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    // 64 / parts lanes a part, the first ones with its largest values.  All
    // loads go out at once (of a row that takes no part they are of no use).
    const int lanes_each = 64 / a.parts, at0 = lane % lanes_each;
    const int64_t first = row * a.parts * a.top + (int64_t)(lane / lanes_each) * a.top;
    const float* v = a.best + first;
    const int32_t* id = a.best_id + first;
    constexpr int U = 8;
    float x[U];
    int32_t xi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = at0 + u * lanes_each;
        x[u] = kNegInf;
        xi[u] = -1;
        if (at < a.top) {
            x[u] = v[at];
            xi[u] = id[at];
        }
    }
    const PartStat p = a.stat[row * a.parts + lane % a.parts];
    const int64_t y = a.target ? a.target[row] : -1;
    const bool live = !a.target || (y >= 0 && y < a.vocab);
    RowEnd e{};
    if (live) {
        const float top = wave_uniform(lanes::max<64>(p.m));
        Sums all{kNegInf, p.s, p.w};
        all.rescale(p.m, top == kNegInf ? 0.0f : top, a.k);
        for (int off = 1; off < a.parts; off <<= 1) {
            all.s += __shfl_xor(all.s, off, 64);
            all.w += __shfl_xor(all.w, off, 64);
        }
        e = row_end(all, top, p.token, y >= 0, a.k);
    }
    if (lane == 0) write_row(a, row, live, e);
    if (a.top == 0) return;
    if (!live) {
        if (lane < a.top) write_top(a, row, lane, 0.0f, -1, e);
        return;
    }
    // the n-th largest of the lanes' first values is reached by little more than n
    const float least = nth_of_wave(x[0], a.top);
    if (lane == 0) kept = 0;
    __syncthreads();
    const auto keep = [&](float f, int i) {
        if (!(f >= least) || f == kNegInf) return false;
        const int at = atomicAdd(&kept, 1);
        lv[at] = f;
        li[at] = i;
        return true;
    };
    bool more = true;  // they come in order
#pragma unroll
    for (int u = 0; u < U; ++u) more = more && keep(x[u], xi[u]);
    for (int i = at0 + U * lanes_each; i < a.top && more; i += lanes_each) more = keep(v[i], id[i]);
    __syncthreads();
    write_best(lv, li, kept, a.top, [&](int rank, float f, int i) { write_top(a, row, rank, f, i, e); });
}

// ---------------------------------------------------------------- gradient

// dz_i = (c ([i = y] - p_i) - b p_i (log p_i + H)) / T for c = dlogp and b =
// dentropy.  With q = E[(m - z) / T], log p_i + H = ln 2 d_i + q, so a value
// takes p_i (slope d_i + level), and the token's own value c (1 - p) from the
// sum of the others.
struct GradRow {
    float m, level, slope, own;
};

// One workgroup per span of a row, as the values lie in memory.  (The last rows
// first, after statistics that leave them in the memory-side cache, gained
// nothing: 511 us for both, 515 so, 550 with all loads kept.)
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

template <int NT, int MODE>
hipError_t launch_stats_mode(const TokenStats& a, hipStream_t s) {
    const unsigned g = grid_of(a.rows * a.parts);
    if (a.f32)
        hipLaunchKernelGGL((stats_kernel<float, NT, MODE>), dim3(g), dim3(NT), 0, s, a);
    else
        hipLaunchKernelGGL((stats_kernel<uint16_t, NT, MODE>), dim3(g), dim3(NT), 0, s, a);
    return hipGetLastError();
}

// The most pieces of any part are part_of()'s: whole lines of 8, behind up to
// 7 pieces of the line that the row starts in.
template <int NT>
hipError_t launch_stats_nt(const TokenStats& a, hipStream_t s) {
    if (a.top == 0) return launch_stats_mode<NT, TOP_NONE>(a, s);
    const int64_t pieces = row_bytes(a.vocab, a.f32) / 16;
    const int64_t most = a.parts == 1 ? pieces : ((pieces + 7 + a.parts - 1) / a.parts + 7) / 8 * 8;
    return most <= kTake * NT ? launch_stats_mode<NT, TOP_HELD>(a, s) : launch_stats_mode<NT, TOP_LONG>(a, s);
}

// Rows of up to this many bytes take one wave each: a workgroup's barriers cost
// more than its threads win on a kilobyte or two each.
constexpr int64_t kWaveRow = 16 << 10;
// Values of a row that one workgroup of the gradient writes.
constexpr int64_t kGradSpan = 4096;

}  // namespace

hipError_t launch_token_stats(const TokenStats& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    hipError_t e = row_bytes(a.vocab, a.f32) <= kWaveRow ? launch_stats_nt<64>(a, s) : launch_stats_nt<256>(a, s);
    if (e != hipSuccess || a.parts == 1) return e;
    hipLaunchKernelGGL(stats_join_kernel, dim3((unsigned)a.rows), dim3(64), 0, s, a);
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
