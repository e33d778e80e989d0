// Tokens to experts and back, for gfx950: a stable counting sort of the
// router's choices by expert, the copy of tokens to their slots, the weighted
// sum of the slots back to tokens, and its gradient.
//
// The sort moves 12 bytes a choice and is bound by its launches (5 us up to
// 1024 choices, 11 us up to 131,072).  The others move rows: a token's row is
// read once for its k slots (dispatch, gradient) or written once from them
// (combine), a wave or workgroup to a token, so everything is read once and
// written once; HBM bounds them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "experts.hpp"
#include "lanes.hpp"
#include "row_common.hpp"

namespace rs {
namespace {

using namespace rows;

// ------------------------------------------------------------------- sort

// Expert of choice i, `experts` for one that is not taken.
__device__ __forceinline__ int choice(const ExpertSort& a, uint32_t i) {
    const uint32_t t = i / (uint32_t)a.k, j = i - t * (uint32_t)a.k;
    if (a.mask && a.mask[t] == 0) return a.experts;
    const int64_t id = a.topk[(int64_t)t * a.ldk + j];
    return id >= 0 && id < a.experts ? (int)id : a.experts;
}

__device__ __forceinline__ int lds_load(const int* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void lds_store(int* p, int v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// Choices [c0, c1) counted per expert by one wave (hist: LDS, may be shared).
__device__ __forceinline__ void count_choices(const ExpertSort& a, int64_t c0, int64_t c1, int* hist) {
    for (int64_t i = c0 + lanes::lane(); i < c1; i += 64) {
        const int id = choice(a, (uint32_t)i);
        if (id < a.experts) atomicAdd(&hist[id], 1);
    }
}

// Slots of 64 consecutive choices, a lane each, by one wave (id: the choice's
// expert): the next of expert e is first[e] + next[e].  Lanes of one expert
// find each other by the bits of its id, and the lowest of them moves next[e]
// on; a wave's LDS accesses take effect in its order.
__device__ __forceinline__ int place(int id, int experts, int bits, const int* first, int* next) {
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
        const bool one = (id >> b) & 1;
        const uint64_t have = __ballot(one);
        same &= one ? have : ~have;
    }
    const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    if (id >= experts) return -1;
    const int at = lds_load(&next[id]);
    if (rank == 0) lds_store(&next[id], at + __popcll(same));
    return first[id] + at + rank;
}
__device__ __forceinline__ int id_bits(int experts) { return 32 - __builtin_clz((unsigned)experts); }

// Slots of choices [c0, c1) by one wave, in order.
__device__ __forceinline__ void place_choices(const ExpertSort& a, int64_t c0, int64_t c1, const int* first,
                                              int* next) {
    const int bits = id_bits(a.experts);
    for (int64_t i0 = c0; i0 < c1; i0 += 64) {
        const int64_t i = i0 + lanes::lane();
        const int slot = place(i < c1 ? choice(a, (uint32_t)i) : a.experts, a.experts, bits, first, next);
        if (i < c1) a.slot[i] = slot;
    }
}

// counts[0 .. experts) to first slots, by one wave; `write`: to d_start too.
__device__ __forceinline__ void first_slots(const ExpertSort& a, int* counts, bool write) {
    const int lane = lanes::lane(), per = (a.experts + 63) / 64;
    const int e0 = lane * per;
    int sum = 0;
    for (int e = e0; e < e0 + per && e < a.experts; ++e) sum += (counts[e] + a.align - 1) / a.align * a.align;
    int before = (int)lanes::sum_upto((uint32_t)sum) - sum;
    for (int e = e0; e < e0 + per && e < a.experts; ++e) {
        const int c = (counts[e] + a.align - 1) / a.align * a.align;
        counts[e] = before;
        if (write) a.start[e] = before;
        before += c;
        if (write && e == a.experts - 1) a.start[a.experts] = before;
    }
}

// All choices in one workgroup of WAVES waves, up to kSmallSteps a lane, which
// are read once.
constexpr int kSmallSteps = 8;
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void sort_small_kernel(ExpertSort a) {
    extern __shared__ int lds[];
    constexpr int NT = 64 * WAVES;
    const int tid = threadIdx.x, wave = lanes::wave(), E = a.experts;
    int* hist = lds + wave * E;  // of the wave
    int* first = lds + WAVES * E;
    const int n = (int)(a.rows * a.k), steps = (n + NT - 1) / NT;
    const int c0 = wave * steps * 64 + lanes::lane();
    int id[kSmallSteps];
#pragma unroll
    for (int s = 0; s < kSmallSteps; ++s) id[s] = s < steps && c0 + s * 64 < n ? choice(a, c0 + s * 64) : E;
    for (int i = tid; i < WAVES * E; i += NT) lds[i] = 0;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSmallSteps; ++s)
        if (id[s] < E) atomicAdd(&hist[id[s]], 1);
    __syncthreads();
    for (int e = tid; e < E; e += NT) {
        int sum = 0;
        for (int w = 0; w < WAVES; ++w) {
            const int c = lds[w * E + e];
            lds[w * E + e] = sum;
            sum += c;
        }
        first[e] = sum;
        a.count[e] = sum;
    }
    __syncthreads();
    if (wave == 0) first_slots(a, first, true);
    __syncthreads();
    const int bits = id_bits(E);
#pragma unroll
    for (int s = 0; s < kSmallSteps; ++s) {
        if (s >= steps) break;
        const int slot = place(id[s], E, bits, first, hist);
        if (c0 + s * 64 < n) a.slot[c0 + s * 64] = slot;
    }
}

// Many choices, first of three launches: chunk c counts its choices.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(ExpertSort a, int64_t chunk) {
    extern __shared__ int hist[];
    const int tid = threadIdx.x, E = a.experts;
    for (int e = tid; e < E; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const int64_t n = a.rows * a.k, c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk);
    const int64_t per = chunk / (kSortThreads / 64), w0 = c0 + lanes::wave() * per;
    count_choices(a, min(w0, c1), min(w0 + per, c1), hist);
    __syncthreads();
    for (int e = tid; e < E; e += kSortThreads) a.part[(int64_t)blockIdx.x * E + e] = hist[e];
}

// Second: an expert's counts to what the chunks before hold, a lane an expert
// and a wave a sixteenth of the chunks, all of a lane's loads in flight at once.
constexpr int kScanWaves = 16;
__global__ __launch_bounds__(64 * kScanWaves) void sort_scan_kernel(ExpertSort a, int chunks) {
    constexpr int EACH = (int)(kSortChunks / kScanWaves);
    __shared__ int sums[kScanWaves][64];
    const int lane = lanes::lane(), wave = lanes::wave(), E = a.experts;
    const int e = blockIdx.x * 64 + lane, c0 = wave * EACH;
    int32_t* part = a.part + (int64_t)c0 * E + e;
    int x[EACH], sum = 0;
#pragma unroll
    for (int c = 0; c < EACH; ++c) x[c] = e < E && c0 + c < chunks ? part[(int64_t)c * E] : 0;
#pragma unroll
    for (int c = 0; c < EACH; ++c) sum += x[c];
    sums[wave][lane] = sum;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kScanWaves; ++w) {
        if (w == wave) before = all;
        all += sums[w][lane];
    }
#pragma unroll
    for (int c = 0; c < EACH; ++c) {
        if (e < E && c0 + c < chunks) part[(int64_t)c * E] = before;
        before += x[c];
    }
    if (wave == 0 && e < E) a.count[e] = all;
}

// Third: the slots.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(ExpertSort a, int64_t chunk) {
    constexpr int WAVES = kSortThreads / 64;
    extern __shared__ int lds[];
    const int tid = threadIdx.x, wave = lanes::wave(), E = a.experts;
    int* hist = lds;
    int* first = lds + WAVES * E;
    for (int i = tid; i < WAVES * E; i += kSortThreads) hist[i] = 0;
    for (int e = tid; e < E; e += kSortThreads) first[e] = a.count[e];
    __syncthreads();
    const int64_t n = a.rows * a.k, b0 = blockIdx.x * chunk, b1 = min(n, b0 + chunk);
    const int64_t per = chunk / WAVES;
    const int64_t c0 = min(b0 + wave * per, b1), c1 = min(c0 + per, b1);
    count_choices(a, c0, c1, hist + wave * E);
    if (wave == 0) first_slots(a, first, blockIdx.x == 0);
    __syncthreads();
    for (int e = tid; e < E; e += kSortThreads) {
        int sum = a.part[(int64_t)blockIdx.x * E + e];
        for (int w = 0; w < WAVES; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = sum;
            sum += c;
        }
    }
    __syncthreads();
    place_choices(a, c0, c1, first, hist + wave * E);
}

// -------------------------------------------------------------------- rows

// A row of `hidden` values in 16-byte pieces and a tail of single values.
// Rows of an odd length start at any element, on either side of a copy.
template <typename T>
struct RowShape {
    static constexpr int N = Vec<T>::n;
    int pieces, tail;
    __device__ __forceinline__ explicit RowShape(int64_t hidden)
        : pieces((int)(hidden / N)), tail((int)(hidden % N)) {}
};

// Rows at 16-byte addresses are written past the caches.  Others share lines
// with their neighbours, which the L2 puts together: 17,300 rows of 1003
// binary32 values 15 us instead of 20.
template <bool LINES, typename T>
__device__ __forceinline__ void put16(T* p, const u32x4& v) {
    if (LINES)
        store16(p, v);
    else
        *reinterpret_cast<u32x4_any*>(p) = v;
}
template <typename T>
bool whole_lines(const T* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)sizeof(T) % 16 == 0;
}

// The padding rows of all experts' segments to 0: the r-th of them by wave r of
// the launch's first kPaddingWaves, then the next ones.  A lane knows an
// expert's, and the lanes' sums where they begin, so that few experts with many
// of them keep as many waves busy as many with few (2 rows of 6421 bf16 values,
// 16 experts' segments of 128: 8.1 us, 33 with a few waves for each expert).
constexpr int64_t kPaddingWaves = 4096;
template <bool LINES, typename T>
__device__ __forceinline__ void zero_padding(const ExpertRows& a, T* y, int64_t ldy, int64_t wave, int64_t waves) {
    constexpr int GROUPS = 4;  // 64 experts each, in flight together
    if (wave >= kPaddingWaves) return;
    waves = min(waves, kPaddingWaves);
    const RowShape<T> shape(a.hidden);
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int lane = lanes::lane();
    int64_t r = wave, before = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64 * GROUPS) {
        int64_t start[GROUPS], next[GROUPS];
        int32_t count[GROUPS];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int e = min(e0 + 64 * g + lane, a.experts - 1);
            start[g] = a.start[e];
            next[g] = a.start[e + 1];
            count[g] = a.count[e];
        }
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            if (e0 + 64 * g >= a.experts) break;
            // whatever the tables hold, rows of [0, slots) only
            const int used = (int)min(max(int64_t(0), min(start[g], a.slots)) + max(0, count[g]), a.slots);
            const int end = (int)max(int64_t(0), min(next[g], a.slots));
            const uint32_t n = e0 + 64 * g + lane < a.experts && end > used ? (uint32_t)(end - used) : 0u;
            const uint32_t upto = lanes::sum_upto(n);
            const uint32_t all = __builtin_amdgcn_readlane(upto, 63);
            for (; r - before < (int64_t)all; r += waves) {
                const uint32_t i = (uint32_t)(r - before);
                const uint64_t later = __ballot(upto > i);
                if (later == 0) break;  // sums that passed 32 bits
                const int l = __builtin_ctzll(later);
                const uint32_t in = i - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l));
                if (in >= (uint32_t)__builtin_amdgcn_readlane(n, l)) continue;
                T* to = y + ((int64_t)__builtin_amdgcn_readlane(used, l) + in) * ldy;
                for (int p = lane; p < shape.pieces; p += 64) put16<LINES>(to + p * shape.N, zero);
                if (lane < shape.tail) to[shape.pieces * shape.N + lane] = T(0);
            }
            before += all;
        }
    }
}

// A wave's share of a row: pieces [p0, p1), at most 64 U of them; the last
// share has the tail.
struct Share {
    int p0, p1;
    bool last;
};
template <int U>
__host__ __device__ __forceinline__ int shares_of(int pieces) {
    return pieces <= 64 * U ? 1 : (pieces + 64 * U - 1) / (64 * U);
}
__device__ __forceinline__ Share share_of(int pieces, int shares, int i) {
    const int per = (pieces + shares - 1) / shares;
    const int p0 = i * per;
    return Share{p0 < pieces ? p0 : pieces, p0 + per < pieces ? p0 + per : pieces, i == shares - 1};
}

constexpr int kRowThreads = 256;

// A wave takes a share of a token's row and writes it to its k slots.  Bound by
// HBM's writes: 16384 x 2880 bf16 to 4 slots 72.5 us (6.5 TB/s), 8192 x 7168 to
// 8 181 us (5.8 TB/s), and 59 us more for 235 MB of padding rows (segments of
// 128).  Weights are free (8192 x 7168 182 us with and without).  Two pieces a
// lane: 16384 x 2880 four 76; 2000 x 4096 binary32 to 6 41.5, four 44.
constexpr int kDispatchPieces = 2;
template <typename T, bool WEIGHTED, bool LINES>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(ExpertRows a, const T* x, int64_t ldx, T* y, int64_t ldy,
                                                               int shares) {
    constexpr int N = Vec<T>::n, U = kDispatchPieces, WAVES = kRowThreads / 64;
    const RowShape<T> shape(a.hidden);
    const int lane = lanes::lane();
    const int64_t items = a.rows * shares, wave0 = blockIdx.x * (int64_t)WAVES + lanes::wave();
    const int64_t waves = gridDim.x * (int64_t)WAVES;
    for (int64_t item = wave0; item < items; item += waves) {
        const int64_t t = item / shares;
        const Share sh = share_of(shape.pieces, shares, (int)(item - t * shares));
        const T* from = x + t * ldx;
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = sh.p0 + u * 64 + lane;
            if (p < sh.p1) v[u] = load16(from + p * N);
        }
        const bool tail = sh.last && lane < shape.tail;
        const int tail_at = shape.pieces * N + lane;
        const T one = tail ? from[tail_at] : T(0);
        const int32_t* slot = a.slot + t * a.k;
        for (int j = 0; j < a.k; ++j) {
            const int s = slot[j];
            if (s < 0 || s >= a.slots) continue;
            T* to = y + s * ldy;
            const float w = WEIGHTED ? a.weight[t * a.ldw + j] : 1.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = sh.p0 + u * 64 + lane;
                if (p >= sh.p1) continue;
                if (WEIGHTED) {
                    float f[N];
                    Vec<T>::open(v[u], f);
#pragma unroll
                    for (int i = 0; i < N; ++i) f[i] *= w;
                    put16<LINES>(to + p * N, Vec<T>::close(f));
                } else {
                    put16<LINES>(to + p * N, v[u]);
                }
            }
            if (tail) to[tail_at] = WEIGHTED ? Vec<T>::pack(Vec<T>::one(one) * w) : one;
        }
    }
    if (a.start) zero_padding<LINES>(a, y, ldy, wave0, waves);
}

// A wave takes a share of a token's row from its k slots, B of them in flight.
// Sums are binary32, in the order of the choices.  Bound by HBM's reads: 8192 x
// 7168 bf16 from 8 slots 178 us, 16384 x 2880 from 4 79 us (5.9 TB/s both; four
// pieces a lane the same; with rows to add 181 and 84).  bf16 rows of one piece
// a lane have eight slots in flight (25534 x 264 from 6 30 us, four 36; binary32
// has none to gain: 8000 x 250 from 8 19 us, four 15).
constexpr int kCombinePieces = 2;
template <typename T, int U, bool LINES>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(ExpertRows a, const T* y, int64_t ldy, const T* add,
                                                              int64_t lda, T* out, int64_t ldo, int shares) {
    constexpr int N = Vec<T>::n, B = 8 / U, WAVES = kRowThreads / 64;
    const RowShape<T> shape(a.hidden);
    const int lane = lanes::lane();
    const int64_t items = a.rows * shares;
    for (int64_t item = blockIdx.x * (int64_t)WAVES + lanes::wave(); item < items; item += gridDim.x * (int64_t)WAVES) {
        const int64_t t = item / shares;
        const Share sh = share_of(shape.pieces, shares, (int)(item - t * shares));
        const bool tail = sh.last && lane < shape.tail;
        const int tail_at = shape.pieces * N + lane;
        const int32_t* slot = a.slot + t * a.k;
        float acc[U][N] = {}, acc_tail = 0.0f;
        if (add) {
            const T* from = add + t * lda;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = sh.p0 + u * 64 + lane;
                if (p < sh.p1) Vec<T>::open(load16(from + p * N), acc[u]);
            }
            if (tail) acc_tail = Vec<T>::one(from[tail_at]);
        }
        for (int j0 = 0; j0 < a.k; j0 += B) {
            u32x4 v[B][U];
            T one[B];
            float w[B];
            bool has[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int j = j0 + b, s = j < a.k ? slot[j] : -1;
                has[b] = s >= 0 && s < a.slots;
                if (!has[b]) continue;
                w[b] = a.weight ? a.weight[t * a.ldw + j] : 1.0f;
                const T* from = y + s * ldy;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int p = sh.p0 + u * 64 + lane;
                    if (p < sh.p1) v[b][u] = load16_once(from + p * N);
                }
                if (tail) one[b] = from[tail_at];
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (!has[b]) continue;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[N];
                    Vec<T>::open(v[b][u], f);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[u][i] = __builtin_fmaf(w[b], f[i], acc[u][i]);
                }
                if (tail) acc_tail = __builtin_fmaf(w[b], Vec<T>::one(one[b]), acc_tail);
            }
        }
        T* to = out + t * ldo;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = sh.p0 + u * 64 + lane;
            if (p < sh.p1) put16<LINES>(to + p * N, Vec<T>::close(acc[u]));
        }
        if (tail) to[tail_at] = Vec<T>::pack(acc_tail);
    }
}

// A workgroup takes `each` choices of a token: its gradient row stays in
// registers while their slots' rows pass, each giving one dot product and taking
// w dout.  All of a token's choices, or two (bf16) or four (binary32) where tokens
// are few (64 x 7168 bf16, 8 slots 7.7 us, all eight 19.5; 600 of them 33.5 and
// 36.8; but 3001 x 1003 binary32, 6 slots 37.4 and 32.4).  Rows
// longer than U NT pieces go in several turns.  A dot product is a lane's
// binary32 chain of up to U N products a turn, then the lanes' in a fixed
// order.  Bound by HBM: 16384 x 2880 bf16, 4 slots 155 us (5.5 TB/s), 8192 x
// 7168, 8 slots and 235 MB of padding 433 us (5.2 TB/s).  Rows of y in flight:
// two of bf16 (four 155 to 158), four of binary32 (2000 x 4096, 6 slots 83 us,
// two 87), eight where a row is one piece a lane (25534 x 264 bf16, 6 slots 72
// us, two 80; 8000 x 250 binary32, 8 slots 34, four 41).
constexpr int kGradPieces = 4;
template <typename T, int U>
constexpr int kGradRows = U == 1 ? 8 : sizeof(T) == 4 ? 4 : 2;
constexpr int64_t kFewTokens = 2048;
template <typename T, int NT, int U, bool LINES>
__global__ __launch_bounds__(NT) void combine_grad_kernel(ExpertRows a, const T* dout, int64_t ldo, const T* y,
                                                          int64_t ldy, T* dy, int64_t lddy, float* dweight,
                                                          int64_t lddw, int each) {
    constexpr int N = Vec<T>::n, WAVES = NT / 64, B = kGradRows<T, U>;
    extern __shared__ float red[];  // WAVES x k
    const RowShape<T> shape(a.hidden);
    const int tid = threadIdx.x, wave = lanes::wave();
    const int groups = (a.k + each - 1) / each;
    const int64_t items = a.rows * groups;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t t = groups == 1 ? item : item / groups;
        const int first = (int)(item - t * groups) * each, end = min(first + each, a.k);
        const T* from = dout + t * ldo;
        const int32_t* slot = a.slot + t * a.k;
        const int turns = shape.pieces > 0 ? (shape.pieces + U * NT - 1) / (U * NT) : 1;
        for (int turn = 0; turn < turns; ++turn) {
            const int p0 = turn * U * NT + tid;
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[u] = u32x4{0u, 0u, 0u, 0u};
                if (p0 + u * NT < shape.pieces) v[u] = load16(from + (p0 + u * NT) * N);
            }
            const bool tail = turn == turns - 1 && tid < shape.tail;
            const int tail_at = shape.pieces * N + tid;
            const float vt = tail ? Vec<T>::one(from[tail_at]) : 0.0f;
            for (int j0 = first; j0 < end; j0 += B) {
                u32x4 q[B][U];
                float qt[B];
                int at[B];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int j = j0 + b, s = j < end ? slot[j] : -1;
                    at[b] = s < a.slots ? s : -1;
                    qt[b] = 0.0f;
                    if (at[b] < 0) continue;
                    const T* row = y + at[b] * ldy;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        q[b][u] = u32x4{0u, 0u, 0u, 0u};
                        if (p0 + u * NT < shape.pieces) q[b][u] = load16_once(row + (p0 + u * NT) * N);
                    }
                    if (tail) qt[b] = Vec<T>::one(row[tail_at]);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int j = j0 + b;
                    if (j >= end) break;
                    float dot = 0.0f;
                    if (at[b] >= 0) {
                        const float w = a.weight ? a.weight[t * a.ldw + j] : 1.0f;
                        T* to = dy + at[b] * lddy;
                        float lo = 0.0f, hi = vt * qt[b];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            float f[N], g[N];
                            Vec<T>::open(v[u], f);
                            Vec<T>::open(q[b][u], g);
#pragma unroll
                            for (int i = 0; i < N; i += 2) {
                                lo = __builtin_fmaf(f[i], g[i], lo);
                                hi = __builtin_fmaf(f[i + 1], g[i + 1], hi);
                            }
                            if (dy && p0 + u * NT < shape.pieces) {
#pragma unroll
                                for (int i = 0; i < N; ++i) f[i] *= w;
                                put16<LINES>(to + (p0 + u * NT) * N, Vec<T>::close(f));
                            }
                        }
                        if (dy && tail) to[tail_at] = Vec<T>::pack(vt * w);
                        dot = lanes::sum<64>(lo + hi);
                    }
                    if (lanes::lane() != 0) continue;
                    if (WAVES == 1)  // rows of one turn
                        dweight[t * lddw + j] = dot;
                    else
                        red[wave * a.k + j] = turn == 0 ? dot : red[wave * a.k + j] + dot;
                }
            }
        }
        if (WAVES == 1) continue;
        __syncthreads();
        for (int j = first + tid; j < end; j += NT) {
            float sum = red[j];
            for (int w = 1; w < WAVES; ++w) sum += red[w * a.k + j];
            dweight[t * lddw + j] = sum;
        }
        __syncthreads();
    }
    if (a.start && dy) zero_padding<LINES>(a, dy, lddy, blockIdx.x * (int64_t)WAVES + wave, gridDim.x * (int64_t)WAVES);
}

// Workgroups of `waves` waves over `items` pieces of work; with padding also
// 2048 waves at least, or one for every slot.
unsigned row_grid(const ExpertRows& a, int64_t items, int waves, bool padding) {
    int64_t n = (items + waves - 1) / waves;
    if (padding) n = std::max(n, (std::min<int64_t>(a.slots, 2048) + waves - 1) / waves);
    return grid_of(n);
}

template <typename T, bool WEIGHTED>
hipError_t dispatch_weighted(const ExpertRows& a, const T* x, int64_t ldx, T* y, int64_t ldy, hipStream_t s) {
    const int shares = shares_of<kDispatchPieces>((int)(a.hidden / Vec<T>::n));
    const unsigned g = row_grid(a, a.rows * shares, kRowThreads / 64, a.start);
    if (g == 0) return hipSuccess;
    if (whole_lines(y, ldy))
        hipLaunchKernelGGL((dispatch_kernel<T, WEIGHTED, true>), dim3(g), dim3(kRowThreads), 0, s, a, x, ldx, y, ldy, shares);
    else
        hipLaunchKernelGGL((dispatch_kernel<T, WEIGHTED, false>), dim3(g), dim3(kRowThreads), 0, s, a, x, ldx, y, ldy, shares);
    return hipGetLastError();
}

template <typename T>
hipError_t dispatch(const ExpertRows& a, const void* x, int64_t ldx, void* y, int64_t ldy, hipStream_t s) {
    return a.weight ? dispatch_weighted<T, true>(a, static_cast<const T*>(x), ldx, static_cast<T*>(y), ldy, s)
                    : dispatch_weighted<T, false>(a, static_cast<const T*>(x), ldx, static_cast<T*>(y), ldy, s);
}

template <typename T, int U>
hipError_t combine_pieces(const ExpertRows& a, const T* y, int64_t ldy, const T* add, int64_t lda, T* out,
                          int64_t ldo, hipStream_t s) {
    const int shares = shares_of<U>((int)(a.hidden / Vec<T>::n));
    const unsigned g = row_grid(a, a.rows * shares, kRowThreads / 64, false);
    if (g == 0) return hipSuccess;
    if (whole_lines(out, ldo))
        hipLaunchKernelGGL((combine_kernel<T, U, true>), dim3(g), dim3(kRowThreads), 0, s, a, y, ldy, add, lda, out, ldo, shares);
    else
        hipLaunchKernelGGL((combine_kernel<T, U, false>), dim3(g), dim3(kRowThreads), 0, s, a, y, ldy, add, lda, out, ldo, shares);
    return hipGetLastError();
}

template <typename T>
hipError_t combine(const ExpertRows& a, const void* y, int64_t ldy, const void* add, int64_t lda, void* out,
                   int64_t ldo, hipStream_t s) {
    const T *from = static_cast<const T*>(y), *more = static_cast<const T*>(add);
    T* to = static_cast<T*>(out);
    if constexpr (sizeof(T) == 2)
        if (a.hidden / Vec<T>::n <= 64) return combine_pieces<T, 1>(a, from, ldy, more, lda, to, ldo, s);
    return combine_pieces<T, kCombinePieces>(a, from, ldy, more, lda, to, ldo, s);
}

template <typename T, int NT, int U>
hipError_t combine_grad_nt(const ExpertRows& a, const void* dout, int64_t ldo, const void* y, int64_t ldy, void* dy,
                           int64_t lddy, float* dweight, int64_t lddw, hipStream_t s) {
    // a workgroup's waves share a token, but not the padding
    const int each = a.rows < kFewTokens ? kGradRows<T, kGradPieces> : a.k;
    const int64_t items = a.rows * ((a.k + each - 1) / each);
    const unsigned g = std::max(row_grid(a, items, 1, false), a.start && dy ? row_grid(a, 0, NT / 64, true) : 0u);
    if (g == 0) return hipSuccess;
    const size_t lds = size_t(NT / 64) * size_t(a.k) * sizeof(float);
    const T *d = static_cast<const T*>(dout), *from = static_cast<const T*>(y);
    T* to = static_cast<T*>(dy);
    if (whole_lines(to, lddy))
        hipLaunchKernelGGL((combine_grad_kernel<T, NT, U, true>), dim3(g), dim3(NT), lds, s, a, d, ldo, from, ldy, to, lddy,
                           dweight, lddw, each);
    else
        hipLaunchKernelGGL((combine_grad_kernel<T, NT, U, false>), dim3(g), dim3(NT), lds, s, a, d, ldo, from, ldy, to, lddy,
                           dweight, lddw, each);
    return hipGetLastError();
}

template <typename T>
hipError_t combine_grad(const ExpertRows& a, const void* dout, int64_t ldo, const void* y, int64_t ldy, void* dy,
                        int64_t lddy, float* dweight, int64_t lddw, hipStream_t s) {
    const int64_t pieces = a.hidden / Vec<T>::n;
    constexpr int U = kGradPieces;
    if (pieces <= 64) return combine_grad_nt<T, 64, 1>(a, dout, ldo, y, ldy, dy, lddy, dweight, lddw, s);
    if (pieces <= 64 * U) return combine_grad_nt<T, 64, U>(a, dout, ldo, y, ldy, dy, lddy, dweight, lddw, s);
    if (pieces <= 128 * U) return combine_grad_nt<T, 128, U>(a, dout, ldo, y, ldy, dy, lddy, dweight, lddw, s);
    return combine_grad_nt<T, 256, U>(a, dout, ldo, y, ldy, dy, lddy, dweight, lddw, s);
}

}  // namespace

hipError_t launch_expert_sort(const ExpertSort& a, hipStream_t s) {
    const int64_t n = a.rows * a.k;
    const size_t row = size_t(a.experts) * sizeof(int);
    // One workgroup as long as its lanes hold all choices, three launches after
    // that (us, one / three: 8192 of 60 experts 9.0 / 10.6, of 256 10.8 / 10.8;
    // 4096 of 1000, whose counters take eight waves, 11.9 / 14.5).
    if (n <= 1024 * kSmallSteps && a.experts <= 512) {
        hipLaunchKernelGGL(sort_small_kernel<16>, dim3(1), dim3(1024), 17 * row, s, a);
        return hipGetLastError();
    }
    if (n <= 512 * kSmallSteps) {
        hipLaunchKernelGGL(sort_small_kernel<8>, dim3(1), dim3(512), 9 * row, s, a);
        return hipGetLastError();
    }
    const int64_t chunk = sort_chunk(n);
    const int chunks = (int)((n + chunk - 1) / chunk);
    hipLaunchKernelGGL(sort_count_kernel, dim3(chunks), dim3(kSortThreads), row, s, a, chunk);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sort_scan_kernel, dim3((a.experts + 63) / 64), dim3(64 * kScanWaves), 0, s, a, chunks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sort_place_kernel, dim3(chunks), dim3(kSortThreads), (kSortThreads / 64 + 1) * row, s, a, chunk);
    return hipGetLastError();
}

hipError_t launch_expert_dispatch(const ExpertRows& a, const void* x, int64_t ldx, void* y, int64_t ldy,
                                  hipStream_t s) {
    return a.f32 ? dispatch<float>(a, x, ldx, y, ldy, s) : dispatch<uint16_t>(a, x, ldx, y, ldy, s);
}

hipError_t launch_expert_combine(const ExpertRows& a, const void* y, int64_t ldy, const void* add, int64_t lda,
                                 void* out, int64_t ldo, hipStream_t s) {
    return a.f32 ? combine<float>(a, y, ldy, add, lda, out, ldo, s)
                 : combine<uint16_t>(a, y, ldy, add, lda, out, ldo, s);
}

hipError_t launch_expert_combine_grad(const ExpertRows& a, const void* dout, int64_t ldo, const void* y, int64_t ldy,
                                      void* dy, int64_t lddy, float* dweight, int64_t lddw, hipStream_t s) {
    return a.f32 ? combine_grad<float>(a, dout, ldo, y, ldy, dy, lddy, dweight, lddw, s)
                 : combine_grad<uint16_t>(a, dout, ldo, y, ldy, dy, lddy, dweight, lddw, s);
}

}  // namespace rs
