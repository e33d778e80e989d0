// C-ABI entry points of the router balance loss: argument checks, scratch
// layout and launches.  Every check happens before the first launch.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "raggedshard.h"
#include "router.hpp"
#include "row_checks.hpp"

namespace {

using namespace rs::rowcheck;

constexpr int64_t kMaxSequences = int64_t(1) << 16;

struct Scratch {
    size_t tokens = 0, part = 0, loss = 0, bytes = 0;
};

Scratch scratch_of(int64_t rows, int32_t experts, int64_t n_seq) {
    // room for the most chunks that up to `rows` rows are cut into, so that a
    // workspace for `rows` serves fewer (32768 rows are 1024 chunks, 34000
    // only 1000)
    const int64_t chunks = rs::router_chunk_room(rows, experts);
    Scratch s;
    s.part = align256(size_t(n_seq) * sizeof(int32_t));
    s.loss = s.part + align256(size_t(chunks + n_seq) * size_t(experts) * sizeof(float));
    s.bytes = s.loss + align256(size_t(chunks) * 2 * sizeof(double));
    return s;
}

bool sizes_ok(int64_t rows, int32_t experts, int64_t n_seq) {
    return rows >= 0 && rows <= kMaxElems && experts >= 1 && experts <= rs::kMaxExperts &&
           n_seq >= 1 && n_seq <= kMaxSequences;
}

}  // namespace

extern "C" {

size_t rs_router_balance_bytes(int64_t rows, int32_t experts, int64_t n_seq) {
    if (!sizes_ok(rows, experts, n_seq)) {
        fail(RS_EINVAL, "sizes out of range");
        return 0;
    }
    return scratch_of(rows, experts, n_seq).bytes;
}

rs_status rs_router_balance(const void* d_logits, int32_t dtype, int64_t rows, int32_t experts,
                            int64_t ld, const int64_t* d_topk, int32_t k, int64_t ldk,
                            const uint8_t* d_mask, const int64_t* d_start, int64_t n_seq,
                            const rs_balance_hparams* hp, void* d_dlogits, int64_t ldd,
                            int32_t* d_counts, float* d_mean_prob, float* d_stats, void* d_work,
                            size_t bytes, void* stream) {
    if (!hp || !d_counts || !d_mean_prob || !d_stats) return fail(RS_EINVAL, "NULL argument");
    if (experts < 1 || experts > rs::kMaxExperts) return fail(RS_EINVAL, "experts outside 1..1024");
    if (n_seq < 1 || n_seq > kMaxSequences) return fail(RS_EINVAL, "number of sequences outside 1..2^16");
    rs_status st = check_logits(d_logits, dtype, rows, experts, ld, d_work);
    if (st != RS_OK) return st;
    if (!d_start && n_seq != 1) return fail(RS_EINVAL, "several sequences need d_start");
    if (k < 1 || k > experts) return fail(RS_EINVAL, "k outside 1..experts");
    if (ldk < k) return fail(RS_EINVAL, "row stride below the row's length");
    if (rows > 0x7fffffff / k || rows > kMaxElems / ldk)
        return fail(RS_EOVERFLOW, "rows * k beyond 2^31 - 1, or rows * ldk beyond 2^50");
    if (rows > 0 && !d_topk) return fail(RS_EINVAL, "NULL argument");
    if (hp->score != RS_SCORE_SOFTMAX && hp->score != RS_SCORE_SIGMOID)
        return fail(RS_EINVAL, "unknown score");
    if (!std::isfinite(hp->balance_coef) || !std::isfinite(hp->z_coef) || hp->balance_coef < 0.0 ||
        hp->z_coef < 0.0 || (hp->score == RS_SCORE_SIGMOID && hp->z_coef != 0.0) || hp->reserved != 0)
        return fail(RS_EINVAL, "hyper-parameters out of range");
    if (!aligned(d_topk, 8) || !aligned(d_start, 8) || !aligned(d_counts, 4) ||
        !aligned(d_mean_prob, 4) || !aligned(d_stats, 4))
        return fail(RS_EINVAL, "misaligned pointer");
    st = check_gradient(d_logits, d_dlogits, dtype, rows, experts, ld, ldd);
    if (st != RS_OK) return st;
    const Scratch sc = scratch_of(rows, experts, n_seq);
    if (bytes < sc.bytes)
        return fail(RS_ENOMEM, "workspace of " + std::to_string(bytes) + " bytes; the call needs " +
                                   std::to_string(sc.bytes));
    const int64_t size = dtype == RS_F32 ? 4 : 2;
    const Extent counts{d_counts, n_seq * experts * 4}, mean = floats(d_mean_prob, n_seq * experts);
    const Extent stats = floats(d_stats, 2), scratch{d_work, int64_t(sc.bytes)};
    st = check_apart({counts, mean, stats, scratch, matrix(d_dlogits, rows, experts, ldd, size)},
                     {matrix(d_topk, rows, k, ldk, 8), Extent{d_mask, rows}, longs(d_start, n_seq + 1)});
    if (st == RS_OK) st = check_apart({counts, mean, stats, scratch}, {matrix(d_logits, rows, experts, ld, size)});
    if (st != RS_OK) return st;
    uint8_t* w = static_cast<uint8_t*>(d_work);
    rs::RouterBalance a;
    a.z = d_logits;
    a.f32 = dtype == RS_F32;
    a.experts = experts;
    a.k = k;
    a.sigmoid = hp->score == RS_SCORE_SIGMOID;
    a.rows = rows;
    a.ld = ld;
    a.topk = d_topk;
    a.ldk = ldk;
    a.mask = d_mask;
    a.start = d_start;
    a.n_seq = n_seq;
    a.balance_coef = hp->balance_coef;
    a.z_coef = hp->z_coef;
    a.d = d_dlogits;
    a.ldd = ldd;
    a.counts = d_counts;
    a.mean_prob = d_mean_prob;
    a.stats = d_stats;
    a.tokens = reinterpret_cast<int32_t*>(w);
    a.part = reinterpret_cast<float*>(w + sc.part);
    a.loss = reinterpret_cast<double*>(w + sc.loss);
    hipError_t e = rs::launch_router_balance(a, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "router_balance launch");
    return RS_OK;
}

}  // extern "C"
