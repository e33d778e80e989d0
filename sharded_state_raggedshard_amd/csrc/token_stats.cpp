// C-ABI entry points of the token statistics: argument checks, scratch layout
// and launches.  Every check happens before the first launch.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <string>

#include "raggedshard.h"
#include "row_checks.hpp"
#include "token_stats.hpp"

namespace {

using namespace rs::rowcheck;

// Scratch of rows in several parts, the same for all vocabularies.
struct Scratch {
    size_t best = 0, best_id = 0, bytes = 0;
};

Scratch scratch_of(int64_t rows, int32_t top) {
    const size_t room = size_t(rs::stats_part_room(rows));
    Scratch s;
    s.best = align256(room * sizeof(rs::PartStat));
    s.best_id = s.best + align256(room * size_t(top) * sizeof(float));
    s.bytes = std::max<size_t>(256, s.best_id + align256(room * size_t(top) * sizeof(int32_t)));
    return s;
}

constexpr double kLog2e = 1.44269504088896340736;
float exponent_scale(double temperature) { return (float)(kLog2e / temperature); }

// What both calls take.
rs_status check_common(const void* z, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld, const int64_t* target,
                       double temperature) {
    if (vocab < 1 || vocab > rs::kMaxVocab) return fail(RS_EINVAL, "vocab outside 1..2^24");
    if (dtype != RS_F32 && dtype != RS_BF16) return fail(RS_EINVAL, "unknown dtype");
    if (rows < 0) return fail(RS_EINVAL, "negative number of rows");
    if (ld < vocab) return fail(RS_EINVAL, "row stride below the row's length");
    if (rows > kMaxElems / ld) return fail(RS_EOVERFLOW, "rows * ld beyond 2^50 elements");
    if (rows > 0 && !z) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(z, dtype == RS_F32 ? 4 : 2) || !aligned(target, 8)) return fail(RS_EINVAL, "misaligned pointer");
    if (!(temperature >= 0x1p-20 && temperature <= 0x1p20))
        return fail(RS_EINVAL, "temperature outside [2^-20, 2^20]");
    return RS_OK;
}

}  // namespace

extern "C" {

size_t rs_token_stats_bytes(int64_t rows, int64_t vocab, int32_t top) {
    if (rows < 0 || vocab < 1 || vocab > rs::kMaxVocab || rows > kMaxElems / vocab || top < 0 || top > rs::kMaxTop) {
        fail(RS_EINVAL, "sizes out of range");
        return 0;
    }
    return scratch_of(rows, top).bytes;
}

rs_status rs_token_stats(const void* d_logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                         const int64_t* d_target, double temperature, float* d_logp, float* d_entropy, int32_t top,
                         int64_t* d_top_id, float* d_top_logp, float* d_saved, void* d_work, size_t bytes,
                         void* stream) {
    rs_status st = check_common(d_logits, dtype, rows, vocab, ld, d_target, temperature);
    if (st != RS_OK) return st;
    if (top < 0 || top > rs::kMaxTop) return fail(RS_EINVAL, "top outside 0..32");
    if (!d_work || (rows > 0 && top > 0 && (!d_top_id || !d_top_logp))) return fail(RS_EINVAL, "NULL argument");
    if (d_logp && !d_target) return fail(RS_EINVAL, "log-probabilities need d_target");
    if (!aligned(d_logp, 4) || !aligned(d_entropy, 4) || !aligned(d_top_id, 8) || !aligned(d_top_logp, 4) ||
        !aligned(d_saved, 4))
        return fail(RS_EINVAL, "misaligned pointer");
    if (!aligned(d_work, 16)) return fail(RS_EINVAL, "workspace not 16-byte aligned");
    const Scratch sc = scratch_of(rows, top);
    if (bytes < sc.bytes)
        return fail(RS_ENOMEM, "workspace of " + std::to_string(bytes) + " bytes; the call needs " + std::to_string(sc.bytes));
    st = check_apart({floats(d_logp, rows), floats(d_entropy, rows), Extent{d_top_id, rows * top * 8},
                      floats(d_top_logp, rows * top), floats(d_saved, rows * 4), Extent{d_work, int64_t(sc.bytes)}},
                     {matrix(d_logits, rows, vocab, ld, dtype == RS_F32 ? 4 : 2), longs(d_target, rows)});
    if (st != RS_OK) return st;
    uint8_t* w = static_cast<uint8_t*>(d_work);
    rs::TokenStats a;
    a.z = d_logits;
    a.f32 = dtype == RS_F32;
    a.rows = rows;
    a.vocab = vocab;
    a.ld = ld;
    a.target = d_target;
    a.k = exponent_scale(temperature);
    a.scale = 1.0 / temperature;
    a.skew = kLog2e * a.scale / (double)a.k - 1.0;
    a.top = top;
    a.logp = d_logp;
    a.entropy = d_entropy;
    a.top_id = d_top_id;
    a.top_logp = d_top_logp;
    a.saved = d_saved;
    a.parts = rs::stats_parts(rows, vocab);
    a.stat = reinterpret_cast<rs::PartStat*>(w);
    a.best = reinterpret_cast<float*>(w + sc.best);
    a.best_id = reinterpret_cast<int32_t*>(w + sc.best_id);
    hipError_t e = rs::launch_token_stats(a, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "token_stats launch");
    return RS_OK;
}

rs_status rs_token_stats_grad(const void* d_logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                              const int64_t* d_target, double temperature, const float* d_saved,
                              const float* d_dlogp, const float* d_dentropy, void* d_dlogits, int64_t ldd,
                              void* stream) {
    rs_status st = check_common(d_logits, dtype, rows, vocab, ld, d_target, temperature);
    if (st != RS_OK) return st;
    if (rows > 0 && (!d_saved || !d_dlogits)) return fail(RS_EINVAL, "NULL argument");
    if (d_dlogp && !d_target) return fail(RS_EINVAL, "gradients of log-probabilities need d_target");
    if (!aligned(d_saved, 4) || !aligned(d_dlogp, 4) || !aligned(d_dentropy, 4)) return fail(RS_EINVAL, "misaligned pointer");
    st = check_gradient(d_logits, d_dlogits, dtype, rows, vocab, ld, ldd);
    if (st != RS_OK) return st;
    st = check_apart({matrix(d_dlogits, rows, vocab, ldd, dtype == RS_F32 ? 4 : 2)},
                     {longs(d_target, rows), floats(d_saved, rows * 4), floats(d_dlogp, rows), floats(d_dentropy, rows)});
    if (st != RS_OK) return st;
    rs::TokenStatsGrad a;
    a.z = d_logits;
    a.f32 = dtype == RS_F32;
    a.rows = rows;
    a.vocab = vocab;
    a.ld = ld;
    a.target = d_target;
    a.k = exponent_scale(temperature);
    a.scale = 1.0 / temperature;
    a.saved = d_saved;
    a.dlogp = d_dlogp;
    a.dentropy = d_dentropy;
    a.d = d_dlogits;
    a.ldd = ldd;
    hipError_t e = rs::launch_token_stats_grad(a, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "token_stats_grad launch");
    return RS_OK;
}

}  // extern "C"
