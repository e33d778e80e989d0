// C-ABI entry points of the training objectives: argument checks, scratch
// layout and launches.  Every check happens before the first launch.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <limits>
#include <string>

#include "objectives.hpp"
#include "raggedshard.h"
#include "row_checks.hpp"

namespace {

using namespace rs::rowcheck;

constexpr int64_t kMaxPairs = int64_t(1) << 21;  // one workgroup each in one launch

// Scratch: row statistics, token logits, the sums of rows or pairs; for the
// preference loss also marks and what the rows' gradients take.
struct Scratch {
    size_t stat = 0, token = 0, mark = 0, grad = 0, terms = 0, slices = 0, bytes = 0;
};

// Statistics of the most demanding call of up to `rows` rows: few rows are
// split into parts, so they may take more than many (512 rows x 128256 have
// 1024 parts, 513 rows one each).  A workspace for `rows` serves fewer.
int64_t stat_room(int64_t rows, int64_t vocab) {
    int64_t room = rows;
    for (int32_t parts = 1; parts <= rs::kMaxParts; parts *= 2) {
        const int64_t r = std::min(rows, rs::kSplitItems / parts);
        room = std::max(room, r * rs::stat_parts(r, vocab));
    }
    return room;
}

Scratch scratch_of(int64_t rows, int64_t vocab, int64_t n_seq) {
    Scratch s;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t p = at;
        at = align256(at + n);
        return p;
    };
    s.stat = take(size_t(stat_room(rows, vocab)) * sizeof(rs::RowStat));
    s.token = take(size_t(rows) * sizeof(float));
    s.terms = take(size_t(std::max(rows, n_seq / 2)) * 3 * sizeof(double));
    s.slices = take(size_t(rs::kTermSlices) * 3 * sizeof(double));
    if (n_seq > 0) {
        s.mark = take(size_t(rows) * sizeof(int32_t));
        s.grad = take(size_t(rows) * sizeof(rs::GradRow));
    }
    s.bytes = std::max<size_t>(at, 256);
    return s;
}

rs_status check_temperature(double t) {
    if (!(t >= 0x1p-20 && t <= 0x1p20)) return fail(RS_EINVAL, "temperature outside [2^-20, 2^20]");
    return RS_OK;
}

rs_status fill_rows(const void* z, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                    const int64_t* target, double temperature, void* work, size_t bytes,
                    int64_t n_seq, rs::LogitRows& a, Scratch& sc) {
    if (vocab < 1 || vocab > rs::kMaxVocab) return fail(RS_EINVAL, "vocab outside 1..2^24");
    rs_status st = check_logits(z, dtype, rows, vocab, ld, work);
    if (st != RS_OK) return st;
    if (rows > 0 && !target) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(target, 8)) return fail(RS_EINVAL, "misaligned pointer");
    st = check_temperature(temperature);
    if (st != RS_OK) return st;
    sc = scratch_of(rows, vocab, n_seq);
    if (bytes < sc.bytes)
        return fail(RS_ENOMEM, "workspace of " + std::to_string(bytes) + " bytes; the call needs " +
                                   std::to_string(sc.bytes));
    uint8_t* w = static_cast<uint8_t*>(work);
    a.z = z;
    a.f32 = dtype == RS_F32;
    a.rows = rows;
    a.vocab = vocab;
    a.ld = ld;
    a.target = target;
    a.weight = nullptr;
    a.scale = 1.0 / temperature;
    const double k = a.scale * 1.44269504088896340736;
    a.k.hi = (float)k;
    if ((double)a.k.hi > k) a.k.hi = std::nextafterf(a.k.hi, 0.0f);
    a.k.lo = std::max((float)(k - (double)a.k.hi), std::numeric_limits<float>::min());
    a.parts = rs::stat_parts(rows, vocab);
    a.stat = reinterpret_cast<rs::RowStat*>(w + sc.stat);
    a.token = reinterpret_cast<float*>(w + sc.token);
    return RS_OK;
}

Extent logits_of(const rs::LogitRows& a) { return matrix(a.z, a.rows, a.vocab, a.ld, a.f32 ? 4 : 2); }
Extent gradient_of(const rs::LogitRows& a, const void* d, int64_t ldd) {
    return matrix(d, a.rows, a.vocab, ldd, a.f32 ? 4 : 2);
}

}  // namespace

extern "C" {

size_t rs_objective_bytes(int64_t rows, int64_t vocab, int64_t n_seq) {
    if (rows < 0 || vocab < 1 || vocab > rs::kMaxVocab || rows > kMaxElems / vocab || n_seq < 0 ||
        n_seq > 2 * kMaxPairs) {
        fail(RS_EINVAL, "sizes out of range");
        return 0;
    }
    return scratch_of(rows, vocab, n_seq).bytes;
}

rs_status rs_token_logp(const void* d_logits, int32_t dtype, int64_t rows, int64_t vocab,
                        int64_t ld, const int64_t* d_target, double temperature, float* d_logp,
                        float* d_lse, void* d_work, size_t bytes, void* stream) {
    rs::LogitRows a;
    Scratch sc;
    rs_status st = fill_rows(d_logits, dtype, rows, vocab, ld, d_target, temperature, d_work, bytes,
                             0, a, sc);
    if (st != RS_OK) return st;
    if (rows > 0 && !d_logp) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(d_logp, 4) || !aligned(d_lse, 4)) return fail(RS_EINVAL, "misaligned pointer");
    const Extent scratch{d_work, int64_t(sc.bytes)};
    st = check_apart({floats(d_logp, rows), floats(d_lse, rows), scratch}, {logits_of(a), longs(d_target, rows)});
    if (st != RS_OK) return st;
    hipError_t e = rs::launch_token_logp(a, d_logp, d_lse, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "token_logp launch");
    return RS_OK;
}

rs_status rs_policy_loss(const void* d_logits, int32_t dtype, int64_t rows, int64_t vocab,
                         int64_t ld, const int64_t* d_target, const float* d_old_logp,
                         const float* d_ref_logp, const float* d_advantage,
                         const float* d_weight, const rs_policy_hparams* hp, void* d_dlogits,
                         int64_t ldd, float* d_logp, float* d_stats, void* d_work, size_t bytes,
                         void* stream) {
    if (!hp || !d_stats) return fail(RS_EINVAL, "NULL argument");
    rs::LogitRows a;
    Scratch sc;
    rs_status st = fill_rows(d_logits, dtype, rows, vocab, ld, d_target, hp->temperature, d_work,
                             bytes, 0, a, sc);
    if (st != RS_OK) return st;
    if (!(hp->clip_low >= 0.0 && hp->clip_low <= 1.0) ||
        !(hp->clip_high >= 0.0 && std::isfinite(hp->clip_high)) ||
        !(hp->kl_coef >= 0.0 && std::isfinite(hp->kl_coef)))
        return fail(RS_EINVAL, "hyper-parameters out of range");
    if (rows > 0 && (!d_old_logp || !d_advantage || !d_weight)) return fail(RS_EINVAL, "NULL argument");
    if (rows > 0 && hp->kl_coef != 0.0 && !d_ref_logp)
        return fail(RS_EINVAL, "a KL term needs d_ref_logp");
    if (!aligned(d_old_logp, 4) || !aligned(d_ref_logp, 4) || !aligned(d_advantage, 4) ||
        !aligned(d_weight, 4) || !aligned(d_logp, 4) || !aligned(d_stats, 4))
        return fail(RS_EINVAL, "misaligned pointer");
    st = check_gradient(d_logits, d_dlogits, dtype, rows, vocab, ld, ldd);
    if (st != RS_OK) return st;
    const Extent logp = floats(d_logp, rows), stats = floats(d_stats, 4);
    const Extent scratch{d_work, int64_t(sc.bytes)};
    st = check_apart({logp, stats, scratch, gradient_of(a, d_dlogits, ldd)},
                     {longs(d_target, rows), floats(d_old_logp, rows), floats(d_ref_logp, rows),
                      floats(d_advantage, rows), floats(d_weight, rows)});
    if (st == RS_OK) st = check_apart({logp, stats, scratch}, {logits_of(a)});
    if (st != RS_OK) return st;
    a.weight = d_weight;
    rs::PolicyTerms t;
    t.old_logp = d_old_logp;
    t.ref_logp = d_ref_logp;
    t.advantage = d_advantage;
    t.lo = 1.0 - hp->clip_low;
    t.hi = 1.0 + hp->clip_high;
    t.kl_coef = hp->kl_coef;
    t.terms = reinterpret_cast<double*>(static_cast<uint8_t*>(d_work) + sc.terms);
    t.slices = reinterpret_cast<double*>(static_cast<uint8_t*>(d_work) + sc.slices);
    hipError_t e = rs::launch_policy(a, t, d_dlogits, ldd, d_logp, d_stats, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "policy_loss launch");
    return RS_OK;
}

rs_status rs_preference_loss(const void* d_logits, int32_t dtype, int64_t rows, int64_t vocab,
                             int64_t ld, const int64_t* d_target, const int64_t* d_start,
                             int64_t n_pairs, const float* d_ref_logp, const float* d_weight,
                             const rs_preference_hparams* hp, void* d_dlogits, int64_t ldd,
                             float* d_seq_logp, float* d_stats, void* d_work, size_t bytes,
                             void* stream) {
    if (!hp || !d_stats || !d_start) return fail(RS_EINVAL, "NULL argument");
    if (n_pairs < 1 || n_pairs > kMaxPairs) return fail(RS_EINVAL, "number of pairs outside 1..2^21");
    rs::LogitRows a;
    Scratch sc;
    rs_status st = fill_rows(d_logits, dtype, rows, vocab, ld, d_target, hp->temperature, d_work,
                             bytes, 2 * n_pairs, a, sc);
    if (st != RS_OK) return st;
    if (hp->kind != RS_PREF_SIGMOID && hp->kind != RS_PREF_HINGE && hp->kind != RS_PREF_IPO)
        return fail(RS_EINVAL, "unknown loss kind");
    if (!(hp->beta > 0.0) || !std::isfinite(hp->beta) || !std::isfinite(hp->margin) ||
        !(hp->label_smoothing >= 0.0 && hp->label_smoothing < 0.5) ||
        (hp->average != 0 && hp->average != 1) ||
        (hp->kind != RS_PREF_SIGMOID && hp->label_smoothing != 0.0) ||
        (hp->kind == RS_PREF_IPO && hp->margin != 0.0))
        return fail(RS_EINVAL, "hyper-parameters out of range");
    if (!aligned(d_start, 8) || !aligned(d_ref_logp, 4) || !aligned(d_weight, 4) ||
        !aligned(d_seq_logp, 4) || !aligned(d_stats, 4))
        return fail(RS_EINVAL, "misaligned pointer");
    st = check_gradient(d_logits, d_dlogits, dtype, rows, vocab, ld, ldd);
    if (st != RS_OK) return st;
    const Extent seq_logp = floats(d_seq_logp, 2 * n_pairs), stats = floats(d_stats, 3);
    const Extent scratch{d_work, int64_t(sc.bytes)};
    st = check_apart({seq_logp, stats, scratch, gradient_of(a, d_dlogits, ldd)},
                     {longs(d_target, rows), longs(d_start, 2 * n_pairs + 1), floats(d_ref_logp, 2 * n_pairs),
                      floats(d_weight, n_pairs)});
    if (st == RS_OK) st = check_apart({seq_logp, stats, scratch}, {logits_of(a)});
    if (st != RS_OK) return st;
    uint8_t* w = static_cast<uint8_t*>(d_work);
    rs::PreferenceTerms t;
    t.start = d_start;
    t.pairs = n_pairs;
    t.ref_logp = d_ref_logp;
    t.weight = d_weight;
    t.beta = hp->beta;
    t.smoothing = hp->label_smoothing;
    t.margin = hp->margin;
    t.kind = hp->kind;
    t.average = hp->average;
    t.mark = reinterpret_cast<int32_t*>(w + sc.mark);
    t.grad = reinterpret_cast<rs::GradRow*>(w + sc.grad);
    t.terms = reinterpret_cast<double*>(w + sc.terms);
    hipError_t e = rs::launch_preference(a, t, d_dlogits, ldd, d_seq_logp, d_stats, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "preference_loss launch");
    return RS_OK;
}

}  // extern "C"
