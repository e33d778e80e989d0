// Training objectives: the launch arguments that objectives.cpp fills after
// its checks, and the launchers of objective_kernels.hip.
#pragma once
#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace rs {

constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kTermSlices = 512;  // slices of rows whose sums come first

// log2(e) / temperature as hi + lo, hi rounded towards 0 and lo > 0 (so that
// -inf times either is -inf).
struct ExpScale {
    float hi, lo;
};

// What the gradient kernels take of a row (grad_row() fills it).
struct GradRow {
    float m, f, own;
    int32_t y;
};

// Maximum and sum of exponentials of (a part of) a row.
struct RowStat {
    double s;
    float m, unused;
};

// Rows of logits and, per row, what the kernels keep of them in scratch.
struct LogitRows {
    const void* z;
    int32_t f32;  // 1: binary32, 0: bf16
    int64_t rows, vocab, ld;
    const int64_t* target;
    const float* weight;  // per row (policy) or nullptr
    double scale;         // 1 / temperature
    ExpScale k;
    // scratch: `parts` (max, sum) pairs and the token's logit per row
    int32_t parts;
    RowStat* stat;
    float* token;
};

struct PolicyTerms {
    const float* old_logp;
    const float* ref_logp;  // nullable: no KL term
    const float* advantage;
    double lo, hi, kl_coef;  // the ratio's bounds
    double* terms;           // scratch: three sums per row, then per slice
    double* slices;
};

struct PreferenceTerms {
    const int64_t* start;
    int64_t pairs;
    const float* ref_logp;  // nullable
    const float* weight;    // nullable
    double beta, smoothing, margin;
    int32_t kind, average;
    int64_t kept_from;  // rows from here on stay cached (launch_preference() sets it)
    // scratch: a mark and a GradRow per row, three sums per pair
    int32_t* mark;
    GradRow* grad;
    double* terms;
};

// Parts a row is split into for its statistics: a power of two up to
// kMaxParts, no more than kSplitItems parts of all rows together.
constexpr int32_t kMaxParts = 32;
constexpr int64_t kSplitItems = 1024;
int32_t stat_parts(int64_t rows, int64_t vocab);

hipError_t launch_token_logp(const LogitRows& a, float* logp, float* lse, hipStream_t s);
hipError_t launch_policy(const LogitRows& a, const PolicyTerms& t, void* d, int64_t ldd,
                         float* logp, float* stats, hipStream_t s);
hipError_t launch_preference(const LogitRows& a, const PreferenceTerms& t, void* d, int64_t ldd,
                             float* seq_logp, float* stats, hipStream_t s);

}  // namespace rs
