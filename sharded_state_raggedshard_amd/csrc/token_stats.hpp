// Token statistics: the launch arguments that token_stats.cpp fills after its
// checks, and the launchers of token_stats_kernels.hip.
#pragma once
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "objectives.hpp"

namespace rs {

constexpr int32_t kMaxTop = 32;

// Statistics of a part of a row, without the row's token: the sums of e = 2^d
// and e d over d = (z - m) k around a reference m; and the token's value.
struct PartStat {
    double s, w;
    float m, token;
};

struct TokenStats {
    const void* z;
    int32_t f32;
    int64_t rows, vocab, ld;
    const int64_t* target;  // nullable: rows have no token, and all take part
    float k;                // log2(e) / temperature
    double scale, skew;     // 1 / temperature; log2(e) scale / k - 1
    int32_t top;
    float* logp;     // nullable
    float* entropy;  // nullable
    int64_t* top_id;
    float* top_logp;
    float* saved;    // nullable: m, 1 / S, E[(m - z) / T], 1 - p of the token
    // scratch of rows in several parts: their statistics and best values
    int32_t parts;
    PartStat* stat;
    float* best;
    int32_t* best_id;
};

// Parts that a row is split into: a power of two up to kMaxParts of at least
// 4096 values each, kStatsItems parts of all rows together at most.
constexpr int64_t kStatsItems = 512;
inline int32_t stats_parts(int64_t rows, int64_t vocab) {
    int32_t parts = 1;
    while (rows > 0 && parts < kMaxParts && rows * 2 * parts <= kStatsItems && vocab >= 2 * parts * 4096) parts *= 2;
    return parts;
}
// Parts of all rows of a call that splits its rows.
inline int64_t stats_part_room(int64_t rows) { return std::min(rows * kMaxParts, kStatsItems); }

struct TokenStatsGrad {
    const void* z;
    int32_t f32;
    int64_t rows, vocab, ld;
    const int64_t* target;
    float k;
    double scale;  // 1 / temperature
    const float* saved;
    const float* dlogp;     // nullable: 0
    const float* dentropy;  // nullable: 0
    void* d;
    int64_t ldd;
};

hipError_t launch_token_stats(const TokenStats& a, hipStream_t s);
hipError_t launch_token_stats_grad(const TokenStatsGrad& a, hipStream_t s);

}  // namespace rs
