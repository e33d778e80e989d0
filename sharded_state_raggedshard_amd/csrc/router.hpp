// Router balance loss: the launch arguments that router.cpp fills after its
// checks, and the launcher of router_kernels.hip.
#pragma once
#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace rs {

constexpr int32_t kMaxExperts = 1024;

struct RouterBalance {
    const void* z;
    int32_t f32;  // 1: binary32, 0: bf16
    int32_t experts, k, sigmoid;
    int64_t rows, ld;
    const int64_t* topk;
    int64_t ldk;
    const uint8_t* mask;   // nullable
    const int64_t* start;  // nullable: one sequence of all rows
    int64_t n_seq;
    double balance_coef, z_coef;
    void* d;  // nullable
    int64_t ldd;
    int32_t* counts;
    float* mean_prob;
    float* stats;
    // scratch: tokens per sequence, probability sums per (chunk, sequence),
    // two loss sums per chunk
    int32_t* tokens;
    float* part;
    double* loss;
};

// Row chunks of the main kernel (one workgroup each) and their length; the
// most chunks that up to `rows` rows are cut into.
constexpr int64_t kRoundChunks = 1024;
struct RouterChunks {
    int64_t n, rows;
};
RouterChunks router_chunks(int64_t rows, int32_t experts, int64_t n_seq);
int64_t router_chunk_room(int64_t rows, int32_t experts);

hipError_t launch_router_balance(const RouterBalance& a, hipStream_t s);

}  // namespace rs
