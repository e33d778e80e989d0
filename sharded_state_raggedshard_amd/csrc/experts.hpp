// Tokens to experts and back: the launch arguments that experts.cpp fills
// after its checks, and the launchers of expert_kernels.hip.
#pragma once
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

namespace rs {

constexpr int32_t kMaxSortExperts = 1024;

// Choices are counted and placed in up to kSortChunks chunks of whole steps of
// a workgroup.
constexpr int64_t kSortChunks = 256;
constexpr int kSortThreads = 256;
inline int64_t sort_chunk(int64_t choices) {
    const int64_t per = (choices + kSortChunks - 1) / kSortChunks;
    return std::max<int64_t>(1, (per + kSortThreads - 1) / kSortThreads) * kSortThreads;
}
// The most chunks that up to `choices` choices are cut into.
inline int64_t sort_chunk_room(int64_t choices) {
    return std::min(kSortChunks, (choices + kSortThreads - 1) / kSortThreads);
}

struct ExpertSort {
    const int64_t* topk;
    int64_t rows, ldk;
    int32_t experts, k, align;
    const uint8_t* mask;  // nullable
    int64_t* start;
    int32_t* count;
    int32_t* slot;
    int32_t* part;  // scratch: choices per chunk and expert
};

// Rows at their slots.  Strides are in elements.
struct ExpertRows {
    int32_t f32;
    int64_t rows, hidden;
    int32_t k, experts;
    const int32_t* slot;
    const float* weight;  // nullable: 1
    int64_t ldw;
    const int64_t* start;  // nullable: padding rows stay as they are
    const int32_t* count;
    int64_t slots;
};

hipError_t launch_expert_sort(const ExpertSort& a, hipStream_t s);
// y[slot] = weight x
hipError_t launch_expert_dispatch(const ExpertRows& a, const void* x, int64_t ldx, void* y, int64_t ldy,
                                  hipStream_t s);
// out = add + sum weight y[slot]; add nullable
hipError_t launch_expert_combine(const ExpertRows& a, const void* y, int64_t ldy, const void* add, int64_t lda,
                                 void* out, int64_t ldo, hipStream_t s);
// dy[slot] = weight dout, dweight = dout . y[slot]; dy nullable
hipError_t launch_expert_combine_grad(const ExpertRows& a, const void* dout, int64_t ldo, const void* y, int64_t ldy,
                                      void* dy, int64_t lddy, float* dweight, int64_t lddw, hipStream_t s);

}  // namespace rs
