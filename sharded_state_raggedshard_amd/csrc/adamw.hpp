// AdamW over many tensors: tables shared by the host plan (adamw.cpp) and the
// kernels (adamw_kernels.hip).  Plain structs and launcher declarations.
#pragma once
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "launch.hpp"

namespace rs {
namespace aw {

constexpr int64_t kChunk = 4096;     // elements of one workgroup's chunk
constexpr int64_t kMaxElems = int64_t(1) << 42;  // of one tensor: chunk indices stay in 32 bits
constexpr int32_t kMaxGroups = 16;   // sets of hyper-parameters of one step
constexpr int kMinBlockLog2 = 6, kMaxBlockLog2 = 12;  // a block lies in one chunk
constexpr int kSumBlocks = 2048;     // most partial sums of the gradients' norm
// Two words each, then on a line of its own the number of the last call (low
// half) and a mark that one of them gave up (high half).
constexpr int kSumWords = 2 * kSumBlocks + 32;

// One tensor: where its arrays are and how they are kept.
struct alignas(16) Tensor {
    void* param;
    const void* grad;
    void* m;
    void* v;
    float* amax_m;   // 8-bit moments only
    float* amax_v;
    uint16_t* out;   // nullable
    int64_t n;       // elements
    int64_t first;   // elements of the tensors before it
    int32_t kind;    // KIND_* bits
    int32_t block_log2;
    int32_t group;
    int32_t pad;
};
static_assert(sizeof(Tensor) == 96, "Tensor layout");

enum { KIND_PARAM_F32 = 1, KIND_GRAD_F32 = 2, KIND_INT8 = 4, KIND_ROOT = 8 };

// Elements [kChunk * index, kChunk * (index + 1)) of a tensor.
struct Chunk {
    int32_t tensor;
    int32_t index;
};

struct Work {
    const Tensor* tensors;
    const Chunk* chunks;
    int64_t n_chunks;
};

struct Scalars {
    StepScalars group[kMaxGroups];
};

hipError_t launch_step(const Work& w, const Scalars& sc, const float* gscale, hipStream_t s);
// slots: kSumWords words, 0 before the first call
hipError_t launch_l2norm(const Work& w, uint64_t* slots, double* sumsq, double max_norm, float* scale,
                         hipStream_t s);
// m, v (nullable): binary32 (f32) or bf16 values of every tensor's moments
hipError_t launch_moments(const Work& w, void* m, void* v, bool f32, hipStream_t s);

}  // namespace aw
}  // namespace rs
