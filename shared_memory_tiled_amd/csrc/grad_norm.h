// grad_norm.h -- the gradients' norm and clipping: the lists the entry points
// hand over and the table a launch takes (not part of the public interface).
#pragma once

#include "launch.h"

namespace gemmf32 {

// Host arrays of `count` tensors, validated by the entry point.
struct GradList {
    int64_t count;
    const void* const* in;
    void* const* out;                  // or null: read only
    const int64_t* size;
    const int* type;                   // 0 bfloat16, 1 binary16, 2 binary32
};

// Tensors of one launch, by value in its arguments (below 4 KB); tensor i's
// chunks of kGradChunk values are numbered first[i] .. first[i + 1] - 1.
constexpr int kGradTensors = 128;
constexpr int64_t kGradChunk = 4096;
constexpr int64_t kGradBlocks = 2048;  // per launch: eight of 256 threads on each CU
struct GradTable {
    int count;
    uint32_t first[kGradTensors + 1];
    const void* in[kGradTensors];
    void* out[kGradTensors];
    int64_t size[kGradTensors];
    unsigned char type[kGradTensors];
};
static_assert(sizeof(GradTable) <= 4000, "kernel arguments");

int64_t grad_partials(int64_t count, const int64_t* size);     // partial sums of launch_grad_squares
hipError_t launch_grad_squares(const GradList& l, double* partials, hipStream_t s);
hipError_t launch_grad_norm(const double* partials, int64_t count, float* norm, hipStream_t s);
// partials null: the norm is read; else computed and written.
hipError_t launch_grad_clip(const GradList& l, const double* partials, int64_t count, float* norm, float max_norm,
                            float eps, hipStream_t s);

}  // namespace gemmf32
