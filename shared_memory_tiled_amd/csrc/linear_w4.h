// linear_w4.h -- the product with a weight held in 4 bits: its arguments and
// launcher (not part of the public interface).
#pragma once

#include "launch.h"

namespace gemmf32 {

struct W4Args {
    int M, N, K;
    const uint16_t* X; int64_t ldx;
    const uint8_t* Q; int64_t ldq;                    // N rows of (K + 1) / 2 bytes
    int group;                                        // 32, 64 or a multiple of 128
    const uint16_t* scales; int64_t ld_scales;        // N rows of ceil(K / group)
    const uint16_t* zeros; int64_t ld_zeros;          // likewise, or null: 8
};
int64_t linear_w4_workspace(int M, int N, int K);
hipError_t launch_linear_w4(const W4Args& p, const EpilogueArgs& e, hipStream_t s, int format, void* workspace);

}  // namespace gemmf32
