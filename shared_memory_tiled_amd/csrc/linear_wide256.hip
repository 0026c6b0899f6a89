// linear_wide256.hip -- linear_wide_kernel.h on 256 x 256 tiles.
#include "linear_wide_kernel.h"

namespace gemmf32 {

hipError_t launch_linear_wide256(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                 int op_b, float* partials) {
    return launch_linear_wide<256>(p, e, s, format, op_a, op_b, partials);
}

}  // namespace gemmf32
