// linear_wide192.hip -- linear_wide_kernel.h on 192 x 192 tiles.
#include "linear_wide_kernel.h"

namespace gemmf32 {

hipError_t launch_linear_wide192(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                 int op_b, float* partials) {
    return launch_linear_wide<192>(p, e, s, format, op_a, op_b, partials);
}

}  // namespace gemmf32
