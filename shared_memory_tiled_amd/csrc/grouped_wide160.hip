// grouped_wide160.hip -- grouped_tiles.h on 160 x 160 tiles of WideCore.
#include "grouped_tiles.h"

namespace gemmf32 {

hipError_t launch_grouped_wide160(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                int format, int op_b) {
    return launch_wide<160>(a, p, e, s, format, op_b);
}

hipError_t launch_grouped_grad_wide160(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                     int format) {
    return launch_grad_wide<160>(a, p, e, s, format);
}

}  // namespace gemmf32
