// rc_paged_tc.cu -- attention of many query rows over pages of E4M3 codes.
#include "rc_paged_tc.cuh"

namespace rc {

cudaError_t launch_paged_tc(PagedAttnParams& p, int D, size_t part_floats_max, cudaStream_t s) {
    return D == 128 ? launch_tc<128, Codes::E4M3>(p, part_floats_max, s) : launch_tc<64, Codes::E4M3>(p, part_floats_max, s);
}

}  // namespace rc
