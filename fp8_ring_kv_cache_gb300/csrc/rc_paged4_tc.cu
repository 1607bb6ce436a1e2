// rc_paged4_tc.cu -- attention of many query rows over pages of E2M1 codes.
#include "rc_paged_tc.cuh"

namespace rc {

cudaError_t launch_paged4_tc(PagedAttnParams& p, int D, size_t part_floats_max, cudaStream_t s) {
    return D == 128 ? launch_tc<128, Codes::E2M1>(p, part_floats_max, s) : launch_tc<64, Codes::E2M1>(p, part_floats_max, s);
}

}  // namespace rc
