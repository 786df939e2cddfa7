// Gated delta rule kernels, 64 values per key.
#define SSM_GDR_INSTANTIATE
#include "gdr_launch.hpp"

namespace ssm_detail {
template hipError_t gdr_prep_launch<64>(const GdrParams &, hipStream_t);
template hipError_t gdr_fwd_launch<64>(const GdrParams &, bool, hipStream_t);
template hipError_t gdr_bwd_launch<64>(const GdrParams &, hipStream_t);
}  // namespace ssm_detail
