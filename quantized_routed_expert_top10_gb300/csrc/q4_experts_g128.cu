// strata_moe_q4_experts with groups of 128 columns.
#include "q4_experts.cuh"

namespace strata {
cudaError_t launch_q4_experts_128(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s) { return q4x::launch_group<128>(ex, a, s); }
}  // namespace strata
