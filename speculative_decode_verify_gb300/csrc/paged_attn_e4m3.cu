// The split kernels of verify_attn_paged_b8 over E4M3 codes.
#include "paged_attn.cuh"

namespace va {
namespace paged {
cudaError_t launch_attn_e4m3(const AttnPagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    return launch_format<false>(a, k, v, stream);
}
}  // namespace paged
}  // namespace va
