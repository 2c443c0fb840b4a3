// The split kernels of verify_attn_paged_b8 over INT8 codes.
#include "paged_attn.cuh"

namespace va {
namespace paged {
cudaError_t launch_attn_int8(const AttnPagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    return launch_format<true>(a, k, v, stream);
}
}  // namespace paged
}  // namespace va
