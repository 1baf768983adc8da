// attn_paged_wide.cu -- the attention over a paged cache for rows of more than 256 dims (a file of its own: the two compile side by
// side).
#include "attn_paged.cuh"

namespace sti {

template cudaError_t launch_attn_paged_nm<3>(const CUtensorMap&, const AttnPagedParams&, cudaStream_t);
template cudaError_t launch_attn_paged_nm<4>(const CUtensorMap&, const AttnPagedParams&, cudaStream_t);

}  // namespace sti
