// Instantiations of the paged decode step for fp16 (attn_paged.cuh).
#include "attn_paged.cuh"

namespace blk {

cudaError_t launch_paged_f16(bool e8, const PagedMapSet& tm, PagedArgs& a, int sms, cudaStream_t s) {
    return e8 ? launch_paged_t<__half, true>(tm, a, sms, s) : launch_paged_t<__half, false>(tm, a, sms, s);
}

}  // namespace blk
