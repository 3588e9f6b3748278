// Instantiations of the paged decode step for bf16 (attn_paged.cuh).
#include "attn_paged.cuh"

namespace blk {

cudaError_t launch_paged_bf16(bool e8, const PagedMapSet& tm, PagedArgs& a, int sms, cudaStream_t s) {
    return e8 ? launch_paged_t<__nv_bfloat16, true>(tm, a, sms, s)
              : launch_paged_t<__nv_bfloat16, false>(tm, a, sms, s);
}

}  // namespace blk
