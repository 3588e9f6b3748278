// K6s kernels for bf16 storage (attn_shared.cuh).
#include "attn_shared.cuh"

namespace blk {

cudaError_t launch_shared_bf16(int d, const SharedMaps& tm, const SharedKernelArgs& a, cudaStream_t s) {
    return launch_shared_t<__nv_bfloat16>(d, tm, a, s);
}

}  // namespace blk
