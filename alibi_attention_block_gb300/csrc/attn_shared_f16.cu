// K6s kernels for f16 storage (attn_shared.cuh).
#include "attn_shared.cuh"

namespace blk {

cudaError_t launch_shared_f16(int d, const SharedMaps& tm, const SharedKernelArgs& a, cudaStream_t s) {
    return launch_shared_t<__half>(d, tm, a, s);
}

}  // namespace blk
