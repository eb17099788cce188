// Instances of the norm after a block's gradient (ssd_block_norm_bwd.cu), by the types of x and of the residual.
#include "ssd_block_norm_bwd.cuh"

namespace ssd {

cudaError_t launch_block_norm_bwd_bf16_f32(BlockNormBwdArgs& a, int* lines, cudaStream_t st) {
    return a.gate ? launch_block_norm_bwd_typed<bf16_t, float, true, true>(a, lines, st)
                  : launch_block_norm_bwd_typed<bf16_t, float, false, true>(a, lines, st);
}

}  // namespace ssd
