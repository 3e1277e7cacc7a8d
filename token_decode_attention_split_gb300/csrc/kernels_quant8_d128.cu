// quantised paged decode-attention kernel instantiations: head dim 128, 8-bit codes, every group size,
// up to 8 and up to 16 query columns per warp.
#include "quant_attn.cuh"

namespace da {

template <>
cudaError_t launch_quant<128, 8>(int groups, bool narrow, const QuantParams& p, int grid,
                                 cudaStream_t st) {
    return launch_quant_any<128, 8>(groups, narrow, p, grid, st);
}

}  // namespace da
