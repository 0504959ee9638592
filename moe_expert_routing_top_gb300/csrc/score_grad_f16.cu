// score_grad_f16.cu -- the gradient's throughput kernels for f16 logits (score_grad_tile.cuh).
#include "score_grad_tile.cuh"

namespace moer {
cudaError_t grad_tile_f16(const ScoreParams& p, cudaStream_t st) { return grad_tile<__half>(p, st); }
}  // namespace moer
