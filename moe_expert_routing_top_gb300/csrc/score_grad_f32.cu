// score_grad_f32.cu -- the gradient's throughput kernels for f32 logits (score_grad_tile.cuh).
#include "score_grad_tile.cuh"

namespace moer {
cudaError_t grad_tile_f32(const ScoreParams& p, cudaStream_t st) { return grad_tile<float>(p, st); }
}  // namespace moer
