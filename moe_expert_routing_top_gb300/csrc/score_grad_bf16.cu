// score_grad_bf16.cu -- the gradient's throughput kernels for bf16 logits (score_grad_tile.cuh).
#include "score_grad_tile.cuh"

namespace moer {
cudaError_t grad_tile_bf16(const ScoreParams& p, cudaStream_t st) { return grad_tile<__nv_bfloat16>(p, st); }
}  // namespace moer
