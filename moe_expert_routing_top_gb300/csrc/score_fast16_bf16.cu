// score_fast16_bf16.cu -- the fast scored top-k kernels of k = 9 .. 16 for bf16 logits (score_fast.cuh).
#include "score_fast.cuh"

namespace moer {
cudaError_t score_fast16_bf16(const ScoreParams& p, cudaStream_t st) { return score_fast16_run<__nv_bfloat16>(p, st); }
}  // namespace moer
