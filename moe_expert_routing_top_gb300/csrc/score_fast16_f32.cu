// score_fast16_f32.cu -- the fast scored top-k kernels of k = 9 .. 16 for f32 logits (score_fast.cuh).
#include "score_fast.cuh"

namespace moer {
cudaError_t score_fast16_f32(const ScoreParams& p, cudaStream_t st) { return score_fast16_run<float>(p, st); }
}  // namespace moer
