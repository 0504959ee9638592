// score_fast_f32.cu -- the fast scored top-k kernels for f32 logits (score_fast.cuh).
#include "score_fast.cuh"

namespace moer {
cudaError_t score_fast_f32(const ScoreParams& p, cudaStream_t st) { return score_fast_run<float>(p, st); }
}  // namespace moer
