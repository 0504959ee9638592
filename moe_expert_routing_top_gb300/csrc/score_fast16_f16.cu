// score_fast16_f16.cu -- the fast scored top-k kernels of k = 9 .. 16 for f16 logits (score_fast.cuh).
#include "score_fast.cuh"

namespace moer {
cudaError_t score_fast16_f16(const ScoreParams& p, cudaStream_t st) { return score_fast16_run<__half>(p, st); }
}  // namespace moer
