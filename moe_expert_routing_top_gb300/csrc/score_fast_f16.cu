// score_fast_f16.cu -- the fast scored top-k kernels for f16 logits (score_fast.cuh).
#include "score_fast.cuh"

namespace moer {
cudaError_t score_fast_f16(const ScoreParams& p, cudaStream_t st) { return score_fast_run<__half>(p, st); }
}  // namespace moer
