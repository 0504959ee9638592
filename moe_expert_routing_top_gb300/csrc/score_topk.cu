// score_topk.cu -- moer_score_topk: scores, choice and weights of the router.
//
// General kernel (any E <= 256 with E % 4 == 0, any k <= 32, any options): one
// warp per row.  A lane holds the quads of neighbouring experts 4 (lane + 32 i),
// as fp32 logits, scores and order-preserving keys of the choice; k rounds of
// a warp maximum over the keys pick the experts, ties to the lower id.
// A unit of work is a span of tokens of one layer; its eight warps take the
// rows in turn, and where score sums are wanted each lane adds up its own
// experts' scores, the warps' sums are joined in warp order and the units' in
// unit order, so the result does not depend on the schedule.
#include "pdl.cuh"
#include "score.cuh"
#include "score_row.cuh"

namespace moer {

cudaError_t score_fast_f32(const ScoreParams& p, cudaStream_t st);
cudaError_t score_fast_bf16(const ScoreParams& p, cudaStream_t st);
cudaError_t score_fast_f16(const ScoreParams& p, cudaStream_t st);

namespace {
constexpr int SC_WARPS = 8;
constexpr int SC_UNITS = 4864;  // units asked for: 152 SMs x 32

constexpr int64_t SC_FAST_ROWS = 4096;  // rows from which the fast kernel is taken
constexpr int SC_FAST_RESIDENT = 5;     // its blocks on an SM

// Tokens of a unit: a multiple of `step`, the rows that a block takes at a time.
int score_span(int64_t T, int L, int step) {
  const int64_t s = (T * L + SC_UNITS - 1) / SC_UNITS;
  return (int)((s + step - 1) / step * step);
}
int score_nspan(int64_t T, int span) { return (int)((T + span - 1) / span); }

// Tokens of a unit of the fast kernel, whose blocks take `step` rows at a time and
// are resident `slots` at once: the fewest rounds, a unit's start counted as one,
// over whole waves of units, and no more units than the general kernel has
// (the workspace holds a partial sum for each).
int fast_span(int64_t T, int L, int step, int64_t slots) {
  const int most = score_nspan(T, score_span(T, L, SC_WARPS));
  int64_t best = -1, cost = 0;
  for (int64_t rounds = 1; rounds <= 64 || best < 0; ++rounds) {
    const int64_t units = (T + rounds * step - 1) / (rounds * step);
    if (units > most) continue;
    const int64_t c = (units * L + slots - 1) / slots * (rounds + 1);
    if (best < 0 || c < cost) best = rounds, cost = c;
    if (units == 1) break;
  }
  return (int)(best * step);
}

// The fast kernel's options (score_fast.cuh): k <= 8, aligned quads, and groups,
// where there are any, that are a power of two of blocks on every lane of a row.
bool fast_supported(const ScoreParams& p) {
  if (p.k > 8 || p.vec == 0 || p.E < 16 || p.L * p.T < SC_FAST_ROWS) return false;
  if (p.n_group == 1) return true;
  const int lanes = p.E <= 64 ? 1 : p.E <= 128 ? 2 : 4, gs = p.E / p.n_group, mb = gs / (8 * lanes);
  return gs % (8 * lanes) == 0 && (mb & (mb - 1)) == 0 && p.n_group <= 8;
}

template <typename X, int NQ>
__global__ void __launch_bounds__(SC_WARPS * 32) score_topk_kernel(const ScoreParams p) {
  __shared__ float part[SC_WARPS][128 * NQ];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = blockIdx.x / p.nspan, u = blockIdx.x - l * p.nspan;
  float bias[4 * NQ], sum[4 * NQ];
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) {
    const int e = 4 * (lane + 32 * (i / 4)) + i % 4;
    bias[i] = p.bias != nullptr && e < p.E ? p.bias[(size_t)l * p.E + e] : 0.f;
    sum[i] = 0.f;
  }
  const int64_t t1 = min64(p.T, (int64_t)(u + 1) * p.span);
  for (int64_t t = (int64_t)u * p.span + warp; t < t1; t += SC_WARPS)
    score_row<X, NQ>(p, static_cast<const X*>(p.logits) + l * p.ld_layer + t * p.ld_token, bias,
                     p.topk + ((int64_t)l * p.T + t) * p.k,
                     p.weights != nullptr ? p.weights + ((int64_t)l * p.T + t) * p.k : nullptr, lane, sum);
  if (p.partial != nullptr) {
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) part[warp][4 * (lane + 32 * (i / 4)) + i % 4] = sum[i];
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += SC_WARPS * 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < SC_WARPS; ++w) v += part[w][e];
      p.partial[(size_t)blockIdx.x * p.E + e] = v;
    }
  }
  pdl_release();
}

// score_sum[l][e]: the units' sums in unit order, split over a block's rows.
__global__ void __launch_bounds__(256) score_sum_kernel(const float* partial, int nspan, int E, float* out) {
  __shared__ float part[8][32];
  pdl_wait();
  const int l = blockIdx.y, e = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float v = 0.f;
  if (e < E)
    for (int u = w; u < nspan; u += 8) v += partial[((size_t)l * nspan + u) * E + e];
  part[w][threadIdx.x & 31] = v;
  __syncthreads();
  if (w == 0 && e < E) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][threadIdx.x];
    out[(size_t)l * E + e] = v;
  }
  pdl_release();
}

template <typename X>
cudaError_t score_run(const ScoreParams& p, cudaStream_t st) {
  const dim3 grid(p.L * p.nspan), block(SC_WARPS * 32);
  return p.E <= 128 ? launch_pdl(score_topk_kernel<X, 1>, grid, block, 0, st, p)
                    : launch_pdl(score_topk_kernel<X, 2>, grid, block, 0, st, p);
}
}  // namespace

// The general kernel's units are the more numerous.
size_t score_scratch_bytes(const moer_dims* d, int64_t T) {
  return (size_t)d->L * (size_t)score_nspan(T, score_span(T, d->L, SC_WARPS)) * (size_t)d->E * 4;
}

moer_status score_topk_launch(ScoreParams p, int dtype, float* score_sum, void* ws, cudaStream_t st) {
  if (p.T == 0)
    return score_sum == nullptr ||
                   cudaMemsetAsync(score_sum, 0, (size_t)p.L * p.E * sizeof(float), st) == cudaSuccess
               ? MOER_OK
               : MOER_ECUDA;
  const bool fast = fast_supported(p);
  if (fast) {
    const int sms = device_sm_count();
    if (sms <= 0) return MOER_ECUDA;
    p.span = fast_span(p.T, p.L, p.E <= 64 ? 128 : p.E <= 128 ? 64 : 32, (int64_t)sms * SC_FAST_RESIDENT);
  } else {
    p.span = score_span(p.T, p.L, SC_WARPS);
  }
  p.nspan = score_nspan(p.T, p.span);
  p.partial = score_sum != nullptr ? reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEADER) : nullptr;
  p.key_mul = 256u;
  const uintptr_t w = reinterpret_cast<uintptr_t>(p.weights);
  p.even = p.k == 8 && w % 16 == 0 ? 2 : p.k % 2 == 0 && w % 8 == 0 ? 1 : 0;
  cudaError_t e;
  if (fast)
    e = dtype == MOER_F32 ? score_fast_f32(p, st) : dtype == MOER_BF16 ? score_fast_bf16(p, st) : score_fast_f16(p, st);
  else
    e = dtype == MOER_F32    ? score_run<float>(p, st)
        : dtype == MOER_BF16 ? score_run<__nv_bfloat16>(p, st)
                             : score_run<__half>(p, st);
  if (e == cudaSuccess && score_sum != nullptr)
    e = launch_pdl(score_sum_kernel, dim3((p.E + 31) / 32, p.L), dim3(256), 0, st, (const float*)p.partial, p.nspan,
                   p.E, score_sum);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
