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

namespace moer {

namespace {
constexpr int SC_WARPS = 8;
constexpr int SC_UNITS = 4864;  // units asked for: 152 SMs x 32

int score_span(int64_t T, int L) {
  const int64_t s = (T * L + SC_UNITS - 1) / SC_UNITS;
  return (int)((s + SC_WARPS - 1) / SC_WARPS * SC_WARPS);
}
int score_nspan(int64_t T, int L) {
  const int s = score_span(T, L);
  return (int)((T + s - 1) / s);
}

// Best and second-best choice key of each group; lane g returns group g's key.
template <int NQ>
__device__ uint32_t group_keys(const ScoreParams& p, const uint32_t (&key)[4 * NQ], int lane) {
  const int gs = p.E / p.n_group;
  uint32_t mine = 0u;
  for (int g = 0; g < p.n_group; ++g) {
    uint32_t a = 0u, b = 0u;  // the lane's two best keys within the group
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) {
      const int e = 4 * (lane + 32 * (i / 4)) + i % 4;
      if (e / gs == g) {
        const uint32_t x = key[i];
        b = max(b, min(a, x));
        a = max(a, x);
      }
    }
    uint32_t gk = __reduce_max_sync(FULL, a);
    if (p.group_best == 2) {
      const int w = __ffs(__ballot_sync(FULL, a == gk)) - 1;  // one instance of the best is used up
      const uint32_t second = __reduce_max_sync(FULL, lane == w ? b : a);
      const float sum = rank_value(gk) + rank_value(second);
      gk = rank_key(sum == sum ? sum : NEG_INF);
    }
    if (lane == g) mine = gk;
  }
  return mine;
}

template <typename X, int NQ>
__device__ void score_row(const ScoreParams& p, const X* row, const float (&bias)[4 * NQ], int64_t out, int lane,
                          float (&sum)[4 * NQ]) {
  const bool soft = p.score == MOER_SCORE_SOFTMAX;
  const bool use_s = p.bias != nullptr || (p.n_group > 1 && p.group_best == 2);  // the choice takes scores
  const bool dense = p.partial != nullptr || use_s || (soft && !p.renorm);
  float x[4 * NQ], s[4 * NQ];
  uint32_t key[4 * NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = 4 * (lane + 32 * q);
    float v[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
    if (e < p.E) load4<X>(row + e, p.vec != 0, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      key[4 * q + j] = e < p.E ? rank_key(v[j]) : 0u;  // of the logit itself
      x[4 * q + j] = live_logit(v[j]);
      s[4 * q + j] = 0.f;
    }
  }
  if (dense) {
    if (soft) {
      float m = NEG_INF;
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) m = fmaxf(m, x[i]);
      m = warp_max(m);
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) {
        s[i] = exp_below(x[i], m);
        z += s[i];
      }
      z = warp_sum(z);
      const float r = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) s[i] *= r;
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) s[i] = sigmoid(x[i]);
    }
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) sum[i] += s[i];
  }
  uint32_t ck[4 * NQ];  // keys of the choice scores where those are scores; masked experts keep their logit's key
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) {
    ck[i] = key[i];
    if (use_s && x[i] != NEG_INF) ck[i] = rank_key(s[i] + bias[i]);
    if (p.bias != nullptr) key[i] = ck[i];
  }
  if (p.n_group > 1) {
    uint32_t gk = group_keys<NQ>(p, ck, lane);
    unsigned keep = 0u;
    for (int r = 0; r < p.top_group; ++r) {
      const uint32_t best = __reduce_max_sync(FULL, gk);
      const int w = __ffs(__ballot_sync(FULL, gk == best && !((keep >> lane) & 1u) && lane < p.n_group)) - 1;
      keep |= 1u << w;
      if (lane == w) gk = 0u;
    }
    const int gs = p.E / p.n_group;
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) {
      const int e = 4 * (lane + 32 * (i / 4)) + i % 4;
      if (e < p.E && !((keep >> (e / gs)) & 1u)) key[i] = 0u;
    }
  }
  // lane r holds the r-th choice: its id and its logit or score
  const bool by_logit = soft && p.renorm;
  int id = 0;
  float val = by_logit ? NEG_INF : 0.f;
  for (int r = 0; r < p.k; ++r) {
    uint32_t best = 0u;
    int be = 0xFFFF;
    float bv = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i)
      if (key[i] > best) {
        best = key[i];
        be = 4 * (lane + 32 * (i / 4)) + i % 4;
        bv = by_logit ? x[i] : (dense ? s[i] : x[i]);
      }
    const uint32_t top = __reduce_max_sync(FULL, best);
    const int e = (int)__reduce_min_sync(FULL, best == top ? (unsigned)be : 0xFFFFu);
    const float v = __shfl_sync(FULL, bv, (e / 4) & 31);
    if (lane == r) id = e, val = v;
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i)
      if (e == 4 * (lane + 32 * (i / 4)) + i % 4) key[i] = 0u;
  }
  if (lane < p.k) p.topk[out * p.k + lane] = (uint8_t)id;
  if (p.weights != nullptr) {
    float w;
    if (by_logit) {
      const float v = lane < p.k ? val : NEG_INF;
      const float m = warp_max(v);
      w = exp_below(v, m);
    } else {
      w = lane < p.k ? (dense ? val : sigmoid(val)) : 0.f;
    }
    if (p.renorm) {
      const float z = warp_sum(w);
      w = z > 0.f ? w / z : 0.f;
    }
    if (lane < p.k) p.weights[out * p.k + lane] = p.scale * w;
  }
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
    score_row<X, NQ>(p, static_cast<const X*>(p.logits) + l * p.ld_layer + t * p.ld_token, bias, (int64_t)l * p.T + t,
                     lane, sum);
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

size_t score_scratch_bytes(const moer_dims* d, int64_t T) {
  return (size_t)d->L * (size_t)score_nspan(T, d->L) * (size_t)d->E * 4;
}

moer_status score_topk_launch(ScoreParams p, int dtype, float* score_sum, void* ws, cudaStream_t st) {
  if (p.T == 0)
    return score_sum == nullptr ||
                   cudaMemsetAsync(score_sum, 0, (size_t)p.L * p.E * sizeof(float), st) == cudaSuccess
               ? MOER_OK
               : MOER_ECUDA;
  p.span = score_span(p.T, p.L);
  p.nspan = score_nspan(p.T, p.L);
  p.partial = score_sum != nullptr ? reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEADER) : nullptr;
  cudaError_t e = dtype == MOER_F32    ? score_run<float>(p, st)
                  : dtype == MOER_BF16 ? score_run<__nv_bfloat16>(p, st)
                                       : score_run<__half>(p, st);
  if (e == cudaSuccess && score_sum != nullptr)
    e = launch_pdl(score_sum_kernel, dim3((p.E + 31) / 32, p.L), dim3(256), 0, st, (const float*)p.partial, p.nspan,
                   p.E, score_sum);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
