// score_grad.cu -- moer_score_topk_grad: the logits' gradient of the router's
// weights and score sums.
//
// With g_j = scale * d_weights_j at the chosen experts i_j and a = d_score_sum:
//   softmax, as it is:      dx_e = p_e (G_e + a_e - sum_j g_j p_ij - sum_e a_e p_e),
//                           G_e the g of the choices of e;
//   softmax, renormalised:  dx_ij = q_j (g_j - sum g q), q the softmax over the
//                           chosen logits, plus p_e (a_e - sum a p);
//   sigmoid:                dx_e = s_e (1 - s_e) (a_e + D_e), D at the chosen ones
//                           g_j, or (g_j - sum g s / S) / S renormalised, S = sum s;
//                           there s_e D_e is q_j (g_j - sum g q) with the shares q = s / S.
// Every form is a dense part (absent without a, but for the plain softmax) and a
// part at the k chosen experts, so a renormalised gate without score sums
// reads its chosen logits alone.
//
// Rows on their vectors' boundaries go to the kernel of score_grad_tile.cuh.
//
// score_grad_kernel (rows off their vectors' boundaries): one warp per row; a lane holds the
// quads 4 (lane + 32 i) and lane j < k the j-th choice.
#include "pdl.cuh"
#include "score.cuh"

namespace moer {

cudaError_t grad_tile_f32(const ScoreParams& p, cudaStream_t st);
cudaError_t grad_tile_bf16(const ScoreParams& p, cudaStream_t st);
cudaError_t grad_tile_f16(const ScoreParams& p, cudaStream_t st);

namespace {
constexpr int SG_WARPS = 8;

template <typename X, int NQ>
__global__ void __launch_bounds__(SG_WARPS * 32) score_grad_kernel(const ScoreParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const bool soft = p.score == MOER_SCORE_SOFTMAX;
  const bool dense = p.d_score_sum != nullptr || (soft && !p.renorm);
  const int64_t rows = (int64_t)p.L * p.T;
  for (int64_t n = (int64_t)blockIdx.x * SG_WARPS + (threadIdx.x >> 5); n < rows; n += (int64_t)gridDim.x * SG_WARPS) {
    const int l = (int)(n / p.T);
    const int64_t t = n - (int64_t)l * p.T;
    const X* row = static_cast<const X*>(p.logits) + l * p.ld_layer + t * p.ld_token;
    X* out = static_cast<X*>(p.d_logits) + l * p.ldg_layer + t * p.ldg_token;
    // the choices
    int id = p.E;
    float g = 0.f, xj = NEG_INF;
    if (lane < p.k) {
      id = p.ids[n * p.k + lane];
      if (id < p.E) {
        g = p.scale * p.d_weights[n * p.k + lane];
        xj = live_logit(Quad<X>::one(row[id]));
      } else {
        atomicOr(p.status, WS_BIT_EDATA);
      }
    }
    float dx[4 * NQ];
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) dx[i] = 0.f;
    float m = NEG_INF, rz = 0.f;  // softmax over the row: largest logit, 1 / sum
    if (dense) {
      float x[4 * NQ], a[4 * NQ];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int e = 4 * (lane + 32 * q);
        float v[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
        if (e < p.E) load4<X>(row + e, p.vec != 0, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[4 * q + j] = live_logit(v[j]);
          a[4 * q + j] = p.d_score_sum != nullptr && e < p.E ? p.d_score_sum[(size_t)l * p.E + e + j] : 0.f;
        }
      }
      if (soft) {
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i) m = fmaxf(m, x[i]);
        m = warp_max(m);
        float z = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i) {
          x[i] = exp_below(x[i], m);
          z += x[i];
          dot = fmaf(a[i], x[i], dot);
        }
        if (!p.renorm) dot = fmaf(g, exp_below(xj, m), dot);
        z = warp_sum(z);
        rz = z > 0.f ? 1.f / z : 0.f;
        dot = warp_sum(dot) * rz;
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i) dx[i] = x[i] * rz * (a[i] - dot);
      } else {
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i) dx[i] = a[i] * sigmoid_slope(x[i]);
      }
    }
    // the part at the chosen experts
    float dj;
    if (soft) {
      if (p.renorm) {
        const float mk = warp_max(xj);
        const float q0 = exp_below(xj, mk), z = warp_sum(q0);
        const float q = z > 0.f ? q0 / z : 0.f;
        dj = q * (g - warp_sum(g * q));
      } else {
        dj = g * exp_below(xj, m) * rz;
      }
    } else {
      if (p.renorm) {
        const float t = expf(-fabsf(xj)), r = rcp_approx(1.f + t), s = sigmoid(xj);
        const float z = warp_sum(s), q = z > 0.f ? s * (1.f / z) : 0.f;
        dj = (g - warp_sum(g * q)) * (q * (xj >= 0.f ? t * r : r));
      } else {
        dj = g * sigmoid_slope(xj);
      }
    }
    for (int j = 0; j < p.k; ++j) {
      const int e = __shfl_sync(FULL, id, j);
      const float v = __shfl_sync(FULL, dj, j);
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i)
        if (e == 4 * (lane + 32 * (i / 4)) + i % 4) dx[i] += v;
    }
    __syncwarp();  // the row is read before it is written (d_logits may be the logits)
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int e = 4 * (lane + 32 * q);
      const float v[4] = {dx[4 * q], dx[4 * q + 1], dx[4 * q + 2], dx[4 * q + 3]};
      if (e < p.E) store4<X>(out + e, p.vec != 0, v);
    }
  }
  pdl_release();
}

template <typename X>
cudaError_t grad_run(const ScoreParams& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.L * p.T;
  const int64_t want = (rows + SG_WARPS - 1) / SG_WARPS;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const dim3 grid((unsigned)min64(want, (int64_t)sms * 8)), block(SG_WARPS * 32);
  return p.E <= 128 ? launch_pdl(score_grad_kernel<X, 1>, grid, block, 0, st, p)
                    : launch_pdl(score_grad_kernel<X, 2>, grid, block, 0, st, p);
}
}  // namespace

moer_status score_grad_launch(ScoreParams p, int dtype, cudaStream_t st) {
  constexpr int SGT_WARPS = 8;  // of the tile kernel
  // units of a layer's tokens, a multiple of the rows that a block takes at a time
  const int STEP = SGT_WARPS * (p.k <= 8 ? 4 : p.k <= 16 ? 2 : 1), UNITS = 152 * 32;
  const int64_t span = ((p.T * p.L + UNITS - 1) / UNITS + STEP - 1) / STEP * STEP;
  p.span = (int)span;
  p.nspan = (int)((p.T + span - 1) / span);
  cudaError_t e;
  if (p.vec != 0)
    e = dtype == MOER_F32 ? grad_tile_f32(p, st) : dtype == MOER_BF16 ? grad_tile_bf16(p, st) : grad_tile_f16(p, st);
  else
    e = dtype == MOER_F32    ? grad_run<float>(p, st)
        : dtype == MOER_BF16 ? grad_run<__nv_bfloat16>(p, st)
                             : grad_run<__half>(p, st);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
