// score_grad.cu -- moer_score_topk_grad: the logits' gradient of the router's
// weights and score sums.
//
// With g_j = scale * d_weights_j at the chosen experts i_j and a = d_score_sum:
//   softmax, as it is:      dx_e = p_e (G_e + a_e - sum_j g_j p_ij - sum_e a_e p_e),
//                           G_e the g of the choices of e;
//   softmax, renormalised:  dx_ij = q_j (g_j - sum g q), q the softmax over the
//                           chosen logits, plus p_e (a_e - sum a p);
//   sigmoid:                dx_e = s_e (1 - s_e) (a_e + D_e), D at the chosen ones
//                           g_j, or (g_j - sum g s / S) / S renormalised, S = sum s.
// Every form is a dense part (absent without a, but for the plain softmax) and a
// part at the k chosen experts, so a renormalised gate without score sums
// reads its chosen logits alone.
//
// score_grad_tile_kernel (aligned rows): a warp takes four rows of a layer (two where
// k > 8, one where k > 16).  The choices go to 8 (16, 32) lanes a row, the dense
// part to LR lanes a row, each with a block of 8 neighbouring experts, so that both
// are coalesced and full; the chosen experts' parts reach their blocks through a
// row of shared memory.
//
// score_grad_kernel (rows off their vectors' boundaries): one warp per row; a lane holds the
// quads 4 (lane + 32 i) and lane j < k the j-th choice.
#include "pdl.cuh"
#include "score.cuh"

namespace moer {

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
      dj = g;
      if (p.renorm) {
        const float s = sigmoid(xj);
        const float z = warp_sum(s), rs = z > 0.f ? 1.f / z : 0.f;
        dj = (g - warp_sum(g * s) * rs) * rs;
      }
      dj *= sigmoid_slope(xj);
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

constexpr int SGT_WARPS = 8;

template <int N>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
template <int N>
__device__ __forceinline__ float part_max(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

template <typename X>
__device__ __forceinline__ void store8(X* p, int room, bool wide, const float (&x)[8]) {
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  if constexpr (sizeof(X) == 2) {
    if (wide && room >= 8) {
      const uint2 u = Quad<X>::put(a), v = Quad<X>::put(b);
      *reinterpret_cast<uint4*>(p) = make_uint4(u.x, u.y, v.x, v.y);
      return;
    }
  }
  if (room >= 4) store4<X>(p, true, a);
  if (room >= 8) store4<X>(p + 4, true, b);
}

// The loads of a warp's next rows are in flight while it works on the present ones:
// ids and weights' gradients two tiles ahead, the chosen logits (which need the
// ids) and the rows one tile ahead.  Rows are read before their own are written,
// so that d_logits may be the logits.
// LR: lanes of a row in the dense part (E <= 8 LR).  KL: lanes of a row for the
// choices (k <= KL <= LR).
template <typename X, int LR, int KL, bool DENSE>
__global__ void __launch_bounds__(SGT_WARPS * 32) score_grad_tile_kernel(const ScoreParams p) {
  constexpr int EB = sizeof(X);
  constexpr int ROWS = 32 / KL;             // of a warp at a time
  constexpr int RS = 32 / LR;               // rows of a step of the dense part
  constexpr int STEPS = ROWS / RS;
  constexpr int PITCH = 8 * LR;
  constexpr int AHEAD = SGT_WARPS * ROWS;  // tokens from a warp's tile to its next
  // expert e of a row lies at (e / 8) * 4 + e % 4, the upper half of its block 4 LR further on:
  // a lane's two vector accesses are then free of bank conflicts
  __shared__ __align__(16) float chosen[SGT_WARPS][ROWS][PITCH];
  __shared__ uint8_t owner[SGT_WARPS][ROWS][PITCH];
  __shared__ float4 scalar[SGT_WARPS][ROWS];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = blockIdx.x / p.nspan, unit = blockIdx.x - l * p.nspan;
  const bool soft = p.score == MOER_SCORE_SOFTMAX;
  const bool has_a = DENSE && p.d_score_sum != nullptr;
  const int rc = lane / KL, j = lane % KL;    // the lane's choice
  const int rd = lane / LR, blk = lane % LR; // its block
  const int room = p.E - 8 * blk;
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = has_a && 8 * blk + i < p.E ? p.d_score_sum[(size_t)l * p.E + 8 * blk + i] : 0.f;
  // positions within the unit, in 32 bits: first tile, end
  const int64_t u0 = (int64_t)unit * p.span;
  const int t1 = (int)min64(p.span, p.T - u0);
  struct Pick {
    int id;   // E and more: no such expert
    float g;
  };
  // addresses of the lane's choice and block in the warp's first tile; `tile` counts tiles from it
  const int t00 = warp * ROWS;
  const uint8_t* ids = p.ids + ((int64_t)l * p.T + u0 + t00 + rc) * p.k + j;
  const float* dw = p.d_weights + ((int64_t)l * p.T + u0 + t00 + rc) * p.k + j;
  const X* crow = static_cast<const X*>(p.logits) + l * p.ld_layer + (u0 + t00 + rc) * p.ld_token;
  const X* brow = static_cast<const X*>(p.logits) + l * p.ld_layer + (u0 + t00 + rd) * p.ld_token + 8 * blk;
  X* orow = static_cast<X*>(p.d_logits) + l * p.ldg_layer + (u0 + t00 + rd) * p.ldg_token + 8 * blk;
  const int kstep = AHEAD * p.k;
  const int64_t cstep = AHEAD * p.ld_token, ostep = AHEAD * p.ldg_token;
  const int64_t rs_in = RS * p.ld_token, rs_out = RS * p.ldg_token;
  const bool chooses = j < p.k;
  auto pick = [&](int t0) {  // at the tile that ids and dw point to, whose first token is t0
    Pick c = {0xFFFF, 0.f};  // no choice at all
    if (chooses && t0 + rc < t1) {
      c.id = *ids;
      c.g = *dw;
    }
    ids += kstep;
    dw += kstep;
    return c;
  };
  auto gather = [&](const Pick& c) {
    X x = Quad<X>::back(NEG_INF);
    if (c.id < p.E) x = crow[c.id];
    crow += cstep;
    return x;
  };
  auto fetch = [&](Raw<EB>(&to)[STEPS], int t0) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      to[s].template load<X>(brow + s * rs_in, t0 + s * RS + rd < t1 ? room : 0, p.wide != 0);
    brow += cstep;
  };
  int t0 = t00;
  if (t0 >= t1) {
    pdl_release();
    return;
  }
  Pick now = pick(t0), then = pick(t0 + AHEAD);
  Raw<EB> raw[DENSE ? STEPS : 1];
  if constexpr (DENSE) fetch(raw, t0);
  X xnow = gather(now);
  for (; t0 < t1; t0 += AHEAD) {
    float v[STEPS][8], rz[STEPS], dot[STEPS];
    if constexpr (DENSE) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) raw[s].template get<X>(v[s]);
      fetch(raw, t0 + AHEAD);
    }
    const X xthen = gather(then);
    const Pick after = pick(t0 + 2 * AHEAD);
    bool ok = now.id < p.E;
    if (now.id >= p.E && now.id != 0xFFFF) atomicOr(p.status, WS_BIT_EDATA);
    const int id = ok ? now.id : 0;
    const float g = ok ? p.scale * now.g : 0.f;
    const float xj = live_logit(Quad<X>::one(xnow));
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      float4* z = reinterpret_cast<float4*>(chosen[warp][s * RS + rd]);
      z[blk] = make_float4(0.f, 0.f, 0.f, 0.f);
      z[LR + blk] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int slot = (id >> 3) * 4 + (id & 3) + ((id & 4) != 0 ? 4 * LR : 0);
    if (ok) owner[warp][rc][slot] = (uint8_t)j;
    if constexpr (DENSE) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        if (soft) {
          float m = LOWEST;  // under every number lies only -inf, whose exponential is 0
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, v[s][i]);
          m = part_max<LR>(m);
          float z = 0.f, e[8];
          const float mm = m * LOG2E;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            e[i] = ex2_approx(fmaf(v[s][i], LOG2E, -mm));
            z += e[i];
          }
          z = part_sum<LR>(z);
          if (__any_sync(FULL, !(z < 3e38f))) {  // a NaN or +inf among the logits, or nothing but masks
            z = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              e[i] = exp_below(live_logit(v[s][i]), m);
              z += e[i];
            }
            z = part_sum<LR>(z);
          }
          rz[s] = z > 0.f ? rcp_approx(z) : 0.f;
          dot[s] = 0.f;
          if (has_a) {
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) d = fmaf(a[i], e[i], d);
            dot[s] = part_sum<LR>(d) * rz[s];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) v[s][i] = e[i];
          if (!p.renorm && blk == 0) scalar[warp][s * RS + rd] = make_float4(m, rz[s], 0.f, 0.f);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[s][i] = a[i] * sigmoid_slope(live_logit(v[s][i]));
        }
      }
    }
    __syncwarp();
    // the part at the chosen expert
    float dj;
    if (soft) {
      const float4 mr = DENSE && !p.renorm ? scalar[warp][rc] : make_float4(0.f, 0.f, 0.f, 0.f);
      const float m = p.renorm ? fmaxf(part_max<KL>(xj), LOWEST) : mr.x;
      const float e = xj == m ? 1.f : ex2_approx(LOG2E * (xj - m));
      if (p.renorm) {
        const float z = part_sum<KL>(e);
        const float q = z > 0.f ? e * rcp_approx(z) : 0.f;
        dj = q * (g - part_sum<KL>(g * q));
      } else {
        dj = g * e * mr.y;
        const float dg = part_sum<KL>(dj);
        __syncwarp();
        if (j == 0) scalar[warp][rc].z = dg;
      }
    } else {
      // s and s (1 - s) from one exponential of -|x|
      const float t = expf(-fabsf(xj)), r = rcp_approx(1.f + t);
      dj = g;
      if (p.renorm) {
        const float s = ok ? (xj >= 0.f ? r : t * r) : 0.f;
        const float z = part_sum<KL>(s), rs = z > 0.f ? 1.f / z : 0.f;
        dj = (g - part_sum<KL>(g * s) * rs) * rs;
      }
      dj *= t * r * r;
    }
    float* at = &chosen[warp][rc][slot];
    const bool lost = ok && owner[warp][rc][slot] != j;  // an id that is repeated in its row
    if (ok) *at = dj;
    if (__any_sync(FULL, lost)) {
      if (ok) *at = 0.f;
      __syncwarp();
      for (int i = 0; i < KL; ++i) {
        if (ok && j == i) *at += dj;
        __syncwarp();
      }
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * RS + rd;
      const float4* z = reinterpret_cast<const float4*>(chosen[warp][r]);
      const float4 lo = z[blk], hi = z[LR + blk];
      float dx[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      if constexpr (DENSE) {
        if (soft) {
          const float d = rz[s] * (dot[s] + (p.renorm ? 0.f : scalar[warp][r].z));
          if (has_a) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dx[i] = fmaf(v[s][i], fmaf(a[i], rz[s], -d), dx[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) dx[i] = fmaf(v[s][i], -d, dx[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dx[i] += v[s][i];
        }
      }
      if (t0 + r < t1) store8<X>(orow + s * rs_out, room, p.wide != 0, dx);
    }
    orow += ostep;
    __syncwarp();
    now = then;
    then = after;
    xnow = xthen;
  }
  pdl_release();
}

template <typename X, int LR, int KL>
cudaError_t grad_tile_run(const ScoreParams& p, cudaStream_t st) {
  const bool dense = p.d_score_sum != nullptr || (p.score == MOER_SCORE_SOFTMAX && !p.renorm);
  const dim3 grid((unsigned)(p.L * p.nspan)), block(SGT_WARPS * 32);
  return dense ? launch_pdl(score_grad_tile_kernel<X, LR, KL, true>, grid, block, 0, st, p)
               : launch_pdl(score_grad_tile_kernel<X, LR, KL, false>, grid, block, 0, st, p);
}

template <typename X>
cudaError_t grad_run(const ScoreParams& p, cudaStream_t st) {
  if (p.vec != 0) {
    if (p.k > 16) return grad_tile_run<X, 32, 32>(p, st);
    if (p.k > 8) return p.E <= 128 ? grad_tile_run<X, 16, 16>(p, st) : grad_tile_run<X, 32, 16>(p, st);
    return p.E <= 64    ? grad_tile_run<X, 8, 8>(p, st)
           : p.E <= 128 ? grad_tile_run<X, 16, 8>(p, st)
                        : grad_tile_run<X, 32, 8>(p, st);
  }
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
  // units of a layer's tokens, a multiple of the rows that a block takes at a time
  const int STEP = SGT_WARPS * (p.k <= 8 ? 4 : p.k <= 16 ? 2 : 1), UNITS = 152 * 32;
  const int64_t span = ((p.T * p.L + UNITS - 1) / UNITS + STEP - 1) / STEP * STEP;
  p.span = (int)span;
  p.nspan = (int)((p.T + span - 1) / span);
  const cudaError_t e = dtype == MOER_F32    ? grad_run<float>(p, st)
                        : dtype == MOER_BF16 ? grad_run<__nv_bfloat16>(p, st)
                                             : grad_run<__half>(p, st);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
