// score_grad_tile.cuh -- the throughput kernel of moer_score_topk_grad (rows on their
// vectors' boundaries); the formulas are in score_grad.cu.
//
// A warp takes four rows of a layer (two where k > 8, one where k > 16).  The
// choices go to 8 (16, 32) lanes a row, the dense part to LR lanes a row, each with
// a block of 8 neighbouring experts, so that both are coalesced and full; the
// chosen experts' parts reach their blocks through a row of shared memory.
//
// Measured (GB300): 30,011 tokens x 26 layers of 64 bf16 logits, k = 6, plain softmax
// and score sums, token-major: 54 us, 4.2 TB/s of algorithmic bytes; issue-bound (3.1
// of 4 instructions a clock).  16,384 x 48 of 256 bf16 logits, renormalised sigmoid
// (chosen logits only): 119 us; ncu counts 395 MB read for 13 MB of chosen logits
// and 31 MB of ids and gradients, for DRAM moves 64-byte pieces, and 350 MB written:
// 82 % of the DRAM's own peak, the bound.
#pragma once

#include "pdl.cuh"
#include "score.cuh"

namespace moer {

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
// choices (k <= KL <= LR).  WHOLE: E = 8 LR and rows on 16 bytes.
template <typename X, int LR, int KL, bool WHOLE, bool SOFT, bool RENORM, bool DENSE>
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
  __shared__ float4 scalar[SGT_WARPS][ROWS];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = blockIdx.x / p.nspan, unit = blockIdx.x - l * p.nspan;
  const bool has_a = DENSE && p.d_score_sum != nullptr;
  const int rc = lane / KL, j = lane % KL;    // the lane's choice
  const int rd = lane / LR, blk = lane % LR; // its block
  const int room = WHOLE ? 8 : p.E - 8 * blk;
  const bool wide = WHOLE || p.wide != 0;
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
      to[s].template load<X>(brow + s * rs_in, t0 + s * RS + rd < t1 ? room : 0, wide);
    brow += cstep;
  };
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    float4* z = reinterpret_cast<float4*>(chosen[warp][s * RS + rd]);
    z[blk] = z[LR + blk] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncwarp();
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
    const int slot = (id >> 3) * 4 + (id & 3) + ((id & 4) != 0 ? 4 * LR : 0);
    float* at = &chosen[warp][rc][slot];
    const float tag = __int_as_float(j + 1);
    if (ok) *at = tag;  // to see whether another choice of the row has the same id
    if constexpr (DENSE) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        if constexpr (SOFT) {
          // exp2(x log2 e - round(m log2 e)): one factor, of the product's rounding, is
          // common to the row, and every use of the exponentials divides it out by z
          float m = LOWEST;  // under every number lies only -inf, whose exponential is 0
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, v[s][i]);
          m = part_max<LR>(m);
          float z = 0.f, e[8], mm = m * LOG2E;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            e[i] = ex2_approx(fmaf(v[s][i], LOG2E, -mm));
            z += e[i];
          }
          z = part_sum<LR>(z);
          // a NaN or +inf among the logits, nothing but masks, or a largest logit so far
          // from 0 that the factor is no small one (without it z is from 1 to E)
          if (__any_sync(FULL, !(z < 1e6f && z > 0.01f))) {
            z = 0.f;
            mm = __uint_as_float(0x7FFFFFFFu);  // tells the chosen ones
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
          if (!RENORM && blk == 0) scalar[warp][s * RS + rd] = make_float4(m, rz[s], 0.f, mm);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[s][i] = a[i] * sigmoid_slope(live_logit(v[s][i]));
        }
      }
    }
    __syncwarp();
    // the part at the chosen expert
    float dj;
    if constexpr (SOFT) {
      const float4 mr = DENSE && !RENORM ? scalar[warp][rc] : make_float4(0.f, 0.f, 0.f, 0.f);
      const float m = RENORM ? fmaxf(part_max<KL>(xj), LOWEST) : mr.x;
      if constexpr (RENORM) {
        const float e = xj == m ? 1.f : ex2_approx(LOG2E * (xj - m));
        const float z = part_sum<KL>(e);
        const float q = z > 0.f ? e * rcp_approx(z) : 0.f;
        dj = q * (g - part_sum<KL>(g * q));
      } else {
        const float e = mr.w == mr.w ? ex2_approx(fmaf(xj, LOG2E, -mr.w)) : exp_below(xj, m);  // as in z
        dj = g * e * mr.y;
        const float dg = part_sum<KL>(dj);
        __syncwarp();
        if (j == 0) scalar[warp][rc].z = dg;
      }
    } else {
      // s and 1 - s from one exponential of -|x|; scores that the gate takes as 0 are 0
      // here too, and the shares q stay below 1 where 1 / sum alone may pass the range
      const float t = expf(-fabsf(xj)), r = rcp_approx(1.f + t);
      if constexpr (RENORM) {
        const bool up = xj >= 0.f;
        const float s = !ok ? 0.f : up ? r : mul_ftz(t, r);
        const float z = part_sum<KL>(s), q = z > 0.f ? s * (1.f / z) : 0.f;
        dj = (g - part_sum<KL>(g * q)) * (q * (up ? t * r : r));
      } else {
        dj = g * mul_ftz(t, r * r);
      }
    }
    const bool lost = ok && __float_as_int(*at) != j + 1;
    const bool repeats = __any_sync(FULL, lost);
    if (ok) *at = repeats ? 0.f : dj;
    if (repeats) {
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
        if constexpr (SOFT) {
          const float d = rz[s] * (dot[s] + (RENORM ? 0.f : scalar[warp][r].z));
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
      if (t0 + r < t1) store8<X>(orow + s * rs_out, room, wide, dx);
    }
    orow += ostep;
    __syncwarp();
    if (ok) *at = 0.f;  // the rows of shared memory stay 0 between tiles
    __syncwarp();
    now = then;
    then = after;
    xnow = xthen;
  }
  pdl_release();
}

template <typename X, int LR, int KL, bool WHOLE>
cudaError_t grad_tile_run(const ScoreParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)(p.L * p.nspan)), block(SGT_WARPS * 32);
  const bool a = p.d_score_sum != nullptr;
  if (p.score == MOER_SCORE_SOFTMAX) {
    if (p.renorm == 0) return launch_pdl(score_grad_tile_kernel<X, LR, KL, WHOLE, true, false, true>, grid, block, 0, st, p);
    return a ? launch_pdl(score_grad_tile_kernel<X, LR, KL, WHOLE, true, true, true>, grid, block, 0, st, p)
             : launch_pdl(score_grad_tile_kernel<X, LR, KL, WHOLE, true, true, false>, grid, block, 0, st, p);
  }
  if (p.renorm == 0)
    return a ? launch_pdl(score_grad_tile_kernel<X, LR, KL, WHOLE, false, false, true>, grid, block, 0, st, p)
             : launch_pdl(score_grad_tile_kernel<X, LR, KL, WHOLE, false, false, false>, grid, block, 0, st, p);
  return a ? launch_pdl(score_grad_tile_kernel<X, LR, KL, WHOLE, false, true, true>, grid, block, 0, st, p)
           : launch_pdl(score_grad_tile_kernel<X, LR, KL, WHOLE, false, true, false>, grid, block, 0, st, p);
}

template <typename X>
cudaError_t grad_tile(const ScoreParams& p, cudaStream_t st) {
  if (p.k > 16) return grad_tile_run<X, 32, 32, false>(p, st);
  if (p.k > 8) return p.E <= 128 ? grad_tile_run<X, 16, 16, false>(p, st) : grad_tile_run<X, 32, 16, false>(p, st);
  if (p.wide != 0) {
    if (p.E == 64) return grad_tile_run<X, 8, 8, true>(p, st);
    if (p.E == 128) return grad_tile_run<X, 16, 8, true>(p, st);
    if (p.E == 256) return grad_tile_run<X, 32, 8, true>(p, st);
  }
  return p.E <= 64    ? grad_tile_run<X, 8, 8, false>(p, st)
         : p.E <= 128 ? grad_tile_run<X, 16, 8, false>(p, st)
                      : grad_tile_run<X, 32, 8, false>(p, st);
}

}  // namespace moer
