// score_fast.cuh -- the scored top-k gate at throughput sizes: G lanes per row
// (E <= 64 G), k <= 8, 32 / G rows of a warp at a time.
//
// Lane i of a row holds the blocks of 8 neighbouring experts 8 (i + G b), b < NB.
// Each block becomes 8 integer keys, sorted by a comparator network; the
// blocks' lists are merged into the lane's top 8 with the 9th key, and the
// lanes' lists across the row (rank.cuh).
//
// Keys: what the choice goes by, v, is mapped to a 23-bit fixed-point number n by a
// saturating multiply-add onto [0, 1] (NaN and -inf to 0) and a second one onto
// the binade [2^23, 2^24), whose mantissa bits are n; a multiply-add puts
// 255 - id below it.  The three steps run on the FMA pipe, while the networks'
// minima and maxima fill the ALU pipe, which is the kernel's bound.  The range is
// +-128 for logits (steps of 2^-15) and [-1, 3) for choice scores (5e-7).
//
// A row's answer is kept only where it is certain: the k-th key above 0, the
// first below the top of the range, no two neighbours among the k + 1 leading keys
// of equal n (of scores: within one step) -- but for neighbours within the k whose
// logits and biases are equal too, a true tie that the id in the key orders
// (16-bit logits of size 2^-5 and more have exact keys, and need no check) --
// and, with groups, the last kept group more
// than the rounding of its keys above the first dropped one.  The warp redoes
// the other rows one by one with the exact keys of score_row.cuh.
//
// The weights are computed from the chosen logits, read again (they are in L1).
// A softmax over the row takes its largest logit from the choice and one pass over
// the registers; score sums take a second pass over the warp's rows from L1, in
// which a lane owns columns, so that no atomics are needed.
#pragma once

#include "pdl.cuh"
#include "score.cuh"
#include "score_row.cuh"

namespace moer {

constexpr int SF_WARPS = 4;

__device__ __forceinline__ float fma_sat(float a, float b, float c) {  // NaN -> 0
  float r;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Whether n holds a logit exactly: 16-bit logits of size 2^-5 to 128 are
// multiples of 2^-15, a step of n, so that equal n mean equal logits there and
// the id in the key orders them.
template <int EB>
__device__ __forceinline__ bool exact_n(int n) {
  return EB == 2 && abs(n - 4194304) > 1024 && n > 0;
}

// Keys of a block's choices v = x or score: n = fixed point of v mul + add.
__device__ __forceinline__ void block_keys(const float (&v)[8], float mul, float add, uint32_t key_mul, int pos,
                                           int (&c)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = fma_sat(v[j], mul, add);
    const float t = fmaf(u, 8388607.f, 8388608.f);
    c[j] = (int)(__float_as_uint(t) * key_mul + (uint32_t)(255 - pos - j));
  }
}

template <int G>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// BY_SCORE: the choice goes by scores (a bias, or groups ranked by two scores)
// or there are groups; without it the logits alone order the experts.
template <typename X, int G, int NB, bool BY_SCORE>
__global__ void __launch_bounds__(SF_WARPS * 32, 4) score_fast_kernel(const ScoreParams p) {
  constexpr int RW = 32 / G;            // rows of a warp at a time
  constexpr int EB = sizeof(X);
  constexpr int NQ = G > 2 ? 2 : 1;     // quads of a lane in the column passes
  constexpr int OUT = 8 / G;            // choices of a lane
  __shared__ float sbias[256];
  __shared__ float part[SF_WARPS][32 * 4 * NQ];
  __shared__ float2 row_mr[SF_WARPS][RW];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane % G, rl = lane / G;
  const int l = blockIdx.x / p.nspan, unit = blockIdx.x - l * p.nspan;
  const bool soft = p.score == MOER_SCORE_SOFTMAX;
  const bool has_bias = BY_SCORE && p.bias != nullptr;
  const bool use_s = BY_SCORE && (has_bias || (p.n_group > 1 && p.group_best == 2));
  const bool sums = p.partial != nullptr;
  const bool dense_soft = soft && (sums || use_s || !p.renorm);
  if (has_bias)
    for (int e = threadIdx.x; e < 256; e += SF_WARPS * 32) sbias[e] = e < p.E ? p.bias[(size_t)l * p.E + e] : 0.f;
  __syncthreads();
  float acc[4 * NQ];
#pragma unroll
  for (int q = 0; q < 4 * NQ; ++q) acc[q] = 0.f;
  const X* base = static_cast<const X*>(p.logits) + l * p.ld_layer;
  const int64_t t1 = min64(p.T, (int64_t)(unit + 1) * p.span);
  for (int64_t t0 = (int64_t)unit * p.span + warp * RW; t0 < t1; t0 += SF_WARPS * RW) {
    const bool live = t0 + rl < t1;
    const int64_t t = live ? t0 + rl : t1 - 1;
    const X* row = base + t * p.ld_token;
    Raw<EB> raw[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int e = 8 * (i + G * b);
      raw[b].template load<X>(row + e, p.E - e, p.wide != 0);
    }
    int top[8], ninth = INT_MIN;
    bool bad = false;
    float m = 0.f, rz = 0.f;
    if constexpr (!BY_SCORE) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float x[8];
        raw[b].template get<X>(x);
        int c[8];
        block_keys(x, 1.f / 256.f, 0.5f, p.key_mul, 8 * G * b, c);
        sort8_desc(c);
        if (b == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) top[j] = c[j];
        } else {
          merge8<true>(top, c, ninth);
        }
      }
    } else {
      float v[NB][8];
#pragma unroll
      for (int b = 0; b < NB; ++b) raw[b].template get<X>(v[b]);
      if (dense_soft) {
        m = NEG_INF;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, v[b][j]);
        m = row_max<G>(m);
        bad = !(fabsf(m) < 128.f);  // nothing but masks, or infinities: left to the exact path
        float z = 0.f;
        const float mm = bad ? 0.f : m * LOG2E;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j) z += ex2_approx(fmaf(fmaxf(v[b][j], NEG_INF), LOG2E, -mm));
        rz = rcp_approx(row_sum<G>(z));
      }
      if (use_s) {
        float sq = 0.f;  // infinite or NaN: some logit is
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j) sq = fmaf(v[b][j], v[b][j], sq);
        // (experts past the row's end are -inf here)
        const bool far = __any_sync(FULL, !(sq < 3e38f));
        const float mm = m * LOG2E;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int e = 8 * (i + G * b);
          float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (has_bias) {
            const float4 b0 = *reinterpret_cast<const float4*>(&sbias[e]), b1 = *reinterpret_cast<const float4*>(&sbias[e + 4]);
            bias[0] = b0.x, bias[1] = b0.y, bias[2] = b0.z, bias[3] = b0.w;
            bias[4] = b1.x, bias[5] = b1.y, bias[6] = b1.z, bias[7] = b1.w;
          }
          float s[8];
          if (soft) {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = ex2_approx(fmaf(v[b][j], LOG2E, -mm)) * rz;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float x = far ? fmaxf(v[b][j], NEG_INF) : v[b][j];  // NaN -> -inf
              s[j] = rcp_approx(1.f + ex2_approx(-LOG2E * x));
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float c = s[j] + bias[j];
            v[b][j] = far && !(v[b][j] > NEG_INF) ? NEG_INF : c;  // masked experts stay out whatever their bias
          }
        }
      }
      int key[NB][8];
      const float mul = use_s ? 0.25f : 1.f / 256.f, add = use_s ? 0.25f : 0.5f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        block_keys(v[b], mul, add, p.key_mul, 8 * G * b, key[b]);
        sort8_desc(key[b]);
      }
      if (p.n_group > 1) {
        // a group is m blocks of every lane of the row
        const int sh = 31 - __clz(p.E / p.n_group / (8 * G)), mb = 1 << sh;
        int g1[8], g2[8], gk[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          g1[b] = b < NB ? key[b < NB ? b : 0][0] >> 8 : -1;
          g2[b] = b < NB ? key[b < NB ? b : 0][1] >> 8 : -1;
        }
#pragma unroll
        for (int s = 1; s < 8; s *= 2)
          if (s < mb)
#pragma unroll
            for (int b = 0; b < 8; b += 2 * s) {
              g2[b] = max(max(g2[b], g2[b + s]), min(g1[b], g1[b + s]));
              g1[b] = max(g1[b], g1[b + s]);
            }
#pragma unroll
        for (int b = 0; b < 8; ++b) {
#pragma unroll
          for (int o = 1; o < G; o *= 2) {
            const int h1 = __shfl_xor_sync(FULL, g1[b], o), h2 = __shfl_xor_sync(FULL, g2[b], o);
            g2[b] = max(max(g2[b], h2), min(g1[b], h1));
            g1[b] = max(g1[b], h1);
          }
          const bool first = (b & (mb - 1)) == 0 && (b >> sh) < p.n_group;
          // the second best counts only where there are two numbers to add
          if (first && p.group_best == 2 && g2[b] <= 0) bad = true;
          g1[b] += p.group_best == 2 ? g2[b] : 0;
          gk[b] = first ? g1[b] * 8 + (7 - (b >> sh)) : INT_MIN;
        }
        sort8_desc(gk);
        int thr = gk[0], nxt = gk[1];
#pragma unroll
        for (int r = 1; r < 7; ++r)
          if (r < p.top_group) thr = gk[r], nxt = gk[r + 1];
        // the sum of two scores' keys can be two steps off either way; equal keys of
        // logits may stand in either order, unless they hold their logits exactly
        if ((thr >> 3) - (nxt >> 3) <= (use_s ? 4 : 0) && (use_s || !exact_n<EB>(thr >> 3))) bad = true;
        int keep = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const bool first = (b & (mb - 1)) == 0;
          keep = first ? (g1[b] * 8 + (7 - (b >> sh)) >= thr ? 1 : 0) : keep;
          if (b < NB)
#pragma unroll
            for (int j = 0; j < 8; ++j) key[b][j] *= keep;  // on the FMA pipe; 0 is below every key
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (b == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) top[j] = key[0][j];
        } else {
          merge8<true>(top, key[b], ninth);
        }
      }
    }
    // ids of the row: the lane's own part comes off the inverted position
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] -= 8 * i;
    ninth -= 8 * i;
#pragma unroll
    for (int o = 1; o < G; o *= 2) {
      int other[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) other[j] = __shfl_xor_sync(FULL, top[j], o);
      const int n9 = __shfl_xor_sync(FULL, ninth, o);
      merge8<true>(top, other, ninth);
      ninth = max(ninth, n9);
    }
    // the lane's choices: j = i, i + G, ...
    float xj[OUT], bj[OUT];
    int mine[OUT];
    const int near = use_s ? 1 : 0;     // steps of n that do not settle an order: a score is rounded before its key is
    int last = top[0], after = top[1];  // the k-th key and the one after it
#pragma unroll
    for (int j = 1; j < 8; ++j)
      if (j < p.k) last = top[j], after = j + 1 < 8 ? top[j + 1 < 8 ? j + 1 : 0] : ninth;
    bad = bad || last < 256 || (top[0] >> 8) >= 8388607 ||
          ((last >> 8) - (after >> 8) <= near && (use_s || !exact_n<EB>(last >> 8)));
#pragma unroll
    for (int jj = 0; jj < OUT; ++jj) {
      int c = top[jj * G];
#pragma unroll
      for (int g = 1; g < G; ++g)
        if (i == g) c = top[jj * G + g];
      mine[jj] = c;
      const int e = 255 - (c & 255);
      const bool on = jj * G + i < p.k && e < p.E;
      xj[jj] = on ? live_logit(Quad<X>::one(row[e])) : NEG_INF;
      bj[jj] = has_bias ? sbias[e] : 0.f;
    }
    // neighbours of equal n have to be a true tie
    bool tie = false;
#pragma unroll
    for (int j = 1; j < 8; ++j)
      if (j < p.k && (top[j - 1] >> 8) - (top[j] >> 8) <= near && (use_s || !exact_n<EB>(top[j] >> 8))) tie = true;
    if (__any_sync(FULL, tie)) {
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        const int from = rl * G + j % G, prev = rl * G + (j - 1) % G;
        const float a = __shfl_sync(FULL, xj[j / G], from), b = __shfl_sync(FULL, xj[(j - 1) / G], prev);
        const float c = __shfl_sync(FULL, bj[j / G], from), d = __shfl_sync(FULL, bj[(j - 1) / G], prev);
        if (j < p.k && (top[j - 1] >> 8) - (top[j] >> 8) <= near && !(a == b && c == d)) bad = true;
      }
    }
    if constexpr (!BY_SCORE) {
      if (dense_soft) {
        m = __shfl_sync(FULL, xj[0], rl * G);  // the first choice is the largest logit
        const float mm = fabsf(m) < 1e30f ? m * LOG2E : 0.f;
        float z = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float x[8];
          raw[b].template get<X>(x);
#pragma unroll
          for (int j = 0; j < 8; ++j) z += ex2_approx(fmaf(fmaxf(x[j], NEG_INF), LOG2E, -mm));
        }
        rz = rcp_approx(row_sum<G>(z));
      }
    }
    const int64_t out = ((int64_t)l * p.T + t) * p.k;
    const bool write = live && !bad;
    if (p.weights != nullptr) {
      float w[OUT], z = 0.f;
      if (soft) {
        float mk = m;
        if (p.renorm) {
          mk = NEG_INF;
#pragma unroll
          for (int jj = 0; jj < OUT; ++jj) mk = fmaxf(mk, xj[jj]);
          mk = row_max<G>(mk);
        }
#pragma unroll
        for (int jj = 0; jj < OUT; ++jj) w[jj] = exp_below(xj[jj], mk);
      } else {
#pragma unroll
        for (int jj = 0; jj < OUT; ++jj) w[jj] = sigmoid(xj[jj]);
      }
#pragma unroll
      for (int jj = 0; jj < OUT; ++jj) z += w[jj];
      float f = soft ? rz : 1.f;
      if (p.renorm) {
        z = row_sum<G>(z);
        f = z > 0.f ? 1.f / z : 0.f;
      }
      f *= p.scale;
#pragma unroll
      for (int jj = 0; jj < OUT; ++jj)
        if (write && jj * G + i < p.k) p.weights[out + jj * G + i] = w[jj] * f;
    }
#pragma unroll
    for (int jj = 0; jj < OUT; ++jj)
      if (write && jj * G + i < p.k) p.topk[out + jj * G + i] = (uint8_t)(255 - (mine[jj] & 255));
    if (sums && i == 0) row_mr[warp][rl] = make_float2(m, rz);
    // rows that are not settled, one by one
    unsigned todo = __ballot_sync(FULL, bad && live && i == 0);
    const bool careful = todo != 0u;
    __syncwarp();
    while (todo != 0u) {
      const int f = (__ffs(todo) - 1) / G;
      todo &= todo - 1;
      float bias[4 * NQ], none[4 * NQ];
#pragma unroll
      for (int q = 0; q < 4 * NQ; ++q) {
        const int e = 4 * (lane + 32 * (q / 4)) + q % 4;
        bias[q] = has_bias ? sbias[e & 255] : 0.f;
        none[q] = 0.f;
      }
      const float2 mr = score_row<X, NQ>(p, base + (t0 + f) * p.ld_token, bias, (int64_t)l * p.T + t0 + f, lane, none);
      if (sums && lane == 0) row_mr[warp][f] = mr;
    }
    if (sums) {
      // a lane's columns: LR lanes hold a row's quads, 32 / LR rows at a time
      const int LR = p.E <= 32 ? 8 : p.E <= 64 ? 16 : 32;
      const int col = lane % LR;
      __syncwarp();
      const int rows = (int)min64(RW, t1 - t0);
      for (int r = lane / LR; r < rows; r += 32 / LR) {
        const X* at = base + (t0 + r) * p.ld_token;
        const float2 mr = soft ? row_mr[warp][r] : make_float2(0.f, 0.f);
        const float mm = mr.x * LOG2E;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const int e = 4 * (col + 32 * q);
          if (e < p.E) {
            float x[4];
            load4<X>(at + e, true, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v = fmaxf(x[j], NEG_INF);  // NaN -> -inf
              float s;
              if (soft)
                s = (careful ? exp_below(v, mr.x) : ex2_approx(fmaf(v, LOG2E, -mm))) * mr.y;
              else
                s = rcp_approx(1.f + ex2_approx(-LOG2E * v));
              acc[4 * q + j] += s;
            }
          }
        }
      }
      __syncwarp();
    }
  }
  if (sums) {
    const int LR = p.E <= 32 ? 8 : p.E <= 64 ? 16 : 32;
#pragma unroll
    for (int q = 0; q < 4 * NQ; ++q) {
      float v = acc[q];
      if (LR <= 16) v += __shfl_xor_sync(FULL, v, 16);
      if (LR <= 8) v += __shfl_xor_sync(FULL, v, 8);
      part[warp][4 * (lane + 32 * (q / 4)) + q % 4] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += SF_WARPS * 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < SF_WARPS; ++w) v += part[w][e];
      p.partial[(size_t)blockIdx.x * p.E + e] = v;
    }
  }
  pdl_release();
}

template <typename X, int G, int NB>
cudaError_t score_fast_shape(const ScoreParams& p, cudaStream_t st) {
  const dim3 grid(p.L * p.nspan), block(SF_WARPS * 32);
  return p.bias != nullptr || p.n_group > 1 ? launch_pdl(score_fast_kernel<X, G, NB, true>, grid, block, 0, st, p)
                                            : launch_pdl(score_fast_kernel<X, G, NB, false>, grid, block, 0, st, p);
}

template <typename X>
cudaError_t score_fast_run(const ScoreParams& p, cudaStream_t st) {
  const int nb = (p.E + 7) / 8;
  if (p.E <= 16) return score_fast_shape<X, 1, 2>(p, st);
  if (p.E <= 32) return score_fast_shape<X, 1, 4>(p, st);
  if (p.E <= 64) return score_fast_shape<X, 1, 8>(p, st);
  if (nb <= 12) return score_fast_shape<X, 2, 6>(p, st);
  if (nb <= 16) return score_fast_shape<X, 2, 8>(p, st);
  if (nb <= 24) return score_fast_shape<X, 4, 6>(p, st);
  return score_fast_shape<X, 4, 8>(p, st);
}

}  // namespace moer
