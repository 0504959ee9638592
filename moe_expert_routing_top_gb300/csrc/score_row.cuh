// score_row.cuh -- one row of the scored top-k gate by one warp, for any E <= 256,
// k <= 32 and any options, with exact keys: the path of the rows that neither kernel's
// fixed-point keys settle (score_fast.cuh).  Some 4 to 8 us of one warp; taken for
// every row it needs 2,367 us where the fast kernel takes 282.
#pragma once

#include "score.cuh"

namespace moer {

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
    gk = max(gk, rank_key(NEG_INF));  // a group of NaN alone ties with one of -inf
    if (lane == g) mine = gk;
  }
  return mine;
}

// One row by one warp: the k ids and weights to `ids` and `weights` (or NULL).
// Returns the row's largest logit where a softmax over the row was formed.
template <typename X, int NQ>
__device__ float score_row(const ScoreParams& p, const X* row, const float (&bias)[4 * NQ], uint8_t* ids,
                           float* weights, int lane) {
  const bool soft = p.score == MOER_SCORE_SOFTMAX;
  const bool use_s = p.bias != nullptr || (p.n_group > 1 && p.group_best == 2);  // the choice takes scores
  const bool dense = p.partial != nullptr || use_s || (soft && !p.renorm);
  float x[4 * NQ], s[4 * NQ], row_m = NEG_INF;
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
      row_m = m;
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
  if (lane < p.k) ids[lane] = (uint8_t)id;
  if (weights != nullptr) {
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
    if (lane < p.k) weights[lane] = p.scale * w;
  }
  return row_m;
}

}  // namespace moer
