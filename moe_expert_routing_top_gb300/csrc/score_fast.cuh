// score_fast.cuh -- the scored top-k gate at throughput sizes: G lanes per row
// (E <= 64 G), k <= KT = 8 or 16, 32 / G rows of a warp at a time.
//
// Lane i of a row holds the blocks of 8 neighbouring experts 8 (i + G b), b < NB.
// Each block becomes 8 integer keys, sorted by a comparator network; the
// blocks' lists are merged into the lane's top KT with the key after them, and the
// lanes' lists across the row (rank.cuh; a top 16 is two lists of 8).
//
// Keys: what the choice goes by, v, is mapped to a 23-bit fixed-point number n by a
// saturating multiply-add onto [0, 1] (NaN and -inf to 0) and a second one onto
// the binade [2^23, 2^24), whose mantissa bits are n; a multiply-add puts
// 255 - id below it.  The three steps run on the FMA pipe, while the networks'
// minima and maxima fill the ALU pipe, which is the kernel's bound.  The range is
// +-128 for logits (steps of 2^-15) and [-1, 3) for choice scores (5e-7; the bias
// comes in with the first step).
//
// A row's answer is kept only where it is certain: the k-th key above 0, the
// first below the top of the range, no run of neighbours among the leading keys of
// equal n (of scores: within two steps) that their values put in another order, but
// for its first two (16-bit logits of size 2^-5 and more have exact keys, which their
// ids order; so have their scores, where all experts share one bias and the slope is
// not small), and, with groups, the last kept group more than the rounding of its keys
// above the first dropped one and no key at the top of the range in a sum of two.  The warp
// redoes the other rows one by one with the exact keys of score_row.cuh.
//
// The weights are computed from the chosen logits, read again (they are in L1).
// A softmax over the row without a renormalisation, and score sums, take a pass
// over the warp's rows from L1 in which a lane owns eight columns: exponentials
// against the row's largest logit (from the choice), their sum across the row's
// lanes, and the columns' sums in registers, so that no atomics are needed.
//
// Measured (GB300): 65,536 tokens x 48 layers of 128 fp32 logits, k = 8, softmax
// weights: 282 us, 6.15 TB/s of algorithmic bytes, 0.91 of the measured copy
// bandwidth (bf16 logits, half the bytes at the same comparators: 277 us).  8,209 x
// 26 of 256 bf16 logits, sigmoid with bias, 4 of 8 groups by their two best: 71 us
// (1.7 TB/s): 247 warp instructions a row, issued at 2.6 of 4 a clock; the networks are
// 30 % of them (580 minima and maxima a lane, 27 us of the ALU pipe at its full rate),
// and with the others the pipe is 63 % busy.  30,011 x 26 of 64 bf16 logits, k = 6,
// softmax weights and score sums: 64 us, of which the column pass is about 20.
// Why lanes by columns of blocks: the networks cost the same per logit in every
// split, but more lanes a row merge more lists (a row of 128 logits: 80 minima and
// maxima for 8 logits with G = 4 and 32 logits a lane, 71 with G = 2 and 64), while one
// lane for 128 and more logits cannot hold them in registers.
#pragma once

#include "pdl.cuh"
#include "score.cuh"
#include "score_row.cuh"

namespace moer {

constexpr int SF_WARPS = 4;

// Keys of a block: t holds n in the low 23 bits of a number in [2^23, 2^24); 255 - id goes below n.
// The upper quad's ids lie `gap` further on.
__device__ __forceinline__ void block_ids(const float (&t)[8], uint32_t key_mul, int pos, int (&c)[8], int gap = 0) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    asm("mad.lo.u32 %0, %1, %2, %3;"
        : "=r"(c[j])
        : "r"(__float_as_uint(t[j])), "r"(key_mul), "r"(255 - pos - j - (j < 4 ? 0 : gap)));
}

// Whether no logit of the blocks is infinite or NaN: the sum of their squares is
// not (16-bit types in pairs; an f16 logit of 256 and more counts as far too).
template <typename X, int N>
__device__ __forceinline__ bool finite_blocks(const Raw<sizeof(X)> (&raw)[N]) {
  if constexpr (sizeof(X) == 4) {
    float sq = 0.f;
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(raw[b].v[j], raw[b].v[j], sq);
    return sq < 3e38f;
  } else {
    using P = typename std::conditional<std::is_same<X, __half>::value, __half2, __nv_bfloat162>::type;
    uint32_t sq = 0u;
#pragma unroll
    for (int b = 0; b < N; ++b) {
      const uint32_t w[4] = {raw[b].v.x, raw[b].v.y, raw[b].v.z, raw[b].v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const P v = *reinterpret_cast<const P*>(&w[j]);
        const P s = __hfma2(v, v, *reinterpret_cast<const P*>(&sq));
        sq = *reinterpret_cast<const uint32_t*>(&s);
      }
    }
    constexpr uint32_t TOP = std::is_same<X, __half>::value ? 0x7C00u : 0x7F80u;  // exponent of infinity and NaN
    return (sq & TOP) != TOP && (sq >> 16 & TOP) != TOP;
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

// A lane's choices, `own` of them (or OUT): in pairs where k is even (`even` 1: the
// weights are on 8 bytes; 2: k = 8 and they are on 16, one store of all).
template <int OUT>
__device__ __forceinline__ void put_weights(float* to, int own, int even, const float (&w)[OUT]) {
  if (even == 2) {
    if constexpr (OUT == 2) {
      *reinterpret_cast<float2*>(to) = make_float2(w[0], w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < OUT; j += 4)
        *reinterpret_cast<float4*>(to + j) = make_float4(w[j], w[j + 1], w[j + 2], w[j + 3]);
    }
  } else if (even == 1) {
#pragma unroll
    for (int j = 0; j < OUT; j += 2)
      if (j < own) *reinterpret_cast<float2*>(to + j) = make_float2(w[j], w[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < OUT; ++j)
      if (j < own) to[j] = w[j];
  }
}
template <int OUT>
__device__ __forceinline__ void put_ids(uint8_t* to, int own, int even, const int (&id)[OUT]) {
  if (even == 2) {  // 8 ids a row, on 8 bytes
    uint32_t v[OUT / 4 + 1];
    if constexpr (OUT == 2) {
      *reinterpret_cast<uint16_t*>(to) = (uint16_t)(id[0] | id[1] << 8);
    } else {
#pragma unroll
      for (int j = 0; j < OUT; j += 4)
        v[j / 4] = (uint32_t)(id[j] | id[j + 1] << 8) | (uint32_t)(id[j + 2] | id[j + 3] << 8) << 16;
      if constexpr (OUT == 4)
        *reinterpret_cast<uint32_t*>(to) = v[0];
      else
        *reinterpret_cast<uint2*>(to) = make_uint2(v[0], v[1]);
    }
  } else if (even == 1) {
#pragma unroll
    for (int j = 0; j < OUT; j += 2)
      if (j < own) *reinterpret_cast<uint16_t*>(to + j) = (uint16_t)(id[j] | id[j + 1] << 8);
  } else {
#pragma unroll
    for (int j = 0; j < OUT; ++j)
      if (j < own) to[j] = (uint8_t)id[j];
  }
}

// Folds a sorted list of 8 into the running top KT: with KT = 16 the upper list takes
// its 8 by Batcher's odd-even merge (25 comparators), whose lower half goes on into
// the lower list.
template <int KT, int N>
__device__ __forceinline__ void fold(int (&top)[8], int (&low)[N], const int (&c)[8], int& next) {
  if constexpr (KT == 8) {
    merge8<true>(top, c, next);
  } else {
    int w[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = top[i], w[8 + i] = c[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) cas(w[i], w[i + 8]);
#pragma unroll
    for (int i = 4; i < 8; ++i) cas(w[i], w[i + 4]);
    cas(w[2], w[4]); cas(w[3], w[5]); cas(w[6], w[8]); cas(w[7], w[9]); cas(w[10], w[12]); cas(w[11], w[13]);
#pragma unroll
    for (int i = 1; i < 14; i += 2) cas(w[i], w[i + 1]);
    int rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = w[i], rest[i] = w[8 + i];
    merge8<true>(low, rest, next);
  }
}

struct Eight {
  float v[8];
};
// u = (c + 1) / 4 of a block's choice scores c = s + b, saturated onto [0, 1].
template <int KIND>
__device__ __forceinline__ Eight choice(Eight x, const Eight& bias, float mm, float rs) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = KIND == BY_SOFTMAX ? ex2_approx(fmaf(x.v[j], LOG2E, -mm)) * rs
                                       : rcp_approx(1.f + ex2_approx(-LOG2E * x.v[j]));
    x.v[j] = fma_sat(s, 0.25f, bias.v[j]);
  }
  return x;
}
// The same where logits are infinite or NaN: masked experts stay out whatever their bias.
template <int KIND>
__device__ __noinline__ Eight far_choice(Eight x, Eight bias, float mm, float rs) {
  Eight y = x;
#pragma unroll
  for (int j = 0; j < 8; ++j) y.v[j] = fmaxf(x.v[j], NEG_INF);  // NaN -> -inf
  const Eight u = choice<KIND>(y, bias, mm, rs);
#pragma unroll
  for (int j = 0; j < 8; ++j) y.v[j] = y.v[j] == NEG_INF ? 0.f : u.v[j];
  return y;
}

// WHOLE: E = 8 G NB and rows on 16 bytes, every block whole.
// SPLIT (groups of gs experts, gs no power of two times 8 G): the lane's blocks go
// group by group, mb to a group, and a block is the quads 2 m G + i and
// (2 m + 1) G + i of its group, so that no block lies in two groups.  Where gs is no
// multiple of 4, a group has the quads that it shares with its neighbours, too, less
// their experts.
template <typename X, int G, int NB, int KT, int KIND, bool WHOLE, bool SPLIT>
__global__ void __launch_bounds__(SF_WARPS * 32, score_resident(sizeof(X), KIND, KT)) score_fast_kernel(const ScoreParams p) {
  constexpr int RW = 32 / G;            // rows of a warp at a time
  constexpr int EB = sizeof(X);
  constexpr int NQ = G > 2 ? 2 : 1;     // quads of a lane on the exact path
  constexpr int OUT = KT / G;           // choices of a lane
  constexpr int CL = 8 * G;             // lanes of a row in the column pass
  constexpr int PF = NB % 4 == 0 ? 4 : NB % 3 == 0 ? 3 : 2;  // blocks in flight: a block's registers take the one PF ahead
  static_assert(NB % PF == 0, "whole rounds of the block buffers");
  constexpr bool LISTS = KIND >= BY_GROUP;     // there may be groups
  constexpr bool SCORES = KIND >= BY_SIGMOID;  // the choice takes scores
  constexpr int ROUNDS = SCORES ? 1 : NB / PF; // unrolled (the longer bodies: rolled, for the instruction cache)
  __shared__ __align__(16) float sbias[SCORES ? 256 : 1];
  __shared__ float part[SF_WARPS][KIND != BY_LOGIT ? 8 * CL : 1];
  __shared__ int4 lists[LISTS ? SF_WARPS : 1][LISTS ? NB : 1][2][32];  // sorted blocks
  __shared__ float2 row_mr[SF_WARPS][RW];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane % G, rl = lane / G;
  const int l = blockIdx.x / p.nspan, unit = blockIdx.x - l * p.nspan;
  const bool soft = KIND == SOFTMAX_SUMS || KIND == BY_SOFTMAX ||
                    (KIND != SIGMOID_SUMS && KIND != BY_SIGMOID && p.score == MOER_SCORE_SOFTMAX);
  const bool sums = KIND != BY_LOGIT && p.partial != nullptr;
  const bool columns = KIND == SOFTMAX_SUMS || KIND == SIGMOID_SUMS || (KIND != BY_LOGIT && (sums || (soft && !p.renorm)));
  bool even_bias = false;  // one bias for all of the layer's experts, and 16-bit logits
  if constexpr (SCORES) {
    const float* b = p.bias + (size_t)l * p.E;
    bool same = EB == 2;
    for (int e = threadIdx.x; e < 256; e += SF_WARPS * 32) {  // u = s / 4 + (b + 1) / 4
      sbias[e] = e < p.E ? fmaf(b[e], 0.25f, 0.25f) : 0.25f;
      same = same && (e >= p.E || b[e] == b[0]);
    }
    even_bias = __syncthreads_and(same);
  }
  constexpr int near = SCORES ? 2 : 0;  // steps of n that do not settle an order: a score is rounded before its key is
  float acc[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] = 0.f;
  const X* base = static_cast<const X*>(p.logits) + l * p.ld_layer;
  const int64_t t1 = min64(p.T, (int64_t)(unit + 1) * p.span);
  int64_t t0 = (int64_t)unit * p.span + warp * RW;
  // rows past the unit's end read its last row again
  auto row_at = [&](int64_t t) { return base + min64(t + rl, t1 - 1) * p.ld_token; };
  Raw<EB> raw[PF];
  const int gs = LISTS ? p.E / p.n_group : 0, per = LISTS ? (group_span(gs) + 8 * G - 1) / (8 * G) : 1;
  const int sh = per > 1 ? 32 - __clz(per - 1) : 0, mb = 1 << sh;  // blocks of a lane to a group
  // first expert of a block's first quad, less the lane's part, and whether its quads lie in the row
  auto split_at = [&](int b) { return ((b >> sh) * gs & ~3) + 8 * G * (b & (mb - 1)); };
  auto split_has = [&](int b, int h) {
    return split_at(b) + 4 * (G * h + i) < ((b >> sh) + 1) * gs && (b >> sh) < p.n_group;
  };
  const bool shared = SPLIT && (gs & 3) != 0;  // quads of two groups; whether expert j of a block is its group's own
  auto split_own = [&](int b, int j) {
    const int r = split_at(b) + 4 * (G * (j / 4) + i) + j % 4 - (b >> sh) * gs;
    return r >= 0 && r < gs;
  };
  auto fetch = [&](Raw<EB>& to, int b, const X* of, float fill = KIND >= BY_SIGMOID ? 0.f : NEG_INF) {
    const int e = 8 * (i + G * b);
    if constexpr (SPLIT) {
      const X* at = of + split_at(b) + 4 * i;
      to.template load2<X>(at, split_has(b, 0), at + 4 * G, split_has(b, 1), fill);
    } else if constexpr (WHOLE) {
      to.template load<X>(of + e, 8, true);
    } else {
      to.template load<X>(of + e, p.E - e, p.wide != 0, fill);
    }
  };
  const X* row = t0 < t1 ? row_at(t0) : base;
  if (t0 < t1)
#pragma unroll
    for (int j = 0; j < PF; ++j) fetch(raw[j], j, row);
  for (; t0 < t1; t0 += SF_WARPS * RW) {
    const bool live = t0 + rl < t1;
    const bool more = t0 + SF_WARPS * RW < t1;
    const X* next = more ? row_at(t0 + SF_WARPS * RW) : row;
    // the running top KT, as sorted lists of 8, and the key after them
    int top[8], low[KT > 8 ? 8 : 1], ninth = KT > 8 ? -1 : INT_MIN;
#pragma unroll
    for (int j = 0; j < (KT > 8 ? 8 : 1); ++j) low[j] = -1;
    bool bad = false;
    float mm = 0.f, rs = 1.f;
    if constexpr (KIND == BY_SOFTMAX) {
      // the softmax first: its largest logit and the sum, from L1
      float m = NEG_INF, z = 0.f;
      for (int b = 0; b < NB; ++b) {
        Raw<EB> again;
        fetch(again, b, row, NEG_INF);
        float x[8];
        again.template get<X>(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, x[j]);
      }
      m = row_max<G>(m);
      bad = !(fabsf(m) < 128.f);  // nothing but masks, or infinities: left to the exact path
      mm = bad ? 0.f : m * LOG2E;
      for (int b = 0; b < NB; ++b) {
        Raw<EB> again;
        fetch(again, b, row, NEG_INF);
        float x[8];
        again.template get<X>(x);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!shared || split_own(b, j)) z += ex2_approx(fmaf(fmaxf(x[j], NEG_INF), LOG2E, -mm));
      }
      rs = rcp_approx(row_sum<G>(z));
    }
#pragma unroll ROUNDS
    for (int g = 0; g < NB; g += PF) {
      const bool last_round = g + PF == NB;
      bool far = false;  // some logit of the round is infinite or NaN
      if constexpr (SCORES) far = __any_sync(FULL, !finite_blocks<X, PF>(raw));
#pragma unroll
      for (int j0 = 0; j0 < PF; ++j0) {
        const int b = g + j0, e = 8 * (i + G * b);
        Eight x;
        raw[j0].template get<X>(x.v);
        if (!last_round)
          fetch(raw[j0], b + PF, row);
        else if (more)
          fetch(raw[j0], j0, next);
        int c[8];
        if constexpr (SCORES) {
          const int f = SPLIT ? split_at(b) + 4 * i : e, f1 = SPLIT ? f + 4 * G : e + 4;  // past 252 is no expert
          const float4 b0 = *reinterpret_cast<const float4*>(&sbias[SPLIT ? min(f, 252) : f]);
          const float4 b1 = *reinterpret_cast<const float4*>(&sbias[SPLIT ? min(f1, 252) : f1]);
          const Eight bias = {{b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w}};
          if (far)
            x = far_choice<KIND>(x, bias, mm, rs);
          else
            x = choice<KIND>(x, bias, mm, rs);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x.v[j] = fma_sat(x.v[j], 1.f / 256.f, 0.5f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x.v[j] = fmaf(x.v[j], 8388607.f, 8388608.f);
        if constexpr (SPLIT)
          block_ids(x.v, p.key_mul, split_at(b), c, 4 * G - 4);
        else
          block_ids(x.v, p.key_mul, 8 * G * b, c);
        if (SCORES && !WHOLE) {  // experts past the row's (or the group's) end
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (SPLIT ? !split_has(b, j / 4) : e + (j & 4) >= p.E) c[j] &= 255;
        }
        if (shared)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!split_own(b, j)) c[j] &= 255;
        sort8_desc(c);
        if (LISTS && p.n_group > 1) {
          lists[warp][b][0][lane] = make_int4(c[0], c[1], c[2], c[3]);
          lists[warp][b][1][lane] = make_int4(c[4], c[5], c[6], c[7]);
        } else if (j0 == 0 && g == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) top[j] = c[j];
        } else {
          fold<KT>(top, low, c, ninth);
        }
      }
    }
    if (LISTS && p.n_group > 1) {
      // a group is mb blocks of every lane of the row, the first of them at group_at
      auto group_at = [&](int b) { return (b & (mb - 1)) == 0 && (b >> sh) < p.n_group; };
      int g1[8], g2[8], gk[8], most = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const int2 two = b < NB ? *reinterpret_cast<const int2*>(&lists[warp][b < NB ? b : 0][0][lane]) : make_int2(0, 0);
        g1[b] = two.x >> 8;
        g2[b] = two.y >> 8;
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
      }
      if (p.group_best == 2) {
        // a best key at the top of the range makes its group's sum too small
        most = g1[0];
#pragma unroll
        for (int b = 1; b < 8; ++b) most = max(most, g1[b]);
        if (most >= 8388607) bad = true;
      }
      if (!SCORES && p.group_best == 2) {  // the scores of the two best logits
        constexpr float STEP = 256.f / 8388607.f * LOG2E;
        auto score = [&](int n) {
          return soft ? ex2_approx((float)(n - most) * STEP)
                      : rcp_approx(1.f + ex2_approx(fmaf((float)(n - 4194304), -STEP, -0.5f * STEP)));
        };
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (g2[b] <= 0 && group_at(b)) bad = true;  // the second best counts only where there are two numbers to add
          g1[b] = (int)((score(g1[b]) + score(g2[b])) * 67108864.f);
        }
      }
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (SCORES && p.group_best == 2) {
          if (g2[b] <= 0 && group_at(b)) bad = true;
          g1[b] += g2[b];
        }
        g1[b] = gk[b] = group_at(b) ? g1[b] * 8 + (7 - (b >> sh)) : INT_MIN;
      }
      sort8_desc(gk);
      int thr = gk[0], nxt = gk[1];
#pragma unroll
      for (int r = 1; r < 7; ++r)
        if (r < p.top_group) thr = gk[r], nxt = gk[r + 1];
      const int kept = thr >> 3, out = nxt >> 3;
      if (!SCORES && p.group_best == 2) {
        // a logit's n is 0.75 steps of 3.1e-5 off at most, which changes each score by
        // 2.3e-5 of itself (of 1 less itself, where that is less): two sums in units of
        // 2^-26 may be 2^-14 of the sum off, and 128 units for the scores' own rounding
        const int part = soft ? kept : min(kept, (1 << 27) - out);
        if (kept - out <= (part >> 14) + 128) bad = true;
      } else if (kept - out <= 3 * near && (SCORES || !exact_n<EB>(kept))) {
        // the sum of two scores' keys can be three steps off either way; equal keys of
        // logits may stand in either order, unless they hold their logits exactly
        bad = true;
      }
      unsigned keep = 0u;  // the first blocks of the kept groups
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (g1[b] >= thr) keep |= 1u << b;
      for (int r = 1; r < mb; r *= 2) keep |= keep << r;  // and the others
      // their lists, each row's own; a single list's eight are all there is
      ninth = KT > 8 ? -1 : 0;
      {
        const int b0 = __ffs(keep) - 1;
        keep &= keep - 1u;
        const int4 u = lists[warp][b0][0][lane], v = lists[warp][b0][1][lane];
        top[0] = u.x, top[1] = u.y, top[2] = u.z, top[3] = u.w;
        top[4] = v.x, top[5] = v.y, top[6] = v.z, top[7] = v.w;
      }
      for (int q = 1; q < p.top_group * mb; ++q) {
        const int b0 = __ffs(keep) - 1;
        keep &= keep - 1u;
        const int4 u = lists[warp][b0][0][lane], v = lists[warp][b0][1][lane];
        const int c[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        fold<KT>(top, low, c, ninth);
      }
    }
    // ids of the row: the lane's own part comes off the inverted position
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top[j] -= (SPLIT ? 4 : 8) * i;
      if (KT > 8) low[KT > 8 ? j : 0] -= (SPLIT ? 4 : 8) * i;
    }
    ninth -= (SPLIT ? 4 : 8) * i;
#pragma unroll
    for (int o = 1; o < G; o *= 2) {
      int other[8];
      if constexpr (KT > 8) {  // the lower lists first: the upper ones' losers join them
#pragma unroll
        for (int j = 0; j < 8; ++j) other[j] = __shfl_xor_sync(FULL, low[j], o);
        merge8<true>(low, other, ninth);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) other[j] = __shfl_xor_sync(FULL, top[j], o);
      const int n9 = __shfl_xor_sync(FULL, ninth, o);
      fold<KT>(top, low, other, ninth);
      ninth = max(ninth, n9);
    }
    int best[KT];
#pragma unroll
    for (int j = 0; j < KT; ++j) best[j] = j < 8 ? top[j & 7] : low[KT > 8 ? j & 7 : 0];
    // the lane's choices: i OUT .. i OUT + OUT - 1
    float xj[OUT];
    int mine[OUT];
    auto take = [&]() {
#pragma unroll
      for (int jj = 0; jj < OUT; ++jj) {
        int c = best[jj];
#pragma unroll
        for (int g = 1; g < G; ++g)
          if (i == g) c = best[g * OUT + jj];
        mine[jj] = 255 - (c & 255);
        xj[jj] = NEG_INF;
        if (i * OUT + jj < p.k && mine[jj] < p.E) xj[jj] = Quad<X>::one(row[mine[jj]]);
      }
    };
    take();
    int after = ninth, least = INT_MAX;  // the key after the k-th, the closest two of the k + 1
#pragma unroll
    for (int j = KT - 1; j >= 1; --j)
      if (j >= p.k) after = best[j];
#pragma unroll
    for (int j = 1; j < KT; ++j)
      if (j < p.k) least = min(least, best[j - 1] - best[j]);
    int last = best[0];
#pragma unroll
    for (int j = 1; j < KT; ++j)
      if (j < p.k) last = best[j];
    least = min(least, last - after);
    bad = bad || last < 256 || (best[0] >> 8) >= 8388607;
    // all leading keys positive logits that their n hold exactly: the ids order equal ones
    const bool sure = EB == 2 && !SCORES && after > (4194304 + 1024) * 256 + 255;
    if (__any_sync(FULL, !sure && least < 256 * (near + 1))) {
      // neighbours that their keys do not settle stand by their own values.  In a run of
      // them the first two may change places, and every later pair has to be in order
      // as it is, which makes the run sorted; other runs, and those that reach the end
      // of the list (a further expert may be as near), are left to the exact path
      auto value = [&](int e) {
        const float x = live_logit(Quad<X>::one(row[e]));
        if (!SCORES || x == NEG_INF) return x;
        return (KIND == BY_SOFTMAX ? ex2_approx(fmaf(x, LOG2E, -mm)) * rs : sigmoid(x)) + p.bias[(size_t)l * p.E + e];
      };
      // with one bias for all: the choices whose 16-bit logit's neighbours have scores 8
      // steps and more from its own, so that keys as near as an open pair's belong to
      // equal logits (a zero bias, 26 x 20,000 rows of 256 bf16 in groups: 198 us, 425
      // without this, for the last choice and the one after it are often equal)
      unsigned alone = 0u;
      if constexpr (SCORES && EB == 2) {
        if (even_bias) {
#pragma unroll
          for (int jj = 0; jj < OUT; ++jj) {
            const float x = xj[jj], next = fabsf(x) * (std::is_same<X, __half>::value ? 1.f / 4096.f : 1.f / 512.f);
            const float slope = KIND == BY_SOFTMAX ? ex2_approx(fmaf(x, LOG2E, -mm)) * rs : sigmoid_slope(x);
            if (slope * next > 8.f * 4.f / 8388607.f) alone |= 1u << (i * OUT + jj);
          }
#pragma unroll
          for (int o = 1; o < G; o *= 2) alone |= __shfl_xor_sync(FULL, alone, o);
        }
      }
      bool before = false;  // the pair before was open
#pragma unroll
      for (int j = 1; j <= KT; ++j) {
        const int hi = best[j - 1], lo = j < KT ? best[j < KT ? j : 0] : ninth;
        bool open = (j <= p.k || before) && (hi >> 8) - (lo >> 8) <= near && (SCORES || !exact_n<EB>(lo >> 8));
        if (SCORES && EB == 2 && (alone >> (j - 1) & 1u) != 0u) open = false;
        if (open && j == KT) bad = true;
        if (j < KT && open) {
          const int e = 255 - (hi & 255), f = 255 - (lo & 255);
          if (max(e, f) < p.E) {
            const float u = value(e), v = value(f);
            if (v > u || (v == u && f < e)) {
              if (before) bad = true;
              best[j - 1] = lo, best[j < KT ? j : 0] = hi;
            }
          }
        }
        before = open;
      }
      take();
    }
    // rows that are not settled, one by one
    float m = KIND < BY_GROUP ? __shfl_sync(FULL, xj[0], rl * G) : 0.f;  // the first choice is the largest logit
    if (LISTS && columns) {
      if (soft) {  // the largest logit may lie in a group that is dropped
        m = NEG_INF;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          Raw<EB> again;
          fetch(again, b, row, NEG_INF);
          float x[8];
          again.template get<X>(x);
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, x[j]);
        }
        m = row_max<G>(m);
        bad = bad || !(fabsf(m) < 128.f);
      }
    }
    if (columns && i == 0) row_mr[warp][rl] = make_float2(m, 0.f);
    unsigned todo = __ballot_sync(FULL, bad && live && i == 0);
    const bool careful = todo != 0u;
    while (todo != 0u) {
      const int f = (__ffs(todo) - 1) / G;
      todo &= todo - 1;
      float bias[4 * NQ];
#pragma unroll
      for (int q = 0; q < 4 * NQ; ++q) {
        const int e = 4 * (lane + 32 * (q / 4)) + q % 4;
        bias[q] = SCORES && e < p.E ? p.bias[(size_t)l * p.E + e] : 0.f;
      }
      __syncwarp();
      const int64_t at = ((int64_t)l * p.T + t0 + f) * p.k;
      const float rm = score_row<X, NQ>(p, base + (t0 + f) * p.ld_token, bias, p.topk + at,
                                        p.weights != nullptr ? p.weights + at : nullptr, lane);
      if (columns && lane == 0) row_mr[warp][f].x = rm;
    }
    const int rows = (int)min64(RW, t1 - t0);
    float rz = 1.f;
    if (columns) {
      __syncwarp();
      const int col = lane % CL, e = 8 * col;
      const X* at = base + t0 * p.ld_token + e;
#pragma unroll 1
      for (int s = 0; s < 8; ++s) {
        const int r = s * (4 / G) + lane / CL;
        float x[8];
        Raw<EB> line;
        if constexpr (WHOLE && CL == NB * G)
          line.template load<X>(at + (int64_t)min(r, rows - 1) * p.ld_token, 8, true);
        else
          line.template load<X>(at + (int64_t)min(r, rows - 1) * p.ld_token, p.E - e, p.wide != 0);
        line.template get<X>(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaxf(x[j], NEG_INF);  // NaN -> -inf
        if (soft) {
          const float mr = row_mr[warp][r].x, mm = mr * LOG2E;
          float z = 0.f;
          if (careful) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = exp_below(x[j], mr);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = ex2_approx(fmaf(x[j], LOG2E, -mm));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) z += x[j];
          z = row_sum<CL>(z);
          const float rr = z > 0.f ? rcp_approx(z) : 0.f;
          if (col == 0) row_mr[warp][r].y = rr;
          if (sums && r < rows)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(x[j], rr, acc[j]);
        } else if (r < rows) {
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += rcp_approx(1.f + ex2_approx(-LOG2E * x[j]));
        }
      }
      __syncwarp();
      if (soft) rz = row_mr[warp][rl].y;
    }
    // ids and weights of the settled rows (their k-th key is above 0: the chosen
    // logits are numbers, or +inf only where the first key is out of range)
    const int64_t out = ((int64_t)l * p.T + t0 + rl) * p.k + i * OUT;
    const bool write = live && !bad;
    const int own = p.k - i * OUT;  // choices of this lane, where below OUT
    float w[OUT];
    if (p.weights != nullptr) {
      if (soft) {
        float mk = m;  // without groups and biases the row's largest logit is the first choice
        if (LISTS && p.renorm) {
          mk = xj[0];
#pragma unroll
          for (int jj = 1; jj < OUT; ++jj) mk = fmaxf(mk, xj[jj]);
          mk = row_max<G>(mk);
        }
        // the form that the row's sum was made with, for either carries the rounding of its
        // own reference; biases may choose logits so low that only the difference is finite
        if (p.renorm || careful) {
#pragma unroll
          for (int jj = 0; jj < OUT; ++jj) w[jj] = ex2_approx(LOG2E * (xj[jj] - mk));
        } else {
          const float mkl = mk * LOG2E;
#pragma unroll
          for (int jj = 0; jj < OUT; ++jj) w[jj] = ex2_approx(fmaf(xj[jj], LOG2E, -mkl));
        }
      } else {
        // expf: a product with log2 e is rounded, which is 2.6e-6 of the score at -85
        // (asking for such logits first and using ex2 for the others took prefill's registers: 283 -> 295 us)
#pragma unroll
        for (int jj = 0; jj < OUT; ++jj) w[jj] = sigmoid(xj[jj]);
      }
      float f = soft ? rz : 1.f;
      if (p.renorm) {
        float z = 0.f;
#pragma unroll
        for (int jj = 0; jj < OUT; ++jj) z += w[jj];
        z = row_sum<G>(z);
        f = z > 0.f ? rcp_approx(z) : 0.f;
      }
      // the scale last: with 1 / sum of tiny scores it may pass the range
#pragma unroll
      for (int jj = 0; jj < OUT; ++jj) w[jj] = w[jj] * f * p.scale;
      if (write) put_weights<OUT>(p.weights + out, own, p.even, w);
    }
    if (write) put_ids<OUT>(p.topk + out, own, p.even, mine);
    row = next;
  }
  if (sums) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float v = acc[q];
#pragma unroll
      for (int o = CL; o < 32; o *= 2) v += __shfl_xor_sync(FULL, v, o);
      if (lane < CL) part[warp][8 * lane + q] = v;
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

template <typename X, int G, int NB, int KT, bool WHOLE>
cudaError_t score_fast_shape(const ScoreParams& p, cudaStream_t st) {
  const dim3 grid(p.L * p.nspan), block(SF_WARPS * 32);
  switch (score_kind(p.bias != nullptr, p.n_group, p.partial != nullptr, p.score == MOER_SCORE_SOFTMAX,
                     p.renorm != 0)) {
    case BY_LOGIT: return launch_pdl(score_fast_kernel<X, G, NB, KT, BY_LOGIT, WHOLE, false>, grid, block, 0, st, p);
    case SOFTMAX_SUMS: return launch_pdl(score_fast_kernel<X, G, NB, KT, SOFTMAX_SUMS, WHOLE, false>, grid, block, 0, st, p);
    case SIGMOID_SUMS: return launch_pdl(score_fast_kernel<X, G, NB, KT, SIGMOID_SUMS, WHOLE, false>, grid, block, 0, st, p);
    case BY_GROUP: return launch_pdl(score_fast_kernel<X, G, NB, KT, BY_GROUP, WHOLE, false>, grid, block, 0, st, p);
    case BY_SIGMOID: return launch_pdl(score_fast_kernel<X, G, NB, KT, BY_SIGMOID, WHOLE, false>, grid, block, 0, st, p);
    default: return launch_pdl(score_fast_kernel<X, G, NB, KT, BY_SOFTMAX, WHOLE, false>, grid, block, 0, st, p);
  }
}

// Groups that are no blocks of 8 on every lane.
template <typename X, int G>
cudaError_t score_fast_split(const ScoreParams& p, cudaStream_t st) {
  const dim3 grid(p.L * p.nspan), block(SF_WARPS * 32);
  switch (score_kind(p.bias != nullptr, p.n_group, false, p.score == MOER_SCORE_SOFTMAX, p.renorm != 0)) {
    case BY_GROUP: return launch_pdl(score_fast_kernel<X, G, 8, 8, BY_GROUP, false, true>, grid, block, 0, st, p);
    case BY_SIGMOID: return launch_pdl(score_fast_kernel<X, G, 8, 8, BY_SIGMOID, false, true>, grid, block, 0, st, p);
    default: return launch_pdl(score_fast_kernel<X, G, 8, 8, BY_SOFTMAX, false, true>, grid, block, 0, st, p);
  }
}

// The lanes of a row and the blocks of a lane by the experts alone.
template <typename X>
cudaError_t score_fast_run(const ScoreParams& p, cudaStream_t st) {
  const int nb = (p.E + 7) / 8, lanes = p.E <= 64 ? 1 : p.E <= 128 ? 2 : 4;
  const int gs = p.E / p.n_group, per = gs / (8 * lanes);
  if (p.n_group > 1 && (gs % (8 * lanes) != 0 || (per & (per - 1)) != 0))
    return lanes == 1   ? score_fast_split<X, 1>(p, st)
           : lanes == 2 ? score_fast_split<X, 2>(p, st)
                        : score_fast_split<X, 4>(p, st);
  if (p.wide != 0) {
    if (p.E == 64) return score_fast_shape<X, 1, 8, 8, true>(p, st);
    if (p.E == 128) return score_fast_shape<X, 2, 8, 8, true>(p, st);
    if (p.E == 256) return score_fast_shape<X, 4, 8, 8, true>(p, st);
  }
  if (p.E <= 32) return score_fast_shape<X, 1, 4, 8, false>(p, st);
  if (p.E <= 64) return score_fast_shape<X, 1, 8, 8, false>(p, st);
  if (nb <= 12) return score_fast_shape<X, 2, 6, 8, false>(p, st);
  if (nb <= 16) return score_fast_shape<X, 2, 8, 8, false>(p, st);
  if (nb <= 24) return score_fast_shape<X, 4, 6, 8, false>(p, st);
  return score_fast_shape<X, 4, 8, 8, false>(p, st);
}

// k = 9 .. 16.
template <typename X>
cudaError_t score_fast16_run(const ScoreParams& p, cudaStream_t st) {
  if (p.E <= 64) return score_fast_shape<X, 1, 8, 16, false>(p, st);
  if (p.E <= 128) return score_fast_shape<X, 2, 8, 16, false>(p, st);
  return score_fast_shape<X, 4, 8, 16, false>(p, st);
}

}  // namespace moer
