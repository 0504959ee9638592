// score_topk.cu -- moer_score_topk: scores, choice and weights of the router.
//
// Batches of two or three thousand rows with k <= 16 go to the fast kernel
// (score_fast.cuh).  The kernel here takes any E <= 256 with E % 4 == 0, any
// k <= 32, options and alignment, and is the faster one for few rows: one warp
// per row, a lane with the quads of neighbouring experts 4 (lane + 32 i).  The
// choice goes by the fast kernel's keys, a fixed-point number above 255 - id:
// a lane sorts its own, and k + 1 rounds of a warp maximum over the lanes' first
// keys take them in order.  Rows that the keys do not settle (see score_fast.cuh)
// are redone with exact keys (score_row.cuh).
// Measured: 32 tokens of 128 fp32 experts, k = 8, 2.4 us on the GPU (launch and
// latency: one row a warp), 5.1 us a call from Python; 16,150 x 16 rows of 160 fp32
// experts, k = 10, sigmoid with bias and score sums: 213 us (0.84 TB/s), bound by
// the k + 1 dependent rounds.
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
cudaError_t score_fast16_f32(const ScoreParams& p, cudaStream_t st);  // k = 9 .. 16
cudaError_t score_fast16_bf16(const ScoreParams& p, cudaStream_t st);
cudaError_t score_fast16_f16(const ScoreParams& p, cudaStream_t st);

namespace {
constexpr int SC_WARPS = 8;
constexpr int SC_UNITS = 4864;  // units asked for: 152 SMs x 32

constexpr int64_t SC_FAST_ROWS = 2048;    // rows from which the fast kernel is taken,
constexpr int64_t SC_FAST16_ROWS = 2816;  // and with k > 8

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
  const int64_t each = (int64_t)most * step;  // tokens of a round of all units: with fewer rounds there are too many
  for (int64_t rounds = (T + each - 1) / each; rounds <= 64 || best < 0; ++rounds) {
    const int64_t units = (T + rounds * step - 1) / (rounds * step);
    const int64_t c = (units * L + slots - 1) / slots * (rounds + 1);
    if (best < 0 || c < cost) best = rounds, cost = c;
    if (units == 1) break;
  }
  return (int)(best * step);
}

// The fast kernel's options (score_fast.cuh): k <= 16, aligned quads, and groups,
// where there are any, that make at most eight blocks of a lane (k > 8: whole ones).
// Few rows leave it idle lanes: at 1,024 / 2,048 / 4,096 rows it took 2.6 / 2.6 / 4.2 us
// (a warp per row: 3.2 / 3.3 / 5.2) with E = 128 fp32, 4.3 / 4.3 / 4.3 (4.5 / 5.6 / 9.7)
// with 256 bf16 experts in groups, 5.3 / 5.6 / 5.3 (4.1 / 5.3 / 8.9) with 64 bf16
// experts and score sums.  With k > 8, at 2,048 / 2,816 / 4,096 rows: 4.0 / 4.0 / 4.1 us
// (a warp per row: 3.7 / 4.2 / 4.8) with E = 128 fp32, k = 10, 6.1 / 6.2 / 6.1 (5.9 / 7.7 /
// 10.3) with 256 bf16 experts in groups, k = 16, 7.7 / 7.6 / 7.5 (5.7 / 7.3 / 9.2) with 64 bf16
// experts and sums, k = 12, 8.7 / 9.3 / 8.9 (6.9 / 8.9 / 11.3) with 160 fp32 ones, bias and
// sums, k = 10.  With k = 10, 48 x 42,076 rows of 72 fp32 experts and score
// sums took 1,072 us a warp per row, about 445 here (k = 9 and 16: 443 and 454).
bool fast_supported(const ScoreParams& p) {
  if (p.k > 16 || p.vec == 0 || p.E < 16 || p.L * p.T < (p.k > 8 ? SC_FAST16_ROWS : SC_FAST_ROWS)) return false;
  if (p.n_group == 1) return true;
  const int lanes = p.E <= 64 ? 1 : p.E <= 128 ? 2 : 4, gs = p.E / p.n_group;
  int mb = 1;  // blocks of a lane to a group
  while (mb * 8 * lanes < group_span(gs)) mb *= 2;
  if (p.k > 8 && (gs % (8 * lanes) != 0 || mb * 8 * lanes != gs)) return false;
  return p.n_group * mb <= 8;
}

// Sorts four keys in descending order.
__device__ __forceinline__ void sort4_desc(int (&c)[4]) {
  cas(c[0], c[2]); cas(c[1], c[3]);
  cas(c[0], c[1]); cas(c[2], c[3]);
  cas(c[1], c[2]);
}

// One row by one warp.  group: the lane's experts' groups; best, second: room for
// 32 keys each in shared memory (with groups).
// x: the lane's logits, -inf past the row's end.
template <typename X, int NQ>
__device__ void row_by_keys(const ScoreParams& p, const X* row, float (&x)[4 * NQ], const float (&bias)[4 * NQ],
                            const int (&group)[4 * NQ], int* best, int* second, int64_t out, int l, int lane,
                            float (&sum)[4 * NQ]) {
  constexpr int EB = sizeof(X);
  const bool soft = p.score == MOER_SCORE_SOFTMAX;
  const bool use_s = p.bias != nullptr || (p.n_group > 1 && p.group_best == 2);  // the choice takes scores
  const bool dense = p.partial != nullptr || use_s || (soft && !p.renorm);
  const int near = use_s ? 2 : 0;
  int key[4 * NQ];
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) x[i] = live_logit(x[i]);
  float m = NEG_INF, rz = 0.f;
  if (dense) {
    float s[4 * NQ];
    if (soft) {
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) m = fmaxf(m, x[i]);
      m = warp_max(m);
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) {
        s[i] = x[i] == m ? 1.f : ex2_approx(LOG2E * (x[i] - m));  // equal infinities share
        if (x[i] == NEG_INF) s[i] = 0.f;
        z += s[i];
      }
      z = warp_sum(z);
      rz = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) s[i] *= rz;
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i) s[i] = rcp_approx(1.f + ex2_approx(-LOG2E * x[i]));
    }
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) {
      sum[i] += s[i];
      if (use_s) key[i] = (int)(__float_as_uint(fmaf(fma_sat(s[i] + bias[i], 0.25f, 0.25f), 8388607.f, 8388608.f)) << 8);
    }
  }
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) {
    const int e = 4 * (lane + 32 * (i / 4)) + i % 4;
    if (!use_s) key[i] = (int)(__float_as_uint(fmaf(fma_sat(x[i], 1.f / 256.f, 0.5f), 8388607.f, 8388608.f)) << 8);
    if (x[i] == NEG_INF) key[i] = 0;  // masked experts stay out whatever their bias
    key[i] = e < p.E ? key[i] | (255 - e) : -1;
  }
  bool bad = false;
  if (p.n_group > 1) {
    best[lane] = second[lane] = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i)
      if (key[i] >= 0) atomicMax(&best[group[i]], key[i]);
    __syncwarp();
    if (p.group_best == 2) {
#pragma unroll
      for (int i = 0; i < 4 * NQ; ++i)
        if (key[i] >= 0 && key[i] != best[group[i]]) atomicMax(&second[group[i]], key[i]);
      __syncwarp();
    }
    const int n2 = second[lane] >> 8;
    const bool real = lane < p.n_group;
    // the second best counts only where there are two numbers to add, and the best one
    // only within the keys' range: a sum with one past it is too small
    if (real && p.group_best == 2 && (n2 <= 0 || best[lane] >> 8 >= 8388607)) bad = true;
    const int gk = real ? ((best[lane] >> 8) + (p.group_best == 2 ? n2 : 0)) * 32 + (31 - lane) : -1;
    int above = 0;
    for (int g = 0; g < p.n_group; ++g) above += __shfl_sync(FULL, gk, g) > gk ? 1 : 0;
    const bool kept = real && above < p.top_group;
    const unsigned keep = __ballot_sync(FULL, kept);
    const int thr = __reduce_min_sync(FULL, kept ? gk : INT_MAX) >> 5;
    const int nxt = __reduce_max_sync(FULL, kept ? -1 : gk) >> 5;
    if (thr - nxt <= 3 * near && (use_s || !exact_n<EB>(thr))) bad = true;
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i)
      if (!((keep >> group[i]) & 1u)) key[i] = -1;
    __syncwarp();
  }
  if constexpr (NQ == 1)
    sort4_desc(key);
  else
    sort8_desc(key);
  // lane r < k holds the r-th key, lane k (or all, if k is 32) the one after
  int mine = INT_MIN, after = INT_MIN;
  for (int r = 0; r <= p.k; ++r) {
    const int top = __reduce_max_sync(FULL, key[0]);
    if (r == p.k) after = top;
    if (lane == r) mine = top;
    if (key[0] == top) {  // keys differ: one lane (or only empty ones are left)
#pragma unroll
      for (int i = 0; i + 1 < 4 * NQ; ++i) key[i] = key[i + 1];
      key[4 * NQ - 1] = -1;
    }
  }
  const bool on = lane < p.k;
  const int id = 255 - (mine & 255);
  const float xj = on && mine >= 0 && id < p.E ? live_logit(Quad<X>::one(row[id])) : NEG_INF;
  const float bj = on && p.bias != nullptr && mine >= 0 ? p.bias[(size_t)l * p.E + id] : 0.f;
  int next = __shfl_down_sync(FULL, mine, 1);
  if (lane == p.k - 1) next = after;
  const float xn = __shfl_down_sync(FULL, xj, 1), bn = __shfl_down_sync(FULL, bj, 1);
  if (on) {
    const bool open = (mine >> 8) - (next >> 8) <= near && (use_s || !exact_n<EB>(mine >> 8));
    bad = bad || mine < 256 || (mine >> 8) >= 8388607;
    bad = bad || (open && (lane == p.k - 1 ? next >= 0 : !(xj == xn && bj == bn)));
  }
  if (__any_sync(FULL, bad)) {
    score_row<X, NQ>(p, row, bias, p.topk + out * p.k, p.weights != nullptr ? p.weights + out * p.k : nullptr, lane);
    return;
  }
  if (on) p.topk[out * p.k + lane] = (uint8_t)id;
  if (p.weights != nullptr) {
    float w = 0.f;
    if (soft)
      w = exp_below(xj, p.renorm ? warp_max(xj) : m) * (p.renorm ? 1.f : rz);
    else if (on)
      w = sigmoid(xj);
    if (p.renorm) {
      const float z = warp_sum(w);
      w = z > 0.f ? w / z : 0.f;
    }
    if (on) p.weights[out * p.k + lane] = p.scale * w;
  }
}

template <typename X, int NQ>
__global__ void __launch_bounds__(SC_WARPS * 32, 3) score_topk_kernel(const ScoreParams p) {
  __shared__ float part[SC_WARPS][128 * NQ];
  __shared__ int group_key[SC_WARPS][2][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = blockIdx.x / p.nspan, u = blockIdx.x - l * p.nspan;
  float bias[4 * NQ], sum[4 * NQ];
  int group[4 * NQ];
  const int gs = p.E / p.n_group;
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) {
    const int e = 4 * (lane + 32 * (i / 4)) + i % 4;
    group[i] = p.n_group > 1 ? min(e / gs, 31) : 0;
    bias[i] = p.bias != nullptr && e < p.E ? p.bias[(size_t)l * p.E + e] : 0.f;
    sum[i] = 0.f;
  }
  const int64_t t1 = min64(p.T, (int64_t)(u + 1) * p.span);
  int64_t t = (int64_t)u * p.span + warp;
  const X* row = static_cast<const X*>(p.logits) + l * p.ld_layer + t * p.ld_token;
  float x[4 * NQ], ahead[4 * NQ];  // the row's logits, and those of the warp's next one
  auto fetch = [&](const X* of, float (&to)[4 * NQ]) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int e = 4 * (lane + 32 * q);
      float v[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
      if (e < p.E) load4<X>(of + e, p.vec != 0, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) to[4 * q + j] = v[j];
    }
  };
  if (t < t1) fetch(row, x);
  for (; t < t1; t += SC_WARPS) {
    const X* next = row + SC_WARPS * p.ld_token;
    if (t + SC_WARPS < t1) fetch(next, ahead);
    row_by_keys<X, NQ>(p, row, x, bias, group, group_key[warp][0], group_key[warp][1], (int64_t)l * p.T + t, l, lane,
                       sum);
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) x[i] = ahead[i];
    row = next;
  }
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

// The general kernel's units are the more numerous.  Their number falls where the span steps;
// the size is a bound of it that grows with T (a span is SC_WARPS and T L / SC_UNITS
// tokens at least), so that a workspace for a batch serves every smaller one.
size_t score_scratch_bytes(const moer_dims* d, int64_t T) {
  const int64_t units = min64((T + SC_WARPS - 1) / SC_WARPS, (SC_UNITS + d->L - 1) / d->L);
  return (size_t)d->L * (size_t)units * (size_t)d->E * 4;
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
    const int kind = score_kind(p.bias != nullptr, p.n_group, score_sum != nullptr, p.score == MOER_SCORE_SOFTMAX, p.renorm != 0);
    p.span = fast_span(p.T, p.L, p.E <= 64 ? 128 : p.E <= 128 ? 64 : 32,
                       (int64_t)sms * score_resident(dtype == MOER_F32 ? 4 : 2, kind, p.k));
  } else {
    p.span = score_span(p.T, p.L, SC_WARPS);
  }
  p.nspan = score_nspan(p.T, p.span);
  p.partial = score_sum != nullptr ? reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEADER) : nullptr;
  p.key_mul = 256u;
  const uintptr_t w = reinterpret_cast<uintptr_t>(p.weights);
  p.even = p.k == 8 && w % 16 == 0 ? 2 : p.k % 2 == 0 && w % 8 == 0 ? 1 : 0;
  cudaError_t e;
  if (fast && p.k <= 8)
    e = dtype == MOER_F32 ? score_fast_f32(p, st) : dtype == MOER_BF16 ? score_fast_bf16(p, st) : score_fast_f16(p, st);
  else if (fast)
    e = dtype == MOER_F32    ? score_fast16_f32(p, st)
        : dtype == MOER_BF16 ? score_fast16_bf16(p, st)
                             : score_fast16_f16(p, st);
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
