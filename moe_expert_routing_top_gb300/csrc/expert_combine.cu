// expert_combine.cu -- moer_expert_combine and its gradient: the experts' rows weighted and summed
// per token.
//
// Forward: a warp takes 256 columns of a token and has its k rows' loads in flight at once.
// Gradient: a warp takes a token, so that the k dot products stay in its lanes; rows that no pair
// takes (padding, dropped pairs) are zeroed by further blocks of the same launch.  Bound by DRAM: 6.3 TB/s forward
// (32,768 tokens of 8 rows of 2,048 bf16: 213 us with four blocks an SM, 244 with fewer), 5.1 in the gradient.
#include "rows.cuh"

namespace moer {

constexpr int COMB_THREADS = 256;
constexpr int COMB_WARPS = COMB_THREADS / 32;
constexpr int COMB_STEP = 256;  // columns a warp takes at once
constexpr int COMB_K = 8;       // rows in flight

// The row of a pair, or -1; a row past the buffer records MOER_EDATA.
__device__ __forceinline__ int pair_row(const moer_expert_combine_args& a, int64_t pair, uint32_t* status) {
  const int r = a.inv[pair];
  if (r >= a.rows) {
    atomicOr(status, WS_BIT_EDATA);
    return -1;
  }
  return r;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(COMB_THREADS, 4) combine_kernel(const __grid_constant__ moer_expert_combine_args a, int nc,
                                                               uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * COMB_WARPS + (threadIdx.x >> 5);
  const int64_t t = u / nc;
  if (t >= a.T) return;
  const int col = (int)(u % nc) * COMB_STEP + lane * 8, n = a.H - col;
  // lane j holds pair j's row and weight
  int row = -1;
  float wt = 1.f;
  if (lane < a.k) {
    row = pair_row(a, t * a.k + lane, status);
    if (a.weights != nullptr) wt = a.weights[t * a.k + lane];
  }
  float s[8];
  {
    Raw8<T> v = load8_rw<T, VEC>(static_cast<const T*>(a.add) + t * a.ld_add + col, a.add != nullptr ? n : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = to_f32(v.v[i]);
  }
  for (int j0 = 0; j0 < a.k; j0 += COMB_K) {
    Raw8<T> v[COMB_K];
    float w[COMB_K];
    int r[COMB_K];
#pragma unroll
    for (int j = 0; j < COMB_K; ++j) {
      r[j] = __shfl_sync(FULL, row, (j0 + j) & 31);
      w[j] = __shfl_sync(FULL, wt, (j0 + j) & 31);
      if (j0 + j >= a.k) r[j] = -1;
      v[j] = load8<T, VEC>(static_cast<const T*>(a.z) + (int64_t)r[j] * a.ld_z + col, r[j] >= 0 ? n : 0);
    }
#pragma unroll
    for (int j = 0; j < COMB_K; ++j)
      if (r[j] >= 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = fmaf(w[j], to_f32(v[j].v[i]), s[i]);
      }
  }
  store8<T, VEC>(static_cast<T*>(a.out) + t * a.ld_out + col, pack8<T>(s), n);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(COMB_THREADS) combine_grad_kernel(const __grid_constant__ moer_expert_combine_args a,
                                                                    unsigned token_blocks, uint32_t* status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= token_blocks) {  // rows that no pair takes: a warp looks at 32 rows' entries at once
    const int64_t nw = (int64_t)(gridDim.x - token_blocks) * COMB_WARPS, pairs = a.T * a.k;
    bool bad = false;
    for (int64_t p0 = ((int64_t)(blockIdx.x - token_blocks) * COMB_WARPS + warp) * 32; p0 < a.rows; p0 += nw * 32) {
      bool none = false;
      if (p0 + lane < a.rows) {
        const int o = a.order[p0 + lane];
        none = o < 0 || o >= pairs;
        bad |= o >= pairs;
        if (!none) {
          const int r = a.inv[o];
          none = r < 0 || r >= a.rows;  // (the latter is said by its token's warp)
          bad |= !none && r != p0 + lane;
        }
      }
      unsigned pad = __ballot_sync(FULL, none);
      for (; pad != 0; pad &= pad - 1) {
        T* o = static_cast<T*>(a.d_z) + (p0 + __ffs(pad) - 1) * a.ld_d_z;
        Raw8<T> zero;
#pragma unroll
        for (int i = 0; i < 8; ++i) zero.v[i] = from_f32<T>(0.f);
        for (int col = lane * 8; col < a.H; col += COMB_STEP) store8<T, VEC>(o + col, zero, a.H - col);
      }
    }
    if (bad) atomicOr(status, WS_BIT_EDATA);
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * COMB_WARPS + warp;
  if (t >= a.T) return;
  int row = -1;
  float wt = 1.f;
  bool owner = false;  // the pair's row is its own: no other pair writes it
  if (lane < a.k) {
    const int64_t pair = t * a.k + lane;
    row = pair_row(a, pair, status);
    if (a.weights != nullptr) wt = a.weights[pair];
    if (row >= 0 && a.d_z != nullptr) {
      owner = a.order[row] == pair;
      if (!owner) atomicOr(status, WS_BIT_EDATA);
    }
  }
  const unsigned owners = __ballot_sync(FULL, owner);
  for (int j0 = 0; j0 < a.k; j0 += COMB_K) {
    float dot[COMB_K], w[COMB_K];
    int r[COMB_K];
#pragma unroll
    for (int j = 0; j < COMB_K; ++j) {
      dot[j] = 0.f;
      r[j] = __shfl_sync(FULL, row, (j0 + j) & 31);
      w[j] = __shfl_sync(FULL, wt, (j0 + j) & 31);
      if (j0 + j >= a.k) r[j] = -1;
    }
    for (int col = lane * 8; col < a.H; col += COMB_STEP) {
      const int n = a.H - col;
      const Raw8<T> dv = load8<T, VEC>(static_cast<const T*>(a.d_out) + t * a.ld_d_out + col, n);
      Raw8<T> v[COMB_K];
      if (a.d_weights != nullptr) {
#pragma unroll
        for (int j = 0; j < COMB_K; ++j)
          v[j] = load8<T, VEC>(static_cast<const T*>(a.z) + (int64_t)r[j] * a.ld_z + col, r[j] >= 0 ? n : 0);
      }
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = to_f32(dv.v[i]);
#pragma unroll
      for (int j = 0; j < COMB_K; ++j) {
        if (r[j] < 0) continue;
        if (a.d_weights != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], to_f32(v[j].v[i]), dot[j]);
        }
        if ((owners >> ((j0 + j) & 31)) & 1u) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = w[j] * d[i];
          store8<T, VEC>(static_cast<T*>(a.d_z) + (int64_t)r[j] * a.ld_d_z + col, pack8<T>(o), n);
        }
      }
    }
    if (a.d_weights != nullptr) {
#pragma unroll
      for (int j = 0; j < COMB_K; ++j) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) dot[j] += __shfl_xor_sync(FULL, dot[j], d);
        if (lane == 0 && j0 + j < a.k) a.d_weights[t * a.k + j0 + j] = dot[j];
      }
    }
  }
}

namespace {
bool comb_vec(const moer_expert_combine_args* a, bool grad, int eb) {
  const void* const p[] = {a->z, grad ? nullptr : a->add, grad ? nullptr : a->out, grad ? a->d_out : nullptr, grad ? a->d_z : nullptr};
  const int64_t ld[] = {a->ld_z, a->ld_add, a->ld_out, a->ld_d_out, a->ld_d_z};
  if (a->H % 8 != 0) return false;
  for (int i = 0; i < 5; ++i)
    if (p[i] != nullptr && (reinterpret_cast<uintptr_t>(p[i]) % 16 != 0 || ld[i] * eb % 16 != 0)) return false;
  return true;
}

template <typename T>
cudaError_t comb_run(const moer_expert_combine_args* a, bool grad, uint32_t* status, int sms, cudaStream_t st) {
  const bool vec = comb_vec(a, grad, sizeof(T));
  if (!grad) {
    const int nc = (a->H + COMB_STEP - 1) / COMB_STEP;
    const unsigned grid = (unsigned)((a->T * nc + COMB_WARPS - 1) / COMB_WARPS);
    if (vec) combine_kernel<T, true><<<grid, COMB_THREADS, 0, st>>>(*a, nc, status);
    else combine_kernel<T, false><<<grid, COMB_THREADS, 0, st>>>(*a, nc, status);
  } else {
    const unsigned tb = (unsigned)((a->T + COMB_WARPS - 1) / COMB_WARPS);
    const unsigned pb = a->d_z != nullptr ? (unsigned)min64((a->rows + 32 * COMB_WARPS - 1) / (32 * COMB_WARPS), 8 * sms) : 0;
    if (tb + pb == 0) return cudaSuccess;
    if (vec) combine_grad_kernel<T, true><<<tb + pb, COMB_THREADS, 0, st>>>(*a, tb, status);
    else combine_grad_kernel<T, false><<<tb + pb, COMB_THREADS, 0, st>>>(*a, tb, status);
  }
  return cudaGetLastError();
}
}  // namespace

moer_status expert_combine_launch(const moer_expert_combine_args* a, bool grad, void* ws, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms <= 0) return MOER_ECUDA;
  uint32_t* status = static_cast<uint32_t*>(ws);
  const cudaError_t e = a->dtype == MOER_F32    ? comb_run<float>(a, grad, status, sms, st)
                        : a->dtype == MOER_BF16 ? comb_run<__nv_bfloat16>(a, grad, status, sms, st)
                                                : comb_run<__half>(a, grad, status, sms, st);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
