// norm.cu -- moer_rms_norm and its gradient: y = s * rstd * weight with s = x + residual, rounded
// to 16 bits and/or to e4m3 with a scale for each block of 128 columns.
//
// A row lies with W warps, eight columns a lane and step, at most four steps (gradient: two), and stays
// in registers between the sum of squares and the outputs: each input is read once.  Bound by DRAM:
// 65,536 rows of 2,048 bf16 with a residual to 16 and 8 bits in 180 us, 6.7 TB/s (eight steps a warp: 248).
// The gradient of 30,011 rows takes 128 us (3.9 TB/s) and is bound by the latency from a row's loads to
// its stores; four steps a warp 144, eight 228, since fewer blocks then fit an SM.
#include "rows.cuh"

namespace moer {

constexpr int NORM_MAX_THREADS = 512;  // a row of 16,384
constexpr int NORM_STEP = 256;  // columns that a warp takes a step: 32 lanes x 8

// Sum over the W warps of a row (W a power of two), in a fixed order.  Every thread of the block
// takes part when W > 1.
__device__ __forceinline__ float row_sum(float v, int W, float* part) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
  if (W == 1) return v;
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[warp] = v;
  __syncthreads();
  const int w0 = warp / W * W;
  v = 0.f;
  for (int i = 0; i < W; ++i) v += part[w0 + i];
  return v;
}

template <typename T, bool VEC, int NC>
__global__ void __launch_bounds__(NORM_MAX_THREADS) rms_norm_kernel(const __grid_constant__ moer_norm_args a, int W) {
  __shared__ float part[NORM_MAX_THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 32 / W) + warp / W;
  const bool live = row < a.T;
  const int H = live ? a.H : 0, c0 = (warp % W) * NORM_STEP + lane * 8, dc = W * NORM_STEP;
  Raw8<T> s[NC];
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
#pragma unroll
  for (int c = 0; c < NC; ++c) s[c] = load8_rw<T, VEC>(x + c0 + c * dc, H - c0 - c * dc);
  if (a.residual != nullptr) {
    const T* r = static_cast<const T*>(a.residual) + row * a.ld_residual;
    Raw8<T> v[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) v[c] = load8_rw<T, VEC>(r + c0 + c * dc, H - c0 - c * dc);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[c].v[i] = from_f32<T>(to_f32(s[c].v[i]) + to_f32(v[c].v[i]));
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = to_f32(s[c].v[i]);
      ss += f * f;
    }
  if (a.sum != nullptr) {
    T* o = static_cast<T*>(a.sum) + row * a.ld_sum;
#pragma unroll
    for (int c = 0; c < NC; ++c) store8<T, VEC>(o + c0 + c * dc, s[c], H - c0 - c * dc);
  }
  ss = row_sum(ss, W, part);
  const float rstd = 1.f / sqrtf(ss / (float)a.H + a.eps);
  if (a.rstd != nullptr && live && c0 == 0) a.rstd[row] = rstd;
  if (a.y == nullptr && a.q == nullptr) return;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = c0 + c * dc, n = H - col;
    const Raw8<T> g = load8<T, VEC>(static_cast<const T*>(a.weight) + col, n);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = to_f32(s[c].v[i]) * rstd * to_f32(g.v[i]);
    if (a.y != nullptr) store8<T, VEC>(static_cast<T*>(a.y) + row * a.ld_y + col, pack8<T>(y), n);
    if (a.q != nullptr)
      store_e4m3<VEC>(y, static_cast<uint8_t*>(a.q) + row * a.ld_q + col, a.scale + row * a.ld_scale + col / 128, lane, n);
  }
}

// Each group of W warps takes every gridDim.x * (groups a block)-th row and keeps its columns' part
// of the weight's gradient in registers; the block's groups add theirs in order into a row of
// `partial` [gridDim.x][H].
template <typename T, bool VEC, int NC>
__global__ void __launch_bounds__(NORM_MAX_THREADS) rms_norm_grad_kernel(const __grid_constant__ moer_norm_args a, int W,
                                                                     float* __restrict__ partial) {
  extern __shared__ float dsum[];  // [H] with a weight's gradient
  __shared__ float part[NORM_MAX_THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = blockDim.x / 32 / W, g = warp / W;
  const int c0 = (warp % W) * NORM_STEP + lane * 8, dc = W * NORM_STEP;
  float acc[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[c][i] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < a.T; r0 += (int64_t)gridDim.x * groups) {
    const int64_t row = r0 + g;
    const bool live = row < a.T;
    const int H = live ? a.H : 0;
    const T* sp = static_cast<const T*>(a.sum) + row * a.ld_sum;
    const T* dp = static_cast<const T*>(a.d_y) + row * a.ld_d_y;
    Raw8<T> s[NC], d[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) s[c] = load8<T, VEC>(sp + c0 + c * dc, H - c0 - c * dc);
#pragma unroll
    for (int c = 0; c < NC; ++c) d[c] = load8_rw<T, VEC>(dp + c0 + c * dc, H - c0 - c * dc);
    Raw8<T> e[NC];
    if (a.d_sum != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        e[c] = load8_rw<T, VEC>(static_cast<const T*>(a.d_sum) + row * a.ld_d_sum + c0 + c * dc, H - c0 - c * dc);
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const Raw8<T> w = load8<T, VEC>(static_cast<const T*>(a.weight) + c0 + c * dc, H - c0 - c * dc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = to_f32(s[c].v[i]) * rstd, dy = to_f32(d[c].v[i]);
        acc[c][i] += dy * n;
        dot += dy * to_f32(w.v[i]) * n;
      }
    }
    dot = row_sum(dot, W, part) / (float)a.H;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = c0 + c * dc, n = H - col;
      const Raw8<T> w = load8<T, VEC>(static_cast<const T*>(a.weight) + col, n);
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dx[i] = rstd * (to_f32(d[c].v[i]) * to_f32(w.v[i]) - to_f32(s[c].v[i]) * rstd * dot);
      if (a.d_sum != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dx[i] += to_f32(e[c].v[i]);
      }
      store8<T, VEC>(static_cast<T*>(a.d_x) + row * a.ld_d_x + col, pack8<T>(dx), n);
    }
  }
  if (partial == nullptr) return;
  for (int t = 0; t < groups; ++t) {
    if (t == g) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int col = c0 + c * dc + i;
          if (col < a.H) dsum[col] = t == 0 ? acc[c][i] : dsum[col] + acc[c][i];
        }
    }
    __syncthreads();
  }
  for (int col = threadIdx.x; col < a.H; col += blockDim.x) partial[(size_t)blockIdx.x * a.H + col] = dsum[col];
}

// d_weight[h] = the sum over the blocks' rows, in a fixed order: a block takes 32 columns, warp w
// every 32nd row from w on (with eight warps, whose chains of loads are four times as long, the gradient of
// 18,055 rows of 120 took 20 us instead of 18).
constexpr int DW_WARPS = 32;
__global__ void __launch_bounds__(DW_WARPS * 32) norm_dweight_kernel(const float* __restrict__ partial, int nb, int H,
                                                                     float* __restrict__ out) {
  __shared__ float sm[DW_WARPS][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < H) {
#pragma unroll 4
    for (int b = warp; b < nb; b += DW_WARPS) v += partial[(size_t)b * H + col];
  }
  sm[warp][lane] = v;
  __syncthreads();
  // warp w adds up column w: its lanes the warps' sums, in pairs
  v = sm[lane][warp];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
  if (lane == 0 && blockIdx.x * 32 + warp < H) out[blockIdx.x * 32 + warp] = v;
}

namespace {
// Steps of 256 columns a warp, and warps a row: as few as hold it.  The gradient, which also keeps its
// part of the weight's gradient, takes two steps a warp while that leaves 16 warps a row.
int norm_steps(int H, bool grad) { return H <= NORM_STEP ? 1 : grad && H <= 16 * 2 * NORM_STEP ? 2 : 4; }
int norm_warps(int H, bool grad) {
  int W = 1;
  while (W * NORM_STEP * norm_steps(H, grad) < H) W *= 2;
  return W;
}
int norm_threads(int H, bool grad) { return norm_warps(H, grad) * 32 > 256 ? norm_warps(H, grad) * 32 : 256; }

bool row_vec(const moer_norm_args* a, int eb) {
  const void* const p[] = {a->x, a->residual, a->weight, a->sum, a->y, a->d_y, a->d_sum, a->d_x};
  const int64_t ld[] = {a->ld_x, a->ld_residual, 16, a->ld_sum, a->ld_y, a->ld_d_y, a->ld_d_sum, a->ld_d_x};
  if (a->H % 8 != 0) return false;
  for (int i = 0; i < 8; ++i)
    if (p[i] != nullptr && (reinterpret_cast<uintptr_t>(p[i]) % 16 != 0 || ld[i] * eb % 16 != 0)) return false;
  return a->q == nullptr || (reinterpret_cast<uintptr_t>(a->q) % 8 == 0 && a->ld_q % 8 == 0);
}

template <typename T, bool VEC, int NC>
cudaError_t norm_run(const moer_norm_args* a, bool grad, float* partial, int blocks, cudaStream_t st) {
  const int W = norm_warps(a->H, grad), threads = norm_threads(a->H, grad), groups = threads / 32 / W;
  if (!grad) {
    if constexpr (NC == 2) return cudaErrorInvalidValue;  // the gradient's alone
    else rms_norm_kernel<T, VEC, NC><<<(unsigned)((a->T + groups - 1) / groups), threads, 0, st>>>(*a, W);
    return cudaGetLastError();
  }
  const size_t smem = partial != nullptr ? (size_t)a->H * 4 : 0;
  if (smem + sizeof(float) * (NORM_MAX_THREADS / 32) > 48 * 1024) {  // with `part`: what a launch has by default
    static std::atomic<unsigned long long> set{0};
    const cudaError_t e = smem_optin(rms_norm_grad_kernel<T, VEC, NC>, 64 * 1024, set);
    if (e != cudaSuccess) return e;
  }
  rms_norm_grad_kernel<T, VEC, NC><<<blocks, threads, smem, st>>>(*a, W, partial);
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_pick(const moer_norm_args* a, bool grad, float* partial, int blocks, cudaStream_t st) {
  const bool vec = row_vec(a, sizeof(T));
  switch (norm_steps(a->H, grad)) {
    case 1: return vec ? norm_run<T, true, 1>(a, grad, partial, blocks, st) : norm_run<T, false, 1>(a, grad, partial, blocks, st);
    case 2: return vec ? norm_run<T, true, 2>(a, grad, partial, blocks, st) : norm_run<T, false, 2>(a, grad, partial, blocks, st);
    default: return vec ? norm_run<T, true, 4>(a, grad, partial, blocks, st) : norm_run<T, false, 4>(a, grad, partial, blocks, st);
  }
}

cudaError_t norm_any(const moer_norm_args* a, bool grad, float* partial, int blocks, cudaStream_t st) {
  if (a->dtype == MOER_F32) return norm_pick<float>(a, grad, partial, blocks, st);
  if (a->dtype == MOER_BF16) return norm_pick<__nv_bfloat16>(a, grad, partial, blocks, st);
  return norm_pick<__half>(a, grad, partial, blocks, st);
}

constexpr int NORM_GRAD_BLOCKS = 2 * 152;  // most blocks of the gradient (two an SM, what fits at 128 registers), and rows of its partial sums
}  // namespace

size_t rms_norm_scratch_bytes(int32_t H) { return (size_t)NORM_GRAD_BLOCKS * H * 4; }

moer_status rms_norm_launch(const moer_norm_args* a, cudaStream_t st) {
  return norm_any(a, false, nullptr, 0, st) == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

moer_status rms_norm_grad_launch(const moer_norm_args* a, void* scratch, cudaStream_t st) {
  const int groups = norm_threads(a->H, true) / 32 / norm_warps(a->H, true);
  const int blocks = (int)min64((a->T + groups - 1) / groups, NORM_GRAD_BLOCKS);
  float* partial = a->d_weight != nullptr ? static_cast<float*>(scratch) : nullptr;
  if (a->T > 0 && norm_any(a, true, partial, blocks, st) != cudaSuccess) return MOER_ECUDA;
  if (a->d_weight != nullptr) norm_dweight_kernel<<<(a->H + 31) / 32, DW_WARPS * 32, 0, st>>>(partial, a->T > 0 ? blocks : 0, a->H, a->d_weight);
  return cudaGetLastError() == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
