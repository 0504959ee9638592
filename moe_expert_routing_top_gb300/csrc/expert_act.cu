// expert_act.cu -- moer_expert_act and its gradient: y = silu(a) * b over the experts' rows, rounded
// to 16 bits and/or to e4m3 with a scale for each block of 128 columns.
//
// Sixteen lanes take a block of 128 columns, eight each; a half-warp has two blocks' loads in flight.
// Bound by DRAM: 5.8 TB/s to 8 bits, 6.7 in the gradient (four blocks an SM: 201 us, three: 213,
// 96,006 rows of 1,408); rows of fp32 6.6 and 6.5 (246 and 414 us, the same rows).
#include "rows.cuh"

namespace moer {

constexpr int ACT_THREADS = 256;
constexpr int ACT_UNROLL = 2;  // blocks in flight a half-warp (four: 204 us where two took 176, 270,208 rows of 768 to 8 bits)

// Rows of fp32: the exponential to a step, then a rounded sum and division.  Rows of 16 bits: to 2 + 1.2 |a| steps
// of the exponential and two of the division, at |a| = 20 a 500th of the output's rounding in bf16 and
// a 70th in fp16; 0 for an exponential past 2^126, from a = -87.3 on.  (An exact division for them: 352 us where this
// took 213, 270,208 rows of 768 to 8 bits.)
template <typename T>
__device__ __forceinline__ float sigmoid_of(float a) {
  if constexpr (sizeof(T) == 4) return 1.f / (1.f + expf(-a));
  else return __fdividef(1.f, 1.f + __expf(-a));
}

template <typename T, bool VEC, bool GRAD>
__global__ void __launch_bounds__(ACT_THREADS, GRAD ? 4 : 1) expert_act_kernel(const __grid_constant__ moer_expert_act_args a) {
  const int lane = threadIdx.x & 31, half = threadIdx.x >> 4;
  const int nb = (a.I + 127) / 128;
  int64_t rows = a.rows;
  if (a.used != nullptr) rows = min64(rows, max64(*a.used, 0));
  const int64_t units = rows * nb;
  const int64_t step = (int64_t)gridDim.x * (ACT_THREADS / 16);
  const int64_t drow = step / nb;
  const int dblk = (int)(step % nb);
  int64_t u = (int64_t)blockIdx.x * (ACT_THREADS / 16) + half;
  int64_t row = u / nb;
  int blk = (int)(u % nb);
  // the two halves of a warp loop together (the shuffles below take both)
  for (int64_t u0 = u & ~int64_t(1); u0 < units; u0 += step * ACT_UNROLL) {
    Raw8<T> va[ACT_UNROLL], vb[ACT_UNROLL], vd[GRAD ? ACT_UNROLL : 1];
    int64_t rw[ACT_UNROLL];
    int col[ACT_UNROLL];
#pragma unroll
    for (int i = 0; i < ACT_UNROLL; ++i) {
      rw[i] = row;
      col[i] = blk * 128 + (lane & 15) * 8;
      const int n = row < rows ? a.I - col[i] : 0;
      const T* h = static_cast<const T*>(a.h) + row * a.ld_h + col[i];
      va[i] = load8_rw<T, VEC>(h, n);
      vb[i] = load8_rw<T, VEC>(h + a.I, n);
      if constexpr (GRAD) vd[i] = load8<T, VEC>(static_cast<const T*>(a.d_y) + row * a.ld_d_y + col[i], n);
      row += drow;
      blk += dblk;
      if (blk >= nb) {
        blk -= nb;
        ++row;
      }
    }
#pragma unroll
    for (int i = 0; i < ACT_UNROLL; ++i) {
      const int n = rw[i] < rows ? a.I - col[i] : 0;
      if constexpr (GRAD) {
        float da[8], db[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = to_f32(va[i].v[j]), d = to_f32(vd[i].v[j]), s = sigmoid_of<T>(x);
          da[j] = d * to_f32(vb[i].v[j]) * s * (1.f + x * (1.f - s));
          db[j] = d * x * s;
        }
        T* o = static_cast<T*>(a.d_h) + rw[i] * a.ld_d_h + col[i];
        store8<T, VEC>(o, pack8<T>(da), n);
        store8<T, VEC>(o + a.I, pack8<T>(db), n);
      } else {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = to_f32(va[i].v[j]);
          y[j] = x * sigmoid_of<T>(x) * to_f32(vb[i].v[j]);
        }
        if (a.y != nullptr) store8<T, VEC>(static_cast<T*>(a.y) + rw[i] * a.ld_y + col[i], pack8<T>(y), n);
        if (a.q != nullptr)
          store_e4m3<VEC>(y, static_cast<uint8_t*>(a.q) + rw[i] * a.ld_q + col[i], a.scale + rw[i] * a.ld_scale + col[i] / 128, lane, n);
      }
    }
  }
}

namespace {
bool act_vec(const moer_expert_act_args* a, bool grad, int eb) {
  const void* const p[] = {a->h, grad ? nullptr : a->y, grad ? a->d_y : nullptr, grad ? a->d_h : nullptr};
  const int64_t ld[] = {a->ld_h, a->ld_y, a->ld_d_y, a->ld_d_h};
  if (a->I % 8 != 0) return false;
  for (int i = 0; i < 4; ++i)
    if (p[i] != nullptr && (reinterpret_cast<uintptr_t>(p[i]) % 16 != 0 || ld[i] * eb % 16 != 0)) return false;
  return grad || a->q == nullptr || (reinterpret_cast<uintptr_t>(a->q) % 8 == 0 && a->ld_q % 8 == 0);
}

template <typename T>
cudaError_t act_run(const moer_expert_act_args* a, bool grad, unsigned grid, cudaStream_t st) {
  const bool vec = act_vec(a, grad, sizeof(T));
  if (grad) {
    if (vec) expert_act_kernel<T, true, true><<<grid, ACT_THREADS, 0, st>>>(*a);
    else expert_act_kernel<T, false, true><<<grid, ACT_THREADS, 0, st>>>(*a);
  } else {
    if (vec) expert_act_kernel<T, true, false><<<grid, ACT_THREADS, 0, st>>>(*a);
    else expert_act_kernel<T, false, false><<<grid, ACT_THREADS, 0, st>>>(*a);
  }
  return cudaGetLastError();
}
}  // namespace

moer_status expert_act_launch(const moer_expert_act_args* a, bool grad, cudaStream_t st) {
  const int sms = device_sm_count();
  if (sms <= 0) return MOER_ECUDA;
  const int64_t blocks = (a->rows * ((a->I + 127) / 128) + ACT_THREADS / 16 - 1) / (ACT_THREADS / 16);
  const unsigned grid = (unsigned)min64(blocks, (int64_t)sms * 16);
  const cudaError_t e = a->dtype == MOER_F32    ? act_run<float>(a, grad, grid, st)
                        : a->dtype == MOER_BF16 ? act_run<__nv_bfloat16>(a, grad, grid, st)
                                                : act_run<__half>(a, grad, grid, st);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
