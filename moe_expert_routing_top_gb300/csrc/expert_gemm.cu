// expert_gemm.cu -- moer_expert_gemm: matrix products grouped by expert, over ragged segments.
//
// The simplest form: a block of 256 threads takes 64 x 64 outputs of one expert, with operand
// tiles of 16 in shared memory as fp32.
#include "rows.cuh"

namespace moer {

constexpr int SG = 64, SK = 16;

struct Segment {
  int64_t lo, hi;
};

// Expert e's rows, held within [0, rows]; a malformed offset records MOER_EDATA.
__device__ __forceinline__ Segment segment(const moer_expert_gemm_args& a, int e, uint32_t* status) {
  const int64_t lo = a.expert_off[e], hi = a.expert_off[e + 1];
  Segment s;
  s.lo = max64(0, min64(lo, a.rows));
  s.hi = max64(s.lo, min64(hi, a.rows));
  if (s.lo != lo || s.hi != hi) atomicOr(status, WS_BIT_EDATA);
  return s;
}

// The row of x behind row p of the lists, or -1.
__device__ __forceinline__ int64_t source_row(const moer_expert_gemm_args& a, int64_t p, uint32_t* status) {
  if (a.order == nullptr) return p;
  const int o = a.order[p];
  if (o < 0) return -1;
  const int64_t r = o / a.k;
  if (r < a.tokens) return r;
  atomicOr(status, WS_BIT_EDATA);
  return -1;
}

__device__ __forceinline__ float elem(const void* p, int dtype, int64_t i) {
  if (dtype == MOER_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == MOER_F16) return __half2float(static_cast<const __half*>(p)[i]);
  __nv_fp8_e4m3 v;
  v.__x = static_cast<const uint8_t*>(p)[i];
  return (float)v;
}

__device__ __forceinline__ void put(void* p, int dtype, int64_t i, float v) {
  if (dtype == MOER_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == MOER_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// out tile rows i, columns j; contraction c.  Rows are list rows (or n of the weights' gradient).
__global__ void __launch_bounds__(256) expert_gemm_kernel(const __grid_constant__ moer_expert_gemm_args a, uint32_t* status) {
  __shared__ float A[SK][SG + 1], B[SK][SG + 1];
  __shared__ int64_t src[SG];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const bool gw = a.op == MOER_GEMM_GRAD_WEIGHT;
  int e = 0;
  Segment sg = {0, 0};
  int64_t i0;
  if (gw) {
    e = blockIdx.z;
    sg = segment(a, e, status);
    i0 = (int64_t)blockIdx.y * SG;
  } else {
    int64_t y = blockIdx.y;
    for (;; ++e) {
      if (e == a.E) return;
      sg = segment(a, e, status);
      const int64_t nt = (sg.hi - sg.lo + SG - 1) / SG;
      if (y < nt) break;
      y -= nt;
    }
    i0 = sg.lo + y * SG;
    if (threadIdx.x < SG) src[threadIdx.x] = i0 + threadIdx.x < sg.hi ? source_row(a, i0 + threadIdx.x, status) : -1;
  }
  const int64_t j0 = (int64_t)blockIdx.x * SG;
  const int64_t C = gw ? sg.hi - sg.lo : (a.op == MOER_GEMM_FORWARD ? a.K : a.N);
  const int64_t NI = gw ? a.N : sg.hi, NJ = a.op == MOER_GEMM_FORWARD ? a.N : a.K;
  const bool fp8 = a.dtype == MOER_E4M3;
  const int nkb = (a.K + 127) / 128, nnb = (a.N + 127) / 128;
  float acc[4][4] = {};
  for (int64_t c0 = 0; c0 < C; c0 += SK) {
    __syncthreads();
    for (int t = threadIdx.x; t < SK * SG; t += 256) {
      float va = 0.f, vb = 0.f;
      if (gw) {
        const int i = t % SG, c = t / SG;
        const int64_t p = sg.lo + c0 + c;
        const int64_t r = p < sg.hi ? source_row(a, p, status) : -1;
        if (r >= 0 && i0 + i < NI) va = elem(a.d_y, a.dtype, p * a.ld_d_y + i0 + i);
        if (r >= 0 && j0 + i < NJ) vb = elem(a.x, a.dtype, r * a.ld_x + j0 + i);
        A[c][i] = va;
        B[c][i] = vb;
      } else {
        {
          const int c = t % SK, i = t / SK;
          const int64_t r = src[i];
          if (r >= 0 && c0 + c < C) {
            va = elem(a.x, a.dtype, r * a.ld_x + c0 + c);
            if (fp8) va *= a.x_scale[r * a.ld_x_scale + (c0 + c) / 128];
          }
          A[c][i] = va;
        }
        const bool fwd = a.op == MOER_GEMM_FORWARD;
        const int c = fwd ? t % SK : t / SG, j = fwd ? t / SK : t % SG;
        if (j0 + j < NJ && c0 + c < C) {
          const int64_t n = fwd ? j0 + j : c0 + c, k = fwd ? c0 + c : j0 + j;
          vb = elem(a.w, a.dtype, e * a.stride_w + n * a.ld_w + k);
          if (fp8) vb *= a.w_scale[((int64_t)e * nnb + n / 128) * nkb + k / 128];
        }
        B[c][j] = vb;
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < SK; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(A[c][ty + 16 * i], B[c][tx + 16 * j], acc[i][j]);
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
      if (r >= NI || c >= NJ) continue;
      const int64_t base = gw ? e * a.stride_out : 0;
      put(a.out, a.out_dtype, base + r * a.ld_out + c, acc[i][j]);
    }
}

moer_status expert_gemm_launch(const moer_expert_gemm_args* a, void* ws, cudaStream_t st) {
  const bool gw = a->op == MOER_GEMM_GRAD_WEIGHT;
  const int NJ = a->op == MOER_GEMM_FORWARD ? a->N : a->K;
  const int64_t ty = gw ? (a->N + SG - 1) / SG : a->rows / SG + a->E;
  if (ty > 65535) return MOER_ERANGE;
  dim3 grid((NJ + SG - 1) / SG, (unsigned)ty, gw ? a->E : 1);
  expert_gemm_kernel<<<grid, 256, 0, st>>>(*a, static_cast<uint32_t*>(ws));
  return cudaGetLastError() == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
