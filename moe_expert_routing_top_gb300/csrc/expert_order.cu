// expert_order.cu -- moer_expert_order: each layer's (token, choice) pairs in
// the order of their experts (a stable counting sort by the expert id), each
// expert's segment padded to a multiple of `align`.
//
// Three kernels over chunks of consecutive pairs of a layer:
//   count    a chunk's histogram of experts;
//   offsets  per layer, the experts' totals, their padded offsets and, in place
//            of each histogram, the row at which the chunk's pairs of an
//            expert start; the padding is set to -1;
//   place    every pair's row: the chunk's start for its expert, the pairs of the
//            chunk's earlier warps, and its rank within its own warp, which
//            takes its pairs 32 at a time and ranks equal ids by a match
//            among the lanes.
#include "common.cuh"
#include "pdl.cuh"

namespace moer {

namespace {
constexpr int EO_WARPS = 8;
constexpr int EO_PAIRS = 4096;                      // of a chunk
constexpr int EO_WPAIRS = EO_PAIRS / EO_WARPS;      // of a warp
constexpr int EO_SCAN = 1024;

struct OrderParams {
  const uint8_t* ids;  // [L][N]
  int N, E, L, align;  // pairs and experts of a layer
  int nchunk;
  uint32_t* hist;      // [L][nchunk][E]
  int32_t* off;        // [L][E+1]
  int32_t* order;      // [L][ld] or NULL
  int64_t ld;
  int32_t* inv;        // [L][N] or NULL
  uint32_t* status;
};

__global__ void __launch_bounds__(EO_WARPS * 32) order_count_kernel(const OrderParams p) {
  __shared__ uint32_t h[256];
  pdl_wait();
  const int l = blockIdx.x / p.nchunk, c = blockIdx.x - l * p.nchunk;
  for (int e = threadIdx.x; e < p.E; e += EO_WARPS * 32) h[e] = 0u;
  __syncthreads();
  const uint8_t* ids = p.ids + (size_t)l * p.N;
  const int i1 = (int)min64((int64_t)(c + 1) * EO_PAIRS, p.N);
  bool bad = false;
  for (int i = c * EO_PAIRS + threadIdx.x; i < i1; i += EO_WARPS * 32) {
    const int e = ids[i];
    if (e < p.E)
      atomicAdd(&h[e], 1u);
    else
      bad = true;
  }
  if (bad) atomicOr(p.status, WS_BIT_EDATA);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += EO_WARPS * 32) p.hist[(size_t)blockIdx.x * p.E + e] = h[e];
  pdl_release();
}

// One block per layer; thread e < E owns an expert.
__global__ void __launch_bounds__(EO_SCAN) order_offsets_kernel(const OrderParams p) {
  __shared__ uint32_t off[257], tot[256];
  pdl_wait();
  const int l = blockIdx.x, e = threadIdx.x;
  uint32_t* h = p.hist + (size_t)l * p.nchunk * p.E;
  if (e < p.E) {
    uint32_t s = 0u;
    for (int c = 0; c < p.nchunk; ++c) s += h[(size_t)c * p.E + e];
    tot[e] = s;
  }
  __syncthreads();
  if (e == 0) {
    uint32_t s = 0u;
    for (int i = 0; i < p.E; ++i) {
      off[i] = s;
      s += (tot[i] + p.align - 1) / p.align * p.align;
    }
    off[p.E] = s;
  }
  __syncthreads();
  for (int i = e; i <= p.E; i += EO_SCAN) p.off[(size_t)l * (p.E + 1) + i] = (int32_t)off[i];
  if (e < p.E) {
    uint32_t s = off[e];
    for (int c = 0; c < p.nchunk; ++c) {
      const uint32_t n = h[(size_t)c * p.E + e];
      h[(size_t)c * p.E + e] = s;
      s += n;
    }
  }
  if (p.order != nullptr) {
    int32_t* order = p.order + (size_t)l * p.ld;
    for (int i = 0; i < p.E; ++i)
      for (uint32_t r = off[i] + tot[i] + e; r < off[i + 1]; r += EO_SCAN) order[r] = -1;
    for (int64_t r = off[p.E] + e; r < p.ld; r += EO_SCAN) order[r] = -1;
  }
  pdl_release();
}

__global__ void __launch_bounds__(EO_WARPS * 32) order_place_kernel(const OrderParams p) {
  __shared__ uint32_t next[EO_WARPS][256];  // the row of each warp's next pair of an expert
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = blockIdx.x / p.nchunk, c = blockIdx.x - l * p.nchunk;
  const uint8_t* ids = p.ids + (size_t)l * p.N;
  int32_t* inv = p.inv != nullptr ? p.inv + (size_t)l * p.N : nullptr;
  int32_t* order = p.order != nullptr ? p.order + (size_t)l * p.ld : nullptr;
  for (int e = lane; e < p.E; e += 32) next[warp][e] = 0u;
  __syncwarp();
  const int64_t i0 = (int64_t)c * EO_PAIRS + warp * EO_WPAIRS;
  for (int64_t i = i0 + lane; i < i0 + EO_WPAIRS; i += 32)
    if (i < p.N && ids[i] < p.E) atomicAdd(&next[warp][ids[i]], 1u);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += EO_WARPS * 32) {
    uint32_t s = p.hist[(size_t)blockIdx.x * p.E + e];
#pragma unroll
    for (int w = 0; w < EO_WARPS; ++w) {
      const uint32_t n = next[w][e];
      next[w][e] = s;
      s += n;
    }
  }
  __syncthreads();
  for (int64_t i = i0 + lane; i - lane < min64(i0 + EO_WPAIRS, p.N); i += 32) {
    const int e = i < p.N ? ids[i] : 0xFFFF;
    const unsigned same = __match_any_sync(FULL, e);
    const bool ok = e < p.E;
    const uint32_t base = ok ? next[warp][e] : 0u;
    __syncwarp();
    const unsigned below = same & ((1u << lane) - 1u);
    if (ok && below == 0u) next[warp][e] = base + __popc(same);
    __syncwarp();
    const int32_t row = ok ? (int32_t)(base + __popc(below)) : -1;
    if (i < p.N) {
      if (inv != nullptr) inv[i] = row;
      if (order != nullptr && ok) order[row] = (int32_t)i;
    }
  }
  pdl_release();
}

__global__ void order_empty_kernel(const OrderParams p) {
  const int l = blockIdx.x;
  for (int i = threadIdx.x; i <= p.E; i += blockDim.x) p.off[(size_t)l * (p.E + 1) + i] = 0;
  if (p.order != nullptr)
    for (int64_t r = threadIdx.x; r < p.ld; r += blockDim.x) p.order[(size_t)l * p.ld + r] = -1;
}

int64_t order_chunks(int64_t N) { return (N + EO_PAIRS - 1) / EO_PAIRS; }
}  // namespace

size_t expert_order_scratch_bytes(const moer_dims* d, int64_t T) {
  return (size_t)d->L * (size_t)order_chunks(T * d->k) * (size_t)d->E * 4;
}

moer_status expert_order_launch(const moer_dims* d, const uint8_t* topk, int64_t T, int32_t align, int32_t* off,
                                int32_t* order, int64_t ld, int32_t* inv, void* ws, cudaStream_t st) {
  OrderParams p;
  p.ids = topk;
  p.N = (int)(T * d->k);
  p.E = d->E;
  p.L = d->L;
  p.align = align;
  p.nchunk = (int)order_chunks(p.N);
  p.hist = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + WS_HEADER);
  p.off = off;
  p.order = order;
  p.ld = ld;
  p.inv = inv;
  p.status = static_cast<uint32_t*>(ws);
  if (p.N == 0) {
    order_empty_kernel<<<p.L, 256, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? MOER_OK : MOER_ECUDA;
  }
  const dim3 grid(p.L * p.nchunk), block(EO_WARPS * 32);
  cudaError_t e = launch_pdl(order_count_kernel, grid, block, 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(order_offsets_kernel, dim3(p.L), dim3(EO_SCAN), 0, st, p);
  if (e == cudaSuccess && (order != nullptr || inv != nullptr)) e = launch_pdl(order_place_kernel, grid, block, 0, st, p);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
