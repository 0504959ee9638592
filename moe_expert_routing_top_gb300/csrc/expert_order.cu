// expert_order.cu -- moer_expert_order: each layer's (token, choice) pairs in
// the order of their experts (a stable counting sort by the expert id), each
// expert's segment padded to a multiple of `align`.
//
// Over chunks of 8,192 consecutive pairs of a layer:
//   count    a chunk's histogram of experts (16 ids to a thread, one load);
//   offsets  per layer, the experts' totals, their padded offsets and, in place
//            of each histogram, the row at which the chunk's pairs of an
//            expert start; the padding is set to -1;
//   place    a chunk is sorted in shared memory and written out from there: every
//            warp takes its pairs 32 at a time in order, finds the lanes with
//            the same expert by a vote on each bit of the id, and adds their
//            number below to the warp's running count; the warps' counts are
//            then scanned, and rows follow.
// Sorting in shared memory first turns the scattered 4-byte writes of `order`
// into runs (a chunk holds 64 pairs of each of 128 experts: 256 bytes).
// A layer that fits one chunk takes one launch, which does all three.
#include "common.cuh"
#include "pdl.cuh"

namespace moer {

namespace {
constexpr int EO_WARPS = 16;
constexpr int EO_THREADS = EO_WARPS * 32;
constexpr int EO_PAIRS = 8192;                  // of a chunk
constexpr int EO_IT = EO_PAIRS / EO_THREADS;    // rounds of 32 pairs of a warp
constexpr int EO_SCAN = 1024;

struct OrderParams {
  const uint8_t* ids;  // [L][N]
  int N, E, L, align;  // pairs and experts of a layer
  int nchunk;
  int vec;             // 1: every layer's ids start on 16 bytes
  uint32_t* hist;      // [L][nchunk][E]
  int32_t* off;        // [L][E+1]
  int32_t* order;      // [L][ld] or NULL
  int64_t ld;
  int32_t* inv;        // [L][N] or NULL
  uint32_t* status;
};

// A chunk's ids to shared memory.
__device__ __forceinline__ void load_ids(const OrderParams& p, const uint8_t* ids, int n, uint8_t* sid) {
  if (p.vec != 0) {
    const int i = (int)threadIdx.x * 16;
    if (i + 16 <= n)
      *reinterpret_cast<uint4*>(sid + i) = *reinterpret_cast<const uint4*>(ids + i);
    else
      for (int j = i; j < n; ++j) sid[j] = ids[j];
  } else {
    for (int i = threadIdx.x; i < n; i += EO_THREADS) sid[i] = ids[i];
  }
}

__global__ void __launch_bounds__(EO_THREADS) order_count_kernel(const OrderParams p) {
  __shared__ uint32_t h[256];
  __shared__ __align__(16) uint8_t sid[EO_PAIRS];
  pdl_wait();
  const int l = blockIdx.x / p.nchunk, c = blockIdx.x - l * p.nchunk;
  const int64_t i0 = (int64_t)c * EO_PAIRS;
  const int n = (int)min64(EO_PAIRS, p.N - i0);
  if (threadIdx.x < 256) h[threadIdx.x] = 0u;
  load_ids(p, p.ids + (size_t)l * p.N + i0, n, sid);
  __syncthreads();
  bool bad = false;
  // a warp's lanes read neighbouring words; each holds four ids
  for (int w = threadIdx.x; 4 * w < n; w += EO_THREADS) {
    const uint32_t q = *reinterpret_cast<const uint32_t*>(sid + 4 * w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = (q >> (8 * j)) & 255;
      if (4 * w + j < n) {
        atomicAdd(&h[e], 1u);
        bad = bad || e >= p.E;
      }
    }
  }
  if (bad) atomicOr(p.status, WS_BIT_EDATA);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += EO_THREADS) p.hist[(size_t)blockIdx.x * p.E + e] = h[e];
  pdl_release();
}

// Exclusive sums of 256 values by one warp group of 256 threads (8 warps);
// every thread of the block calls it.  total: the sum of all.
__device__ __forceinline__ uint32_t scan256(uint32_t v, uint32_t* wsum, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31 && warp < 8) wsum[warp] = x;
  __syncthreads();
  uint32_t before = 0u;
  total = 0u;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  __syncthreads();
  return before + x - v;
}

// -1 in the rows of a layer's `order` that hold no pair, by `nwarps` warps.
__device__ __forceinline__ void fill_padding(const OrderParams& p, int l, const uint32_t* off, const uint32_t* tot,
                                             int nwarps) {
  int32_t* order = p.order + (size_t)l * p.ld;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = warp; e < p.E; e += nwarps)
    for (uint32_t r = off[e] + tot[e] + lane; r < off[e + 1]; r += 32) order[r] = -1;
  for (int64_t r = (int64_t)off[p.E] + threadIdx.x; r < p.ld; r += nwarps * 32) order[r] = -1;
}

// One block per layer: four threads to an expert, each with a quarter of the chunks.
__global__ void __launch_bounds__(EO_SCAN) order_offsets_kernel(const OrderParams p) {
  __shared__ uint32_t off[257], tot[256], wsum[8], quarter[4][256];
  pdl_wait();
  const int l = blockIdx.x, e = threadIdx.x & 255, q = threadIdx.x >> 8;
  uint32_t* h = p.hist + (size_t)l * p.nchunk * p.E;
  const int c0 = (int)((int64_t)p.nchunk * q / 4), c1 = (int)((int64_t)p.nchunk * (q + 1) / 4);
  uint32_t s = 0u;
  if (e < p.E) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) s += h[(size_t)c * p.E + e];
  }
  quarter[q][e] = s;
  __syncthreads();
  const uint32_t all = quarter[0][e] + quarter[1][e] + quarter[2][e] + quarter[3][e];
  const uint32_t padded = (all + p.align - 1) / p.align * p.align;
  uint32_t total;
  const uint32_t at = scan256(q == 0 ? padded : 0u, wsum, total);
  if (q == 0) {
    off[e] = at;
    tot[e] = all;
    if (e == 0) off[256] = total;  // E = 256; a smaller E's end is its next, empty expert's start
  }
  __syncthreads();
  if ((int)threadIdx.x <= p.E) p.off[(size_t)l * (p.E + 1) + threadIdx.x] = (int32_t)off[threadIdx.x];
  if (e < p.E) {
    uint32_t r = off[e];
    for (int i = 0; i < q; ++i) r += quarter[i][e];
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
      const uint32_t n = h[(size_t)c * p.E + e];
      h[(size_t)c * p.E + e] = r;
      r += n;
    }
  }
  if (p.order != nullptr) fill_padding(p, l, off, tot, EO_SCAN / 32);
  pdl_release();
}

// BITS: of an expert id (E <= 2^BITS).  ALONE: the layer is one chunk, and this
// launch also makes the offsets and the padding.
template <int BITS, bool ALONE>
__global__ void __launch_bounds__(EO_THREADS) order_place_kernel(const OrderParams p) {
  constexpr int EM = 1 << BITS;
  __shared__ uint32_t count[EO_WARPS][EM];  // pairs of each expert: the warp's, then those before it in the chunk
  __shared__ uint32_t shift[256];           // row of an expert's first pair, less its place in the sorted chunk
  __shared__ uint32_t wsum[8];
  __shared__ __align__(16) uint8_t sid[EO_PAIRS];
  __shared__ uint16_t sorted[EO_PAIRS];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = blockIdx.x / p.nchunk, c = blockIdx.x - l * p.nchunk;
  const int64_t i0 = (int64_t)c * EO_PAIRS;
  const int n = (int)min64(EO_PAIRS, p.N - i0);
  load_ids(p, p.ids + (size_t)l * p.N + i0, n, sid);
  for (int e = lane; e < EM; e += 32) count[warp][e] = 0u;
  __syncthreads();
  uint32_t rank[EO_IT];
  // a warp's pairs: whole rounds of 32, spread over the warps where the chunk is short
  const int span = (n + EO_THREADS - 1) / EO_THREADS * 32;
  const int w0 = warp * span;
  bool bad = false;
#pragma unroll
  for (int it = 0; it < EO_IT; ++it) {
    if (it * 32 >= span) break;
    const int i = w0 + it * 32 + lane;
    const int e = i < n ? sid[i] : 256;
    const bool ok = e < p.E;
    bad = bad || (i < n && !ok);
    unsigned same = __ballot_sync(FULL, ok);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
      const unsigned v = __ballot_sync(FULL, (e >> b) & 1);
      same &= ((e >> b) & 1) ? v : ~v;
    }
    const unsigned below = same & ((1u << lane) - 1u);
    const uint32_t before = ok ? count[warp][e & (EM - 1)] : 0u;
    __syncwarp();
    if (ok && below == 0u) count[warp][e & (EM - 1)] = before + __popc(same);
    __syncwarp();
    rank[it] = before + __popc(below);
  }
  if (ALONE && bad) atomicOr(p.status, WS_BIT_EDATA);
  __syncthreads();
  // the warps' counts become the pairs of earlier warps; the experts' totals are scanned
  uint32_t mine = 0u;
  const int e = threadIdx.x;
  if (e < EM) {
#pragma unroll
    for (int w = 0; w < EO_WARPS; ++w) {
      const uint32_t v = count[w][e];
      count[w][e] = mine;
      mine += v;
    }
  }
  uint32_t total;
  const uint32_t start = scan256(e < 256 ? mine : 0u, wsum, total);
  uint32_t row = 0u;
  if constexpr (ALONE) {
    __shared__ uint32_t off[257], tot[256];
    const uint32_t padded = (mine + p.align - 1) / p.align * p.align;
    uint32_t end;
    row = scan256(e < 256 ? padded : 0u, wsum, end);
    if (e < 256) off[e] = row, tot[e] = mine;
    if (e == 0) off[256] = end;
    __syncthreads();
    if (e <= p.E) p.off[(size_t)l * (p.E + 1) + e] = (int32_t)off[e];
    if (p.order != nullptr) fill_padding(p, l, off, tot, EO_WARPS);
  } else if (e < p.E) {
    row = p.hist[(size_t)blockIdx.x * p.E + e];
  }
  if (e < EM) {
    shift[e] = row - start;
#pragma unroll
    for (int w = 0; w < EO_WARPS; ++w) count[w][e] += start;
  }
  __syncthreads();
  int32_t* inv = p.inv != nullptr ? p.inv + (size_t)l * p.N + i0 : nullptr;
#pragma unroll
  for (int it = 0; it < EO_IT; ++it) {
    if (it * 32 >= span) break;
    const int i = w0 + it * 32 + lane;
    if (i < n) {
      const int x = sid[i];
      const bool ok = x < p.E;
      const uint32_t place = ok ? rank[it] + count[warp][x & (EM - 1)] : 0u;
      if (ok) sorted[place] = (uint16_t)i;
      if (inv != nullptr) inv[i] = ok ? (int32_t)(place + shift[x & (EM - 1)]) : -1;
    }
  }
  if (p.order != nullptr) {
    __syncthreads();
    int32_t* order = p.order + (size_t)l * p.ld;
    for (int s = threadIdx.x; s < (int)total; s += EO_THREADS) {
      const int i = sorted[s];
      order[(uint32_t)s + shift[sid[i]]] = (int32_t)(i0 + i);
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

template <bool ALONE>
cudaError_t place(const OrderParams& p, cudaStream_t st) {
  const dim3 grid(p.L * p.nchunk), block(EO_THREADS);
  return p.E <= 64    ? launch_pdl(order_place_kernel<6, ALONE>, grid, block, 0, st, p)
         : p.E <= 128 ? launch_pdl(order_place_kernel<7, ALONE>, grid, block, 0, st, p)
                      : launch_pdl(order_place_kernel<8, ALONE>, grid, block, 0, st, p);
}
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
  p.vec = reinterpret_cast<uintptr_t>(topk) % 16 == 0 && (p.L == 1 || p.N % 16 == 0);
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
  if (p.nchunk == 1) return place<true>(p, st) == cudaSuccess ? MOER_OK : MOER_ECUDA;
  const dim3 grid(p.L * p.nchunk), block(EO_THREADS);
  cudaError_t e = launch_pdl(order_count_kernel, grid, block, 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(order_offsets_kernel, dim3(p.L), dim3(EO_SCAN), 0, st, p);
  if (e == cudaSuccess && (order != nullptr || inv != nullptr)) e = place<false>(p, st);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
