// expert_order.cu -- moer_expert_order: each layer's (token, choice) pairs in
// the order of their experts (a stable counting sort by the expert id), each
// expert's segment padded to a multiple of `align`.
//
// Over chunks of up to 32 tiles of 32 tokens (8,192 pairs):
//   count    a chunk's histogram of experts (16 ids to a thread, one load);
//   offsets  per layer, the experts' totals, their padded offsets and, in place
//            of each histogram, the row at which the chunk's pairs of an
//            expert start;
//   place    a chunk is sorted in shared memory and written out from there.  For
//            every tile and expert a word holds which of the tile's 32 tokens
//            chose the expert, one bit each, set by an atomic or: a pair's rank
//            in its tile is the number of lower bits, whatever the order in which
//            the bits came.  The words' counts are summed over the tiles, and
//            rows follow.  (Ranking by votes on the ids' bits took 124
//            instructions for 32 pairs; this takes about a third.)
// Sorting in shared memory first turns the scattered 4-byte writes of `order`
// into runs (a chunk holds 64 pairs of each of 128 experts: 256 bytes).
// A token that names an expert twice has one bit for two pairs: the chunk is
// then placed by a thread to an expert that reads the pairs in order.
// A layer that fits one chunk takes one launch, which does all three.
// Measured (GB300): 65,536 tokens x 48 layers, E = 128, k = 8, segments padded to 128:
// 92 us, 2.46 TB/s of algorithmic bytes (9 a pair); the place kernel is bound by
// shared memory, 22 passes over its banks for 32 pairs (random words: the ors 4,
// the reads 12, the sorted pairs' writes 5) at 82 % of its rate.  64 tokens, one layer: 4.0 us.
#include "common.cuh"
#include "pdl.cuh"

namespace moer {

namespace {
constexpr int EO_WARPS = 16;
constexpr int EO_THREADS = EO_WARPS * 32;
constexpr int EO_PAIRS = 8192;                  // of a chunk, at most
constexpr int EO_TILES = 32;                    // of a chunk, at most (16 for E > 128)
constexpr int EO_SCAN = 1024;

struct OrderParams {
  const uint8_t* ids;  // [L][N]
  int N, E, L, align;  // pairs and experts of a layer
  int k, T, ctok;      // ids of a token, tokens of a layer and of a chunk
  int nchunk;
  int vec;             // 1: every layer's ids and inv start on 16 bytes
  int pairs;           // 1: k is even and inv takes pairs
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
  pdl_wait();
  const int l = blockIdx.x / p.nchunk, c = blockIdx.x - l * p.nchunk;
  const int64_t i0 = (int64_t)c * p.ctok * p.k;
  const int n = (int)min64((int64_t)p.ctok * p.k, p.N - i0);
  const uint8_t* ids = p.ids + (size_t)l * p.N + i0;
  const int i = (int)threadIdx.x * 16;
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  const bool whole = p.vec != 0 && i + 16 <= n;
  if (whole) q = *reinterpret_cast<const uint4*>(ids + i);
  if (threadIdx.x < 256) h[threadIdx.x] = 0u;
  __syncthreads();
  if (whole) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 16; ++j) atomicAdd(&h[w[j / 4] >> (8 * (j % 4)) & 255u], 1u);
  } else if (p.vec != 0) {
    for (int j = i; j < n; ++j) atomicAdd(&h[ids[j]], 1u);
  } else {
    for (int j = threadIdx.x; j < n; j += EO_THREADS) atomicAdd(&h[ids[j]], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 256; e += EO_THREADS) {
    if (e < p.E)
      p.hist[(size_t)blockIdx.x * p.E + e] = h[e];
    else if (h[e] != 0u)
      atomicOr(p.status, WS_BIT_EDATA);
  }
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

// -1 in the rows of a layer's `order` that hold no pair, by the layer's last
// chunk: `end` [E] the rows after the experts' last pairs, `off` [E+1].
template <typename Off>
__device__ __forceinline__ void fill_padding(const OrderParams& p, int l, const Off* off, const uint32_t* end) {
  int32_t* order = p.order + (size_t)l * p.ld;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = warp; e < p.E; e += EO_WARPS)
    for (uint32_t r = end[e] + lane; r < (uint32_t)off[e + 1]; r += 32) order[r] = -1;
  for (int64_t r = (int64_t)(uint32_t)off[p.E] + threadIdx.x; r < p.ld; r += EO_THREADS) order[r] = -1;
}

// One block per layer: four threads to an expert, each with a quarter of the chunks.
__global__ void __launch_bounds__(EO_SCAN) order_offsets_kernel(const OrderParams p) {
  __shared__ uint32_t off[257], wsum[8], quarter[4][256];
  pdl_wait();
  pdl_release();  // the place kernel's blocks rank their pairs meanwhile, and wait before they read what this one writes
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
}

// EM: room for the experts, 64, 128 or 256.  ALONE: the layer is one chunk, and this
// launch also makes the offsets.
template <int EM>
struct PlaceGeo {
  static constexpr int TILES = EM > 128 ? 16 : EO_TILES;
  static constexpr int PAIRS = EM > 128 ? EO_PAIRS / 2 : EO_PAIRS;
  static constexpr size_t OFF_SORTED = (size_t)TILES * EM * 8;
  static constexpr size_t OFF_IDS = OFF_SORTED + (size_t)PAIRS * 4;
  static constexpr size_t SMEM8 = OFF_IDS, SMEM = OFF_IDS + PAIRS;  // k = 8, any k
};

// The word of a tile that holds expert e's tokens, and the one that holds the place
// of its first pair: neighbours, in turns, so that either spreads over all banks.
__device__ __forceinline__ int bits_at(int e) { return 2 * e + (e >> 4 & 1); }
__device__ __forceinline__ int place_at(int e) { return 2 * e + 1 - (e >> 4 & 1); }

template <int EM, bool ALONE, bool K8>
__global__ void __launch_bounds__(EO_THREADS) order_place_kernel(const OrderParams p) {
  constexpr int SEG = EO_THREADS / EM;  // threads to an expert in the sums
  constexpr int MINE = 2;               // tiles of a warp
  extern __shared__ __align__(16) char smem[];
  uint32_t(*tiles)[2 * EM] = reinterpret_cast<uint32_t(*)[2 * EM]>(smem);
  uint32_t* sorted = reinterpret_cast<uint32_t*>(smem + PlaceGeo<EM>::OFF_SORTED);  // expert, pair
  uint8_t* sid = reinterpret_cast<uint8_t*>(smem + PlaceGeo<EM>::OFF_IDS);          // the ids, where k is not 8
  __shared__ uint32_t shift[256];       // row of an expert's first pair, less its place in the sorted chunk
  __shared__ uint32_t end[256];         // row after its last pair
  __shared__ uint32_t part[SEG][EM];
  __shared__ uint32_t wsum[8];
  __shared__ uint32_t off[257];
  __shared__ uint32_t strangers;        // ids of no expert
  // Not ALONE, the ids are final already: the offsets kernel releases this one only
  // after the kernels before it have ended, and only its offsets are waited for, below.
  if (ALONE) pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = blockIdx.x / p.nchunk, c = blockIdx.x - l * p.nchunk;
  const int k = K8 ? 8 : p.k;
  const int64_t t0 = (int64_t)c * p.ctok;
  const int ntok = (int)min64(p.ctok, p.T - t0), ntile = (ntok + 31) >> 5, n = ntok * k;
  const int64_t i0 = t0 * k;
  const uint8_t* ids = p.ids + (size_t)l * p.N + i0;
  const unsigned below = (1u << lane) - 1u;
  if (threadIdx.x == 0) strangers = 0u;
  uint2 eight[MINE];
#pragma unroll
  for (int q = 0; q < MINE; ++q) {
    const int tile = warp + q * EO_WARPS, t = tile * 32 + lane;
    eight[q] = make_uint2(0u, 0u);
    if (K8 && t < ntok) eight[q] = *reinterpret_cast<const uint2*>(ids + t * 8);
    if (tile < ntile)
      for (int e = lane; e < EM; e += 32) reinterpret_cast<uint2*>(tiles[tile])[e] = make_uint2(0u, 0u);
  }
  if (!K8) load_ids(p, ids, n, sid);
  __syncthreads();
  auto id_of = [&](int q, int t, int j) {
    if (K8) return (int)(__byte_perm(eight[q].x, eight[q].y, j) & 255u);
    return (int)sid[t * k + j];
  };
  // each lane begins with another choice: tokens often rank the same expert first
  const int turn = K8 ? lane & 7 : lane % k;
  uint32_t none = 0u;
#pragma unroll
  for (int q = 0; q < MINE; ++q) {
    const int tile = warp + q * EO_WARPS, t = tile * 32 + lane;
    if (t < ntok) {
      int j = turn;
#pragma unroll 8
      for (int i = 0; i < k; ++i) {
        const int e = id_of(q, t, j);
        if (e < p.E)
          atomicOr(&tiles[tile][bits_at(e)], 1u << lane);
        else
          ++none;
        j = K8 ? (j + 1) & 7 : j + 1 < k ? j + 1 : 0;
      }
    }
  }
  if (none != 0u) {
    atomicAdd(&strangers, none);
    if (ALONE) atomicOr(p.status, WS_BIT_EDATA);
  }
  __syncthreads();
  // the pairs of each expert: in earlier tiles, and in all
  const int e = threadIdx.x % EM, seg = threadIdx.x / EM;
  const int s0 = ntile * seg / SEG, s1 = ntile * (seg + 1) / SEG;
  constexpr int EACH = PlaceGeo<EM>::TILES / SEG;  // tiles of a thread, at most
  uint32_t count = 0u, in_tile[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    in_tile[i] = s0 + i < s1 ? __popc(tiles[s0 + i][bits_at(e)]) : 0u;
    count += in_tile[i];
  }
  uint32_t mine, before, total, start;
  auto sum = [&]() {
    part[seg][e] = count;
    __syncthreads();
    mine = before = 0u;
#pragma unroll
    for (int i = 0; i < SEG; ++i) {
      if (i < seg) before += part[i][e];
      mine += part[i][e];
    }
    start = scan256((int)threadIdx.x < EM ? mine : 0u, wsum, total);
  };
  sum();
  const bool serial = total + strangers != (uint32_t)n;  // some token names an expert twice
  if (serial) {
    count = 0u;
    if (seg == 0 && e < p.E)
      for (int i = 0; i < n; ++i) count += ids[i] == e ? 1u : 0u;
    sum();
  }
  if (!ALONE) pdl_wait();
  uint32_t row = 0u;
  if constexpr (ALONE) {
    const uint32_t padded = (mine + p.align - 1) / p.align * p.align;
    uint32_t last;
    row = scan256((int)threadIdx.x < EM ? padded : 0u, wsum, last);
    if (threadIdx.x < 256) off[threadIdx.x] = row;
    if (threadIdx.x == 0) off[256] = last;
    __syncthreads();
    if ((int)threadIdx.x <= p.E) p.off[(size_t)l * (p.E + 1) + threadIdx.x] = (int32_t)off[threadIdx.x];
  } else if ((int)threadIdx.x < p.E) {
    row = p.hist[(size_t)blockIdx.x * p.E + threadIdx.x];
  }
  if ((int)threadIdx.x < EM) {
    shift[threadIdx.x] = row - start;
    end[threadIdx.x] = row + mine;
    part[0][threadIdx.x] = start;
  }
  __syncthreads();
  start = part[0][e];
  int32_t* inv = p.inv != nullptr ? p.inv + (size_t)l * p.N + i0 : nullptr;
  if (!serial) {
    uint32_t at = start + before;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (s0 + i < s1) tiles[s0 + i][place_at(e)] = at;
      at += in_tile[i];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < MINE; ++q) {
      const int tile = warp + q * EO_WARPS, t = tile * 32 + lane;
      if (t < ntok) {
        auto row_of = [&](int j) {
          const int x = id_of(q, t, j);
          int32_t r = -1;
          if (x < p.E) {
            const uint2 w = reinterpret_cast<const uint2*>(tiles[tile])[x];
            const bool odd = (x >> 4 & 1) != 0;
            const uint32_t place = (odd ? w.x : w.y) + __popc((odd ? w.y : w.x) & below);
            sorted[place] = (uint32_t)x << 16 | (uint32_t)(t * k + j);
            r = (int32_t)(place + shift[x]);
          }
          return r;
        };
        if constexpr (K8) {
          int32_t rows[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) rows[j] = row_of(j);
          if (inv != nullptr) {
            if (p.vec != 0) {
              *reinterpret_cast<int4*>(inv + t * 8) = make_int4(rows[0], rows[1], rows[2], rows[3]);
              *reinterpret_cast<int4*>(inv + t * 8 + 4) = make_int4(rows[4], rows[5], rows[6], rows[7]);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) inv[t * 8 + j] = rows[j];
            }
          }
        } else if (p.pairs != 0) {
          for (int j = 0; j < k; j += 2) {
            const int32_t a = row_of(j), b = row_of(j + 1);
            if (inv != nullptr) *reinterpret_cast<int2*>(inv + t * k + j) = make_int2(a, b);
          }
        } else {
          for (int j = 0; j < k; ++j) {
            const int32_t a = row_of(j);
            if (inv != nullptr) inv[t * k + j] = a;
          }
        }
      }
    }
  } else {
    if (seg == 0 && e < p.E) {
      uint32_t at = start;
      for (int i = 0; i < n; ++i)
        if (ids[i] == e) {
          if (inv != nullptr) inv[i] = (int32_t)(at + shift[e]);
          sorted[at++] = (uint32_t)e << 16 | (uint32_t)i;
        }
    }
    if (inv != nullptr)
      for (int i = threadIdx.x; i < n; i += EO_THREADS)
        if (ids[i] >= p.E) inv[i] = -1;
  }
  if (p.order != nullptr) {
    __syncthreads();
    int32_t* order = p.order + (size_t)l * p.ld;
    for (int s = threadIdx.x; s < (int)total; s += EO_THREADS) {
      const uint32_t w = sorted[s];
      order[(uint32_t)s + shift[w >> 16]] = (int32_t)(i0 + (w & 0xFFFFu));
    }
    if (c == p.nchunk - 1) {
      if constexpr (ALONE)
        fill_padding(p, l, off, end);
      else
        fill_padding(p, l, p.off + (size_t)l * (p.E + 1), end);
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

// Tokens of a chunk: as many tiles of 32 as the pairs and the tiles allow.
int order_ctok(int E, int k) {
  const int tiles = E > 128 ? 16 : EO_TILES, pairs = E > 128 ? EO_PAIRS / 2 : EO_PAIRS;
  const int fit = pairs / (32 * k);
  return 32 * (fit < tiles ? fit : tiles);
}
int64_t order_chunks(int E, int k, int64_t T) {
  const int ctok = order_ctok(E, k);
  return (T + ctok - 1) / ctok;
}

template <int EM, bool ALONE, bool K8>
cudaError_t place_run(const OrderParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> set{0};
  constexpr size_t smem = K8 ? PlaceGeo<EM>::SMEM8 : PlaceGeo<EM>::SMEM;
  const cudaError_t e = smem_optin(order_place_kernel<EM, ALONE, K8>, (int)smem, set);
  if (e != cudaSuccess) return e;
  return launch_pdl(order_place_kernel<EM, ALONE, K8>, dim3(p.L * p.nchunk), dim3(EO_THREADS), smem, st, p);
}
template <bool ALONE>
cudaError_t place(const OrderParams& p, cudaStream_t st) {
  if (p.k == 8)
    return p.E <= 64    ? place_run<64, ALONE, true>(p, st)
           : p.E <= 128 ? place_run<128, ALONE, true>(p, st)
                        : place_run<256, ALONE, true>(p, st);
  return p.E <= 64    ? place_run<64, ALONE, false>(p, st)
         : p.E <= 128 ? place_run<128, ALONE, false>(p, st)
                      : place_run<256, ALONE, false>(p, st);
}
}  // namespace

size_t expert_order_scratch_bytes(const moer_dims* d, int64_t T) {
  return (size_t)d->L * (size_t)order_chunks(d->E, d->k, T) * (size_t)d->E * 4;
}

moer_status expert_order_launch(const moer_dims* d, const uint8_t* topk, int64_t T, int32_t align, int32_t* off,
                                int32_t* order, int64_t ld, int32_t* inv, void* ws, cudaStream_t st) {
  OrderParams p;
  p.ids = topk;
  p.N = (int)(T * d->k);
  p.E = d->E;
  p.L = d->L;
  p.k = d->k;
  p.T = (int)T;
  p.ctok = order_ctok(d->E, d->k);
  p.align = align;
  p.nchunk = (int)order_chunks(d->E, d->k, T);
  p.vec = reinterpret_cast<uintptr_t>(topk) % 16 == 0 && reinterpret_cast<uintptr_t>(inv) % 16 == 0 &&
          (p.L == 1 || p.N % 16 == 0);
  p.pairs = p.k % 2 == 0 && reinterpret_cast<uintptr_t>(inv) % 8 == 0;
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
