// block_plan.cu -- moer_block_plan: the tables of a batch from its requests'
// lengths ([ELDR] section "Key idea / structure / operation": counts per KV
// block, co-indexed with the KV cache).
//
// With c_r tokens held and n_r new ones, page size B and h_r = ceil(c_r / B):
//   tokens   req_off      exclusive sums of n_r
//   blocks   req_blk_off  exclusive sums of ceil((c_r mod B + n_r) / B), 0 if n_r = 0
//   cached   req_cache_off exclusive sums of floor(c_r / B)
//   taken    exclusive sums of ceil((c_r + n_r) / B) - h_r: where a request's
//            new pages start in free_pages.
// Block i of a request lies on page floor(c_r / B) + i; a token's slot follows
// from its position.  A page's id is read from the table where the request
// held it and from free_pages otherwise, so nothing waits for the table's new
// entries to be written.
//
// Two kernels: the sums, then one pass over tokens, blocks and cached blocks.
#include "common.cuh"
#include "pdl.cuh"

namespace moer {

namespace {
constexpr int BP_SCAN = 1024;
constexpr int BP_FILL = 256;

struct Sums {
  int64_t v[4];  // tokens, blocks, cached blocks, pages taken
};

__device__ __forceinline__ int64_t ceil_div(int64_t a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ void request(const moer_block_plan_args& a, int r, int64_t& c, int64_t& n, bool& bad) {
  n = a.new_len[r];
  c = a.ctx_len != nullptr ? a.ctx_len[r] : 0;
  if (n < 0 || c < 0) bad = true;
  n = max64(n, 0);
  c = max64(c, 0);
}

__device__ __forceinline__ Sums sums_of(int64_t c, int64_t n, int B) {
  Sums s;
  s.v[0] = n;
  s.v[1] = n > 0 ? ceil_div(c % B + n, B) : 0;
  s.v[2] = c / B;
  s.v[3] = ceil_div(c + n, B) - ceil_div(c, B);
  return s;
}

__device__ __forceinline__ int32_t clamp32(int64_t v) { return (int32_t)min64(v, 0x7FFFFFFF); }

// One block scans all requests, 1,024 at a time.
__global__ void __launch_bounds__(BP_SCAN) plan_scan_kernel(const moer_block_plan_args a, int32_t* taken_off,
                                                            uint32_t* status) {
  __shared__ int64_t wsum[4][BP_SCAN / 32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t base[4] = {0, 0, 0, 0};
  bool bad = false;
  for (int r0 = 0; r0 < a.R; r0 += BP_SCAN) {
    const int r = r0 + (int)threadIdx.x;
    int64_t c = 0, n = 0;
    if (r < a.R) request(a, r, c, n, bad);
    const Sums s = sums_of(c, n, a.block);
    int64_t x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[q] = s.v[q];
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x[q], o);
        if (lane >= o) x[q] += y;
      }
      if (lane == 31) wsum[q][warp] = x[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      int64_t before = 0, all = 0;
      for (int w = 0; w < BP_SCAN / 32; ++w) {
        if (w < warp) before += wsum[q][w];
        all += wsum[q][w];
      }
      x[q] += base[q] + before - s.v[q];
      base[q] += all;
    }
    if (r < a.R) {
      a.req_off[r] = clamp32(x[0]);
      a.req_blk_off[r] = clamp32(x[1]);
      if (a.req_cache_off != nullptr) a.req_cache_off[r] = clamp32(x[2]);
      taken_off[r] = clamp32(x[3]);
      if (a.pages != nullptr && ceil_div(c + n, a.block) > a.ld_pages) bad = true;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    a.req_off[a.R] = clamp32(base[0]);
    a.req_blk_off[a.R] = clamp32(base[1]);
    if (a.req_cache_off != nullptr) a.req_cache_off[a.R] = clamp32(base[2]);
    taken_off[a.R] = clamp32(base[3]);
    if (a.totals != nullptr)
      for (int q = 0; q < 4; ++q) a.totals[q] = clamp32(base[q]);
    if (base[0] > a.T || base[1] > a.nblk || (a.cache_idx != nullptr && base[2] > a.ncached) ||
        (a.free_pages != nullptr && base[3] > a.n_free))
      bad = true;
  }
  if (bad) atomicOr(status, WS_BIT_EDATA);
  pdl_release();
}

// Largest r with off[r] <= i, for i < off[R].
__device__ __forceinline__ int find(const int32_t* off, int R, int64_t i) {
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The page of a request's page number: held pages from the table, new ones
// from free_pages (or from the table where that is complete); -1 if there is none.
__device__ __forceinline__ int page_of(const moer_block_plan_args& a, const int32_t* taken_off, int r, int64_t c,
                                       int64_t i) {
  if (i >= a.ld_pages) return -1;
  const int64_t h = ceil_div(c, a.block);
  if (a.free_pages != nullptr && i >= h) {
    const int64_t f = taken_off[r] + (i - h);
    return f < a.n_free ? a.free_pages[f] : -1;
  }
  return a.pages[(int64_t)r * a.ld_pages + i];
}

__global__ void __launch_bounds__(BP_FILL) plan_fill_kernel(const moer_block_plan_args a, const int32_t* taken_off) {
  pdl_wait();
  const int64_t T = a.req_off[a.R], nblk = a.req_blk_off[a.R];
  const int64_t step = (int64_t)gridDim.x * BP_FILL, first = (int64_t)blockIdx.x * BP_FILL + threadIdx.x;
  bool bad;
  if (a.slot_map != nullptr || a.tok_req != nullptr || a.tok_pos != nullptr)
    for (int64_t t = first; t < a.T; t += step) {
      int64_t slot = -1, pos = -1;
      int r = -1;
      if (t < T) {
        r = find(a.req_off, a.R, t);
        int64_t c, n;
        request(a, r, c, n, bad);
        pos = c + (t - a.req_off[r]);
        if (a.slot_map != nullptr) {
          const int page = page_of(a, taken_off, r, c, pos / a.block);
          if (page >= 0) slot = (int64_t)page * a.block + pos % a.block;
        }
      }
      if (a.slot_map != nullptr) a.slot_map[t] = slot;
      if (a.tok_req != nullptr) a.tok_req[t] = r;
      if (a.tok_pos != nullptr) a.tok_pos[t] = (int32_t)pos;
    }
  for (int64_t b = first; b < a.nblk; b += step) {
    int tok0 = clamp32(T), len = 0, slot = -1;
    if (b < nblk) {
      const int r = find(a.req_blk_off, a.R, b);
      int64_t c, n;
      request(a, r, c, n, bad);
      const int64_t i = c / a.block + (b - a.req_blk_off[r]);
      const int64_t lo = max64(i * a.block, c), hi = min64((i + 1) * a.block, c + n);
      tok0 = clamp32(a.req_off[r] + (lo - c));
      len = (int)(hi - lo);
      const int page = page_of(a, taken_off, r, c, i);
      if (len == a.block) slot = page;
      if (a.free_pages != nullptr && i >= ceil_div(c, a.block) && i < a.ld_pages)
        a.pages[(int64_t)r * a.ld_pages + i] = page;
    }
    a.blk_tab[2 * b] = tok0;
    a.blk_tab[2 * b + 1] = len;
    if (a.insert_slot != nullptr) a.insert_slot[b] = slot;
  }
  if (a.cache_idx != nullptr) {
    const int64_t nc = a.req_cache_off[a.R];
    for (int64_t j = first; j < a.ncached; j += step) {
      int page = -1;
      if (j < nc) {
        const int r = find(a.req_cache_off, a.R, j);
        const int64_t i = j - a.req_cache_off[r];
        if (i < a.ld_pages) page = a.pages[(int64_t)r * a.ld_pages + i];
      }
      a.cache_idx[j] = page;
    }
  }
  pdl_release();
}
}  // namespace

size_t block_plan_scratch_bytes(int32_t R) { return ((size_t)R + 1) * 4; }

moer_status block_plan_launch(const moer_block_plan_args* a, void* ws, cudaStream_t st) {
  uint32_t* status = static_cast<uint32_t*>(ws);
  int32_t* taken = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + WS_HEADER);
  if (launch_pdl(plan_scan_kernel, dim3(1), dim3(BP_SCAN), 0, st, *a, taken, status) != cudaSuccess)
    return MOER_ECUDA;
  const int64_t n = max64(max64(a->T, a->nblk), a->ncached);
  const int sms = device_sm_count();
  if (sms <= 0) return MOER_ECUDA;
  const int64_t grid = max64(1, min64((n + BP_FILL - 1) / BP_FILL, (int64_t)sms * 8));
  return launch_pdl(plan_fill_kernel, dim3((unsigned)grid), dim3(BP_FILL), 0, st, *a, (const int32_t*)taken) ==
                 cudaSuccess
             ? MOER_OK
             : MOER_ECUDA;
}

}  // namespace moer
