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
// Two kernels.  The sums: a block scans 4,096 requests, four to a thread, after
// adding up the lengths of all requests before them by itself (a few
// thousand requests are a few reads of L2; a chain of blocks would cost more).
// The fill: a block takes 2,048 neighbouring tokens (then blocks, then cached
// blocks); two warps find the first and the last one's request by a 32-way
// search, and a thread searches between them only, once for the four tokens
// that it writes with vector stores.  It is bound by the stores (16 bytes a token).
#include "common.cuh"
#include "pdl.cuh"

namespace moer {

namespace {
constexpr int BP_SCAN = 1024;
constexpr int BP_EACH = 4;                     // requests of a thread in the scan
constexpr int BP_CHUNK = BP_SCAN * BP_EACH;
constexpr int BP_FILL = 256;
constexpr int BP_ITEMS = 2048;                 // tokens or blocks of a fill block
constexpr int BP_SMALL = 4;                    // fill blocks that one block does by itself

struct PlanParams {
  moer_block_plan_args a;
  uint32_t mul, shift;     // x / B = (x mul) >> (32 + shift) for x < 2^31; shift 32: B = 1
  int32_t* taken_off;      // [R+1]
  uint32_t* status;
  int vec;                 // 1: the token maps take vector stores
  int tok_blocks, blk_blocks;  // fill blocks of tokens, of blocks
};

// x / B for x < 2^31: with s = ceil(log2 B) the multiplier is floor(2^(31 + s) / B) + 1,
// whose excess over 2^(31 + s) / B, at most 1, times x / 2^(31 + s) stays below 1 / B.
__device__ __forceinline__ uint32_t div_b(const PlanParams& p, uint32_t x) {
  return p.shift < 32u ? __umulhi(x, p.mul) >> p.shift : x;
}

struct Request {
  uint32_t c, n;  // tokens held, tokens computed: their sum is below 2^31
};

__device__ __forceinline__ Request request(const PlanParams& p, int r, bool& bad) {
  const int n = p.a.new_len[r], c = p.a.ctx_len != nullptr ? p.a.ctx_len[r] : 0;
  if (n < 0 || c < 0 || max(n, 0) > 0x7FFFFFFF - max(c, 0)) bad = true;
  const uint32_t held = (uint32_t)max(c, 0);
  return {held, min((uint32_t)max(n, 0), 0x7FFFFFFFu - held)};  // positions are int32
}

// Pages that x tokens touch, x < 2^31.
__device__ __forceinline__ uint32_t pages_of(const PlanParams& p, uint32_t x) {
  return x > 0u ? div_b(p, x - 1u) + 1u : 0u;
}

// Tokens, blocks, cached blocks and pages taken of a request.
__device__ __forceinline__ void sums_of(const PlanParams& p, const Request& q, uint32_t (&s)[4]) {
  const uint32_t whole = div_b(p, q.c), rest = q.c - whole * (uint32_t)p.a.block;
  s[0] = q.n;
  s[1] = q.n > 0u ? pages_of(p, rest + q.n) : 0u;  // rest + n <= c + n
  s[2] = whole;
  s[3] = pages_of(p, q.c + q.n) - pages_of(p, q.c);
}

__device__ __forceinline__ int32_t clamp32(int64_t v) { return (int32_t)min64(v, 0x7FFFFFFF); }

// The sums, by gridDim.x blocks of 1,024 threads.
__device__ __forceinline__ void scan_requests(const PlanParams& p) {
  __shared__ int64_t wsum[2][4][BP_SCAN / 32];
  const moer_block_plan_args& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = (int)blockIdx.x * BP_CHUNK + (int)threadIdx.x * BP_EACH;
  bool bad = false;
  // the thread's requests, and its share of those before the block's
  uint32_t s[BP_EACH][4];
  int64_t x[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < BP_EACH; ++i) {
    Request q = {0u, 0u};
    if (r0 + i < a.R) {
      q = request(p, r0 + i, bad);
      if (a.pages != nullptr && pages_of(p, q.c + q.n) > (uint32_t)a.ld_pages) bad = true;
    }
    sums_of(p, q, s[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] += s[i][k];
  }
  for (int r = threadIdx.x; r < (int)blockIdx.x * BP_CHUNK; r += BP_SCAN) {
    uint32_t v[4];
    sums_of(p, request(p, r, bad), v);
#pragma unroll
    for (int k = 0; k < 4; ++k) before[k] += v[k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    int64_t y = x[k], b = before[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(FULL, y, o);
      if (lane >= o) y += z;
    }
    if (blockIdx.x > 0)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(FULL, b, o);
    if (lane == 31) wsum[0][k][warp] = y, wsum[1][k][warp] = b;
    x[k] = y - x[k];  // of the warp's earlier threads
  }
  __syncthreads();
  // one warp for each of the four: the warps' sums, scanned from the sum before the block
  if (warp < 4) {
    const int64_t y = wsum[0][warp][lane];
    int64_t z = y, b = wsum[1][warp][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(FULL, z, o);
      if (lane >= o) z += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(FULL, b, o);
    wsum[0][warp][lane] = b + z - y;
    if (lane == 31) wsum[1][warp][0] = b + z;  // up to the block's end
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] += wsum[0][k][warp];
#pragma unroll
  for (int i = 0; i < BP_EACH; ++i)
    if (r0 + i < a.R) {
      a.req_off[r0 + i] = clamp32(x[0]);
      a.req_blk_off[r0 + i] = clamp32(x[1]);
      if (a.req_cache_off != nullptr) a.req_cache_off[r0 + i] = clamp32(x[2]);
      p.taken_off[r0 + i] = clamp32(x[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] += s[i][k];
    }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
    const int64_t t[4] = {wsum[1][0][0], wsum[1][1][0], wsum[1][2][0], wsum[1][3][0]};
    a.req_off[a.R] = clamp32(t[0]);
    a.req_blk_off[a.R] = clamp32(t[1]);
    if (a.req_cache_off != nullptr) a.req_cache_off[a.R] = clamp32(t[2]);
    p.taken_off[a.R] = clamp32(t[3]);
    if (a.totals != nullptr)
      for (int k = 0; k < 4; ++k) a.totals[k] = clamp32(t[k]);
    if (t[0] > a.T || t[1] > a.nblk || (a.cache_idx != nullptr && t[2] > a.ncached) ||
        (a.free_pages != nullptr && t[3] > a.n_free))
      bad = true;
  }
  if (bad) atomicOr(p.status, WS_BIT_EDATA);
}

__global__ void __launch_bounds__(BP_SCAN) plan_scan_kernel(const PlanParams p) {
  pdl_wait();
  scan_requests(p);
  pdl_release();
}

// Largest r in [lo, hi) with off[r] <= i, where off[lo] <= i.
__device__ __forceinline__ int find(const int32_t* off, int lo, int hi, int i) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The same over [0, R) by a warp: 32 probes at a time, each step leaves one of
// 32 parts.  Every lane returns the result.
__device__ __forceinline__ int find_warp(const int32_t* off, int R, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = R;
  while (n > 1) {
    const int part = (n + 31) >> 5;
    const int at = lo + lane * part;
    const bool le = lane * part < n && off[at] <= i;
    const int last = 31 - __clz(__ballot_sync(FULL, le) | 1u);
    lo += last * part;
    n = min(part, n - last * part);
  }
  return lo;
}

// The page of a request's page number: held pages from the table, new ones
// from free_pages (or from the table where that is complete); -1 if there is none.
__device__ __forceinline__ int page_of(const PlanParams& p, int r, uint32_t held, uint32_t i) {
  const moer_block_plan_args& a = p.a;
  if (i >= (uint32_t)a.ld_pages) return -1;
  if (a.free_pages != nullptr && i >= held) {
    const int64_t f = (int64_t)p.taken_off[r] + (i - held);
    return f < a.n_free ? a.free_pages[f] : -1;
  }
  return a.pages[(int64_t)r * a.ld_pages + i];
}

// Walks over neighbouring tokens: the request, and the slot on its page.
struct Walk {
  int r;
  int64_t end;             // first token past the request
  uint32_t pos, page_no, held, rest;
  int page;
  __device__ __forceinline__ void enter(const PlanParams& p, int request_no, int t) {
    bool bad;
    r = request_no;
    const Request q = request(p, r, bad);
    const int at = p.a.req_off[r];
    end = (int64_t)at + q.n;
    pos = q.c + (uint32_t)(t - at);
    held = pages_of(p, q.c);
    page_no = div_b(p, pos);
    rest = pos - page_no * (uint32_t)p.a.block;
    page = p.a.slot_map != nullptr ? page_of(p, r, held, page_no) : -1;
  }
  // to token t, the one after the last
  __device__ __forceinline__ void next(const PlanParams& p, int t) {
    ++pos;
    if (t >= end) {
      int q = r + 1;
      while (p.a.req_off[q + 1] <= t) ++q;  // requests without tokens
      enter(p, q, t);
    } else if (++rest == (uint32_t)p.a.block) {
      rest = 0u;
      ++page_no;
      if (p.a.slot_map != nullptr) page = page_of(p, r, held, page_no);
    }
  }
};

__device__ void fill_tokens(const PlanParams& p, int64_t i0, int* range) {
  const moer_block_plan_args& a = p.a;
  const int T = a.req_off[a.R];
  const int n_in = (int)max64(0, min64(BP_ITEMS, T - i0));  // of the block's tokens
  if (threadIdx.x < 64 && n_in > 0) {
    const int w = threadIdx.x >> 5;
    const int r = find_warp(a.req_off, a.R, (int)i0 + (w == 0 ? 0 : n_in - 1));
    if ((threadIdx.x & 31) == 0) range[w] = r;
  }
  __syncthreads();
  for (int k = (int)threadIdx.x * 4; k < BP_ITEMS; k += (int)blockDim.x * 4) {
    const int64_t t0 = i0 + k;
    if (t0 >= a.T) break;
    int64_t slot[4] = {-1, -1, -1, -1};
    int req[4] = {-1, -1, -1, -1}, pos[4] = {-1, -1, -1, -1};
    if (k < n_in) {
      Walk w;
      w.enter(p, find(a.req_off, range[0], range[1] + 1, (int)t0), (int)t0);
      if (t0 + 4 <= w.end && w.rest + 4u <= (uint32_t)a.block) {
        // all four on one page of one request
        const int64_t s0 = w.page >= 0 ? (int64_t)w.page * a.block + w.rest : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          req[j] = w.r;
          pos[j] = (int)w.pos + j;
          slot[j] = s0 >= 0 ? s0 + j : -1;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k + j < n_in) {
            if (j > 0) w.next(p, (int)t0 + j);
            req[j] = w.r;
            pos[j] = (int)w.pos;
            if (w.page >= 0) slot[j] = (int64_t)w.page * a.block + w.rest;
          }
      }
    }
    if (p.vec != 0 && t0 + 4 <= a.T) {
      if (a.slot_map != nullptr) {
        *reinterpret_cast<longlong2*>(a.slot_map + t0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(a.slot_map + t0 + 2) = make_longlong2(slot[2], slot[3]);
      }
      if (a.tok_req != nullptr) *reinterpret_cast<int4*>(a.tok_req + t0) = make_int4(req[0], req[1], req[2], req[3]);
      if (a.tok_pos != nullptr) *reinterpret_cast<int4*>(a.tok_pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t0 + j < a.T) {
          if (a.slot_map != nullptr) a.slot_map[t0 + j] = slot[j];
          if (a.tok_req != nullptr) a.tok_req[t0 + j] = req[j];
          if (a.tok_pos != nullptr) a.tok_pos[t0 + j] = pos[j];
        }
    }
  }
}

__device__ void fill_blocks(const PlanParams& p, int64_t i0, int* range) {
  const moer_block_plan_args& a = p.a;
  const int T = a.req_off[a.R], nblk = a.req_blk_off[a.R];
  const int n_in = (int)max64(0, min64(BP_ITEMS, nblk - i0));
  if (threadIdx.x < 64 && n_in > 0) {
    const int w = threadIdx.x >> 5;
    const int r = find_warp(a.req_blk_off, a.R, (int)i0 + (w == 0 ? 0 : n_in - 1));
    if ((threadIdx.x & 31) == 0) range[w] = r;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < BP_ITEMS && i0 + k < a.nblk; k += (int)blockDim.x) {
    const int64_t b = i0 + k;
    int tok0 = T, len = 0, slot = -1;
    if (k < n_in) {
      bool bad;
      const int r = find(a.req_blk_off, range[0], range[1] + 1, (int)b);
      const Request q = request(p, r, bad);
      const uint32_t B = (uint32_t)a.block, i = div_b(p, q.c) + (uint32_t)(b - a.req_blk_off[r]);
      const uint32_t lo = max(i * B, q.c), hi = min(i * B + B, q.c + q.n);
      tok0 = clamp32((int64_t)a.req_off[r] + (lo - q.c));
      len = (int)(hi - lo);
      if (a.pages != nullptr) {
        const uint32_t held = pages_of(p, q.c);
        const int page = page_of(p, r, held, i);
        if (len == a.block) slot = page;
        if (a.free_pages != nullptr && i >= held && i < (uint32_t)a.ld_pages)
          a.pages[(int64_t)r * a.ld_pages + i] = page;
      }
    }
    a.blk_tab[2 * b] = tok0;
    a.blk_tab[2 * b + 1] = len;
    if (a.insert_slot != nullptr) a.insert_slot[b] = slot;
  }
}

__device__ void fill_cached(const PlanParams& p, int64_t i0, int* range) {
  const moer_block_plan_args& a = p.a;
  const int nc = a.req_cache_off[a.R];
  const int n_in = (int)max64(0, min64(BP_ITEMS, nc - i0));
  if (threadIdx.x < 64 && n_in > 0) {
    const int w = threadIdx.x >> 5;
    const int r = find_warp(a.req_cache_off, a.R, (int)i0 + (w == 0 ? 0 : n_in - 1));
    if ((threadIdx.x & 31) == 0) range[w] = r;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < BP_ITEMS && i0 + k < a.ncached; k += (int)blockDim.x) {
    int page = -1;
    if (k < n_in) {
      const int r = find(a.req_cache_off, range[0], range[1] + 1, (int)i0 + k);
      const int i = (int)i0 + k - a.req_cache_off[r];
      if (i < a.ld_pages) page = a.pages[(int64_t)r * a.ld_pages + i];
    }
    a.cache_idx[i0 + k] = page;
  }
}

__global__ void __launch_bounds__(BP_FILL) plan_fill_kernel(const PlanParams p) {
  __shared__ int range[2];  // requests of the block's first and last item
  pdl_wait();
  const int b = (int)blockIdx.x;
  if (b < p.tok_blocks)
    fill_tokens(p, (int64_t)b * BP_ITEMS, range);
  else if (b < p.tok_blocks + p.blk_blocks)
    fill_blocks(p, (int64_t)(b - p.tok_blocks) * BP_ITEMS, range);
  else
    fill_cached(p, (int64_t)(b - p.tok_blocks - p.blk_blocks) * BP_ITEMS, range);
  pdl_release();
}

// Small batches: one block makes the sums and then fills the tables itself.
__global__ void __launch_bounds__(BP_SCAN) plan_small_kernel(const PlanParams p) {
  __shared__ int range[2];
  pdl_wait();
  scan_requests(p);
  __syncthreads();  // the sums in global memory are this block's own
  for (int b = 0; b < p.tok_blocks; ++b) {
    fill_tokens(p, (int64_t)b * BP_ITEMS, range);
    __syncthreads();
  }
  for (int b = 0; b < p.blk_blocks; ++b) {
    fill_blocks(p, (int64_t)b * BP_ITEMS, range);
    __syncthreads();
  }
  if (p.a.cache_idx != nullptr)
    for (int64_t i = 0; i < p.a.ncached; i += BP_ITEMS) {
      fill_cached(p, i, range);
      __syncthreads();
    }
  pdl_release();
}

bool on16(const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }
}  // namespace

size_t block_plan_scratch_bytes(int32_t R) { return ((size_t)R + 1) * 4; }

moer_status block_plan_launch(const moer_block_plan_args* a, void* ws, cudaStream_t st) {
  PlanParams p;
  p.a = *a;
  const unsigned long long B = (unsigned long long)a->block;
  uint32_t log = 0u;
  while ((1ull << log) < B) ++log;
  p.mul = B == 1 ? 0u : (uint32_t)((1ull << (31u + log)) / B + 1ull);
  p.shift = B == 1 ? 32u : log - 1u;
  p.status = static_cast<uint32_t*>(ws);
  p.taken_off = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + WS_HEADER);
  p.vec = on16(a->slot_map) && on16(a->tok_req) && on16(a->tok_pos);
  const bool tokens = a->slot_map != nullptr || a->tok_req != nullptr || a->tok_pos != nullptr;
  auto blocks = [](int64_t n) { return (n + BP_ITEMS - 1) / BP_ITEMS; };
  p.tok_blocks = tokens ? (int)blocks(a->T) : 0;
  p.blk_blocks = (int)blocks(a->nblk);
  const int64_t fill = (int64_t)p.tok_blocks + p.blk_blocks + (a->cache_idx != nullptr ? blocks(a->ncached) : 0);
  if (a->R <= BP_CHUNK && fill <= BP_SMALL)
    return launch_pdl(plan_small_kernel, dim3(1), dim3(BP_SCAN), 0, st, p) == cudaSuccess ? MOER_OK : MOER_ECUDA;
  const int scan = a->R > BP_CHUNK ? (a->R + BP_CHUNK - 1) / BP_CHUNK : 1;
  cudaError_t e = launch_pdl(plan_scan_kernel, dim3(scan), dim3(BP_SCAN), 0, st, p);
  if (e == cudaSuccess && fill > 0) e = launch_pdl(plan_fill_kernel, dim3((unsigned)fill), dim3(BP_FILL), 0, st, p);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
