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
// The sums: a block scans 1,024 requests (four to a thread) from the sum of those
// before them, which it makes by itself in batches of up to 4,096 requests; in
// larger ones a launch before it has summed every block's own.
// The fill: a block of 256 threads takes 256 KV blocks.  A thread to a KV block
// finds its request (two warps bracket the block's requests by a 32-way search,
// the thread searches between them), its page and its first token; then the
// tokens are written by as many lanes to a KV block as it has tokens (a power of
// two, 32 at most), from what was found once.  Finding request and page for
// every four tokens instead took five times the instructions.
// Measured (GB300): 14,000 requests, 12.9 M tokens in 0.8 M KV blocks with slots, owners
// and positions (227 MB): 50 us, 4.6 TB/s, 0.67 of the copy bandwidth; the sums take
// 8 us of it, the fill's stores (16 bytes a token) the rest.  256 requests with one
// new token each: 6.0 us in the small form, a chain of dependent steps.
// Small batches take one launch: one block does it all, in shared memory.
#include "common.cuh"
#include "pdl.cuh"

namespace moer {

namespace {
constexpr int BP_THREADS = 256;
constexpr int BP_EACH = 4;                       // requests of a thread in the scan
constexpr int BP_CHUNK = BP_THREADS * BP_EACH;   // of a block
constexpr int SMALL_R = BP_CHUNK;                // requests of a small batch,
constexpr int BP_ALONE = 4;                      // chunks up to which a block sums those before it by itself
constexpr int64_t SMALL_ITEMS = 8192;            // its tokens and blocks

// What the fill reads of the requests: the caller's arrays and the sums, or a
// small batch's copies in shared memory.
struct Tables {
  const int32_t *new_len, *ctx_len;  // ctx_len may be NULL
  const int32_t *req, *blk, *cac, *taken;  // [R+1]
};

struct PlanParams {
  moer_block_plan_args a;
  uint32_t mul, shift;     // x / B = (x mul) >> (32 + shift) for x < 2^31; shift 32: B = 1
  int32_t* taken_off;      // [R+1]
  uint32_t* status;
  int64_t* partial;        // [chunks][4] sums of each chunk of requests, where
  int summed;              // 1: a launch of its own has made them
  int vec_len;             // 1: the lengths take vector loads
  int vec_tab;             // 1: blk_tab's pairs are on 8 bytes
  int lanes;               // to a KV block when tokens are written: a power of two
  // blocks that have room, or whose tokens have (b blocks hold b tokens at least): a batch
  // of absurd lengths has up to 2^31 more, of which only pages are written
  int limit;
};

// x / B for x < 2^31: with s = ceil(log2 B) the multiplier is floor(2^(31 + s) / B) + 1,
// whose excess over 2^(31 + s) / B, at most 1, times x / 2^(31 + s) stays below 1 / B.
__device__ __forceinline__ uint32_t div_b(const PlanParams& p, uint32_t x) {
  return p.shift < 32u ? __umulhi(x, p.mul) >> p.shift : x;
}

struct Request {
  uint32_t c, n;  // tokens held, tokens computed: their sum is below 2^31
};

__device__ __forceinline__ Request request(int n, int c, bool& bad) {
  if (n < 0 || c < 0 || max(n, 0) > 0x7FFFFFFF - max(c, 0)) bad = true;
  const uint32_t held = (uint32_t)max(c, 0);
  return {held, min((uint32_t)max(n, 0), 0x7FFFFFFFu - held)};  // positions are int32
}

__device__ __forceinline__ Request request(const Tables& t, int r) {
  bool bad;
  return request(t.new_len[r], t.ctx_len != nullptr ? t.ctx_len[r] : 0, bad);
}

// Four neighbouring lengths from r on, 0 past the end or where there are none.
__device__ __forceinline__ int4 four(const int32_t* len, int R, int r, int vec) {
  if (len == nullptr) return make_int4(0, 0, 0, 0);
  if (vec != 0 && r + 4 <= R) return *reinterpret_cast<const int4*>(len + r);
  return make_int4(r < R ? len[r] : 0, r + 1 < R ? len[r + 1] : 0, r + 2 < R ? len[r + 2] : 0,
                   r + 3 < R ? len[r + 3] : 0);
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

// Sums of four values over the block; every thread returns them.
__device__ __forceinline__ void block_sums(int64_t (&x)[4], int64_t (*wsum)[BP_THREADS / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x[k] += __shfl_xor_sync(FULL, x[k], o);
    if (lane == 0) wsum[k][warp] = x[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[k] = 0;
#pragma unroll
    for (int w = 0; w < BP_THREADS / 32; ++w) x[k] += wsum[k][w];
  }
  __syncthreads();
}

// The four requests of a thread, and whether their lengths or tables are bad.
struct Four {
  uint32_t s[BP_EACH][4];
  int n[BP_EACH], c[BP_EACH];
  bool bad;
};
__device__ __forceinline__ Four four_requests(const PlanParams& p, int r0) {
  const moer_block_plan_args& a = p.a;
  const int4 n4 = four(a.new_len, a.R, r0, p.vec_len), c4 = four(a.ctx_len, a.R, r0, p.vec_len);
  Four f = {{}, {n4.x, n4.y, n4.z, n4.w}, {c4.x, c4.y, c4.z, c4.w}, false};
#pragma unroll
  for (int i = 0; i < BP_EACH; ++i) {
    const Request q = request(f.n[i], f.c[i], f.bad);
    if (a.pages != nullptr && pages_of(p, q.c + q.n) > (uint32_t)a.ld_pages) f.bad = true;
    sums_of(p, q, f.s[i]);
  }
  return f;
}

__global__ void __launch_bounds__(BP_THREADS) plan_sum_kernel(const PlanParams p) {
  __shared__ int64_t wsum[4][BP_THREADS / 32];
  pdl_wait();
  const Four f = four_requests(p, (int)blockIdx.x * BP_CHUNK + (int)threadIdx.x * BP_EACH);
  int64_t x[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < BP_EACH; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] += f.s[i][k];
  block_sums(x, wsum);
  if (threadIdx.x == 0)
#pragma unroll
    for (int k = 0; k < 4; ++k) p.partial[(int64_t)blockIdx.x * 4 + k] = x[k];
  pdl_release();
}

// The offsets of the block's requests; `keep` (a small batch): copies of the lengths
// and offsets in shared memory, SMALL_R + 1 of each.
__device__ __forceinline__ void scan_requests(const PlanParams& p, int32_t* keep) {
  __shared__ int64_t wsum[4][BP_THREADS / 32];
  const moer_block_plan_args& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = (int)blockIdx.x * BP_CHUNK + (int)threadIdx.x * BP_EACH;
  int64_t base[4] = {0, 0, 0, 0};
  if (blockIdx.x > 0) {
    if (p.summed != 0) {
      for (int c = threadIdx.x; c < (int)blockIdx.x; c += BP_THREADS)
#pragma unroll
        for (int k = 0; k < 4; ++k) base[k] += p.partial[(int64_t)c * 4 + k];
    } else {
      for (int r = (int)threadIdx.x * BP_EACH; r < (int)blockIdx.x * BP_CHUNK; r += BP_CHUNK) {
        const Four f = four_requests(p, r);
#pragma unroll
        for (int i = 0; i < BP_EACH; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) base[k] += f.s[i][k];
      }
    }
    block_sums(base, wsum);
  }
  const Four f = four_requests(p, r0);
  bool bad = f.bad;
  int64_t x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t own = (int64_t)f.s[0][k] + f.s[1][k] + f.s[2][k] + f.s[3][k];
    int64_t y = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(FULL, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) wsum[k][warp] = y;
    x[k] = y - own;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[k] += base[k];
#pragma unroll
    for (int w = 0; w < BP_THREADS / 32; ++w) {
      if (w < warp) x[k] += wsum[k][w];
      base[k] += wsum[k][w];
    }
  }
#pragma unroll
  for (int i = 0; i < BP_EACH; ++i)
    if (r0 + i < a.R) {
      const int r = r0 + i;
      a.req_off[r] = clamp32(x[0]);
      a.req_blk_off[r] = clamp32(x[1]);
      if (a.req_cache_off != nullptr) a.req_cache_off[r] = clamp32(x[2]);
      if (keep != nullptr) {
        keep[r] = f.n[i];
        keep[SMALL_R + 1 + r] = f.c[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) keep[(2 + k) * (SMALL_R + 1) + r] = clamp32(x[k]);
      } else {
        p.taken_off[r] = clamp32(x[3]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] += f.s[i][k];
    }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
    a.req_off[a.R] = clamp32(base[0]);
    a.req_blk_off[a.R] = clamp32(base[1]);
    if (a.req_cache_off != nullptr) a.req_cache_off[a.R] = clamp32(base[2]);
    p.taken_off[a.R] = clamp32(base[3]);
    if (keep != nullptr)
      for (int k = 0; k < 4; ++k) keep[(2 + k) * (SMALL_R + 1) + a.R] = clamp32(base[k]);
    if (a.totals != nullptr)
      for (int k = 0; k < 4; ++k) a.totals[k] = clamp32(base[k]);
    if (base[0] > a.T || base[1] > a.nblk || (a.cache_idx != nullptr && base[2] > a.ncached) ||
        (a.free_pages != nullptr && base[3] > a.n_free))
      bad = true;
  }
  if (bad) atomicOr(p.status, WS_BIT_EDATA);
}

__global__ void __launch_bounds__(BP_THREADS) plan_scan_kernel(const PlanParams p) {
  pdl_wait();
  scan_requests(p, nullptr);
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
__device__ __forceinline__ int page_of(const PlanParams& p, const Tables& tb, int r, uint32_t held, uint32_t i) {
  const moer_block_plan_args& a = p.a;
  if (i >= (uint32_t)a.ld_pages) return -1;
  if (a.free_pages != nullptr && i >= held) {
    const int64_t f = (int64_t)tb.taken[r] + (i - held);
    return f < a.n_free ? a.free_pages[f] : -1;
  }
  return a.pages[(int64_t)r * a.ld_pages + i];
}

// The requests of items i0 and i0 + n - 1, by two warps; every thread calls it.
__device__ __forceinline__ void find_range(const int32_t* off, int R, int i0, int n, int* range) {
  if (threadIdx.x < 64) {
    const int w = threadIdx.x >> 5;
    const int r = find_warp(off, R, i0 + (w == 0 ? 0 : n - 1));
    if ((threadIdx.x & 31) == 0) range[w] = r;
  }
  __syncthreads();
}

// A KV block's tokens: the first one's slot (-1: no page), number and position, how
// many there is room for, and their request.
struct Run {
  int64_t slot;
  int tok0, len, pos, req;
};

// New pages of the blocks from `last` on, as far as the table reaches.
__device__ __forceinline__ void fill_pages(const PlanParams& p, const Tables& tb, int last) {
  const moer_block_plan_args& a = p.a;
  for (int64_t r = (int64_t)blockIdx.x * BP_THREADS + threadIdx.x; r < a.R; r += (int64_t)gridDim.x * BP_THREADS) {
    const Request q = request(tb, (int)r);
    const uint32_t held = pages_of(p, q.c), end = min(pages_of(p, q.c + q.n), (uint32_t)a.ld_pages);
    const uint32_t past = (uint32_t)max(last - tb.blk[r], 0);  // its blocks that are done
    for (uint32_t i = max(held, div_b(p, q.c) + past); i < end; ++i)
      a.pages[r * a.ld_pages + i] = page_of(p, tb, (int)r, held, i);
  }
}

// The batch's KV blocks, and with each its tokens.
__device__ void fill_blocks(const PlanParams& p, const Tables& tb) {
  __shared__ Run runs[BP_THREADS];
  __shared__ int range[2];
  const moer_block_plan_args& a = p.a;
  const int nblk = tb.blk[a.R];
  const bool tokens = a.slot_map != nullptr || a.tok_req != nullptr || a.tok_pos != nullptr;
  const uint32_t B = (uint32_t)a.block;
  const int room = (int)min64(a.T, 0x7FFFFFFF);
  const int last = min(nblk, p.limit);
  for (int64_t b0 = (int64_t)blockIdx.x * BP_THREADS; b0 < last; b0 += (int64_t)gridDim.x * BP_THREADS) {
    const int n = (int)min64(BP_THREADS, last - b0);
    find_range(tb.blk, a.R, (int)b0, n, range);
    if ((int)threadIdx.x < n) {
      const int b = (int)b0 + (int)threadIdx.x;
      const int r = find(tb.blk, range[0], range[1] + 1, b);
      const Request q = request(tb, r);
      const uint32_t i = div_b(p, q.c) + (uint32_t)(b - tb.blk[r]);
      const uint32_t lo = max(i * B, q.c), hi = min(i * B + B, q.c + q.n);
      const int tok0 = clamp32((int64_t)tb.req[r] + (lo - q.c)), len = (int)(hi - lo);
      int page = -1;
      if (a.pages != nullptr) {
        const uint32_t held = pages_of(p, q.c);
        page = page_of(p, tb, r, held, i);
        if (a.free_pages != nullptr && i >= held && i < (uint32_t)a.ld_pages)
          a.pages[(int64_t)r * a.ld_pages + i] = page;
      }
      if (b < a.nblk) {
        if (p.vec_tab != 0) {
          *reinterpret_cast<int2*>(a.blk_tab + 2 * (int64_t)b) = make_int2(tok0, len);
        } else {
          a.blk_tab[2 * (int64_t)b] = tok0;
          a.blk_tab[2 * (int64_t)b + 1] = len;
        }
        if (a.insert_slot != nullptr) a.insert_slot[b] = len == a.block ? page : -1;
      }
      runs[threadIdx.x] = {page >= 0 ? (int64_t)page * a.block + (lo - i * B) : -1, tok0,
                           min(len, max(room - tok0, 0)), (int)lo, r};
    }
    __syncthreads();
    if (tokens) {
      // W lanes to a KV block, and all its tokens in one go unless it has more than 32
      const int W = p.lanes, o0 = (int)threadIdx.x & (W - 1), step = BP_THREADS / W;
      auto write = [&](const Run& u, int o) {
        const int t = u.tok0 + o;
        if (a.slot_map != nullptr) a.slot_map[t] = u.slot >= 0 ? u.slot + o : -1;
        if (a.tok_req != nullptr) a.tok_req[t] = u.req;
        if (a.tok_pos != nullptr) a.tok_pos[t] = u.pos + o;
      };
      if (a.block <= 32) {
#pragma unroll 4
        for (int k = (int)threadIdx.x / W; k < n; k += step) {
          const Run u = runs[k];
          if (o0 < u.len) write(u, o0);
        }
      } else {
        for (int k = (int)threadIdx.x / W; k < n; k += step) {
          const Run u = runs[k];
          for (int o = o0; o < u.len; o += W) write(u, o);
        }
      }
    }
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * BP_THREADS, first = (int64_t)blockIdx.x * BP_THREADS + threadIdx.x;
  if (last < nblk && a.pages != nullptr && a.free_pages != nullptr) fill_pages(p, tb, last);
  // room that the batch leaves
  for (int64_t t = tb.req[a.R] + first; t < a.T; t += step) {
    if (a.slot_map != nullptr) a.slot_map[t] = -1;
    if (a.tok_req != nullptr) a.tok_req[t] = -1;
    if (a.tok_pos != nullptr) a.tok_pos[t] = -1;
  }
  for (int64_t b = nblk + first; b < a.nblk; b += step) {
    a.blk_tab[2 * b] = tb.req[a.R];
    a.blk_tab[2 * b + 1] = 0;
    if (a.insert_slot != nullptr) a.insert_slot[b] = -1;
  }
}

__device__ void fill_cached(const PlanParams& p, const Tables& tb) {
  __shared__ int range[2];
  const moer_block_plan_args& a = p.a;
  const int nc = tb.cac[a.R];
  constexpr int ITEMS = BP_THREADS * 4;
  for (int64_t i0 = (int64_t)blockIdx.x * ITEMS; i0 < a.ncached; i0 += (int64_t)gridDim.x * ITEMS) {
    const int n = (int)max64(0, min64(ITEMS, nc - i0));
    if (n > 0) find_range(tb.cac, a.R, (int)i0, n, range);
    for (int k = threadIdx.x; k < ITEMS && i0 + k < a.ncached; k += BP_THREADS) {
      int page = -1;
      if (k < n) {
        const int r = find(tb.cac, range[0], range[1] + 1, (int)i0 + k);
        const int i = (int)i0 + k - tb.cac[r];
        if (i < a.ld_pages) page = a.pages[(int64_t)r * a.ld_pages + i];
      }
      a.cache_idx[i0 + k] = page;
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(BP_THREADS) plan_fill_kernel(const PlanParams p) {
  pdl_wait();
  const Tables tb = {p.a.new_len, p.a.ctx_len, p.a.req_off, p.a.req_blk_off, p.a.req_cache_off, p.taken_off};
  fill_blocks(p, tb);
  if (p.a.cache_idx != nullptr) fill_cached(p, tb);
  pdl_release();
}

__global__ void __launch_bounds__(BP_THREADS) plan_small_kernel(const PlanParams p) {
  __shared__ int32_t keep[6 * (SMALL_R + 1)];
  pdl_wait();
  scan_requests(p, keep);
  __syncthreads();
  constexpr int S = SMALL_R + 1;
  const Tables tb = {keep, keep + S, keep + 2 * S, keep + 3 * S, keep + 4 * S, keep + 5 * S};
  fill_blocks(p, tb);
  if (p.a.cache_idx != nullptr) fill_cached(p, tb);
  pdl_release();
}

bool on16(const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }
}  // namespace

// The pages taken before each request, then the chunks' sums.
size_t block_plan_scratch_bytes(int32_t R) {
  const size_t chunks = ((size_t)R + BP_CHUNK - 1) / BP_CHUNK;
  return (((size_t)R + 1) * 4 + 15) / 16 * 16 + chunks * 4 * sizeof(int64_t);
}

moer_status block_plan_launch(const moer_block_plan_args* a, void* ws, cudaStream_t st) {
  PlanParams p;
  p.a = *a;
  const unsigned long long B = (unsigned long long)a->block;
  uint32_t log = 0u;
  while ((1ull << log) < B) ++log;
  p.mul = B == 1 ? 0u : (uint32_t)((1ull << (31u + log)) / B + 1ull);
  p.shift = B == 1 ? 32u : log - 1u;
  p.lanes = 1 << (log < 5u ? log : 5u);
  const bool tokens = a->slot_map != nullptr || a->tok_req != nullptr || a->tok_pos != nullptr;
  p.limit = (int)max64(a->nblk, tokens ? a->T : 0);
  p.status = static_cast<uint32_t*>(ws);
  char* scratch = static_cast<char*>(ws) + WS_HEADER;
  p.taken_off = reinterpret_cast<int32_t*>(scratch);
  p.partial = reinterpret_cast<int64_t*>(scratch + (((size_t)a->R + 1) * 4 + 15) / 16 * 16);
  p.vec_len = on16(a->new_len) && on16(a->ctx_len);
  p.vec_tab = reinterpret_cast<uintptr_t>(a->blk_tab) % 8 == 0;
  const dim3 block(BP_THREADS);
  if (a->R <= SMALL_R && a->T + a->nblk + a->ncached <= SMALL_ITEMS)
    return launch_pdl(plan_small_kernel, dim3(1), block, 0, st, p) == cudaSuccess ? MOER_OK : MOER_ECUDA;
  const int chunks = a->R > BP_CHUNK ? (a->R + BP_CHUNK - 1) / BP_CHUNK : 1;
  p.summed = chunks > BP_ALONE;
  cudaError_t e = p.summed != 0 ? launch_pdl(plan_sum_kernel, dim3(chunks), block, 0, st, p) : cudaSuccess;
  if (e == cudaSuccess) e = launch_pdl(plan_scan_kernel, dim3(chunks), block, 0, st, p);
  // a block to 256 KV blocks (their number is at most nblk where the batch fits)
  const int64_t fill = max64(1, (max64(a->nblk, a->ncached / 4) + BP_THREADS - 1) / BP_THREADS);
  if (e == cudaSuccess) e = launch_pdl(plan_fill_kernel, dim3((unsigned)fill), block, 0, st, p);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
