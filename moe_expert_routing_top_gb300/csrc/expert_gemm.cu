// expert_gemm.cu -- moer_expert_gemm: matrix products grouped by expert, over the ragged segments of
// the experts' token lists, on the 5th-generation tensor cores.
//
// Every product is formed as D[m][j] = sum_c A[m][c] * B[j][c], with the output's contiguous
// dimension as m and its rows as j:
//   FORWARD       m = n,  j = list rows, c = k:  A = w[e]      B = x by row
//   GRAD_INPUT    m = k,  j = list rows, c = n:  A = w[e]^T    B = d_out by row
//   GRAD_WEIGHT   m = k,  j = n, c = list rows:  A = x^T       B = d_y^T
// so that the weights fill the wide side of the instruction (256 over a CTA pair) whatever the
// segment's length, and a tile of list rows is as narrow as the segment needs: 16 .. 256 in
// steps of 16.  Transposed operands are not copied: the instruction takes them as they lie
// (m or j contiguous) from 64 x 64 panels.
//
// Clusters of two CTAs, persistent over tiles of 256 m x up to 256 j (tcgen05.mma.cta_group::2,
// M = 256), c in blocks of 128 bytes, six stages of 32 KB.  A CTA loads its 128 of m and half
// of the j rows, all by TMA: listed rows of x by its row gather, which follows the list's entries, so
// no permuted copy of x exists (one made first, in the workspace: 1,432 us for 262,144 rows of
// 2,048 x 1,536, against 1,291), rows without a list in boxes of 32.  Where rows are contracted
// (GRAD_WEIGHT), those past the segment or of padding are gathered from past the map's end, in both
// operands: zeros.  Bound by the operands' arrival: 1.26 to 1.32 PFLOP/s there, 1.37 to 1.46 without a list
// (1.74 sustained by a large library product).
// Accumulators are fp32 in TMEM, two of 256 columns, drained by sixteen warps while the MMAs go
// on.  TMEM sums are cut, not rounded, so that their error grows with their length: after
// 8 blocks (512 terms) a sum is added to fp32 registers (weights' gradient over 1,500 rows: relative
// error 2.2e-6 without that, 5e-7 with it).
// E4M3 adds up after each block of 128, times its two scales.  There the rows of x are the
// instruction's 256 m and the weights its 256 columns, so that a thread, which reads one TMEM lane,
// has one scale of either operand a block; with the scales along the columns their loads from
// shared memory, 1,024 clocks a block, took twice the MMAs' time (2,626 us for 262,144 rows of
// 2,048 x 1,536; this way 1,211).
// Every wait is bounded; on expiry the kernel records MOER_ETIMEOUT and returns.
#include "rows.cuh"
#include "umma.cuh"

namespace moer {

constexpr int EG_STAGES = 6;
constexpr int EG_HALF = 16384;               // one operand's part of a stage: 128 rows (or 2 panels of 64) x 128 bytes
constexpr int EG_STAGE_BYTES = 2 * EG_HALF;
constexpr int EG_PANEL = 8192;               // 64 rows x 128 bytes
constexpr int EG_EPI_WARPS = 16;
constexpr int EG_THREADS = (8 + EG_EPI_WARPS) * 32;
constexpr int EG_J = 256;                    // most j of a tile
constexpr int EG_COLS = EG_J / (EG_EPI_WARPS / 4);  // columns that an epilogue warp holds
constexpr int EG_TMEM_COLS = 512;
constexpr int EG_ROUND = 8;                  // blocks summed in TMEM (not E4M3)
constexpr size_t EG_OFF_BAR = (size_t)EG_STAGES * EG_STAGE_BYTES;
constexpr int EG_LISTS = 8;                            // row lists under way: of tiles, or (GRAD_WEIGHT) of blocks
constexpr int EG_LIST = 128;                           // entries of a list
constexpr size_t EG_OFF_LIST = EG_OFF_BAR + 512;       // [list][EG_LIST] ints
constexpr int EG_SLOTS = 8, EG_SLOT_KB = 4;            // E4M3: ring of x's scales, blocks a slot
constexpr size_t EG_OFF_SCALE = EG_OFF_LIST + (size_t)EG_LISTS * EG_LIST * 4;  // [slot][block][128 rows]
constexpr size_t EG_SCALE_BYTES = (size_t)EG_SLOTS * EG_SLOT_KB * 128 * 4;
constexpr size_t EG_OFF_TABLE = EG_OFF_SCALE + EG_SCALE_BYTES;  // the experts' tiles: 3 x (E + 1) ints
// Barriers, as byte offsets from the stages' start.
constexpr uint32_t EG_FULL = (uint32_t)EG_OFF_BAR;            // [stage] in the leader: both operands of both CTAs
constexpr uint32_t EG_EMPTY = EG_FULL + 8 * EG_STAGES;        // [stage] the MMAs have read it
constexpr uint32_t EG_TFULL = EG_EMPTY + 8 * EG_STAGES;       // [2] an accumulator is complete
constexpr uint32_t EG_TEMPTY = EG_TFULL + 16;                 // [2] in the leader: it is drained in both CTAs
constexpr uint32_t EG_DRAIN = EG_TEMPTY + 16;
constexpr uint32_t EG_LFULL = EG_DRAIN + 8;                   // [list] written
constexpr uint32_t EG_LEMPTY = EG_LFULL + 8 * EG_LISTS;       // [list] read
constexpr uint32_t EG_SFULL = EG_LEMPTY + 8 * EG_LISTS;       // [slot] E4M3: scales written
constexpr uint32_t EG_SEMPTY = EG_SFULL + 8 * EG_SLOTS;       // [slot] read
constexpr uint32_t EG_TMEM = EG_SEMPTY + 8 * EG_SLOTS;        // TMEM address, failure flag
constexpr uint32_t EG_DIRTY = EG_TMEM + 8;                    // [list] GRAD_WEIGHT: whether one of the block's rows is none
static_assert(EG_DIRTY + 4 * EG_LISTS <= EG_OFF_LIST, "barrier area");

struct GemmParams {
  CUtensorMap tmx;   // x by single rows: boxes of 128 bytes of one
  CUtensorMap tmw;   // w [E][N][K], or d_y [rows][N]
  CUtensorMap tmy;   // GRAD_WEIGHT: d_y by single rows
  CUtensorMap tmr;   // without an order: x by 32 rows
  const int32_t* off;
  const int32_t* order;
  int64_t rows, tokens;
  int E, k;
  uint64_t div_m;    // o / k = (o * div_m) >> div_s for 0 <= o < 2^31: div_m = 2^div_s / k, rounded up past it,
  int div_s;         // div_s = 32 + ceil(log2 k), so that o times the excess (k at most) stays below 2^div_s
  int M, C, J;       // extents of m, c (FORWARD, GRAD_INPUT) and j (GRAD_WEIGHT)
  int nmb, njb;      // blocks of 256 of m, and of j (GRAD_WEIGHT)
  int one_w;         // the experts share one matrix
  void* out;
  int64_t ld_out, stride_out;
  int out_dtype;
  uint32_t idesc;    // instruction descriptor without N
  const float* sx;   // E4M3
  const float* sw;
  int64_t ld_sx;
  uint32_t* status;
};

// ------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// 128 bytes from column c0 on of four rows of a row-by-row map, one after the other; a row past the
// map's end gives zeros.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap* tm, int c0, const int4& r, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
      : "memory");
}

// The operands' descriptors come as 32-bit halves: the high one is the same for every stage.
template <bool FP8>
__device__ __forceinline__ void umma_pair(uint32_t dt, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accum) {
  if constexpr (FP8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %4, p;\n\t}" ::"r"(dt),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accum));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(dt),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accum));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Descriptor of an operand whose m (or j) is contiguous: panels of 64 of it, EG_PANEL bytes
// apart, rows of c of 128 bytes, groups of eight rows 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t umma_desc_panels(uint32_t saddr) {
  return (umma_desc_sw128(saddr) & ~(0x3FFFull << 16)) | ((uint64_t)(EG_PANEL >> 4) << 16);
}

// Bounded wait by one thread on a barrier of this CTA.  Scope: the block.  What the other CTA of the
// pair hands over through a barrier is read by the tensor cores alone (each from its own SM's
// shared memory), after the writer's proxy fence; nothing that threads wrote is read across the
// pair.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool one_wait(uint32_t bar, uint32_t parity, uint32_t* status) {
  if (try_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (try_wait(bar, parity)) return true;
    if ((it & 63u) == 63u) {
      const unsigned long long t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > WAIT_LIMIT_NS || it >= WAIT_LIMIT_ITERS) {
        atomicOr(status, WS_BIT_ETIMEOUT);
        return false;
      }
    }
  }
}

// Waits by the epilogue's warps: one thread polls (sixteen polling warps took the issue slots of the
// thread that issues the MMAs), the others stand at a named barrier, which passes its answer on.
__device__ __forceinline__ bool epilogue_wait(uint32_t bar, uint32_t parity, uint32_t* status) {
  uint32_t ok = 1;
  if (threadIdx.x == 256) ok = one_wait(bar, parity, status);
  __syncwarp();
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok), "n"(EG_EPI_WARPS * 32)
      : "memory");
  return all != 0;
}

// Arrival on a barrier of either CTA, with the same scope: released at cluster scope each
// arrival would first wait for the thread's memory operations (1.7 us a stage instead of 0.3).
__device__ __forceinline__ void pair_arrive(uint32_t caddr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

// Arrival on the leader's barrier of a stage, with the bytes that this thread brings to it, perhaps none:
// a stage fills only when every thread that brings to stages has come by.  One that could stay behind
// or run ahead (having nothing to bring to a narrow tile, say) would lose its place, since a
// barrier's parity tells neighbouring rounds apart and no more.
__device__ __forceinline__ void stage_arrive(uint32_t caddr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(caddr), "r"(bytes) : "memory");
}

// One lane of the warp, which the compiler knows to be one: descriptors then go to uniform registers
// without a loop over lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Waits by a whole warp.  MEM: the lanes then read, or overwrite, shared memory that the barrier stands for, so
// each of them waits itself.  Else lane 0 polls and its answer is everyone's: loads from TMEM, which the whole
// warp makes behind a fence.  (A shuffle orders no memory; with a barrier of the warp behind lane 0's wait
// the registers that it cost made the 8-bit product of 262,144 rows of 2,048 x 1,536 take 1,285 us instead of 1,210.)
template <bool MEM>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t* status, int lane) {
  if constexpr (MEM) return __all_sync(FULL, one_wait(bar, parity, status)) != 0;
  bool ok = true;
  if (lane == 0) ok = one_wait(bar, parity, status);
  return __shfl_sync(FULL, (int)ok, 0) != 0;
}

// ------------------------------------------------------------ tiles
// The experts' rows and tiles, in shared memory: lo[e] .. lo[e + 1] are e's rows (offsets held
// within [0, rows] and non-decreasing), first[e] its first tile column, high[e] the rows of each of its
// tiles but the last.
struct TileTable {
  const int* lo;
  const int* first;
  const int* high;
};

// One warp.  With `by_rows` an expert has as few tile columns as hold its rows, of equal height
// (in steps of 16) but for the last.
__device__ __forceinline__ void make_tile_table(const GemmParams& p, bool by_rows, int* lo, int lane) {
  int* first = lo + p.E + 1;
  int* high = first + p.E + 1;
  int most = 0, sum = 0;  // running maximum of the offsets, tile columns so far
  bool bad = false;
  for (int e0 = 0; e0 <= p.E; e0 += 32) {
    const int e = e0 + lane;
    const int64_t raw = e <= p.E ? p.off[e] : 0;
    int v = (int)max64(0, min64(raw, p.rows));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(FULL, v, d);
      if (lane >= d) v = max(v, u);
    }
    v = max(v, most);
    bad |= e <= p.E && v != raw;
    int prev = __shfl_up_sync(FULL, v, 1);
    if (lane == 0) prev = most;
    most = __shfl_sync(FULL, v, 31);
    // tile columns of expert e - 1, whose rows are prev .. v
    const uint32_t n = (uint32_t)(v - prev), nt = (n + EG_J - 1) / EG_J;
    int t = e >= 1 && e <= p.E ? (by_rows ? (int)nt : p.njb) : 0;
    if (e >= 1 && e <= p.E) high[e - 1] = nt > 0 ? (int)(((n + nt - 1) / nt + 15) & ~15u) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(FULL, t, d);
      if (lane >= d) t += u;
    }
    if (e <= p.E) {
      lo[e] = v;
      first[e] = sum + t;
    }
    sum += __shfl_sync(FULL, t, 31);
  }
  if (bad) atomicOr(p.status, WS_BIT_EDATA);
}

struct Tile {
  int e, mb;
  int p0;     // first list row (GRAD_WEIGHT: of the segment)
  int hi;     // end of the segment
  int j0;     // GRAD_WEIGHT: first n
  int rows;   // valid j
  int ncol;   // N of the instruction: j rounded up to 16 (E4M3: 256 of m)
  int nkb;    // blocks of c
};

// A cluster's tiles, every t_step-th, m blocks first.  Kept by each warp for itself; steps take no
// division and no search, since a division and a binary search a tile left gaps between tiles.
template <int OP, bool FP8>
struct TileWalk {
  int left;  // tiles that remain, this one included
  int col, mb, e, dcol, dmb;
  __device__ __forceinline__ TileWalk(const GemmParams& p, const TileTable& tt) {
    const int t = blockIdx.x >> 1, step = gridDim.x >> 1, n = tt.first[p.E] * p.nmb;
    left = t < n ? (n - t + step - 1) / step : 0;
    col = t / p.nmb;
    mb = t - col * p.nmb;
    dcol = step / p.nmb;
    dmb = step - dcol * p.nmb;
    e = 0;
  }
  __device__ __forceinline__ void advance(const GemmParams& p) {
    --left;
    col += dcol;
    mb += dmb;
    if (mb >= p.nmb) {
      mb -= p.nmb;
      ++col;
    }
  }
  // Of the present position, when tiles remain.
  __device__ __forceinline__ Tile tile(const GemmParams& p, const TileTable& tt) {
    constexpr int KE = FP8 ? 128 : 64;
    while (tt.first[e + 1] <= col) ++e;
    Tile x;
    x.e = e;
    x.mb = mb;
    const int lo = tt.lo[e], i = col - tt.first[e];
    x.hi = tt.lo[e + 1];
    if (OP == MOER_GEMM_GRAD_WEIGHT) {
      x.p0 = lo;
      x.j0 = i * EG_J;
      x.rows = min(EG_J, p.J - x.j0);
      x.ncol = EG_J;
      x.nkb = (int)(((uint32_t)(x.hi - lo) + KE - 1) / KE);
    } else {
      const int h = tt.high[e];
      x.p0 = lo + i * h;
      x.j0 = 0;
      x.rows = min(h, x.hi - x.p0);
      x.ncol = FP8 ? EG_J : (x.rows + 15) & ~15;
      x.nkb = (p.C + KE - 1) / KE;
    }
    return x;
  }
};

// The row of x behind a list row's entry, or -1; `bad`: it names no token.
__device__ __forceinline__ int entry_row(const GemmParams& p, int o, bool& bad) {
  if (p.order == nullptr || o < 0) return o;
  const int r = (int)(((uint64_t)(uint32_t)o * p.div_m) >> p.div_s);
  if (r < p.tokens) return r;
  bad = true;
  return -1;
}
__device__ __forceinline__ int list_entry(const GemmParams& p, int q) { return p.order == nullptr ? q : p.order[q]; }

// ------------------------------------------------------------ rows of x
// The lister, one warp: turns the lists' entries into rows of x, well ahead of their use.  FORWARD,
// GRAD_INPUT: a list of this CTA's rows for each tile (those past the tile repeat its last one;
// padding takes any row).  GRAD_WEIGHT: a list of 64 for each block; a row past the segment or of
// padding is given as the map's end, which reads as zeros.
template <int OP, bool FP8>
__device__ __forceinline__ bool write_lists(const GemmParams& p, const TileTable& tt, char* sm, uint32_t base, int rank, int lane) {
  constexpr bool GW = OP == MOER_GEMM_GRAD_WEIGHT;
  int* const lists = reinterpret_cast<int*>(sm + EG_OFF_LIST);
  uint32_t i = 0;  // lists written
  bool bad = false;
  auto take = [&]() { return i < EG_LISTS || warp_wait<true>(base + EG_LEMPTY + 8u * (i % EG_LISTS), (i / EG_LISTS - 1) & 1u, p.status, lane); };
  auto give = [&]() {
    __syncwarp();
    if (lane == 0) pair_arrive(mapa_u32(base + EG_LFULL + 8u * (i % EG_LISTS), (uint32_t)rank));
    ++i;
  };
  for (TileWalk<OP, FP8> walk(p, tt); walk.left > 0; walk.advance(p)) {
    const Tile x = walk.tile(p, tt);
    if constexpr (!GW) {
      const int part = FP8 ? 128 : x.ncol >> 1;
      int v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = 32 * c < part ? list_entry(p, x.p0 + min(rank * part + 32 * c + lane, x.rows - 1)) : 0;
      if (!take()) return false;
      int* d = lists + (i % EG_LISTS) * EG_LIST + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c) d[32 * c] = max(entry_row(p, v[c], bad), 0);
      give();
    } else {
      constexpr int AHEAD = 4;  // blocks whose entries are fetched in one go, while the four before are written
      int v[2 * AHEAD];
      auto fetch = [&](int kb) {
#pragma unroll
        for (int c = 0; c < 2 * AHEAD; ++c) {
          const uint32_t q = (uint32_t)kb * 64 + 32 * c + lane;
          v[c] = q < (uint32_t)(x.hi - x.p0) ? list_entry(p, x.p0 + (int)q) : -1;
        }
      };
      fetch(0);
      for (int k0 = 0; k0 < x.nkb; k0 += AHEAD) {
        int r[2 * AHEAD];
#pragma unroll
        for (int c = 0; c < 2 * AHEAD; ++c) r[c] = entry_row(p, v[c], bad);
        if (k0 + AHEAD < x.nkb) fetch(k0 + AHEAD);
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) {
          if (k0 + b >= x.nkb) break;
          const bool dirty = __any_sync(FULL, r[2 * b] < 0 || r[2 * b + 1] < 0);
          if (!take()) return false;
          int* d = lists + (i % EG_LISTS) * EG_LIST + lane;
          d[0] = r[2 * b] < 0 ? (int)p.tokens : r[2 * b];
          d[32] = r[2 * b + 1] < 0 ? (int)p.tokens : r[2 * b + 1];
          if (lane == 0) *reinterpret_cast<int*>(sm + EG_DIRTY + 4 * (i % EG_LISTS)) = dirty;
          give();
        }
      }
    }
  }
  if (GW && bad) atomicOr(p.status, WS_BIT_EDATA);  // (else the epilogue says it)
  return true;
}

// One thread of each of four warps brings a quarter of a stage's rows, by TMA, eight gathers of four.
// (One warp with a gather in each lane took 72 clocks a gather and 3,408 us; the rows by cp.async,
// with their proxy fences and two more barriers, 1,301 us; this way 1,291, and the weights' gradient
// 914 instead of 1,894.)
constexpr int EG_GATHERS = 8;

template <int OP, bool FP8>
__device__ __forceinline__ bool gather_rows(const GemmParams& p, const TileTable& tt, char* sm, uint32_t base, int w, int rank) {
  constexpr bool GW = OP == MOER_GEMM_GRAD_WEIGHT;
  constexpr int KE = FP8 ? 128 : 64;
  const uint32_t bar0 = mapa_u32(base + EG_FULL, 0);
  uint32_t i = 0;  // lists read
  int s = 0;
  uint32_t fills = 0, ph = 1;  // parity of the release that the next fill of stage s waits for
  int4 r[EG_GATHERS];
  auto list = [&](int first) {  // this thread's entries, from list entry `first` on
    const int4* d = reinterpret_cast<const int4*>(sm + EG_OFF_LIST + (i % EG_LISTS) * EG_LIST * 4) + first / 4;
#pragma unroll
    for (int g = 0; g < EG_GATHERS; ++g) r[g] = d[g];
  };
  auto wait_list = [&]() { return one_wait(base + EG_LFULL + 8u * (i % EG_LISTS), (i / EG_LISTS) & 1u, p.status); };
  auto done = [&]() {
    pair_arrive(mapa_u32(base + EG_LEMPTY + 8u * (i % EG_LISTS), (uint32_t)rank));
    ++i;
  };
  for (TileWalk<OP, FP8> walk(p, tt); walk.left > 0; walk.advance(p)) {
    const Tile x = walk.tile(p, tt);
    int n = EG_GATHERS;  // gathers that this thread makes a stage
    if constexpr (!GW) {
      const int part = FP8 ? max(0, min(128, x.rows - rank * 128)) : x.ncol >> 1;
      n = min(EG_GATHERS, max(0, ((part + 3) >> 2) - w * EG_GATHERS));
      if (!wait_list()) return false;
      list(w * 4 * EG_GATHERS);
      done();
    }
    for (int kb = 0; kb < x.nkb; ++kb) {
      bool dirty = false;
      if constexpr (GW) {  // warps 0, 1: the first panel's rows 0 .. 31 and 32 .. 63, 2, 3: the second panel's
        if (!wait_list()) return false;
        list((w & 1) * 32);
        dirty = *reinterpret_cast<const volatile int*>(sm + EG_DIRTY + 4 * (i % EG_LISTS)) != 0;
        done();
      }
      if (fills >= EG_STAGES && !one_wait(base + EG_EMPTY + 8u * s, ph, p.status)) return false;
      fills += fills < EG_STAGES;
      const uint32_t st = base + (uint32_t)(s * EG_STAGE_BYTES), bar = bar0 + 8u * s;
      stage_arrive(bar, 512u * (uint32_t)(dirty ? 2 * n : n));
      if constexpr (!GW) {
        if (p.order == nullptr && n == EG_GATHERS)  // 32 neighbouring rows at once
          tma_load_2d_pair(st + EG_HALF + 4096u * w, &p.tmr, kb * KE, x.p0 + rank * (FP8 ? 128 : x.ncol >> 1) + 32 * w, bar);
        else
#pragma unroll
        for (int g = 0; g < EG_GATHERS; ++g)
          if (g < n) tma_gather4_pair(st + EG_HALF + 512u * (w * EG_GATHERS + g), &p.tmx, kb * KE, r[g], bar);
      } else {
        const uint32_t dst = st + (uint32_t)((w >> 1) * EG_PANEL + (w & 1) * 4096);
        const int col = rank * 128 + (w >> 1) * 64;
        if (p.order == nullptr && !dirty) tma_load_2d_pair(dst, &p.tmr, x.mb * 256 + col, x.p0 + kb * 64 + (w & 1) * 32, bar);
        else
#pragma unroll
          for (int g = 0; g < EG_GATHERS; ++g) tma_gather4_pair(dst + 512u * g, &p.tmx, x.mb * 256 + col, r[g], bar);
        if (dirty) {  // d_y's rows one by one too, those that are none as zeros (else warp 0 brings them)
          const int first = x.p0 + kb * 64 + (w & 1) * 32, none = (int)p.rows, end = (int)p.tokens;
#pragma unroll
          for (int g = 0; g < EG_GATHERS; ++g) {
            const int q = first + 4 * g;
            const int4 y = {r[g].x < end ? q : none, r[g].y < end ? q + 1 : none, r[g].z < end ? q + 2 : none, r[g].w < end ? q + 3 : none};
            tma_gather4_pair(dst + EG_HALF + 512u * g, &p.tmy, x.j0 + col, y, bar);
          }
        }
      }
      if (++s == EG_STAGES) {
        s = 0;
        ph ^= 1u;
      }
    }
  }
  return true;
}

// ------------------------------------------------------------ epilogue
// a.x += r0 * x, a.y += r1 * y (two lanes of one instruction).
__device__ __forceinline__ void fma2(float2& a, uint32_t r0, uint32_t r1, float x, float y) {
  asm("{\n\t.reg .b64 d, u, v;\n\tmov.b64 d, {%0, %1};\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t"
      "fma.rn.f32x2 d, u, v, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(r0), "r"(r1), "f"(x), "f"(y));
}
__device__ __forceinline__ void add2(float2& a, uint32_t r0, uint32_t r1) {
  asm("{\n\t.reg .b64 d, u;\n\tmov.b64 d, {%0, %1};\n\tmov.b64 u, {%2, %3};\n\t"
      "add.rn.f32x2 d, u, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(r0), "r"(r1));
}

template <typename T>
__device__ __forceinline__ void store_cols(T* o, int64_t ld, const float2* v, int n, uint32_t zero) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (c < n) o[(int64_t)c * ld] = from_f32<T>((zero >> c) & 1u ? 0.f : (c & 1 ? v[c / 2].y : v[c / 2].x));
}

// 32 columns (output rows) of one m; `first`: element of the first; n: valid rows; zero: rows that
// are padding.
__device__ __forceinline__ void store_chunk(const GemmParams& p, int64_t first, const float2* v, int n, uint32_t zero) {
  if (p.out_dtype == MOER_F32) store_cols(static_cast<float*>(p.out) + first, p.ld_out, v, n, zero);
  else if (p.out_dtype == MOER_BF16) store_cols(static_cast<__nv_bfloat16*>(p.out) + first, p.ld_out, v, n, zero);
  else store_cols(static_cast<__half*>(p.out) + first, p.ld_out, v, n, zero);
}

// A thread's neighbouring columns of one row (E4M3).  n: columns that exist.
template <typename T, int N>
__device__ __forceinline__ void store_row(T* o, const float2 (&v)[N], int n, bool zero) {
  constexpr int PER = 16 / (int)sizeof(T);
  const bool wide = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
#pragma unroll
  for (int c = 0; c < 2 * N; c += PER) {
    T t[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) t[i] = from_f32<T>(zero ? 0.f : ((c + i) & 1 ? v[(c + i) / 2].y : v[(c + i) / 2].x));
    if (wide && c + PER <= n) {
      *reinterpret_cast<uint4*>(o + c) = *reinterpret_cast<const uint4*>(t);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (c + i < n) o[c + i] = t[i];
    }
  }
}

template <int OP>
__device__ __forceinline__ int64_t out_first(const GemmParams& p, const Tile& x, int m) {
  return OP == MOER_GEMM_GRAD_WEIGHT ? x.e * p.stride_out + (int64_t)x.j0 * p.ld_out + m : (int64_t)x.p0 * p.ld_out + m;
}

// Which of the tile's rows 32 c .. 32 c + 31 are padding, by the warp.
template <int OP>
__device__ __forceinline__ uint32_t pad_mask(const GemmParams& p, const Tile& x, int c, int lane) {
  if (OP == MOER_GEMM_GRAD_WEIGHT || p.order == nullptr) return 0u;
  bool bad = false;
  const int j = c * 32 + lane;
  const bool pad = j < x.rows && entry_row(p, list_entry(p, x.p0 + j), bad) < 0;
  if (bad) atomicOr(p.status, WS_BIT_EDATA);
  return __ballot_sync(FULL, pad);
}

// ------------------------------------------------------------ the kernel
// Warps: 0 loads whole tiles, 1 allocates TMEM and issues the MMAs (in the leader), 2 lists rows, 4 to 7
// gather them, 8 to 23 drain the accumulators, each 64 columns of its TMEM lanes.  Registers go to
// the last sixteen: the six warpgroups' shares, 64 + 64 + 4 x 88 (E4M3, whose epilogue has two loads
// from TMEM under way: 48 + 48 + 4 x 96), are the block's 6 x 80.  With the latter for all, prefill
// takes 1,397 instead of 1,291 us; with the former for all, E4M3 1,281 instead of 1,211.
template <int OP, bool FP8>
__global__ void __launch_bounds__(EG_THREADS, 1) expert_gemm_kernel(const __grid_constant__ GemmParams p) {
  constexpr int EB = FP8 ? 1 : 2, KE = 128 / EB;  // bytes of an element, elements of c a block
  constexpr bool GW = OP == MOER_GEMM_GRAD_WEIGHT;
  constexpr bool A_PANELS = OP != MOER_GEMM_FORWARD, B_PANELS = GW;
  constexpr int ROUND = FP8 ? 1 : EG_ROUND;
  extern __shared__ __align__(1024) char eg_raw[];
  const uint32_t base = (smem_u32(eg_raw) + 1023) & ~1023u;  // the same in both CTAs, as the MMA's descriptors require
  char* sm = eg_raw + (base - smem_u32(eg_raw));
  volatile int& failed = *reinterpret_cast<int*>(sm + EG_TMEM + 4);
  int* lo = reinterpret_cast<int*>(sm + EG_OFF_TABLE);
  const TileTable tt{lo, lo + p.E + 1, lo + 2 * (p.E + 1)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();

  if (threadIdx.x == 32) {
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm);
    for (int s = 0; s < EG_STAGES; ++s) {
      mbar_init(bar + EG_FULL / 8 + s, 2 * 5);  // of either CTA: the tiles' thread and the four that gather
      mbar_init(bar + EG_EMPTY / 8 + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + EG_TFULL / 8 + i, 1);
      mbar_init(bar + EG_TEMPTY / 8 + i, 2 * EG_EPI_WARPS);
    }
    mbar_init(bar + EG_DRAIN / 8, 1);
    for (int i = 0; i < EG_LISTS; ++i) {
      mbar_init(bar + EG_LFULL / 8 + i, 1);
      mbar_init(bar + EG_LEMPTY / 8 + i, GW ? 5 : 4);  // the gathering threads, and warp 0's for `dirty`
    }
    for (int i = 0; i < EG_SLOTS; ++i) {
      mbar_init(bar + EG_SFULL / 8 + i, 1);
      mbar_init(bar + EG_SEMPTY / 8 + i, EG_EPI_WARPS);
    }
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 0) make_tile_table(p, !GW, lo, lane);
  cluster_sync();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + EG_TMEM), "r"(EG_TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();

  if (warp < 4) {
    if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // -------------------------------------------------------- TMA: w, or d_y
      if (elect_one()) {
        const uint32_t bar0 = mapa_u32(base + EG_FULL, 0);
        int s = 0;
        uint32_t fills = 0, ph = 1, i = 0;  // lists looked at
        bool ok = true;
        for (TileWalk<OP, FP8> walk(p, tt); walk.left > 0 && ok; walk.advance(p)) {
          const Tile x = walk.tile(p, tt);
          const int m0 = x.mb * 256 + rank * 128, n0 = x.j0 + rank * 128;
          const int e = p.one_w ? 0 : x.e;
          for (int kb = 0; kb < x.nkb; ++kb) {
            bool dirty = false;
            if constexpr (GW) {
              ok = one_wait(base + EG_LFULL + 8u * (i % EG_LISTS), (i / EG_LISTS) & 1u, p.status);
              if (!ok) break;
              dirty = *reinterpret_cast<const volatile int*>(sm + EG_DIRTY + 4 * (i % EG_LISTS)) != 0;
              pair_arrive(mapa_u32(base + EG_LEMPTY + 8u * (i % EG_LISTS), (uint32_t)rank));
              ++i;
            }
            if (fills >= EG_STAGES && !one_wait(base + EG_EMPTY + 8u * s, ph, p.status)) {
              ok = false;
              break;
            }
            fills += fills < EG_STAGES;
            const uint32_t st = base + (uint32_t)(s * EG_STAGE_BYTES), bar = bar0 + 8u * s;
            stage_arrive(bar, dirty ? 0u : (uint32_t)EG_HALF);
            if (OP == MOER_GEMM_FORWARD) {
              tma_load_3d_pair(st, &p.tmw, kb * KE, m0, e, bar);
            } else if (OP == MOER_GEMM_GRAD_INPUT) {
              tma_load_3d_pair(st, &p.tmw, m0, kb * KE, e, bar);
              tma_load_3d_pair(st + EG_PANEL, &p.tmw, m0 + 64, kb * KE, e, bar);
            } else if (!dirty) {
              tma_load_3d_pair(st + EG_HALF, &p.tmw, n0, x.p0 + kb * KE, 0, bar);
              tma_load_3d_pair(st + EG_HALF + EG_PANEL, &p.tmw, n0 + 64, x.p0 + kb * KE, 0, bar);
            }
            if (++s == EG_STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        // the last fills' stages have been released: no MMA still reads them
        for (uint32_t q = 0; q < fills && ok; ++q) {
          if (fills < EG_STAGES) {  // the ring was never full: stages 0 .. fills - 1, first round
            ok = one_wait(base + EG_EMPTY + 8u * q, 0, p.status);
            continue;
          }
          ok = one_wait(base + EG_EMPTY + 8u * s, ph, p.status);
          if (++s == EG_STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) failed = 1;
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA
      if (elect_one()) {
        bool ok = true;
        if (rank == 0) {
          int s = 0;
          uint32_t ph = 0, j = 0;  // parity of the full barriers; rounds begun
          // E4M3 has the rows of x as the instruction's m and the weights as its columns
          const uint32_t at_w = base, at_x = base + EG_HALF;
          const uint64_t d0 = FP8 ? umma_desc_sw128(at_x) : A_PANELS ? umma_desc_panels(at_w) : umma_desc_sw128(at_w);
          const uint64_t d1 = FP8 ? umma_desc_sw128(at_w) : B_PANELS ? umma_desc_panels(at_x) : umma_desc_sw128(at_x);
          const uint32_t hi = (uint32_t)(d0 >> 32);  // the same for both
          // one instruction takes 32 bytes of a row of c, or 16 rows of panels (16-byte units)
          constexpr uint32_t A_STEP = A_PANELS ? 128 : 2, B_STEP = B_PANELS ? 128 : 2;
          const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + EG_TMEM);
          TileWalk<OP, FP8> walk(p, tt);
          int nkb = 0;
          uint32_t idesc = 0;
          auto look = [&]() {
            const Tile x = walk.tile(p, tt);
            nkb = x.nkb;
            idesc = p.idesc | ((uint32_t)(x.ncol >> 3) << 17);
          };
          if (walk.left > 0) look();
          while (walk.left > 0 && ok) {
            const int nk = nkb;
            const uint32_t id = idesc;
            if (nk == 0) {
              walk.advance(p);
              if (walk.left > 0) look();
              continue;
            }
            for (int kb = 0, r = 0; kb < nk; ++kb) {
              const uint32_t a = j & 1u;
              if (r == 0 && j >= 2 && !one_wait(base + EG_TEMPTY + 8u * a, ((j >> 1) - 1) & 1u, p.status)) {
                ok = false;
                break;
              }
              if (!one_wait(base + EG_FULL + 8u * s, ph, p.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t da = (uint32_t)d0 + (uint32_t)s * (EG_STAGE_BYTES >> 4), db = (uint32_t)d1 + (uint32_t)s * (EG_STAGE_BYTES >> 4);
              const uint32_t dt = tmem + a * EG_J;
#pragma unroll
              for (int i = 0; i < 4; ++i) umma_pair<FP8>(dt, da + A_STEP * i, db + B_STEP * i, hi, id, (i > 0 || r > 0) ? 1u : 0u);
              umma_commit_pair(base + EG_EMPTY + 8u * s);
              if (++r == ROUND || kb == nk - 1) {
                umma_commit_pair(base + EG_TFULL + 8u * a);
                ++j;
                r = 0;
              }
              if (++s == EG_STAGES) {
                s = 0;
                ph ^= 1u;
              }
              if (kb == 0) {  // the next tile, while this one's MMAs run
                walk.advance(p);
                if (walk.left > 0) look();
              }
            }
          }
          umma_commit_pair(base + EG_DRAIN);
        }
        if (!ok) failed = 1;
      }
    } else if (warp == 2) {
      if (!write_lists<OP, FP8>(p, tt, sm, base, rank, lane) && lane == 0) failed = 1;
    } else if (FP8) {
      // -------------------------------------------------------- x's scales (E4M3), four rows a lane
      uint32_t it = 0;
      bool ok = true;
      const bool quad = p.ld_sx % 4 == 0 && reinterpret_cast<uintptr_t>(p.sx) % 16 == 0;
      for (TileWalk<OP, FP8> walk(p, tt); walk.left > 0 && ok; walk.advance(p)) {
        const Tile x = walk.tile(p, tt);
        const float* sx[4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // rows past the tile repeat its last one
          const int r = entry_row(p, list_entry(p, x.p0 + min(rank * 128 + 32 * i + lane, x.rows - 1)), bad);
          sx[i] = p.sx + (int64_t)max(r, 0) * p.ld_sx;
        }
        for (int k0 = 0; k0 < x.nkb; k0 += EG_SLOT_KB, ++it) {
          float v[4][EG_SLOT_KB];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (quad && k0 + EG_SLOT_KB <= x.nkb) {
              const float4 f = __ldg(reinterpret_cast<const float4*>(sx[i] + k0));
              v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
            } else {
#pragma unroll
              for (int b = 0; b < EG_SLOT_KB; ++b) v[i][b] = k0 + b < x.nkb ? __ldg(sx[i] + k0 + b) : 0.f;
            }
          }
          const uint32_t slot = it % EG_SLOTS;
          if (it >= EG_SLOTS && !warp_wait<true>(base + EG_SEMPTY + 8u * slot, (it / EG_SLOTS - 1) & 1u, p.status, lane)) {
            ok = false;
            break;
          }
          float* d = reinterpret_cast<float*>(sm + EG_OFF_SCALE) + slot * EG_SLOT_KB * 128 + lane;
#pragma unroll
          for (int b = 0; b < EG_SLOT_KB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[b * 128 + 32 * i] = v[i][b];
          __syncwarp();
          if (lane == 0) pair_arrive(mapa_u32(base + EG_SFULL + 8u * slot, (uint32_t)rank));
        }
      }
      if (!ok && lane == 0) failed = 1;
    }
  } else if (warp < 8) {
    if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (elect_one() && !gather_rows<OP, FP8>(p, tt, sm, base, warp - 4, rank)) failed = 1;
  } else {
    // ---------------------------------------------------------- epilogue
    if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    const int h0 = ((warp - 8) >> 2) * EG_COLS;  // first of the warp's columns
    const uint32_t tempty = mapa_u32(base + EG_TEMPTY, 0);
    // the TMEM lane quarter that this warp may access
    const uint32_t t0 = *reinterpret_cast<const uint32_t*>(sm + EG_TMEM) + ((uint32_t)((warp & 3) * 32) << 16) + h0;
    uint32_t j = 0, it = 0;
    bool ok = true;
    for (TileWalk<OP, FP8> walk(p, tt); walk.left > 0 && ok; walk.advance(p)) {
      const Tile x = walk.tile(p, tt);
      const int l = rank * 128 + (warp & 3) * 32 + lane;  // this thread's m in the tile (E4M3: its row)
      float2 acc[EG_COLS / 2];
#pragma unroll
      for (int c = 0; c < EG_COLS / 2; ++c) acc[c] = make_float2(0.f, 0.f);
      if constexpr (FP8) {
        // a thread has one row and 64 neighbouring columns: one scale of either operand a block
        const int nkw = x.nkb, nnb = (p.M + 127) / 128;
        bool bad = false;
        const int row = l < x.rows ? entry_row(p, list_entry(p, x.p0 + l), bad) : -1;
        if (bad) atomicOr(p.status, WS_BIT_EDATA);
        const bool some = rank * 128 + (warp & 3) * 32 < x.rows;  // (a warp without rows only hands buffers back)
        const float* sw = p.sw + ((int64_t)x.e * nnb + min(x.mb * 2 + h0 / 128, nnb - 1)) * nkw;
        const float* sx = reinterpret_cast<const float*>(sm + EG_OFF_SCALE) + (warp & 3) * 32 + lane;
        float fw = __ldg(sw);
        for (int kb = 0; kb < nkw; ++kb, ++j) {
          const uint32_t a = j & 1u, slot = it % EG_SLOTS;
          if (kb % EG_SLOT_KB == 0 && !warp_wait<true>(base + EG_SFULL + 8u * slot, (it / EG_SLOTS) & 1u, p.status, lane)) ok = false;
          const float f = fw * sx[(slot * EG_SLOT_KB + kb % EG_SLOT_KB) * 128];
          if (kb + 1 < nkw) fw = __ldg(sw + kb + 1);  // the next block's, under way
          if (!ok || !warp_wait<false>(base + EG_TFULL + 8u * a, (j >> 1) & 1u, p.status, lane)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (some) {
            uint32_t r[2][16];
            tmem_ld16(t0 + a * EG_J, r[0]);
#pragma unroll
            for (int c = 0; c < EG_COLS / 16; ++c) {
              tmem_ld_wait();
              if (c + 1 < EG_COLS / 16) tmem_ld16(t0 + a * EG_J + 16u * (c + 1), r[(c + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 8; ++i) fma2(acc[c * 8 + i], r[c & 1][2 * i], r[c & 1][2 * i + 1], f, f);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) pair_arrive(tempty + 8u * a);
          if (kb % EG_SLOT_KB == EG_SLOT_KB - 1 || kb == nkw - 1) {
            if (lane == 0) pair_arrive(mapa_u32(base + EG_SEMPTY + 8u * slot, (uint32_t)rank));
            ++it;
          }
        }
        if (!ok) break;
        const int m = x.mb * 256 + h0;
        if (l < x.rows && m < p.M) {
          const int64_t o = ((int64_t)x.p0 + l) * p.ld_out + m;
          const int n = min(EG_COLS, p.M - m);
          if (p.out_dtype == MOER_F32) store_row(static_cast<float*>(p.out) + o, acc, n, row < 0);
          else if (p.out_dtype == MOER_BF16) store_row(static_cast<__nv_bfloat16*>(p.out) + o, acc, n, row < 0);
          else store_row(static_cast<__half*>(p.out) + o, acc, n, row < 0);
        }
      } else {
        const int nch = max(0, min(EG_COLS / 16, (x.ncol - h0) >> 4));  // chunks of 16 columns that this warp holds
        for (int kb = 0; kb < x.nkb; kb += ROUND, ++j) {
          const uint32_t a = j & 1u;
          if (!epilogue_wait(base + EG_TFULL + 8u * a, (j >> 1) & 1u, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < EG_COLS / 16; ++c) {
            if (c < nch) {
              uint32_t r[16];
              tmem_ld16(t0 + a * EG_J + 16u * c, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) add2(acc[c * 8 + i], r[2 * i], r[2 * i + 1]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) pair_arrive(tempty + 8u * a);
        }
        if (!ok) break;
        const int m = x.mb * 256 + l;
#pragma unroll
        for (int c = 0; c < EG_COLS / 32; ++c) {
          const int j0 = h0 + c * 32;
          if (j0 < x.rows) {
            const uint32_t zero = pad_mask<OP>(p, x, j0 / 32, lane);
            if (m < p.M) store_chunk(p, out_first<OP>(p, x, m) + (int64_t)j0 * p.ld_out, &acc[c * 16], x.rows - j0, zero);
          }
        }
      }
    }
    if (!ok && lane == 0) failed = 1;
  }
  __syncthreads();
  // The last MMAs, once this CTA has drained its accumulators, when they are done or nearly so: the other CTA's
  // thread that waited for them from its start on gave up in calls of more than two seconds.
  bool late = failed;
  if (warp == 1) {
    if (lane == 0 && !one_wait(base + EG_DRAIN, 0, p.status)) late = true;
    __syncwarp();
  }
  if (late) {
    // a wait expired: give copies still in flight into this CTA time to land
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(*reinterpret_cast<const uint32_t*>(sm + EG_TMEM)), "r"(EG_TMEM_COLS));
  cluster_sync();
}

// No row of x to take: zeros in every row of a segment, or in the weights' gradient.  One warp a row.
template <typename T>
__global__ void __launch_bounds__(256) expert_gemm_zero_kernel(T* out, int64_t ld, int64_t stride, int cols, int64_t rows, const int32_t* off,
                                                               int E, const int32_t* order, int64_t list_rows, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  int64_t first = 0, most = 0;  // of the segments' rows; the offsets' running maximum, as in the tile table
  bool bad = false;
  for (int e0 = 0; e0 <= E; e0 += 32) {
    const int64_t raw = off[min(e0 + lane, E)];
    int64_t v = max64(0, min64(raw, list_rows));
    if (e0 == 0) first = __shfl_sync(FULL, v, 0);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(FULL, v, d);
      if (lane >= d) v = max64(v, u);
    }
    v = max64(v, most);
    bad |= v != raw;
    most = __shfl_sync(FULL, v, 31);
  }
  const int64_t step = (int64_t)gridDim.x * 8;
  const int64_t r0 = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  for (int64_t r = first + r0; r < most; r += step) bad |= order != nullptr && order[r] >= 0;
  if (bad) atomicOr(status, WS_BIT_EDATA);
  const int64_t from = stride == 0 ? first : 0, end = stride == 0 ? most : rows;  // list rows, or the gradient's
  for (int64_t r = from + r0; r < end; r += step) {
    T* o = stride == 0 ? out + r * ld : out + r / (rows / E) * stride + r % (rows / E) * ld;
    for (int c = lane; c < cols; c += 32) o[c] = from_f32<T>(0.f);
  }
}

// --------------------------------------------------------------- host side
namespace {
bool map_of(CUtensorMap* m, const void* base, int dtype, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const CUtensorMapDataType type = dtype == MOER_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : dtype == MOER_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cuuint64_t d[3], s[2];
  cuuint32_t b[3], one[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i > 0) s[i - 1] = strides[i - 1];
  }
  return enc(m, type, (cuuint32_t)rank, const_cast<void*>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t smem_bytes(int E) { return EG_OFF_TABLE + (size_t)3 * (E + 1) * 4 + 1024; }

cudaLaunchConfig_t pair_config(int clusters, size_t smem, cudaStream_t st, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)clusters);
  cfg.blockDim = dim3(EG_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <int OP, bool FP8>
cudaError_t gemm_run(const GemmParams& p, int64_t most_tiles, cudaStream_t st) {
  static std::atomic<unsigned long long> set{0};
  static std::atomic<int> cached[64];
  cudaError_t e = smem_optin(expert_gemm_kernel<OP, FP8>, (int)smem_bytes(1024), set);
  if (e != cudaSuccess) return e;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  int most = dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (most <= 0) {  // clusters that fit on the device at once, one CTA an SM
    const cudaLaunchConfig_t cfg = pair_config(1, smem_bytes(1024), nullptr, at);
    e = cudaOccupancyMaxActiveClusters(&most, expert_gemm_kernel<OP, FP8>, &cfg);
    if (e != cudaSuccess) return e;
    if (most <= 0) return cudaErrorInvalidConfiguration;
    if (dev < 64) cached[dev].store(most, std::memory_order_relaxed);
  }
  const cudaLaunchConfig_t cfg = pair_config((int)min64(most_tiles, most), smem_bytes(p.E), st, at);
  e = cudaLaunchKernelEx(&cfg, expert_gemm_kernel<OP, FP8>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t zero_run(const moer_expert_gemm_args* a, uint32_t* status, cudaStream_t st) {
  const bool gw = a->op == MOER_GEMM_GRAD_WEIGHT;
  const int64_t rows = gw ? (int64_t)a->E * a->N : a->rows;
  const int64_t stride = a->E > 1 ? a->stride_out : (int64_t)a->N * a->ld_out;
  const unsigned grid = (unsigned)min64((rows + 7) / 8, 152 * 8);
  expert_gemm_zero_kernel<T><<<grid, 256, 0, st>>>(static_cast<T*>(a->out), a->ld_out, gw ? stride : 0, a->op == MOER_GEMM_FORWARD ? a->N : a->K,
                                                   rows, a->expert_off, a->E, a->order, a->rows, status);
  return cudaGetLastError();
}
}  // namespace

moer_status expert_gemm_launch(const moer_expert_gemm_args* a, void* ws, cudaStream_t st) {
  const bool gw = a->op == MOER_GEMM_GRAD_WEIGHT, fwd = a->op == MOER_GEMM_FORWARD, fp8 = a->dtype == MOER_E4M3;
  uint32_t* status = static_cast<uint32_t*>(ws);
  if (a->rows == 0 || a->tokens == 0) {
    const cudaError_t e = a->out_dtype == MOER_F32    ? zero_run<float>(a, status, st)
                          : a->out_dtype == MOER_BF16 ? zero_run<__nv_bfloat16>(a, status, st)
                                                      : zero_run<__half>(a, status, st);
    return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
  }
  const uint64_t eb = fp8 ? 1 : 2, ke = 128 / eb;
  GemmParams p = {};
  p.off = a->expert_off;
  p.order = a->order;
  p.rows = a->rows;
  p.tokens = a->tokens;
  p.E = a->E;
  if (a->order != nullptr) {
    p.div_s = 32;
    while ((int64_t(1) << (p.div_s - 32)) < a->k) ++p.div_s;
    p.div_m = (uint64_t(1) << p.div_s) / (uint64_t)a->k + 1;
  }
  p.M = fwd ? a->N : a->K;
  p.C = fwd ? a->K : a->N;
  p.J = a->N;
  p.nmb = (p.M + 255) / 256;
  p.njb = (a->N + EG_J - 1) / EG_J;
  p.one_w = a->E > 1 && a->stride_w == 0;
  p.out = a->out;
  p.ld_out = a->ld_out;
  p.stride_out = a->E > 1 ? a->stride_out : 0;
  p.out_dtype = a->out_dtype;
  p.sx = a->x_scale;
  p.sw = a->w_scale;
  p.ld_sx = a->ld_x_scale;
  p.status = status;
  // D fp32; A and B bf16, fp16 or e4m3; transposed operands; M = 256
  const uint32_t fmt = a->dtype == MOER_BF16 ? 1u : 0u;
  p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((fwd ? 0u : 1u) << 15) | ((gw ? 1u : 0u) << 16) | ((256u >> 4) << 24);
  {
    const uint64_t dims[2] = {(uint64_t)(a->op == MOER_GEMM_GRAD_INPUT ? a->N : a->K), (uint64_t)a->tokens}, str[1] = {(uint64_t)a->ld_x * eb};
    const uint32_t box[2] = {(uint32_t)ke, 1};
    if (!map_of(&p.tmx, a->x, a->dtype, 2, dims, str, box)) return MOER_ECUDA;
    const uint32_t box32[2] = {(uint32_t)ke, 32};
    if (a->order == nullptr && !map_of(&p.tmr, a->x, a->dtype, 2, dims, str, box32)) return MOER_ECUDA;
  }
  if (gw) {
    const uint64_t dims[3] = {(uint64_t)a->N, (uint64_t)a->rows, 1}, str[2] = {(uint64_t)a->ld_d_y * eb, (uint64_t)a->ld_d_y * eb};
    const uint32_t box[3] = {64, 64, 1};
    if (!map_of(&p.tmw, a->d_y, a->dtype, 3, dims, str, box)) return MOER_ECUDA;
    const uint32_t row[2] = {64, 1};
    if (!map_of(&p.tmy, a->d_y, a->dtype, 2, dims, str, row)) return MOER_ECUDA;
  } else {
    const bool one = a->E == 1 || p.one_w;
    const uint64_t dims[3] = {(uint64_t)a->K, (uint64_t)a->N, (uint64_t)(one ? 1 : a->E)};
    const uint64_t str[2] = {(uint64_t)a->ld_w * eb, (uint64_t)(one ? a->ld_w : a->stride_w) * eb};
    const uint32_t box[3] = {(uint32_t)ke, fwd ? 128u : 64u, 1};
    if (!map_of(&p.tmw, a->w, a->dtype, 3, dims, str, box)) return MOER_ECUDA;
  }
  // tiles are counted in 32 bits
  const int64_t most = (gw ? (int64_t)a->E * p.njb : (a->rows + EG_J - 1) / EG_J + min64(a->E, a->rows)) * p.nmb;
  if (most >= (int64_t(1) << 30)) return MOER_ERANGE;
  const cudaError_t e = fp8   ? gemm_run<MOER_GEMM_FORWARD, true>(p, most, st)
                        : fwd ? gemm_run<MOER_GEMM_FORWARD, false>(p, most, st)
                        : gw  ? gemm_run<MOER_GEMM_GRAD_WEIGHT, false>(p, most, st)
                              : gemm_run<MOER_GEMM_GRAD_INPUT, false>(p, most, st);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
