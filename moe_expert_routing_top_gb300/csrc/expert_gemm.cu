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
// M = 256), K in blocks of 128 bytes, six stages of 32 KB.  A CTA loads its 128 of m and half
// of the j rows.  Rows of x are fetched by the list's entries, four at a time (TMA gather), so no
// permuted copy of x exists; where rows are contracted (GRAD_WEIGHT) the last block of
// a segment, and any block with padding, is cleared of other rows in shared memory before
// its MMAs.  Accumulators are fp32 in TMEM, two of 256 columns, drained while the next tile runs.
// E4M3: the sum of each block of 128 is taken out of TMEM and added in fp32 registers, times its
// two scales, by eight warps.
// Every wait is bounded; on expiry the kernel records MOER_ETIMEOUT and returns.
#include "rows.cuh"
#include "umma.cuh"

namespace moer {

constexpr int EG_STAGES = 6;
constexpr int EG_HALF = 16384;               // one operand's part of a stage: 128 rows (or 2 panels of 64) x 128 bytes
constexpr int EG_STAGE_BYTES = 2 * EG_HALF;
constexpr int EG_PANEL = 8192;               // 64 rows x 128 bytes
constexpr int EG_J = 256;                    // most j of a tile
constexpr int EG_SLOTS = 4, EG_SLOT_KB = 4;  // E4M3: ring of the scales' products, blocks a slot
constexpr int EG_SCALE_BYTES = EG_SLOTS * EG_SLOT_KB * EG_J * 4;
constexpr int EG_TMEM_COLS = 512;
constexpr size_t EG_OFF_BAR = (size_t)EG_STAGES * EG_STAGE_BYTES;
constexpr size_t EG_OFF_SCALE = EG_OFF_BAR + 512;

struct GemmParams {
  CUtensorMap tmx;   // x, fetched row by row: box of one row x 128 bytes
  CUtensorMap tmw;   // w [E][N][K], or d_y [rows][N]
  const int32_t* off;
  const int32_t* order;
  int64_t rows, tokens;
  int E, k;
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

// Four rows r[0..3] of a row-by-row map, 128 bytes each from column c0 on, one after the other.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap* tm, int c0, const int (&r)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}

template <bool FP8>
__device__ __forceinline__ void umma_pair(uint32_t dt, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  if constexpr (FP8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(dt),
        "l"(a), "l"(b), "r"(idesc), "r"(accum));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dt),
        "l"(a), "l"(b), "r"(idesc), "r"(accum));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Descriptor of an operand whose m (or j) is contiguous: panels of 64 of it, EG_PANEL bytes
// apart, rows of c of 128 bytes, groups of eight rows 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t umma_desc_panels(uint32_t saddr) {
  return (umma_desc_sw128(saddr) & ~(0x3FFFull << 16)) | ((uint64_t)(EG_PANEL >> 4) << 16);
}

// Waits by a whole warp, with one answer for it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  return __all_sync(FULL, mbar_wait_cl(bar, parity, status));
}

// ------------------------------------------------------------ tiles
// The experts' rows and tiles, in shared memory: lo[e] .. lo[e + 1] are e's rows (offsets
// held within [0, rows] and non-decreasing), first[e] its first tile column.
struct TileTable {
  const int* lo;
  const int* first;
};

// One warp.  With `by_rows` an expert has a tile column for each 256 of its rows.
__device__ __forceinline__ void make_tile_table(const GemmParams& p, bool by_rows, int* lo, int* first, int lane) {
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
    int t = e >= 1 && e <= p.E ? (by_rows ? (int)(((uint32_t)(v - prev) + EG_J - 1) / EG_J) : p.njb) : 0;
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
  int ncol;   // j rounded up to 16: N of the instruction
  int nkb;    // blocks of c
};

template <int OP, int KE>
__device__ __forceinline__ Tile tile_of(const GemmParams& p, const TileTable& tt, int64_t t) {
  Tile x;
  const int col = (int)(t / p.nmb);
  x.mb = (int)(t - (int64_t)col * p.nmb);
  int a = 0, b = p.E - 1;  // the last expert with first[e] <= col: the one that has tile column col
  while (a < b) {
    const int m = (a + b + 1) >> 1;
    if (tt.first[m] <= col) a = m;
    else b = m - 1;
  }
  x.e = a;
  const int lo = tt.lo[a], i = col - tt.first[a];
  x.hi = tt.lo[a + 1];
  const uint32_t n = (uint32_t)(x.hi - lo);
  if (OP == MOER_GEMM_GRAD_WEIGHT) {
    x.p0 = lo;
    x.j0 = i * EG_J;
    x.rows = min(EG_J, p.J - x.j0);
    x.ncol = EG_J;
    x.nkb = (int)((n + KE - 1) / KE);
  } else {
    // as few tiles as hold the segment, of equal height but for the last
    const uint32_t nt = (n + EG_J - 1) / EG_J;
    const int h = (int)(((n + nt - 1) / nt + 15) & ~15u);
    x.p0 = lo + i * h;
    x.j0 = 0;
    x.rows = min(h, x.hi - x.p0);
    x.ncol = (x.rows + 15) & ~15;
    x.nkb = (p.C + KE - 1) / KE;
  }
  return x;
}

// The row of x behind list row q, or -1; `bad`: its entry names no token.
__device__ __forceinline__ int source_row(const GemmParams& p, int q, bool& bad) {
  if (p.order == nullptr) return q;
  const int o = p.order[q];
  if (o < 0) return -1;
  const int r = o / p.k;
  if (r < p.tokens) return r;
  bad = true;
  return -1;
}

// ------------------------------------------------------------ epilogue
template <typename T>
__device__ __forceinline__ void store_cols(T* o, int64_t ld, const uint32_t* v, int n, uint32_t zero) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (c < n) o[(int64_t)c * ld] = from_f32<T>((zero >> c) & 1u ? 0.f : __uint_as_float(v[c]));
}

// 32 columns (output rows) of one m; `first`: element of the first; n: valid rows; zero: rows that
// are padding.
__device__ __forceinline__ void store_chunk(const GemmParams& p, int64_t first, const uint32_t* v, int n, uint32_t zero) {
  if (p.out_dtype == MOER_F32) store_cols(static_cast<float*>(p.out) + first, p.ld_out, v, n, zero);
  else if (p.out_dtype == MOER_BF16) store_cols(static_cast<__nv_bfloat16*>(p.out) + first, p.ld_out, v, n, zero);
  else store_cols(static_cast<__half*>(p.out) + first, p.ld_out, v, n, zero);
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
  const bool pad = j < x.rows && source_row(p, x.p0 + j, bad) < 0;
  if (bad) atomicOr(p.status, WS_BIT_EDATA);
  return __ballot_sync(FULL, pad);
}

// ------------------------------------------------------------ the kernel
// Warps: 0 loads, 1 allocates TMEM and issues the MMAs (in the leader), 2 and 3 form the scales'
// products (E4M3), the last four (E4M3: eight) drain the accumulators.
template <bool FP8>
constexpr int eg_threads() {
  return FP8 ? 384 : 192;
}

template <int OP, bool FP8>
__global__ void __launch_bounds__(eg_threads<FP8>(), 1) expert_gemm_kernel(const __grid_constant__ GemmParams p) {
  constexpr int KE = FP8 ? 128 : 64;         // elements of c a block: 128 bytes
  constexpr bool GW = OP == MOER_GEMM_GRAD_WEIGHT;
  constexpr bool A_PANELS = OP != MOER_GEMM_FORWARD, B_PANELS = GW;
  constexpr int EPI0 = FP8 ? 4 : 2, EPI_WARPS = FP8 ? 8 : 4;
  extern __shared__ __align__(1024) char eg_raw[];
  char* sm = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(eg_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + EG_OFF_BAR);  // used in the leader
  uint64_t* empty = full + EG_STAGES;
  uint64_t* tfull = empty + EG_STAGES;
  uint64_t* tempty = tfull + 2;   // used in the leader
  uint64_t* drain = tempty + 2;
  uint64_t* fix = drain + 1;      // GRAD_WEIGHT: this CTA's copies of a block that has to be cleared
  uint64_t* sfull = fix + 1;
  uint64_t* sempty = sfull + EG_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + EG_SLOTS);
  volatile int& failed = *reinterpret_cast<int*>(tmem_slot + 1);
  float* scales = reinterpret_cast<float*>(sm + EG_OFF_SCALE);  // [slot][block][j]
  int* lo = reinterpret_cast<int*>(sm + EG_OFF_SCALE + (FP8 ? EG_SCALE_BYTES : 0));
  int* first = lo + p.E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int64_t cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

  if (threadIdx.x == 32) {
    for (int s = 0; s < EG_STAGES; ++s) {
      mbar_init(&full[s], GW ? 2 : 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(fix, 1);
    for (int i = 0; i < EG_SLOTS; ++i) {
      mbar_init(&sfull[i], 2);
      mbar_init(&sempty[i], EPI_WARPS);
    }
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 0) make_tile_table(p, !GW, lo, first, lane);
  cluster_sync();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(EG_TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const TileTable tt{lo, first};
  const int64_t ntiles = (int64_t)first[p.E] * p.nmb;

  if (warp == 0) {
    // ---------------------------------------------------------- loads
    const uint32_t bar0 = mapa_u32(smem_u32(full), 0), base = smem_u32(sm);
    const uint32_t fixc = mapa_u32(smem_u32(fix), rank);
    int64_t g = 0;     // stages filled so far
    int s = 0;
    uint32_t ph = 1;   // parity of the release that the next fill of stage s waits for
    uint32_t fph = 0;
    bool ok = true;
    for (int64_t t = cluster; t < ntiles && ok; t += nclusters) {
      const Tile x = tile_of<OP, KE>(p, tt, t);
      const int m0 = x.mb * 256 + (int)rank * 128;
      if constexpr (!GW) {
        const int half = x.ncol >> 1;
        int r[4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // rows past the tile repeat its last one; padding takes any row
          const int j = min((int)rank * half + 4 * lane + i, x.rows - 1);
          r[i] = max(source_row(p, x.p0 + j, bad), 0);
        }
        const uint32_t tx = 2u * EG_HALF + (uint32_t)x.ncol * 128u;
        for (int kb = 0; kb < x.nkb; ++kb, ++g) {
          if (g >= EG_STAGES && !warp_wait(&empty[s], ph, p.status)) {
            ok = false;
            break;
          }
          const uint32_t st = base + (uint32_t)(s * EG_STAGE_BYTES), bar = bar0 + 8u * s;
          if (lane == 0) {
            if (leader) mbar_arrive_expect_tx(&full[s], tx);
            const int e = p.one_w ? 0 : x.e;
            if (OP == MOER_GEMM_FORWARD) {
              tma_load_3d_pair(st, &p.tmw, kb * KE, m0, e, bar);
            } else {
              tma_load_3d_pair(st, &p.tmw, m0, kb * KE, e, bar);
              tma_load_3d_pair(st + EG_PANEL, &p.tmw, m0 + 64, kb * KE, e, bar);
            }
          }
          if (4 * lane < half) tma_gather4_pair(st + EG_HALF + 512u * lane, &p.tmx, kb * KE, r, bar);
          if (++s == EG_STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      } else {
        // lane: panel lane / 16 of A, rows 4 (lane % 16) .. + 3 of the block
        const int r0 = 4 * (lane & 15), pan = lane >> 4;
        int r[4], nx[4];
        bool bad = false;
        auto rows_of = [&](int kb, int (&v)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t q = (uint32_t)kb * KE + r0 + i;
            v[i] = q < (uint32_t)(x.hi - x.p0) ? source_row(p, x.p0 + (int)q, bad) : -1;
          }
        };
        if (x.nkb > 0) rows_of(0, nx);
        for (int kb = 0; kb < x.nkb; ++kb, ++g) {
          uint32_t dead = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dead |= nx[i] < 0 ? 1u << i : 0u;
            r[i] = max(nx[i], 0);
          }
          const bool dirty = __any_sync(FULL, dead != 0);
          if (kb + 1 < x.nkb) rows_of(kb + 1, nx);
          if (g >= EG_STAGES && !warp_wait(&empty[s], ph, p.status)) {
            ok = false;
            break;
          }
          const uint32_t st = base + (uint32_t)(s * EG_STAGE_BYTES);
          const uint32_t bar = dirty ? fixc : bar0 + 8u * s;
          if (lane == 0) {
            if (dirty) mbar_arrive_expect_tx(fix, EG_STAGE_BYTES);
            else if (leader) mbar_arrive_expect_tx(&full[s], 2u * EG_STAGE_BYTES);
            else mbar_arrive_cluster(bar0 + 8u * s);
          }
          __syncwarp();
          if (lane < 2)
            tma_load_3d_pair(st + EG_HALF + EG_PANEL * lane, &p.tmw, x.j0 + (int)rank * 128 + 64 * lane, x.p0 + kb * KE, 0, bar);
          tma_gather4_pair(st + EG_PANEL * pan + 128u * r0, &p.tmx, m0 + 64 * pan, r, bar);
          if (dirty) {
            if (!warp_wait(fix, fph, p.status)) {
              ok = false;
              break;
            }
            fph ^= 1u;
            char* row = sm + (size_t)s * EG_STAGE_BYTES + (lane >> 3) * EG_PANEL + (lane & 7) * 16;
            for (int i = 0; i < KE; ++i)
              if ((__shfl_sync(FULL, dead, i >> 2) >> (i & 3)) & 1u) *reinterpret_cast<uint4*>(row + i * 128) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(bar0 + 8u * s);
          }
          if (++s == EG_STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (bad) atomicOr(p.status, WS_BIT_EDATA);
      }
    }
    // the last fills' stages have been released: no MMA still reads them
    for (int64_t q = (g > EG_STAGES ? g - EG_STAGES : 0); q < g && ok; ++q)
      if (!mbar_wait_cl(&empty[q % EG_STAGES], (uint32_t)((q / EG_STAGES) & 1), p.status)) ok = false;
    if (!ok && lane == 0) failed = 1;
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA
    if (lane == 0) {
      bool ok = true;
      if (leader) {
        const uint32_t base = smem_u32(sm);
        const uint64_t da0 = A_PANELS ? umma_desc_panels(base) : umma_desc_sw128(base);
        const uint64_t db0 = B_PANELS ? umma_desc_panels(base + EG_HALF) : umma_desc_sw128(base + EG_HALF);
        // one instruction takes 32 bytes of a row of c, or 16 rows of panels (16-byte units)
        constexpr uint64_t A_STEP = A_PANELS ? 128 : 2, B_STEP = B_PANELS ? 128 : 2;
        int s = 0;
        uint32_t ph = 0;
        int64_t j = 0;  // accumulators begun
        for (int64_t t = cluster; t < ntiles && ok; t += nclusters) {
          const Tile x = tile_of<OP, KE>(p, tt, t);
          const uint32_t idesc = p.idesc | ((uint32_t)(x.ncol >> 3) << 17);
          for (int kb = 0; kb < x.nkb; ++kb) {
            const int a = (int)(j & 1);
            if (FP8 || kb == 0) {
              if (j >= 2 && !mbar_wait_cl(&tempty[a], (uint32_t)(((j >> 1) - 1) & 1), p.status)) {
                ok = false;
                break;
              }
            }
            if (!mbar_wait_cl(&full[s], ph, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t da = da0 + (uint64_t)(s * (EG_STAGE_BYTES >> 4)), db = db0 + (uint64_t)(s * (EG_STAGE_BYTES >> 4));
            const uint32_t dt = tmem + (uint32_t)(a * EG_J);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_pair<FP8>(dt, da + A_STEP * i, db + B_STEP * i, idesc, (i > 0 || (!FP8 && kb > 0)) ? 1u : 0u);
            umma_commit_pair(&empty[s]);
            if (FP8 || kb == x.nkb - 1) {
              umma_commit_pair(&tfull[a]);
              ++j;
            }
            if (++s == EG_STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        umma_commit_pair(drain);
      }
      if (!mbar_wait_cl(drain, 0, p.status)) ok = false;
      if (!ok) failed = 1;
    }
  } else if (FP8 && warp < EPI0) {
    // ---------------------------------------------------------- scales (E4M3)
    if constexpr (FP8) {
      const int th = threadIdx.x - 64;  // 64 threads, four j each
      const int nkw = (p.C + 127) / 128, nnb = (p.M + 127) / 128;
      int64_t it = 0;
      bool ok = true;
      for (int64_t t = cluster; t < ntiles && ok; t += nclusters) {
        const Tile x = tile_of<OP, KE>(p, tt, t);
        const float* sx[4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = th + 64 * i;
          const int r = j < x.rows ? source_row(p, x.p0 + j, bad) : -1;
          sx[i] = r >= 0 ? p.sx + (int64_t)r * p.ld_sx : nullptr;
        }
        const int mb = x.mb * 2 + (int)rank;
        const float* sw = mb < nnb ? p.sw + ((int64_t)x.e * nnb + mb) * nkw : nullptr;
        for (int k0 = 0; k0 < x.nkb; k0 += EG_SLOT_KB, ++it) {
          const int slot = (int)(it % EG_SLOTS);
          float v[EG_SLOT_KB][4];
#pragma unroll
          for (int b = 0; b < EG_SLOT_KB; ++b) {
            const bool in = k0 + b < x.nkb;
            const float w = in && sw != nullptr ? sw[k0 + b] : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[b][i] = in && sx[i] != nullptr ? sx[i][k0 + b] * w : 0.f;
          }
          if (it >= EG_SLOTS && !warp_wait(&sempty[slot], (uint32_t)((it / EG_SLOTS - 1) & 1), p.status)) {
            ok = false;
            break;
          }
          float* d = scales + slot * EG_SLOT_KB * EG_J + th;
#pragma unroll
          for (int b = 0; b < EG_SLOT_KB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[b * EG_J + 64 * i] = v[b][i];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[slot]);
        }
      }
      if (!ok && lane == 0) failed = 1;
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t tempty0 = mapa_u32(smem_u32(tempty), 0);
    int64_t j = 0, it = 0;
    bool ok = true;
    for (int64_t t = cluster; t < ntiles && ok; t += nclusters) {
      const Tile x = tile_of<OP, KE>(p, tt, t);
      const int m = x.mb * 256 + (int)rank * 128 + q * 32 + lane;
      const bool mine = m < p.M;
      const int64_t o = out_first<OP>(p, x, m);
      if constexpr (FP8) {
        const int h = (warp - EPI0) >> 2;  // columns h * 128 .. + 127
        float acc[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) acc[c] = 0.f;
        for (int kb = 0; kb < x.nkb; ++kb, ++j) {
          const int slot = (int)(it % EG_SLOTS), b = kb % EG_SLOT_KB;
          if (b == 0 && !warp_wait(&sfull[slot], (uint32_t)((it / EG_SLOTS) & 1), p.status)) ok = false;
          const int a = (int)(j & 1);
          if (!ok || !warp_wait(&tfull[a], (uint32_t)((j >> 1) & 1), p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * EG_J + h * 128);
          const float4* sc = reinterpret_cast<const float4*>(scales + (slot * EG_SLOT_KB + b) * EG_J + h * 128);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (h * 128 + c * 16 < x.ncol) {
              uint32_t r[16];
              tmem_ld16(ta + 16u * c, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = sc[c * 4 + i];
                acc[c * 16 + 4 * i + 0] = fmaf(__uint_as_float(r[4 * i + 0]), f.x, acc[c * 16 + 4 * i + 0]);
                acc[c * 16 + 4 * i + 1] = fmaf(__uint_as_float(r[4 * i + 1]), f.y, acc[c * 16 + 4 * i + 1]);
                acc[c * 16 + 4 * i + 2] = fmaf(__uint_as_float(r[4 * i + 2]), f.z, acc[c * 16 + 4 * i + 2]);
                acc[c * 16 + 4 * i + 3] = fmaf(__uint_as_float(r[4 * i + 3]), f.w, acc[c * 16 + 4 * i + 3]);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_cluster(tempty0 + (uint32_t)(a * 8));
            if (b == EG_SLOT_KB - 1 || kb == x.nkb - 1) mbar_arrive(&sempty[slot]);
          }
          if (b == EG_SLOT_KB - 1 || kb == x.nkb - 1) ++it;
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j0 = h * 128 + c * 32;
          if (j0 < x.rows) {
            const uint32_t zero = pad_mask<OP>(p, x, j0 / 32, lane);
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(acc[c * 32 + i]);
            if (mine) store_chunk(p, o + (int64_t)j0 * p.ld_out, v, x.rows - j0, zero);
          }
        }
      } else {
        if (GW && x.nkb == 0) {  // an expert without rows
          uint32_t z[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) z[c] = 0u;
          if (mine)
            for (int j0 = 0; j0 < x.rows; j0 += 32) store_chunk(p, o + (int64_t)j0 * p.ld_out, z, x.rows - j0, 0u);
          continue;
        }
        const int a = (int)(j & 1);
        uint32_t zero[EG_J / 32];
#pragma unroll
        for (int c = 0; c < EG_J / 32; ++c) zero[c] = c * 32 < x.rows ? pad_mask<OP>(p, x, c, lane) : 0u;
        if (!warp_wait(&tfull[a], (uint32_t)((j >> 1) & 1), p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * EG_J);
#pragma unroll
        for (int c = 0; c < EG_J / 32; ++c) {
          if (c * 32 < x.rows) {
            uint32_t r[32];
            tmem_ld32(ta + 32u * c, r);
            tmem_ld_wait();
            if (mine) store_chunk(p, o + (int64_t)(c * 32) * p.ld_out, r, x.rows - c * 32, zero[c]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + (uint32_t)(a * 8));
        ++j;
      }
    }
    if (!ok && lane == 0) failed = 1;
  }
  __syncthreads();
  if (failed) {
    // a wait expired: give copies still in flight into this CTA time to land
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(EG_TMEM_COLS));
  cluster_sync();
}

// No row of x to take: zeros in every row of a segment, or in the weights' gradient.  One warp a row.
template <typename T>
__global__ void __launch_bounds__(256) expert_gemm_zero_kernel(T* out, int64_t ld, int64_t stride, int cols, int64_t rows, const int32_t* off,
                                                               int E, const int32_t* order, int64_t list_rows, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  int64_t most = 0, end = rows;
  bool bad = false;
  for (int e = lane; e <= E; e += 32) {
    const int64_t v = max64(0, min64(off[e], list_rows));
    bad |= v != off[e];
    most = max64(most, v);
  }
  for (int d = 16; d >= 1; d >>= 1) most = max64(most, __shfl_xor_sync(FULL, most, d));
  const int64_t step = (int64_t)gridDim.x * 8;
  const int64_t r0 = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (stride == 0) end = most;  // list rows
  for (int64_t r = r0; r < most; r += step) bad |= order != nullptr && order[r] >= 0;
  if (bad) atomicOr(status, WS_BIT_EDATA);
  for (int64_t r = r0; r < end; r += step) {
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

size_t smem_bytes(int E, bool fp8) { return EG_OFF_SCALE + (fp8 ? EG_SCALE_BYTES : 0) + (size_t)2 * (E + 1) * 4 + 1024; }

cudaLaunchConfig_t pair_config(int clusters, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)clusters);
  cfg.blockDim = dim3(threads);
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
  constexpr int threads = eg_threads<FP8>();
  cudaError_t e = smem_optin(expert_gemm_kernel<OP, FP8>, (int)smem_bytes(1024, FP8), set);
  if (e != cudaSuccess) return e;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  int most = dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (most <= 0) {  // clusters that fit on the device at once, one CTA an SM
    const cudaLaunchConfig_t cfg = pair_config(1, threads, smem_bytes(1024, FP8), nullptr, at);
    e = cudaOccupancyMaxActiveClusters(&most, expert_gemm_kernel<OP, FP8>, &cfg);
    if (e != cudaSuccess) return e;
    if (most <= 0) return cudaErrorInvalidConfiguration;
    if (dev < 64) cached[dev].store(most, std::memory_order_relaxed);
  }
  const cudaLaunchConfig_t cfg = pair_config((int)min64(most_tiles, most), threads, smem_bytes(p.E, FP8), st, at);
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
  p.k = a->k;
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
  }
  if (gw) {
    const uint64_t dims[3] = {(uint64_t)a->N, (uint64_t)a->rows, 1}, str[2] = {(uint64_t)a->ld_d_y * eb, (uint64_t)a->ld_d_y * eb};
    const uint32_t box[3] = {64, 64, 1};
    if (!map_of(&p.tmw, a->d_y, a->dtype, 3, dims, str, box)) return MOER_ECUDA;
  } else {
    const bool one = a->E == 1 || p.one_w;
    const uint64_t dims[3] = {(uint64_t)a->K, (uint64_t)a->N, (uint64_t)(one ? 1 : a->E)};
    const uint64_t str[2] = {(uint64_t)a->ld_w * eb, (uint64_t)(one ? a->ld_w : a->stride_w) * eb};
    const uint32_t box[3] = {(uint32_t)ke, fwd ? 128u : 64u, 1};
    if (!map_of(&p.tmw, a->w, a->dtype, 3, dims, str, box)) return MOER_ECUDA;
  }
  const int64_t most = (gw ? (int64_t)a->E * p.njb : (a->rows + EG_J - 1) / EG_J + min64(a->E, a->rows)) * p.nmb;
  const cudaError_t e = fp8   ? gemm_run<MOER_GEMM_FORWARD, true>(p, most, st)
                        : fwd ? gemm_run<MOER_GEMM_FORWARD, false>(p, most, st)
                        : gw  ? gemm_run<MOER_GEMM_GRAD_WEIGHT, false>(p, most, st)
                              : gemm_run<MOER_GEMM_GRAD_INPUT, false>(p, most, st);
  return e == cudaSuccess ? MOER_OK : MOER_ECUDA;
}

}  // namespace moer
