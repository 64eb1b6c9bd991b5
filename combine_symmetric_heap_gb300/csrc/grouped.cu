// grouped.cu -- matrix products grouped by expert with ragged row counts, the
// products that training an MoE layer needs besides the fused forward FFN:
//
//   product   out[r][f] = sum_c x[r][c] * w[e][f][c]     (forward; K = C)
//             out[r][f] = sum_c x[r][c] * w[e][c][f]     (trans: data gradient)
//   wgrad     dw[e][f][c] (+)= sum_{r of e} dy[r][f] * x[r][c]  (K = the rows)
//
// for the rows r of group e, a contiguous range [off_e, off_e + cnt_e) of its
// slot, read from device memory by the kernels (no host sync).  bf16 or fp16
// operands, fp32 accumulation in TMEM, one rounding of the result.
//
// Both run on CTA pairs (tcgen05 cta_group::2, M = 256, N <= 256; the pair
// protocol of gemm2sm.cuh: each CTA stages its half of both operands, copies
// of both count on the leader's full barrier, its commits free the stage in
// both).  The product keeps weights on the M side and rows on N, so a ragged
// group shortens N; wgrad has features on both sides and the ragged axis is
// K: whole MMA steps of 16 rows stream through the ring, and the last cnt mod
// 16 rows of a group take a step of their own from a side buffer, where the
// rows past the group's end (they belong to another group, or to nobody, and
// may hold anything) are zeroed first.
//
// An operand whose contraction index is the outer one in memory (trans
// weights, both operands of wgrad) is staged as it lies: boxes of 64
// contraction rows x 64 features, a tile the tensor core reads in its
// "MN-major" form, so no operand is ever transposed by a copy.
//
// Measured (bf16; measured rates: copy 6.69 TB/s, library GEMM 1867 TFLOP/s in a burst, 1710 under
// the power cap): product of 8192 rows in 256 groups, 7168 -> 2048, 1.17 ms (6.57
// TB/s, bound by the weights' read); of 65536 rows 1.49 ms for a pass by itself, 1.64 to
// 1.68 ms back to back under the power cap (the narrow second MMA of groups of 257..288
// rows then bounds half the tiles); data gradient 32768 rows, 8 groups, 4096 ->
// 14336, 2.41 to 2.49 ms (1540 to 1600 TFLOP/s, the power cap).  Weight gradient of the
// 65536 rows (7.5 GB written) 1.95 to 1.99 ms; where every count is a multiple of 16 1.65
// ms in runs of three, 1.83 under the power cap.  No single unit bounds it: at 64 of these
// groups DRAM is 65% busy, L1 and shared memory 76%, the tensor pipe 49% (58, 68 and 45
// with ragged counts), and the same bytes written by themselves take 1.10 ms.  Into
// fp32 2.73 ms, added to what is there 6.2 ms (15 GB read, 15 written).  8 groups of
// 4096 rows, 4096 x 14336: 2.02 ms in runs of three (1.91 PFLOP/s), 2.31 ms
// back to back (1.67 PFLOP/s at the 1.54 GHz that the power cap leaves).
#include <algorithm>

#include "pair_ops.cuh"

namespace symmoe {
namespace grouped {

using namespace pair;

constexpr int PRODUCT_THREADS = 192;  // producer, MMA issuer, 4 epilogue warps
constexpr int WG_EPI_WARPS = 8;       // two per TMEM lane quarter, each with half of a tile's columns
constexpr int WGRAD_THREADS = 32 * (3 + WG_EPI_WARPS);  // ... and the warp of the groups' last rows
constexpr int CTRL_BYTES = 512;
// A call's most groups.  The product's tables take their 12 KB whatever the call's
// number: one shared-memory size for the kernel, so that calls from several host
// threads set the same limit and the resident pairs are looked up once.
constexpr int MAX_GROUPS = 1024;
constexpr int WG_STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int WG_STAGES = 6;
constexpr int WG_OUT_BYTES = 32 * 64;  // staged output of a warp: 32 rows of 64 bytes

struct Groups {
  const int32_t *cnt, *off;
  int64_t cnt_ss, off_ss;  // elements between slots
  int G, per_slot;
  int64_t cap;  // rows per slot
  int32_t *status;
  uint32_t tmo;
};

struct Out {
  void *ptr;
  int64_t ld, stride;  // elements between rows, and between slots (product) or groups (wgrad)
};

__device__ __forceinline__ void tma_load_3d_pair_hint(void *dst, const CUtensorMap *m, uint32_t bar_cluster, int x,
                                                      int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// ---------------------------------------------------------------------------
// group tables: rows, first row and prefix of row tiles of every group.  A
// group whose range does not lie in its slot is taken as empty and flagged.
// ---------------------------------------------------------------------------
__device__ inline void build_tables(const Groups &g, const TokTables &tb, bool report) {
  for (int e = threadIdx.x; e < g.G; e += blockDim.x) {
    const int d = e / g.per_slot, l = e - d * g.per_slot;
    int c = g.cnt[d * g.cnt_ss + l], o = g.off[d * g.off_ss + l];
    if (c < 0 || o < 0 || (int64_t)o + c > g.cap) {
      if (report) raise(g.status, SYM_STATUS_OVERFLOW);
      c = 0;
      o = 0;
    }
    tb.cnt[e] = c;
    tb.roff[e] = o;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    if (lane == 0) tb.tokprefix[0] = 0;
    for (int e0 = 0; e0 < g.G; e0 += 32) {
      const int e = e0 + lane;
      int incl = e < g.G ? ntok_of(tb.cnt[e]) : 0;
#pragma unroll
      for (int step = 1; step < 32; step <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, step);
        if (lane >= step) incl += o;
      }
      if (e < g.G) tb.tokprefix[e + 1] = carry + incl;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}

struct Tile {
  int e, d, f, row0, valid, single;
};

// Tile t of the product: per group, row tiles in runs of `run`, feature tile
// major inside a run (consecutive tiles share weight rows).
__device__ inline Tile decode_product(const Groups &g, const TokTables &tb, int nf, int run, int t) {
  const int key = t / nf;
  int lo = 0, hi = g.G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tb.tokprefix[mid] <= key) lo = mid; else hi = mid;
  }
  Tile ti;
  ti.e = lo;
  ti.d = lo / g.per_slot;
  const int c = tb.cnt[lo], ntok = ntok_of(c);
  const int local = t - tb.tokprefix[lo] * nf;
  const int R = min(run, ntok);
  const int r = local / (R * nf), in_run = local - r * R * nf;
  const int w = min(R, ntok - r * R);
  ti.f = in_run / w;
  const int n = r * R + in_run % w;
  ti.row0 = tb.roff[lo] + n * BN;
  ti.valid = n == ntok - 1 ? c - n * BN : BN;
  ti.single = ntok == 1;
  return ti;
}

// ---------------------------------------------------------------------------
// product kernel
// ---------------------------------------------------------------------------
using Ring = RingOf<STAGES>;

// K loop of the producer for one tile; TWO: with a remainder part
template <bool TRANS, bool TWO>
__device__ __forceinline__ bool product_load(Ring &rg, const Ctl &ctl, uint32_t rank, const CUtensorMap *ma,
                                             const CUtensorMap *mb0, const CUtensorMap *mb1, int e, int d, int f0,
                                             int r0, int r1, uint32_t tx, int nk, uint64_t pol) {
  const uint32_t full_leader = map_to(rg.full, 0);
  for (int kb = 0; kb < nk; ++kb) {
    if (!bar_wait(&rg.empty[rg.stage], rg.phase ^ 1u, ctl)) return false;
    uint8_t *sb = rg.base + (size_t)rg.stage * STAGE_BYTES;
    const uint32_t bar = full_leader + (uint32_t)(rg.stage * sizeof(uint64_t));
    if (rank == 0) mbar_arrive_expect_tx(&rg.full[rg.stage], tx);
    if (TRANS) {  // 64 contraction rows of 2 x 64 features
      tma_load_3d_pair_hint(sb, ma, bar, f0, kb * BK, e, pol);
      tma_load_3d_pair_hint(sb + CHUNK_BYTES, ma, bar, f0 + 64, kb * BK, e, pol);
    } else {  // 128 feature rows of 64 contraction columns
      tma_load_3d_pair_hint(sb, ma, bar, kb * BK, f0, e, pol);
    }
    tma_load_3d_pair(sb + A_BYTES, mb0, bar, kb * BK, r0, d);
    if (TWO) tma_load_3d_pair(sb + A_BYTES + B_BYTES, mb1, bar, kb * BK, r1, d);
    rg.next();
  }
  return true;
}

template <bool TRANS, bool TWO>
__device__ __forceinline__ bool product_mma(Ring &rg, const Ctl &ctl, uint32_t d0, uint32_t d1, uint32_t i0,
                                            uint32_t i1, int nk) {
  constexpr uint64_t astep = TRANS ? MN_STEP : K_STEP;
  for (int kb = 0; kb < nk; ++kb) {
    if (!bar_wait(&rg.full[rg.stage], rg.phase, ctl)) return false;
    tc_fence_after();
    uint8_t *sb = rg.base + (size_t)rg.stage * STAGE_BYTES;
    const uint64_t da = TRANS ? smem_desc_mn(sb) : smem_desc_sw128(sb);
    const uint64_t db0 = smem_desc_sw128(sb + A_BYTES), db1 = smem_desc_sw128(sb + A_BYTES + B_BYTES);
#pragma unroll
    for (int kk = 0; kk < BK / UK; ++kk) {
      const uint32_t acc = (kb > 0 || kk > 0) ? 1u : 0u;
      mma2(d0, da + kk * astep, db0 + kk * K_STEP, i0, acc);
      if (TWO) mma2(d1, da + kk * astep, db1 + kk * K_STEP, i1, acc);
    }
    commit2_both(&rg.empty[rg.stage]);
    rg.next();
  }
  return true;
}

// Rows [row, row + n) of a tile: this lane's feature of each
template <bool FP16, typename Head>
__device__ __forceinline__ void product_store(uint32_t tcol, uint16_t *out, int64_t ld, bool live, int n, Head head) {
  for (int c0 = 0; c0 < n; c0 += 32) {
    uint32_t v[32];
    tmem_ld32(tcol + c0, v);
    tmem_ld_wait();
    if (c0 == 0) head();
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (live && c0 + c < n) out[(int64_t)(c0 + c) * ld] = narrow<FP16>(__uint_as_float(v[c]));
  }
}

template <bool TRANS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PRODUCT_THREADS, 1)
    grouped_product_kernel(const Groups g, const Out o, int F, int C, int fp16, int run,
                           const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ BMaps tm_x) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *ctrl = smem + (size_t)STAGES * STAGE_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(ctrl);
  uint64_t *acc_full = bars + 2 * STAGES, *acc_empty = acc_full + 2, *acc_head = acc_full + 4;
  uint64_t *drained = acc_full + 6;
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base_s + 1);
  int *tab = reinterpret_cast<int *>(ctrl + CTRL_BYTES);
  const TokTables tb{tab, tab + g.G, tab + 2 * g.G};
  const int wid = warp_id(), lane = lane_id();
  const uint32_t rank = cta_rank();
  const int pair = (int)cluster_id_x(), npairs = (int)num_clusters_x();
  const Ctl ctl{abort_flag, g.status, g.tmo};
  Ring rg{smem, bars, bars + STAGES};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&rg.full[s], 1);
      mbar_init(&rg.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);  // 4 epilogue warps of each CTA
      mbar_init(&acc_head[b], 8);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w);
    for (int i = 0; i < NBOX; ++i) tma_prefetch_desc(&tm_x.m[i]);
  }
  if (wid == 1) {
    tmem_alloc2(tmem_base_s, TMEM_COLS);
    tmem_relinquish2();
  }
  build_tables(g, tb, blockIdx.x == 0);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const int nf = (F + 255) / 256, nk = (C + BK - 1) / BK;
  const int total = tb.tokprefix[g.G] * nf;

  if (wid == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      const uint64_t normal = l2_evict_normal_policy(), once = l2_evict_first_policy();
      for (int i = 0, t; (t = pair_tile(i, pair, npairs)) < total; ++i) {
        const Tile ti = decode_product(g, tb, nf, run, t);
        const TileGeom gm = geom(ti.valid);
        const int half0 = gm.n0 / 2, half1 = gm.n1 / 2;
        const int b0 = box_index(half0), b1 = box_index(max(half1, 1));
        const uint32_t rows = (uint32_t)(BOX_MIN_ROWS << b0) + (gm.n1 ? (uint32_t)(BOX_MIN_ROWS << b1) : 0u);
        const uint32_t tx = 2u * ((uint32_t)A_BYTES + rows * BK * 2);
        const int f0 = ti.f * 256 + (int)rank * 128;
        const int r0 = ti.row0 + (int)rank * half0, r1 = ti.row0 + BN + (int)rank * half1;
        // weights that no other tile reads leave L2 to the rows and outputs
        const uint64_t pol = ti.single && ti.valid >= BN / 2 ? once : normal;
        const bool ok = gm.n1 ? product_load<TRANS, true>(rg, ctl, rank, &tm_w, &tm_x.m[b0], &tm_x.m[b1], ti.e, ti.d,
                                                          f0, r0, r1, tx, nk, pol)
                              : product_load<TRANS, false>(rg, ctl, rank, &tm_w, &tm_x.m[b0], &tm_x.m[b1], ti.e,
                                                           ti.d, f0, r0, r1, tx, nk, pol);
        if (!ok) break;
      }
    }
  } else if (wid == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------------------------------------------- MMA issuer (leader)
      // acquisition n of a barrier waits for its release n - 1
      uint32_t ne[2] = {0, 0}, nh[2] = {0, 0};
      auto acquire = [&](uint64_t *bar, uint32_t &n) { return bar_wait(bar, (n++ & 1u) ^ 1u, ctl); };
      int b = 0;
      for (int i = 0, t; (t = pair_tile(i, pair, npairs)) < total; ++i, b ^= 1) {
        const Tile ti = decode_product(g, tb, nf, run, t);
        const TileGeom gm = geom(ti.valid);
        // the main part takes all of accumulator b, a remainder the head of the other
        if (!acquire(&acc_empty[b], ne[b]) || !acquire(&acc_head[b], nh[b])) break;
        if (gm.n1 && !acquire(&acc_head[b ^ 1], nh[b ^ 1])) break;
        tc_fence_after();
        const uint32_t d0 = tmem + (uint32_t)(b * ACC_COLS), d1 = tmem + (uint32_t)((b ^ 1) * ACC_COLS);
        const uint32_t i0 = idesc(fp16, TRANS, false, gm.n0);
        const bool ok = gm.n1 ? product_mma<TRANS, true>(rg, ctl, d0, d1, i0, idesc(fp16, TRANS, false, gm.n1), nk)
                              : product_mma<TRANS, false>(rg, ctl, d0, d1, i0, i0, nk);
        if (!ok) break;
        commit2_both(&acc_full[b]);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = wid & 3;  // TMEM lane quarter of this warp
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    uint32_t used[2] = {0, 0};
    int b = 0;
    for (int i = 0, t; (t = pair_tile(i, pair, npairs)) < total; ++i, b ^= 1) {
      const Tile ti = decode_product(g, tb, nf, run, t);
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full[b], used[b]++ & 1u, ctl))) break;
      tc_fence_after();
      const int f = ti.f * 256 + (int)rank * 128 + q * 32 + lane;
      // the remainder (head of the other accumulator) first; the first 32
      // columns are handed back as soon as they are read
      for (int part = ti.valid > BN ? 1 : 0; part >= 0; --part) {
        const int buf = part ? (b ^ 1) : b;
        const int row = ti.row0 + part * BN, n = part ? ti.valid - BN : min(ti.valid, BN);
        uint16_t *out = reinterpret_cast<uint16_t *>(o.ptr) + ti.d * o.stride + (int64_t)row * o.ld + f;
        const uint32_t tcol = lanes + (uint32_t)(buf * ACC_COLS);
        auto head = [&]() { give_back(&acc_head[buf], rank, lane); };
        if (fp16) product_store<true>(tcol, out, o.ld, f < F, n, head);
        else product_store<false>(tcol, out, o.ld, f < F, n, head);
        if (part == 0) give_back(&acc_empty[buf], rank, lane);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) settle(drained, wid == 1 && lane == 0 && rank == 0);
  __syncwarp();
  cluster_sync();  // no remote arrive or MMA of the pair is still in flight
  tc_fence_after();
  if (wid == 1) tmem_dealloc2(tmem, TMEM_COLS);
}

// ---------------------------------------------------------------------------
// weight gradient kernel: tile (e, f, c) = 256 x tile_c of dw[e], K = cnt_e rows.
// tile_c is 256, or 128 where every pair still has one tile at most: the time is
// then one tile's K axis, whose blocks take less (one group of 56548 rows, 1096 x
// 872: 371 -> 285 us; 8 groups, 4096 rows, 512 x 512: 18.4 -> 15.4; the wide
// tile's are bound by the pair's tensor cores, the narrow one's by six loads in
// flight).  With more tiles the wide one's operands are read less often.
// ---------------------------------------------------------------------------
// Row boxes of a K block: a group's last block loads 16, 32 or 64 rows,
// whichever holds what is left of its whole steps.
constexpr int WG_BOXES = 3;
// The side buffer of a group's last cnt mod 16 rows: 16 rows of the CTA's four
// chunks.  Cutting the last K block in the ring instead held its slot through
// copy, zeroing and two barriers: 0.3 of 1.98 ms on the prefill shape.
constexpr int REST_CHUNK = UK * 128;
constexpr int REST_BYTES = 4 * REST_CHUNK;
struct WMaps {
  CUtensorMap m[WG_BOXES];
};

struct WTile {
  int e, d, f, c, row0, cnt;
};
// Tile t, with the group's range read (and checked) when the group changes:
// one role's walk of the tiles.
struct WWalk {
  const Groups &g;
  int nf, nc;
  WTile ti;
  __device__ WWalk(const Groups &g_, int nf_, int nc_) : g(g_), nf(nf_), nc(nc_) { ti.e = -1; }
  __device__ __forceinline__ const WTile &at(int t) {
    const int e = t / (nf * nc), r = t - e * nf * nc;
    ti.f = r / nc;  // the x tiles of a group pass under each dy tile
    ti.c = r - ti.f * nc;
    if (e != ti.e) {
      ti.e = e;
      ti.d = e / g.per_slot;
      const int l = e - ti.d * g.per_slot;
      const int c = __ldg(g.cnt + ti.d * g.cnt_ss + l), o = __ldg(g.off + ti.d * g.off_ss + l);
      const bool ok = c >= 0 && o >= 0 && (int64_t)o + c <= g.cap;
      ti.cnt = ok ? c : 0;
      ti.row0 = ok ? o : 0;
    }
    return ti;
  }
};

enum OutType { OUT_BF16, OUT_FP16, OUT_FP32 };

// 32 columns of this thread's output row; vec: 16-byte stores are aligned and
// all 32 columns exist
template <int OT>
__device__ __forceinline__ void wgrad_store(void *row, const uint32_t (&v)[32], int n, bool vec, bool add) {
  float a[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) a[i] = __uint_as_float(v[i]);
  if (OT == OUT_FP32) {
    float *p = reinterpret_cast<float *>(row);
    if (vec) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float4 s = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
        if (add) {
          const float4 old = *reinterpret_cast<const float4 *>(p + i);
          s.x += old.x, s.y += old.y, s.z += old.z, s.w += old.w;
        }
        *reinterpret_cast<float4 *>(p + i) = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < n) p[i] = add ? a[i] + p[i] : a[i];
    }
    return;
  }
  constexpr bool H = OT == OUT_FP16;
  uint16_t *p = reinterpret_cast<uint16_t *>(row);
  if (vec) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      if (add) {
        const uint4 old = *reinterpret_cast<const uint4 *>(p + i);
        const uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[i + 2 * j] += widen(H, (uint16_t)w[j]);
          a[i + 2 * j + 1] += widen(H, (uint16_t)(w[j] >> 16));
        }
      }
      *reinterpret_cast<uint4 *>(p + i) =
          make_uint4(narrow2<H>(a[i], a[i + 1]), narrow2<H>(a[i + 2], a[i + 3]), narrow2<H>(a[i + 4], a[i + 5]),
                     narrow2<H>(a[i + 6], a[i + 7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) p[i] = narrow<H>(add ? a[i] + widen(H, p[i]) : a[i]);
  }
}

// This lane's row of a staged box (64 bytes: 16 floats or 32 16-bit values), in
// the 64-byte swizzle: 16-byte word j of row r sits at word j ^ (r / 2 mod 4).
template <int OT>
__device__ __forceinline__ void stage_row(uint8_t *box, int lane, const uint32_t *v) {
  uint8_t *row = box + lane * 64;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 w;
    if (OT == OUT_FP32) {
      w = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
      constexpr bool H = OT == OUT_FP16;
      const uint32_t *s = v + 8 * j;
      w = make_uint4(narrow2<H>(__uint_as_float(s[0]), __uint_as_float(s[1])),
                     narrow2<H>(__uint_as_float(s[2]), __uint_as_float(s[3])),
                     narrow2<H>(__uint_as_float(s[4]), __uint_as_float(s[5])),
                     narrow2<H>(__uint_as_float(s[6]), __uint_as_float(s[7])));
    }
    *reinterpret_cast<uint4 *>(row + ((j ^ ((lane >> 1) & 3)) << 4)) = w;
  }
}

// by_tma: the output's rows are 16-byte aligned and written (fp32: or added)
// by tensor copies from a staged box per warp.  Direct stores of each lane's
// row touch 32 lines per instruction with half a sector each: the prefill
// shape (256 experts, 2048 x 7168, bf16) took 4.57 ms that way.
template <int OT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WGRAD_THREADS, 1)
    grouped_wgrad_kernel(const Groups g, const Out o, int F, int C, int fp16, int add, int by_tma, int tile_c,
                         const __grid_constant__ WMaps tm_dy, const __grid_constant__ WMaps tm_x,
                         const __grid_constant__ CUtensorMap tm_dw) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *rest = smem + (size_t)WG_STAGES * WG_STAGE_BYTES;  // [2]
  uint8_t *boxes = rest + 2 * REST_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(boxes + WG_EPI_WARPS * WG_OUT_BYTES);
  uint64_t *rest_in = bars + 2 * WG_STAGES;  // [2] this CTA's copies of a group's last rows have landed
  uint64_t *rest_peer = rest_in + 2;         // [2] (the leader's) the peer's half is zeroed past the end
  uint64_t *rest_full = rest_in + 4;         // [2] (the leader's) both halves are
  uint64_t *rest_empty = rest_in + 6;        // [2] the MMA has read it
  uint64_t *acc_full = rest_in + 8, *acc_empty = acc_full + 2;
  uint64_t *drained = acc_full + 4;
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base_s + 1);
  const int wid = warp_id(), lane = lane_id();
  const uint32_t rank = cta_rank();
  const int pair = (int)cluster_id_x(), npairs = (int)num_clusters_x();
  const Ctl ctl{abort_flag, g.status, g.tmo};
  RingOf<WG_STAGES> rg{smem, bars, bars + WG_STAGES};

  if (threadIdx.x == 0) {
    for (int s = 0; s < WG_STAGES; ++s) {
      mbar_init(&rg.full[s], 1);
      mbar_init(&rg.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      for (int k = 0; k < 8; k += 2) mbar_init(&rest_in[k + b], 1);
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * WG_EPI_WARPS);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < WG_BOXES; ++i) {
      tma_prefetch_desc(&tm_dy.m[i]);
      tma_prefetch_desc(&tm_x.m[i]);
    }
    if (by_tma) tma_prefetch_desc(&tm_dw);
  }
  if (wid == 1) {
    tmem_alloc2(tmem_base_s, TMEM_COLS);
    tmem_relinquish2();
  }
  if (blockIdx.x == 0 && g.status)  // groups outside their slot: taken as empty, and flagged
    for (int e = threadIdx.x; e < g.G; e += blockDim.x) {
      const int d = e / g.per_slot, l = e - d * g.per_slot;
      const int c = g.cnt[d * g.cnt_ss + l], o = g.off[d * g.off_ss + l];
      if (c < 0 || o < 0 || (int64_t)o + c > g.cap) raise(g.status, SYM_STATUS_OVERFLOW);
    }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const int nf = (F + 255) / 256, nc = (C + tile_c - 1) / tile_c;
  const int total = g.G * nf * nc;
  const int own_c = tile_c / 2;  // columns of x that this CTA stages: one or two chunks
  WWalk walk(g, nf, nc);

  if (wid == 0) {
    if (lane == 0) {
      // ------------------------------------------- producer of the whole steps
      const uint32_t full_leader = map_to(rg.full, 0);
      bool ok = true;
      for (int i = 0, t; ok && (t = pair_tile(i, pair, npairs)) < total; ++i) {
        const WTile &ti = walk.at(t);
        const int whole = ti.cnt & ~(UK - 1);
        const int f0 = ti.f * 256 + (int)rank * 128, c0 = ti.c * tile_c + (int)rank * own_c;
        for (int k0 = 0; k0 < whole; k0 += BK) {
          if (!(ok = bar_wait(&rg.empty[rg.stage], rg.phase ^ 1u, ctl))) break;
          uint8_t *sb = rg.base + (size_t)rg.stage * WG_STAGE_BYTES;
          const int row = ti.row0 + k0, left = whole - k0;
          const int box = left > 32 ? 2 : left > 16 ? 1 : 0;
          const CUtensorMap *my = &tm_dy.m[box], *mx = &tm_x.m[box];
          const uint32_t bar = full_leader + (uint32_t)(rg.stage * sizeof(uint64_t));
          if (rank == 0) mbar_arrive_expect_tx(&rg.full[rg.stage], (4u + (uint32_t)tile_c / 64u) * 128u * (16u << box));  // both CTAs' chunks
          for (int h = 0; h < 2; ++h) {
            tma_load_3d_pair(sb + h * CHUNK_BYTES, my, bar, f0 + h * 64, row, ti.d);
            if (h * 64 < own_c) tma_load_3d_pair(sb + A_BYTES + h * CHUNK_BYTES, mx, bar, c0 + h * 64, row, ti.d);
          }
          rg.next();
        }
      }
    }
  } else if (wid == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------------------------------------------- MMA issuer (leader)
      uint32_t ne[2] = {0, 0}, nr = 0;  // accumulators acquired, side buffers read
      const uint32_t id = idesc(fp16, true, true, tile_c);
      int b = 0;
      bool ok = true;
      for (int i = 0, t; ok && (t = pair_tile(i, pair, npairs)) < total; ++i) {
        const WTile &ti = walk.at(t);
        if (ti.cnt == 0) continue;
        const int whole = ti.cnt & ~(UK - 1);
        if (!(ok = bar_wait(&acc_empty[b], (ne[b]++ & 1u) ^ 1u, ctl))) break;
        tc_fence_after();
        const uint32_t d0 = tmem + (uint32_t)(b * ACC_COLS);
        for (int k0 = 0; k0 < whole; k0 += BK) {
          if (!(ok = bar_wait(&rg.full[rg.stage], rg.phase, ctl))) break;
          tc_fence_after();
          uint8_t *sb = rg.base + (size_t)rg.stage * WG_STAGE_BYTES;
          const uint64_t da = smem_desc_mn(sb), db = smem_desc_mn(sb + A_BYTES);
          const int steps = min(BK, whole - k0) / UK;
#pragma unroll
          for (int kk = 0; kk < BK / UK; ++kk)
            if (kk < steps) mma2(d0, da + kk * MN_STEP, db + kk * MN_STEP, id, (k0 > 0 || kk > 0) ? 1u : 0u);
          commit2_both(&rg.empty[rg.stage]);
          rg.next();
        }
        if (!ok) break;
        if (ti.cnt != whole) {
          const int j = nr & 1;
          if (!(ok = bar_wait(&rest_full[j], (nr >> 1) & 1u, ctl))) break;
          ++nr;
          tc_fence_after();
          uint8_t *sb = rest + j * REST_BYTES;
          mma2(d0, smem_desc_mn(sb, REST_CHUNK), smem_desc_mn(sb + 2 * REST_CHUNK, REST_CHUNK), id, whole ? 1u : 0u);
          commit2_both(&rest_empty[j]);
        }
        commit2_both(&acc_full[b]);
        b ^= 1;
      }
    }
  } else if (wid == 2 + WG_EPI_WARPS) {
    // --------------------------------------------- the groups' last cnt mod 16
    // rows: loaded one tile ahead, zeroed past the end, reported to the leader.
    // This warp runs ahead over the tiles without such rows, so what it waits for
    // may come only after all of the pair's tiles so far.
    // Only these steps cross the pair by a release at cluster scope (as part
    // of every K block it held each to 0.8 us).
    auto load = [&](int i, uint32_t n) {  // tile i's rows as use n of the side buffers
      const WTile &ti = walk.at(pair_tile(i, pair, npairs));
      const int j = n & 1, row = ti.row0 + (ti.cnt & ~(UK - 1));
      const int f0 = ti.f * 256 + (int)rank * 128, c0 = ti.c * tile_c + (int)rank * own_c;
      if (!__all_sync(0xffffffffu, bar_wait(&rest_empty[j], ((n >> 1) & 1u) ^ 1u, ctl, i + 1))) return false;
      if (lane == 0) {
        uint8_t *sb = rest + j * REST_BYTES;
        mbar_arrive_expect_tx(&rest_in[j], (2u + (uint32_t)own_c / 64u) * REST_CHUNK);
        for (int h = 0; h < 2; ++h) {
          tma_load_3d(sb + h * REST_CHUNK, &tm_dy.m[0], &rest_in[j], f0 + h * 64, row, ti.d);
          if (h * 64 < own_c) tma_load_3d(sb + (2 + h) * REST_CHUNK, &tm_x.m[0], &rest_in[j], c0 + h * 64, row, ti.d);
        }
      }
      return true;
    };
    // the next tile from i on that has such rows
    auto next = [&](int i) {
      for (int t; (t = pair_tile(i, pair, npairs)) < total; ++i)
        if (walk.at(t).cnt & (UK - 1)) return i;
      return -1;
    };
    int i = next(0);
    uint32_t n = 0;
    bool ok = i < 0 || load(i, 0);
    while (ok && i >= 0) {
      const int r = walk.at(pair_tile(i, pair, npairs)).cnt & (UK - 1), j = n & 1;
      const uint32_t parity = (n >> 1) & 1u;
      const int after = next(i + 1);
      if (after >= 0 && !(ok = load(after, n + 1))) break;
      if (!(ok = __all_sync(0xffffffffu, bar_wait(&rest_in[j], parity, ctl)))) break;
      // a row past the end: 8 lanes x 16 bytes in each of the four chunks
      uint8_t *sb = rest + j * REST_BYTES + (lane >> 3) * REST_CHUNK + (lane & 7) * 16;
      for (int row = r; row < UK; ++row) *reinterpret_cast<uint4 *>(sb + row * 128) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_shared();  // the zeros before the tensor core's reads
      __syncwarp();
      if (rank != 0) {
        if (lane == 0) mbar_arrive_remote(map_to(&rest_peer[j], 0));
      } else {
        if (!(ok = __all_sync(0xffffffffu, bar_wait(&rest_peer[j], parity, ctl, i + 1)))) break;
        if (lane == 0) mbar_arrive(&rest_full[j]);
      }
      i = after;
      ++n;
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = wid & 3;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    constexpr int OB = OT == OUT_FP32 ? 4 : 2, BOX = 64 / OB;  // bytes of an element, columns of a box
    const bool aligned = ((reinterpret_cast<uintptr_t>(o.ptr) | (uintptr_t)(o.ld * OB) | (uintptr_t)(o.stride * OB)) & 15u) == 0;
    const int half = (wid - 2) / 4;
    uint8_t *box = boxes + (size_t)(wid - 2) * WG_OUT_BYTES;
    uint32_t used[2] = {0, 0};
    int b = 0;
    for (int i = 0, t; (t = pair_tile(i, pair, npairs)) < total; ++i) {
      const WTile &ti = walk.at(t);
      const int fw = ti.f * 256 + (int)rank * 128 + q * 32, f = fw + lane, c0 = ti.c * tile_c + half * own_c;  // the warp's rows, columns
      const int cols = min(own_c, C - c0);
      const bool empty = ti.cnt == 0;  // zeros, or nothing to add
      if (empty && add) continue;
      if (!empty && !__all_sync(0xffffffffu, bar_wait(&acc_full[b], used[b]++ & 1u, ctl))) break;
      tc_fence_after();
      const uint32_t acc = lanes + (uint32_t)(b * ACC_COLS + half * own_c);
      if (by_tma) {
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          uint32_t v[32];
          if (empty) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          } else {
            tmem_ld32(acc + (uint32_t)c, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int j = 0; j < 32; j += BOX) {
            if (lane == 0) bulk_wait_read<0>();  // the last copy has left the box
            __syncwarp();
            stage_row<OT>(box, lane, v + j);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (fw < F && c + j < cols) {
                if (OT == OUT_FP32 && add) tma_add_3d(&tm_dw, box, c0 + c + j, fw, ti.e);
                else tma_store_3d(&tm_dw, box, c0 + c + j, fw, ti.e);
              }
              bulk_commit();
            }
          }
        }
      } else {
        uint8_t *row = reinterpret_cast<uint8_t *>(o.ptr) + ((int64_t)ti.e * o.stride + (int64_t)f * o.ld + c0) * OB;
        for (int c = 0; c < cols; c += 32) {
          uint32_t v[32] = {};
          if (!empty) {
            tmem_ld32(acc + (uint32_t)c, v);
            tmem_ld_wait();
          }
          if (f < F) wgrad_store<OT>(row + c * OB, v, cols - c, aligned && c + 32 <= cols, add != 0);
        }
      }
      if (empty) continue;
      give_back(&acc_empty[b], rank, lane);
      b ^= 1;
    }
    if (lane == 0) bulk_wait_all();  // the copies have read their shared memory before the block ends
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) settle(drained, wid == 1 && lane == 0 && rank == 0);
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (wid == 1) tmem_dealloc2(tmem, TMEM_COLS);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// rows of a sym_rows, boxes of [box_rows][64]
static bool encode_rows(CUtensorMap *m, const sym_rows &r, uint32_t box_rows) {
  const int64_t slot = r.slots > 1 ? r.slot_stride : r.ld * r.rows;
  return encode(m, r.ptr, (uint64_t)r.cols, (uint64_t)r.rows, (uint64_t)r.slots, r.ld, slot, BK, box_rows);
}

static Groups groups_of(const sym_groups &g, const sym_rows &rows) {
  return Groups{g.cnt, g.off, g.cnt_slot_stride, g.off_slot_stride, g.groups, g.groups / g.slots, rows.rows,
                g.status, g.wait_timeout_us};
}

}  // namespace grouped

cudaError_t launch_grouped_matmul(const sym_groups &sg, int fp16, const sym_rows &x, const void *w, int64_t w_group,
                                  int64_t w_ld, int trans, const sym_rows &out, int num_sms, cudaStream_t st) {
  using namespace grouped;
  const int F = out.cols, C = x.cols;
  CUtensorMap mw;
  BMaps mx;
  const uint64_t wp = reinterpret_cast<uint64_t>(w);
  const int64_t wg = sg.groups > 1 ? w_group : w_ld * (trans ? C : F);
  if (!(trans ? encode(&mw, wp, F, C, sg.groups, w_ld, wg, 64, BK) : encode(&mw, wp, C, F, sg.groups, w_ld, wg, BK, 128)))
    return cudaErrorInvalidValue;
  for (int i = 0; i < NBOX; ++i)
    if (!encode_rows(&mx.m[i], x, (uint32_t)(BOX_MIN_ROWS << i))) return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)STAGES * STAGE_BYTES + CTRL_BYTES + tok_tables_bytes(MAX_GROUPS);
  // row tiles of a run: their rows fit 64 MB, so a wave's rows stay in L2
  // while the feature tiles pass (the expert FFN's budget for wide rows)
  const int run = (int)std::max<int64_t>(1, GROUP_H_BYTES / ((int64_t)BN * C * 2));
  const Groups g = groups_of(sg, x);
  const Out o{reinterpret_cast<void *>(out.ptr), out.ld, out.slots > 1 ? out.slot_stride : 0};
  return trans ? launch_pairs(grouped_product_kernel<true>, PRODUCT_THREADS, smem, num_sms, st, g, o, F, C, fp16, run, mw, mx)
               : launch_pairs(grouped_product_kernel<false>, PRODUCT_THREADS, smem, num_sms, st, g, o, F, C, fp16, run, mw, mx);
}

cudaError_t launch_grouped_wgrad(const sym_groups &sg, int fp16, const sym_rows &dy, const sym_rows &x, void *dw,
                                 int64_t dw_group, int64_t dw_ld, int out_type, int add, int num_sms,
                                 cudaStream_t st) {
  using namespace grouped;
  WMaps md, mx;
  sym_rows ry = dy, rx = x;
  if (x.rows == 0) {  // no rows at all: nothing is loaded; maps over the output keep the encoder content
    ry.ptr = rx.ptr = reinterpret_cast<uint64_t>(dw) & ~uint64_t(15);
    ry.rows = rx.rows = 1;
  }
  for (int i = 0; i < WG_BOXES; ++i)
    if (!encode_rows(&md.m[i], ry, 16u << i) || !encode_rows(&mx.m[i], rx, 16u << i)) return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)WG_STAGES * WG_STAGE_BYTES + 2 * REST_BYTES + WG_EPI_WARPS * WG_OUT_BYTES + CTRL_BYTES;
  const Groups g = groups_of(sg, x);
  const Out o{dw, dw_ld, dw_group};
  // Tensor copies need 16-byte aligned rows.  16-bit sums onto old values are
  // stored directly: they are rounded once, a copy would add rounded values.
  const bool fp32 = out_type == OUT_FP32;
  const int64_t per16 = fp32 ? 4 : 8, gs = sg.groups > 1 ? dw_group : dw_ld * dy.cols;
  const int by_tma = reinterpret_cast<uintptr_t>(dw) % 16 == 0 && dw_ld % per16 == 0 && gs % per16 == 0 && (fp32 || !add);
  CUtensorMap mo = md.m[0];
  if (by_tma && !encode(&mo, reinterpret_cast<uint64_t>(dw), x.cols, dy.cols, sg.groups, dw_ld, gs, fp32 ? 16 : 32, 32, fp32,
                        CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const int64_t narrow = (int64_t)sg.groups * ((dy.cols + 255) / 256) * ((x.cols + 127) / 128);
  const int tile_c = narrow <= num_sms / 2 ? 128 : 256;
  auto go = [&](auto kern) {
    return launch_pairs(kern, WGRAD_THREADS, smem, num_sms, st, g, o, dy.cols, x.cols, fp16, add, by_tma, tile_c, md, mx, mo);
  };
  return fp32 ? go(grouped_wgrad_kernel<OUT_FP32>)
              : fp16 ? go(grouped_wgrad_kernel<OUT_FP16>) : go(grouped_wgrad_kernel<OUT_BF16>);
}

}  // namespace symmoe
