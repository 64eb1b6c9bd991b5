// orthogonalize.cu -- Newton-Schulz products that bring the singular values of a
// batch of matrices towards one:
//
//   X = g / (|g| + eps);   steps times  A = X X^T,  B = b A + c A A,  X = a X + B X
//
// (tall matrices: A = X^T X and X B; A is square with the shorter side m).
//
// How the numbers are held.  The products take fp16 operands (11 bits; bf16's 8
// would leave an error of 1e-2 in the result, where a bf16 result's own rounding is
// 1.7e-3).  What a product multiplies may be rounded; what is carried from step to
// step may not, since small singular values grow by a = 3.4 a step and errors
// beside them likewise:
//   - X is hi + lo, two fp16 numbers (22 bits): a X is taken of both, B X of hi or of both;
//   - A and B are their diagonal in fp32 and the rest in fp16, one number or two.  With D and O for
//     the two, A A = D D + D O + O D + O O: only O O is a product of matrices, the
//     rest belongs to one element each.  As X comes near to orthogonality the
//     diagonals come near to constants and the rests to zero, and so does what
//     their rounding leaves.
// The first two steps of matrices that are wider than tall (or the other way) share one
// update: with P = a I + B, the second's Gram matrix is A' = P A P, and X goes to P' P X.  All
// of these commute and are symmetric, and their products, of the shorter side, cost less than an update and a Gram
// matrix.  It is for the first two only: what rounding leaves in A is taken times P
// squared, up to a^2 = 12, where singular values are small; beside an A of at most one
// that adds 2e-4 of a result's norm or less (with the third and fourth step so too the error
// is 3e-3).  Not where products take both parts (PRECISE_SIDE): the shared factors are rounded to 11 bits.
//
// All are held times a power of two that keeps them in fp16's range: X (entries at
// most its largest singular value; 1 / sqrt(m n) at first) times 2^13, A times 2^10, B
// times 2^8.
#include <algorithm>

#include "pair_ops.cuh"
#include "rows_dev.cuh"

namespace symmoe {
namespace orth {

using namespace rows;
using namespace pair;

// A bf16 result rounds by 1.7e-3 of its norm, an fp16 result by 2.1e-4; products of 11-bit
// operands add 3e-4 to 6e-4 where a gradient has a broad rest.  Beside strong directions with little else
// they add more: what they leave in the other directions, like everything small, grows 3.4 times
// a step, 480 times in five.  Of a gradient of rank one (the worst) 3e-2 of the norm at a shorter side of 8,
// 1.1e-2 at 40, 5e-3 at 64, 2e-3 at 256, 8e-4 at 512, 7e-4 at 700.  So products are taken of both parts
// (hi hi + hi lo + lo hi) in all steps for fp16 results, and for bf16 results of a shorter side up
// to PRECISE_SIDE in all but the last two, whose errors grow little.  With / without, us: bf16 1 x 256 x
// 7168 196 / 155, 24 x 512 x 2048 653 / 450, 24 x 512 x 7168 1679 / 997; fp16 (without: in the last three
// steps) 5 x 1031 x 519 344 / 289, 8 x 2048 x 7168 8011 / 5560.
constexpr int PRECISE_SIDE = 512, ROUGH_STEPS = 2;
constexpr float X_SCALE = 8192.f, A_SCALE = 1024.f, B_SCALE = 256.f;

// A matrix' part of the workspace
struct Layout {
  int64_t ld_x, ld_a;                      // rows of X, of A and B: multiples of 64 elements
  size_t x_bytes, a_bytes;                 // one copy of X's hi or lo, of A or B
  // offsets: two copies of X's hi and lo; A's and B's (b: B's, a: A's, each hi, lo)
  size_t hi, lo, a, b, diag_a, diag_b, diag_a2, diag_b2, sums, parts, total;
  int splits;  // parts that a Gram product's K axis may be cut into
};
constexpr int SUMS = 256;  // partial sums of squares
// A Gram matrix of few tiles with a long K axis is made of parts (joined in their
// order): of one tile, a pair of SMs takes 0.37 us for each 64 columns of X.
constexpr int MOST_SPLITS = 16, SPLIT_SIDE = 512, SPLIT_K = 512;
static Layout layout_of(int rows, int cols) {
  Layout l;
  const int m = std::min(rows, cols);
  auto up = [](size_t v, size_t to) { return (v + to - 1) / to * to; };
  l.ld_x = up(cols, 64), l.ld_a = up(m, 64);
  l.x_bytes = up((size_t)rows * l.ld_x * 2, 256), l.a_bytes = up((size_t)m * l.ld_a * 2, 256);
  l.hi = 0, l.lo = 2 * l.x_bytes, l.a = 4 * l.x_bytes, l.b = l.a + 2 * l.a_bytes;
  l.diag_a = l.b + 2 * l.a_bytes, l.diag_b = l.diag_a + up((size_t)m * 4, 256);
  l.diag_a2 = l.diag_b + up((size_t)m * 4, 256), l.diag_b2 = l.diag_a2 + up((size_t)m * 4, 256);
  l.sums = l.diag_b2 + up((size_t)m * 4, 256), l.parts = l.sums + SUMS * 8;
  l.splits = m > SPLIT_SIDE ? 1 : std::max(1, std::min(MOST_SPLITS, std::max(rows, cols) / SPLIT_K));
  l.total = up(l.parts + (l.splits > 1 ? (size_t)l.splits * m * l.ld_a * 4 : 0), 256);
  return l;
}

struct Call {
  const void *g;
  void *out;
  char *work;
  Layout l;
  int64_t g_stride, ldg, out_stride, ld_out;
  int rows, cols, m, tall;
  float a, b, c, eps, scale;
};
struct State {
  __half *hi, *lo;
};
__device__ __forceinline__ State state_of(const Call &p, int matrix, int copy) {
  char *w = p.work + matrix * p.l.total;
  return State{reinterpret_cast<__half *>(w + p.l.hi + copy * p.l.x_bytes), reinterpret_cast<__half *>(w + p.l.lo + copy * p.l.x_bytes)};
}

// Eight columns of a row, those past the end zeros
template <typename T, bool VEC>
__device__ __forceinline__ void eight(const T *row, int c, int cols, float (&f)[8]) {
  if (VEC && c + 8 <= cols) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4 *>(row + c), b = *reinterpret_cast<const float4 *>(row + c + 4);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
      unpack<T, 8>(*reinterpret_cast<const uint4 *>(row + c), f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? Elem<T>::get(row[c + i]) : 0.f;
  }
}
// Eights that a thread has in flight; the SMs are full of threads (2 / 4 / 8: squares of 4 x 2048 x 7168
// 32 / 45 / 62 us, the first X 60 / 67 / 105).
constexpr int AT_ONCE = 2;
// Partial sums of squares, grid (SUMS, matrices): eight at a time in 32 bits where they
// stay in range there, in 64 bits where not; added up in 64 bits.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) squares_kernel(const Call p) {
  __shared__ double part[8];
  pdl_launch_dependents();
  const T *g = reinterpret_cast<const T *>(p.g) + blockIdx.y * p.g_stride;
  const uint32_t each = (p.cols + 7) / 8, all = p.rows * each, step = SUMS * 256;  // eights of a row, of the matrix
  double s = 0;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < all; i += AT_ONCE * step) {
    float f[AT_ONCE][8], run = 0.f;
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const uint32_t k = i + u * step, r = k / each, c = (k - r * each) * 8;
      if (k < all) eight<T, VEC>(g + r * p.ldg, c, p.cols, f[u]);
      else
#pragma unroll
        for (int v = 0; v < 8; ++v) f[u][v] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      float q = 0.f, most = 0.f;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        q += f[u][v] * f[u][v];
        most = fmaxf(most, fabsf(f[u][v]));
      }
      if (most <= 1e15f && (most >= 1e-15f || most == 0.f) && q == q) {
        run += q;
      } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) s += (double)f[u][v] * f[u][v];
      }
    }
    s += run;
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) s += part[i];
    reinterpret_cast<double *>(p.work + blockIdx.y * p.l.total + p.l.sums)[blockIdx.x] = s;
  }
}
// X_SCALE / (|g| + eps) as two factors, the first a power of two that brings the
// largest g into range; by the whole block of SUMS threads (one of them does what
// runs in 64 bits: a block's would keep the few units for that busy for microseconds)
__device__ __forceinline__ float2 normaliser(const double *sums, float eps) {
  __shared__ double part[SUMS / 32];
  __shared__ float2 f;
  double s = sums[threadIdx.x];
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < SUMS / 32; ++i) s += part[i];
    const double norm = sqrt(s) + (double)eps;
    f = make_float2(1.f, norm == 0 ? 0.f : NAN);
    if (norm > 0 && norm <= 1.7e308) {
      const int e = max(-126, min(126, -ilogb(norm)));
      f = make_float2(ldexpf(1.f, e), (float)(X_SCALE / ldexp(norm, e)));
    }
  }
  __syncthreads();
  return f;
}
// The first X, grid (groups of rows, matrices).  (What lies past a row's end, up to
// its pitch, may be written: nothing reads it.)
template <typename T, bool VEC>
__global__ void __launch_bounds__(SUMS) start_kernel(const Call p) {
  pdl_launch_dependents();
  const T *g = reinterpret_cast<const T *>(p.g) + blockIdx.y * p.g_stride;
  const State s = state_of(p, blockIdx.y, 0);
  pdl_wait();
  const float2 f = normaliser(reinterpret_cast<const double *>(p.work + blockIdx.y * p.l.total + p.l.sums), p.eps);
  const uint32_t each = (p.cols + 7) / 8, all = p.rows * each, step = gridDim.x * SUMS;
  for (uint32_t i = blockIdx.x * SUMS + threadIdx.x; i < all; i += AT_ONCE * step) {
    float v[AT_ONCE][8];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const uint32_t k = i + u * step, r = k / each, c = (k - r * each) * 8;
      if (k < all) eight<T, VEC>(g + r * p.ldg, c, p.cols, v[u]);
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const uint32_t k = i + u * step, r = k / each, c = (k - r * each) * 8;
      if (k >= all) break;
      float h[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) v[u][w] = v[u][w] * f.x * f.y;
      const uint4 hi = pack<__half, 8>(v[u]);
      unpack<__half, 8>(hi, h);
#pragma unroll
      for (int w = 0; w < 8; ++w) v[u][w] -= h[w];
      *reinterpret_cast<uint4 *>(s.hi + r * p.l.ld_x + c) = hi;
      *reinterpret_cast<uint4 *>(s.lo + r * p.l.ld_x + c) = pack<__half, 8>(v[u]);
    }
  }
}
template <typename T>
__global__ void __launch_bounds__(256) finish_kernel(const Call p, int copy) {
  T *out = reinterpret_cast<T *>(p.out) + blockIdx.y * p.out_stride;
  const State s = state_of(p, blockIdx.y, copy);
  pdl_wait();
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x)
    for (int c = threadIdx.x; c < p.cols; c += 256) {
      const int64_t i = r * p.l.ld_x + c;
      out[r * p.ld_out + c] = Elem<T>::put((__half2float(s.hi[i]) + __half2float(s.lo[i])) * (p.scale / X_SCALE));
    }
}

// ---------------------------------------------------------------------------
// The three products on CTA pairs (tcgen05 cta_group::2, tiles of 256 x 256; the
// pair protocol of gemm2sm.cuh), for all matrices of a turn at once:
//   GRAM    A = X X^T (X^T X)          X from both sides
//   POLY    B = b A + c A A
//   UPDATE  X = a X + B X (X B)
//   MIX     the product of two symmetric matrices that commute
// All but X are symmetric: only tiles on and below the diagonal are made, each
// written twice, as it is and turned over.
//
// What a product adds to (A for POLY, X for UPDATE) comes into an epilogue
// warp's own boxes of 32 x 32 one box ahead (cp.async), is turned there from rows of
// memory to rows of a lane, and the result back the same way.  Tensor copies of the
// boxes were no faster where products are large (8 x 2048 x 7168 UPDATE 308 to 335 us, 316
// to 328 now; four warps with three boxes ahead 316) and slower where they are small, each issued by
// one lane while the others wait (POLY 75 us, now 61; 5 x 1031 x 519 370 us in all, now 300).
//
// X X^T of wide matrices and products with A or B read K-major tiles; X^T X and the X of
// B X lie the other way and are read as they lie.
//
// What bounds them (8 x 2048 x 7168): a CTA takes in 32 KB for each 64 of K, 64 bytes a
// cycle at the tensor cores' full rate, which is what an SM takes in at most.  GRAM 160 us
// (1.69 PFLOP/s of the tiles it makes, tensor pipe 82% busy), UPDATE 316 (1.52, 67%): its
// X in and out, 8 bytes an element, shares that way (without either half of it 216); POLY 61.
// ---------------------------------------------------------------------------
enum Kind { GRAM, POLY, UPDATE, MIX };
constexpr int EPI_WARPS = 8;  // two per TMEM lane quarter, each with half of a tile's columns
constexpr int THREADS = 32 * (2 + EPI_WARPS);
constexpr int BOX = 32 * 64;  // 32 rows of 32 fp16
constexpr int CTRL = 512;
// Tiles of 256 columns, or 128 where that leaves a pair of SMs one tile at most.  Such small
// products' blocks take half of an SM's shared memory and TMEM, so that the next one's
// start up beside them.
template <bool SMALL>
struct Shape {
  static constexpr int TILE_N = SMALL ? 128 : 256;
  static constexpr int RING = SMALL ? 3 : 5;
  static constexpr int BUFS = SMALL ? 1 : 2;  // boxes (hi and lo) of an epilogue warp
  static constexpr int OPERANDS = A_BYTES + TILE_N / 2 * BK * 2;  // of a stage
  static constexpr int SMEM = 1024 + RING * OPERANDS + EPI_WARPS * BUFS * 2 * BOX + CTRL;
};
static_assert(Shape<true>::SMEM <= 113 * 1024 && Shape<false>::SMEM <= 227 * 1024, "blocks an SM");

struct Maps {
  CUtensorMap a[2], b[2];  // operands: hi, lo
};
struct Prod {
  char *work;  // of the turn's first matrix
  size_t stride;        // between matrices
  size_t in[2], out[2]; // what is added to and the result: hi, lo
  size_t diag_in, diag; // the diagonals: of what is multiplied, of the result
  size_t diag_in2;      // MIX: the second factor's
  float shift, shift2;  // added to them
  float f0, f1, f2;     // MIX: scales of the factors' elements and of the sums in the result's
  int64_t ld;           // of those rows
  int M, N, K, tiles_m, tiles, count, tall;
  int splits, split_kb;  // GRAM: parts of the K axis, K blocks of one (parts: where their sums go)
  size_t parts;
  // 1: hi hi;  3: and hi lo, lo hi before it: the accumulator drops what is below its last
  // bit at every 16 of K, so the small sums come first (2048 x 7168 of rank one, fp16: off by
  // 3e-4 of the norm, with hi hi first 1.1e-3)
  int passes;
  int last;    // the result is the user's: 1 bf16, 2 fp16
  int vec;     // ... with rows of 16-byte vectors
  char *user;
  int64_t user_stride, user_ld;
  float a, b, c, scale;
  int32_t *status;
  uint32_t tmo;
};

struct Tile {
  int z, i, j, part;
  bool turned;  // also written turned over
};
template <int KIND, int TILE_N>
__device__ __forceinline__ Tile tile_of(const Prod &p, int t) {
  Tile ti;
  ti.part = 0;
  if (KIND == GRAM && p.splits > 1) {
    ti.part = t % p.splits;
    t /= p.splits;
  }
  ti.z = t / p.tiles;
  int k = t - ti.z * p.tiles;
  if (KIND == UPDATE) {  // consecutive tiles share columns
    ti.j = k / p.tiles_m;
    ti.i = k - ti.j * p.tiles_m;
    ti.turned = false;
  } else {  // row i of the lower triangle holds squares [i (i + 1) / 2, ...), of one or two tiles
    constexpr int in_square = 256 / TILE_N;
    const int first = k % in_square;
    k /= in_square;
    int i = (int)((sqrtf(8.f * k + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > k) --i;
    while ((i + 1) * (i + 2) / 2 <= k) ++i;
    const int j = k - i * (i + 1) / 2;
    ti.i = i;
    ti.j = j * in_square + first;
    ti.turned = i != j;
  }
  return ti;
}

// This lane's row of a box (64-byte swizzle: 16-byte word w of row r at w ^ (r / 2 mod 4))
__device__ __forceinline__ uint4 *box_word(uint8_t *box, int lane, int w) {
  return reinterpret_cast<uint4 *>(box + lane * 64 + ((w ^ ((lane >> 1) & 3)) << 4));
}
// Eight lanes' rows of eight 16-bit columns turned over among them: lane i's result is column
// i mod 8 of its eight lanes' rows.  (Stores of 2 bytes, a column at a time, instead: POLY
// 38 us at 4 x 2048 x 7168, 31 without them, 35 so.)
__device__ __forceinline__ uint4 turned8(const uint4 &q, int lane) {
  uint32_t t[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // lanes 1 apart: columns 2j (even lanes) or 2j + 1 of two rows
    const uint32_t o = __shfl_xor_sync(0xffffffffu, t[j], 1);
    t[j] = lane & 1 ? __byte_perm(o, t[j], 0x7632) : __byte_perm(t[j], o, 0x5410);
  }
  const bool b = lane & 2, c = lane & 4;
  // lanes 2 apart: j = b and j = 2 + b, of four rows
  const uint32_t r0 = __shfl_xor_sync(0xffffffffu, b ? t[0] : t[1], 2), r1 = __shfl_xor_sync(0xffffffffu, b ? t[2] : t[3], 2);
  const uint32_t k0 = b ? t[1] : t[0], k1 = b ? t[3] : t[2];
  const uint32_t u[2][2] = {{b ? r0 : k0, b ? k0 : r0}, {b ? r1 : k1, b ? k1 : r1}};
  // lanes 4 apart: one of the two, of eight rows
  const uint32_t s0 = __shfl_xor_sync(0xffffffffu, c ? u[0][0] : u[1][0], 4), s1 = __shfl_xor_sync(0xffffffffu, c ? u[0][1] : u[1][1], 4);
  const uint32_t m0 = c ? u[1][0] : u[0][0], m1 = c ? u[1][1] : u[0][1];
  return c ? make_uint4(s0, s1, m0, m1) : make_uint4(m0, m1, s0, s1);
}
// 8 consecutive fp32 columns of this thread's TMEM lane (as tmem_ld32)
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

template <int KIND, bool A_MN, bool B_MN, bool SMALL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, SMALL ? 2 : 1)
    product_kernel(const Prod p, const __grid_constant__ Maps maps) {
  using S = Shape<SMALL>;
  constexpr int RING = S::RING, BUFS = S::BUFS, OPERANDS = S::OPERANDS, tile_n = S::TILE_N;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *boxes = smem + (size_t)RING * OPERANDS;
  uint64_t *bars = reinterpret_cast<uint64_t *>(boxes + EPI_WARPS * BUFS * 2 * BOX);
  uint64_t *acc_full = bars + 2 * RING, *acc_empty = acc_full + 2, *drained = acc_full + 4;
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base_s + 1);
  const int wid = warp_id(), lane = lane_id();
  const uint32_t rank = cta_rank();
  const int pair_id = (int)cluster_id_x(), npairs = (int)num_clusters_x();
  const Ctl ctl{abort_flag, p.status, p.tmo};
  RingOf<RING> rg{smem, bars, bars + RING};

  if (threadIdx.x == 0) {
    for (int s = 0; s < RING; ++s) {
      mbar_init(&rg.full[s], 1);
      mbar_init(&rg.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * EPI_WARPS);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  if (wid == 1) {
    tmem_alloc2(tmem_base_s, 2 * tile_n);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const int nk = (p.K + BK - 1) / BK, total = p.tiles * p.count * p.splits;
  if (KIND != UPDATE || !p.last) pdl_launch_dependents();  // (what follows the call waits for all of it)
  pdl_wait();           // the kernel before this one has written what this one reads,
  fence_proxy_async();  // some of it by plain stores
  auto blocks = [&](const Tile &ti, int &kb0, int &kb1) {  // K blocks of a tile
    kb0 = ti.part * p.split_kb;
    kb1 = min(nk, kb0 + p.split_kb);
  };

  if (wid == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      const uint32_t full_leader = map_to(rg.full, 0);
      bool ok = true;
      for (int n = 0, t; ok && (t = pair_tile(n, pair_id, npairs)) < total; ++n) {
        const Tile ti = tile_of<KIND, tile_n>(p, t);
        const int m0 = ti.i * 256 + (int)rank * 128, n0 = ti.j * tile_n + (int)rank * (tile_n / 2);
        int kb0, kb1;
        blocks(ti, kb0, kb1);
        for (int pass = p.passes; ok && pass-- > 0;) {  // lo hi, hi lo, and hi hi last (Prod::passes)
          const CUtensorMap *ma = &maps.a[pass == 2], *mb = &maps.b[pass == 1];
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!(ok = bar_wait(&rg.empty[rg.stage], rg.phase ^ 1u, ctl))) break;
            uint8_t *sb = rg.base + (size_t)rg.stage * OPERANDS;
            const uint32_t bar = full_leader + (uint32_t)(rg.stage * sizeof(uint64_t));
            if (rank == 0) mbar_arrive_expect_tx(&rg.full[rg.stage], 2u * A_BYTES + (uint32_t)tile_n * BK * 2);  // both CTAs'
            if (A_MN) {
              tma_load_3d_pair(sb, ma, bar, m0, kb * BK, ti.z);
              tma_load_3d_pair(sb + CHUNK_BYTES, ma, bar, m0 + 64, kb * BK, ti.z);
            } else {
              tma_load_3d_pair(sb, ma, bar, kb * BK, m0, ti.z);
            }
            if (B_MN) {
              tma_load_3d_pair(sb + A_BYTES, mb, bar, n0, kb * BK, ti.z);
              if (tile_n > 128) tma_load_3d_pair(sb + A_BYTES + CHUNK_BYTES, mb, bar, n0 + 64, kb * BK, ti.z);
            } else {
              tma_load_3d_pair(sb + A_BYTES, mb, bar, kb * BK, n0, ti.z);
            }
            rg.next();
          }
        }
      }
    }
  } else if (wid == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------------------------------------------- MMA issuer (leader)
      constexpr uint64_t astep = A_MN ? MN_STEP : K_STEP, bstep = B_MN ? MN_STEP : K_STEP;
      const uint32_t id = idesc(true, A_MN, B_MN, tile_n);
      uint32_t ne[2] = {0, 0};
      int b = 0;
      bool ok = true;
      for (int n = 0, t; ok && (t = pair_tile(n, pair_id, npairs)) < total; ++n, b ^= 1) {
        if (!(ok = bar_wait(&acc_empty[b], (ne[b]++ & 1u) ^ 1u, ctl))) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * tile_n);
        int kb0, kb1;
        blocks(tile_of<KIND, tile_n>(p, t), kb0, kb1);
        for (int kb = 0; kb < (kb1 - kb0) * p.passes; ++kb) {
          if (!(ok = bar_wait(&rg.full[rg.stage], rg.phase, ctl))) break;
          tc_fence_after();
          uint8_t *sb = rg.base + (size_t)rg.stage * OPERANDS;
          const uint64_t da = A_MN ? smem_desc_mn(sb) : smem_desc_sw128(sb);
          const uint64_t db = B_MN ? smem_desc_mn(sb + A_BYTES) : smem_desc_sw128(sb + A_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / UK; ++kk) mma2(d, da + kk * astep, db + kk * bstep, id, (kb > 0 || kk > 0) ? 1u : 0u);
          commit2_both(&rg.empty[rg.stage]);
          rg.next();
        }
        if (ok) commit2_both(&acc_full[b]);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    constexpr int SHARES = EPI_WARPS / 4;  // of a tile's columns
    const int q = wid & 3, share = (wid - 2) / 4;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    uint8_t *my_boxes = boxes + (size_t)(wid - 2) * BUFS * 2 * BOX;  // [BUFS][hi, lo]
    // two boxes in: hi and lo of one matrix (MIX: both factors'); out: hi and lo
    const int two_in = KIND == UPDATE || KIND == MIX || p.passes > 1, two_out = KIND == UPDATE ? !p.last : p.passes > 1;
    // memory's rows: lane 4r + w has word w of rows r, 8 + r, ...
    const int r8 = lane >> 2, w4 = lane & 3;
    auto in_box = [&](uint8_t *box, int r) { return reinterpret_cast<uint4 *>(box + r * 64 + ((w4 ^ ((r >> 1) & 3)) << 4)); };
    uint32_t used[2] = {0, 0};
    uint32_t boxno = 0;
    int b = 0;
    bool ok = true;
    for (int n = 0, t; ok && (t = pair_tile(n, pair_id, npairs)) < total; ++n, b ^= 1) {
      const Tile ti = tile_of<KIND, tile_n>(p, t);
      const int row0 = ti.i * 256 + (int)rank * 128 + q * 32, row = row0 + lane, col0 = ti.j * tile_n + share * (tile_n / SHARES);
      const int chunks = row0 < p.M ? min(tile_n / SHARES / 32, (p.N - col0 + 31) / 32) : 0;  // (negative: none)
      char *w = p.work + ti.z * p.stride;
      float *diag = reinterpret_cast<float *>(w + p.diag);
      const float *diag_in = reinterpret_cast<const float *>(w + p.diag_in);
      const bool by_column = KIND == POLY || KIND == MIX || (KIND == UPDATE && p.tall);
      const float *diag_col = KIND == MIX ? reinterpret_cast<const float *>(w + p.diag_in2) : diag_in;
      auto fetch = [&](int c) {  // the tile's box c
        if (KIND == GRAM) return;
        if (c >= chunks) {
          cp_async_commit();
          return;
        }
        uint8_t *box = my_boxes + (boxno + c) % BUFS * 2 * BOX;
        const int64_t at = (int64_t)(row0 + r8) * p.ld + col0 + 32 * c + 8 * w4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row0 + 8 * i + r8 < p.M) {
            cp_async16(in_box(box, 8 * i + r8), reinterpret_cast<const __half *>(w + p.in[0]) + at + 8 * i * p.ld);
            if (two_in) cp_async16(in_box(box + BOX, 8 * i + r8), reinterpret_cast<const __half *>(w + p.in[1]) + at + 8 * i * p.ld);
          }
        cp_async_commit();
      };
#pragma unroll
      for (int c = 0; c < max(1, BUFS - 1); ++c) fetch(c);
      // the next box's columns' diagonal elements, one a lane (padded to whole boxes)
      float d_next = by_column && chunks > 0 ? diag_col[col0 + lane] : 0.f;
      const float d_row = KIND != GRAM && row < p.M && !(KIND == UPDATE && p.tall) ? diag_in[row] : 0.f;
      if (!(ok = __all_sync(0xffffffffu, bar_wait(&acc_full[b], used[b]++ & 1u, ctl)))) break;
      tc_fence_after();
      const uint32_t acc = lanes + (uint32_t)(b * tile_n + share * (tile_n / SHARES));
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int col = col0 + 32 * c;
        uint8_t *box = my_boxes + (boxno + c) % BUFS * 2 * BOX;
        const float d_col = d_next;
        if (by_column && c + 1 < chunks) d_next = diag_col[col + 32 + lane];
        if (KIND != GRAM) {
          if (BUFS > 1 || c > 0) fetch(c + BUFS - 1);
          cp_async_wait<BUFS - 1>();
          __syncwarp();
        }
        const bool users = KIND == UPDATE && p.last;
        // Eight columns at a time in a loop that is not unrolled: a tile runs this code a few
        // times, and small products are bound by its way to the SM (with 32 columns unrolled the
        // three kernels of a step took 7.6 us each for one 64 x 64 tile, now 4.6).
#pragma unroll 1
        for (int o = 0; o < 4; ++o) {
          uint32_t v[8];
          float x[8], l[8];
          tmem_ld8(acc + 32 * c + 8 * o, v);
          uint4 *const hi_word = box_word(box, lane, o), *const lo_word = box_word(box + BOX, lane, o);
          if (KIND != GRAM) {
            unpack<__half, 8>(*hi_word, x);
            if (two_in) {
              unpack<__half, 8>(*lo_word, l);
              if (KIND != MIX)
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] += l[k];
            }
          }
          tmem_ld_wait();
          const int at = col + 8 * o;
          if (KIND == GRAM && p.splits > 1) {  // a part's sums, for join_kernel
            if (row < p.M) {
              float *to = reinterpret_cast<float *>(w + p.parts) + ((int64_t)ti.part * p.M + row) * p.ld + at;
#pragma unroll
              for (int k = 0; k < 8; k += 4)
                *reinterpret_cast<float4 *>(to + k) = make_float4(__uint_as_float(v[k]), __uint_as_float(v[k + 1]),
                                                                  __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
            }
            continue;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float sum = __uint_as_float(v[k]);
            const float d = by_column ? __shfl_sync(0xffffffffu, d_col, 8 * o + k) : 0.f;
            if (KIND == GRAM) x[k] = sum * (A_SCALE / (X_SCALE * X_SCALE));
            else if (KIND == MIX) x[k] = (d_row + p.shift) * (l[k] * p.f1) + (d + p.shift2) * (x[k] * p.f0) + sum * p.f2;
            else if (KIND == POLY)
              x[k] = (p.b + p.c * (d_row + d)) * (x[k] * (B_SCALE / A_SCALE)) + p.c * (sum * (B_SCALE / (A_SCALE * A_SCALE)));
            else x[k] = (p.a + (p.tall ? d : d_row)) * x[k] + sum * (1.f / B_SCALE);
          }
          if (KIND != UPDATE && row0 == col) {  // 32 elements of the diagonal, one for each lane
            float own = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (8 * o + k == lane) {
                own = x[k];
                x[k] = 0.f;
              }
            // (the factors' own parts of x are zero here)
            if (lane / 8 == o && row < p.M)
              diag[row] = KIND == GRAM  ? own * (1.f / A_SCALE)
                          : KIND == MIX ? (d_row + p.shift) * (d_col + p.shift2) + own / (p.f0 * p.f1 / p.f2)
                                        : d_row * (p.b + p.c * d_row) + own * (1.f / B_SCALE);
          }
          if (users) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] *= p.scale / X_SCALE;
            *hi_word = p.last == 1 ? pack<__nv_bfloat16, 8>(x) : pack<__half, 8>(x);
            continue;
          }
          const uint4 hi = pack<__half, 8>(x);
          uint4 lo = make_uint4(0u, 0u, 0u, 0u);
          *hi_word = hi;
          if (two_out) {
            float h[8];
            unpack<__half, 8>(hi, h);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] -= h[k];
            lo = pack<__half, 8>(x);
            *lo_word = lo;
          }
          if (ti.turned) {  // turned over: a lane has a column of eight rows (past the last row: the pitch's end)
            const int64_t to = (int64_t)(at + (lane & 7)) * p.ld + row0 + (lane & ~7);
            const bool there = at + (lane & 7) < p.N;
            const uint4 th = turned8(hi, lane);
            if (there) *reinterpret_cast<uint4 *>(reinterpret_cast<__half *>(w + p.out[0]) + to) = th;
            if (two_out) {
              const uint4 tl = turned8(lo, lane);
              if (there) *reinterpret_cast<uint4 *>(reinterpret_cast<__half *>(w + p.out[1]) + to) = tl;
            }
          }
        }
        if (KIND == GRAM && p.splits > 1) continue;
        __syncwarp();
        if (!users) {  // (whole words: rows' pitches are whole boxes)
          const int64_t at = (int64_t)(row0 + r8) * p.ld + col + 8 * w4;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row0 + 8 * i + r8 < p.M) {
              *reinterpret_cast<uint4 *>(reinterpret_cast<__half *>(w + p.out[0]) + at + 8 * i * p.ld) = *in_box(box, 8 * i + r8);
              if (two_out)
                *reinterpret_cast<uint4 *>(reinterpret_cast<__half *>(w + p.out[1]) + at + 8 * i * p.ld) = *in_box(box + BOX, 8 * i + r8);
            }
        } else if (p.vec && col + 32 <= p.N) {
          uint16_t *to = reinterpret_cast<uint16_t *>(p.user) + ti.z * p.user_stride + (row0 + r8) * p.user_ld + col + 8 * w4;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row0 + 8 * i + r8 < p.M) *reinterpret_cast<uint4 *>(to + 8 * i * p.user_ld) = *in_box(box, 8 * i + r8);
        } else if (col + lane < p.N) {  // a row at a time, a column a lane
          uint16_t *to = reinterpret_cast<uint16_t *>(p.user) + ti.z * p.user_stride + row0 * p.user_ld + col + lane;
#pragma unroll 8
          for (int r = 0; r < min(32, p.M - row0); ++r)
            to[r * p.user_ld] =
                *reinterpret_cast<const uint16_t *>(box + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
        }
        __syncwarp();  // the box has been read
      }
      boxno += (uint32_t)max(chunks, 0);
      give_back(&acc_empty[b], rank, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) settle(drained, wid == 1 && lane == 0 && rank == 0);
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (wid == 1) tmem_dealloc2(tmem, 2 * tile_n);
}

// A Gram matrix of its parts, grid (rows, matrices)
__global__ void __launch_bounds__(128) join_kernel(const Prod p) {
  pdl_launch_dependents();
  pdl_wait();
  char *w = p.work + blockIdx.y * p.stride;
  const int i = blockIdx.x, end = min(p.M, (i / 256 + 1) * 256);  // the squares below the diagonal's, and that
  const float *part = reinterpret_cast<const float *>(w + p.parts);
  auto put = [&](int r, int c, float x) {
    const int64_t at = r * p.ld + c;
    const uint16_t h = to_half(x);
    reinterpret_cast<uint16_t *>(w + p.out[0])[at] = h;
    if (p.passes > 1) reinterpret_cast<uint16_t *>(w + p.out[1])[at] = to_half(x - widen(true, h));
  };
  for (int j = threadIdx.x; j < end; j += 128) {
    float v = 0.f;
    for (int k = 0; k < p.splits; ++k) v += part[((int64_t)k * p.M + i) * p.ld + j];
    float x = v * (A_SCALE / (X_SCALE * X_SCALE));
    if (i == j) {
      reinterpret_cast<float *>(w + p.diag)[i] = x * (1.f / A_SCALE);
      x = 0.f;
    }
    put(i, j, x);
    if (j / 256 < i / 256) put(j, i, x);
  }
}

// A launch that may begin while the kernel before it ends
template <int KIND, bool A_MN, bool B_MN, bool SMALL>
static cudaError_t launch_product(int num_sms, cudaStream_t st, const Prod &p, const Maps &maps) {
  constexpr int SMEM = Shape<SMALL>::SMEM;
  auto kern = product_kernel<KIND, A_MN, B_MN, SMALL>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (err != cudaSuccess) return err;
  // No more pairs than tiles: the next kernel's blocks find room sooner.  (All large
  // products have the same shared memory and threads: one of them is asked for its resident pairs.)
  const int pairs = SMALL ? num_sms / 2
                          : max_resident_pairs((const void *)product_kernel<POLY, false, false, false>, THREADS, SMEM, num_sms);
  const int64_t tiles = (int64_t)p.tiles * p.count * p.splits;
  if (pairs <= 0) return cudaErrorInvalidConfiguration;
  return launch_pdl(kern, dim3(2 * (unsigned)std::min<int64_t>(pairs, tiles)), dim3(THREADS), SMEM, st, p, maps);
}
template <int KIND, bool A_MN, bool B_MN>
static cudaError_t launch_product(bool small, int num_sms, cudaStream_t st, const Prod &p, const Maps &maps) {
  return small ? launch_product<KIND, A_MN, B_MN, true>(num_sms, st, p, maps) : launch_product<KIND, A_MN, B_MN, false>(num_sms, st, p, maps);
}

}  // namespace orth

// (bytes of one matrix, bytes that the call runs best with: all matrices, or as many as make
// eight waves of the square products' tiles, and any number up to a gigabyte)
void orthogonalize_workspace(int count, int rows, int cols, int num_sms, size_t *least, size_t *best) {
  *least = orth::layout_of(rows, cols).total;
  const int64_t tm = (std::min(rows, cols) + 255) / 256, squares = tm * (tm + 1) / 2;
  const int64_t enough = std::max<int64_t>((4 * num_sms + squares - 1) / squares, (int64_t(1) << 30) / (int64_t)*least);
  *best = *least * (size_t)std::max<int64_t>(1, std::min<int64_t>(count, enough));
}

cudaError_t launch_orthogonalize(const sym_orthogonalize &o, int num_sms, cudaStream_t st) {
  using namespace orth;
  Call p{};
  const Layout l = p.l = layout_of(o.rows, o.cols);
  p.g_stride = o.g_stride, p.ldg = o.ld_g, p.out_stride = o.out_stride, p.ld_out = o.ld_out;
  p.work = reinterpret_cast<char *>(o.work);
  p.rows = o.rows, p.cols = o.cols, p.m = std::min(o.rows, o.cols), p.tall = o.rows > o.cols;
  p.a = o.coeffs[0], p.b = o.coeffs[1], p.c = o.coeffs[2], p.eps = o.eps, p.scale = o.scale;
  const int each = (int)std::min<uint64_t>(o.work_bytes / l.total, o.count), m = p.m;
  const int64_t gs = o.g_dtype == SYM_FP32 ? 4 : 2, between = l.total / 2;
  const uint64_t work = reinterpret_cast<uint64_t>(o.work);
  cudaError_t err = cudaSuccess;
  for (int at = 0; at < o.count; at += each) {
    const unsigned n = std::min(each, o.count - at);
    p.g = reinterpret_cast<const char *>(o.g) + at * o.g_stride * gs;
    p.out = reinterpret_cast<char *>(o.out) + at * o.out_stride * 2;
    // 16-byte vectors of g where every row starts on their boundary
    const bool vec = reinterpret_cast<uintptr_t>(p.g) % 16 == 0 && (o.rows == 1 || o.ld_g * gs % 16 == 0) && (n == 1 || o.g_stride * gs % 16 == 0);
    auto start = [&](auto t, auto v) {
      using T = decltype(t);
      constexpr bool VEC = decltype(v)::value;
      squares_kernel<T, VEC><<<dim3(SUMS, n), 256, 0, st>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      const int64_t blocks = ((int64_t)o.rows * ((o.cols + 7) / 8) + AT_ONCE * SUMS - 1) / (AT_ONCE * SUMS);
      // (each block adds up the partial sums for itself: no more blocks than keep the SMs full)
      const int64_t most = std::max<int64_t>(1, 16 * num_sms / n);
      return launch_pdl(start_kernel<T, VEC>, dim3((unsigned)std::min(blocks, most), n), dim3(SUMS), 0, st, p);
    };
    auto typed = [&](auto t) { return vec ? start(t, std::true_type()) : start(t, std::false_type()); };
    err = o.g_dtype == SYM_BF16 ? typed(__nv_bfloat16()) : o.g_dtype == SYM_FP16 ? typed(__half()) : typed(float());
    if (err != cudaSuccess) return err;

    // maps of the operands' rows: K-major (64 columns of 128 rows, or of half a tile's)
    // or as they lie (64 of 64)
    bool ok = true;
    auto map = [&](size_t at_, int rows, int cols, int64_t ld, uint32_t b0, uint32_t b1) {
      CUtensorMap t;
      ok = encode(&t, work + at_, cols, rows, n, ld, between, b0, b1) && ok;
      return t;
    };
    auto both = [&](CUtensorMap(&t)[2], size_t hi, size_t lo, int rows, int cols, int64_t ld, uint32_t b0, uint32_t b1) {
      t[0] = map(hi, rows, cols, ld, b0, b1);
      t[1] = map(lo, rows, cols, ld, b0, b1);
    };
    const size_t a_lo = l.a + l.a_bytes, b_lo = l.b + l.a_bytes;
    Prod q{};
    q.work = p.work, q.stride = l.total, q.count = n, q.tall = p.tall;
    q.a = p.a, q.b = p.b, q.c = p.c, q.scale = p.scale, q.status = o.status;
    q.tmo = o.wait_timeout_us ? o.wait_timeout_us : 2000000u;
    q.user = reinterpret_cast<char *>(p.out), q.user_stride = o.out_stride, q.user_ld = o.ld_out;
    const int tm = (m + 255) / 256, pairs = num_sms / 2;
    const int squares = tm * (tm + 1) / 2, tr = (p.rows + 255) / 256;
    // which products are small (Shape)
    const bool sq_small = (int64_t)2 * squares * n <= pairs, up_small = (int64_t)tr * ((p.cols + 127) / 128) * n <= pairs;
    const int sq_n = sq_small ? 128 : 256, up_n = up_small ? 128 : 256;
    const int sq_tiles = squares * (256 / sq_n), up_tiles = tr * ((p.cols + up_n - 1) / up_n);
    const int nk = (std::max(p.rows, p.cols) + BK - 1) / BK;
    int splits = std::max(1, std::min(l.splits, pairs / (sq_tiles * (int)std::min<unsigned>(n, 4096))));
    const int split_kb = (nk + splits - 1) / splits;
    splits = (nk + split_kb - 1) / split_kb;  // none without K blocks
    Maps gram[2], poly, update[2], mix[3], update2;
    for (int k = 0; k < 2; ++k) {  // from copy k of X
      const size_t hi = l.hi + k * l.x_bytes, lo = l.lo + k * l.x_bytes;
      both(gram[k].a, hi, lo, p.rows, p.cols, l.ld_x, 64, p.tall ? 64 : 128);
      both(gram[k].b, hi, lo, p.rows, p.cols, l.ld_x, 64, p.tall ? 64 : sq_n / 2);
      CUtensorMap x[2], sq[2];
      both(x, hi, lo, p.rows, p.cols, l.ld_x, 64, p.tall ? 128 : 64);
      both(sq, l.b, b_lo, m, m, l.ld_a, 64, p.tall ? up_n / 2 : 128);
      for (int h = 0; h < 2; ++h) {
        update[k].a[h] = p.tall ? x[h] : sq[h];
        update[k].b[h] = p.tall ? sq[h] : x[h];
      }
    }
    // products of both parts (PRECISE_SIDE)
    auto passes_of = [&](int i) { return o.out_dtype == SYM_FP16 || (m <= PRECISE_SIDE && i + ROUGH_STEPS < o.steps) ? 3 : 1; };
    // Two steps with one update (of single parts: the low ones' places are free): an update and a
    // Gram matrix, 3 m^2 n operations, against three products of 3 m^3.
    // One launch more, so small products only where n is far from m.  With / without, us: 8 x 2048 x
    // 7168 2792 / 3190, 4096 x 14336 2500 / 2843, 3 x 600 x 6000 367 / 399, 520 x 7168 314 / 337; 5 x 1031 x 519 219 / 209.
    const int n_side = std::max(p.rows, p.cols);
    const bool twice = (sq_small ? n_side >= 8 * (int64_t)m : n_side * 2 >= 3 * m) &&
                       o.steps >= 2 && passes_of(0) == 1;
    if (twice) {
      const size_t left[3] = {l.a, a_lo, b_lo};
      for (int k = 0; k < 3; ++k) {
        both(mix[k].a, left[k], left[k], m, m, l.ld_a, 64, 128);
        both(mix[k].b, l.b, l.b, m, m, l.ld_a, 64, sq_n / 2);
      }
      update2 = update[0];
      both(p.tall ? update2.b : update2.a, l.a, a_lo, m, m, l.ld_a, 64, p.tall ? up_n / 2 : 128);
    }
    both(poly.a, l.a, a_lo, m, m, l.ld_a, 64, 128);
    both(poly.b, l.a, a_lo, m, m, l.ld_a, 64, sq_n / 2);
    const int user_vec = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && (p.rows == 1 || o.ld_out % 8 == 0) && (n == 1 || o.out_stride % 8 == 0);
    if (!ok) return cudaErrorInvalidValue;
    for (int i = 0, k = 0; i < o.steps; k ^= 1) {
      const bool both_steps = i == 0 && twice;
      q.passes = passes_of(i);
      q.M = q.N = m, q.K = std::max(p.rows, p.cols), q.tiles_m = tm, q.tiles = sq_tiles;
      q.diag = l.diag_a, q.out[0] = l.a, q.out[1] = a_lo, q.ld = l.ld_a;
      q.splits = splits, q.split_kb = split_kb, q.parts = l.parts;
      err = p.tall ? launch_product<GRAM, true, true>(sq_small, num_sms, st, q, gram[k])
                   : launch_product<GRAM, false, false>(sq_small, num_sms, st, q, gram[k]);
      if (err == cudaSuccess && splits > 1) err = launch_pdl(join_kernel, dim3(m, n), dim3(128), 0, st, q);
      if (err != cudaSuccess) return err;
      q.splits = 1, q.split_kb = 1 << 30;
      q.K = m, q.diag_in = l.diag_a, q.diag = l.diag_b;
      q.in[0] = l.a, q.in[1] = a_lo, q.out[0] = l.b, q.out[1] = b_lo;
      err = launch_product<POLY, false, false>(sq_small, num_sms, st, q, poly);
      if (err != cudaSuccess) return err;
      q.a = p.a;
      if (both_steps) {
        // W = A P, A' = W P over A, P' from A', P' P over A'
        auto mix_of = [&](int which, size_t first, size_t first_diag, float shift, float first_scale, size_t to, size_t to_diag, float scale) {
          q.in[0] = first, q.in[1] = l.b, q.diag_in = first_diag, q.diag_in2 = l.diag_b, q.shift = shift, q.shift2 = p.a;
          q.out[0] = to, q.diag = to_diag;
          q.f0 = scale / first_scale, q.f1 = scale / B_SCALE, q.f2 = scale / (first_scale * B_SCALE);
          return launch_product<MIX, false, false>(sq_small, num_sms, st, q, mix[which]);
        };
        if ((err = mix_of(0, l.a, l.diag_a, 0.f, A_SCALE, a_lo, l.diag_a2, A_SCALE)) != cudaSuccess ||
            (err = mix_of(1, a_lo, l.diag_a2, 0.f, A_SCALE, l.a, l.diag_a, A_SCALE)) != cudaSuccess)
          return err;
        q.in[0] = l.a, q.diag_in = l.diag_a, q.out[0] = b_lo, q.diag = l.diag_b2;
        if ((err = launch_product<POLY, false, false>(sq_small, num_sms, st, q, poly)) != cudaSuccess ||
            (err = mix_of(2, b_lo, l.diag_b2, p.a, B_SCALE, l.a, l.diag_a, B_SCALE)) != cudaSuccess)
          return err;
        q.a = 0.f;  // (P' P has all of it)
      }
      i += both_steps ? 2 : 1;
      q.M = p.rows, q.N = p.cols, q.diag_in = both_steps ? l.diag_a : l.diag_b;
      q.tiles_m = tr, q.tiles = up_tiles;
      q.last = i < o.steps ? 0 : o.out_dtype == SYM_BF16 ? 1 : 2, q.vec = user_vec;
      q.in[0] = l.hi + k * l.x_bytes, q.in[1] = l.lo + k * l.x_bytes, q.ld = l.ld_x;
      q.out[0] = l.hi + (k ^ 1) * l.x_bytes, q.out[1] = l.lo + (k ^ 1) * l.x_bytes;
      const Maps &maps = both_steps ? update2 : update[k];
      err = p.tall ? launch_product<UPDATE, false, false>(up_small, num_sms, st, q, maps)
                   : launch_product<UPDATE, false, true>(up_small, num_sms, st, q, maps);
      if (err != cudaSuccess) return err;
      q.last = 0, q.a = p.a;
    }
    if (o.steps == 0) {
      const dim3 lines(std::min(o.rows, 1024), n);
      err = o.out_dtype == SYM_BF16 ? launch_pdl(finish_kernel<__nv_bfloat16>, lines, dim3(256), 0, st, p, 0)
                                    : launch_pdl(finish_kernel<__half>, lines, dim3(256), 0, st, p, 0);
      if (err != cudaSuccess) return err;
    }
  }
  return cudaSuccess;
}

}  // namespace symmoe
