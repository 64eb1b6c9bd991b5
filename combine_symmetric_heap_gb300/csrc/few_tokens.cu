// few_tokens.cu -- a whole MoE layer for up to 32 tokens: routing, the chosen
// experts' SwiGLU and the weighted sum, without a heap.
//
//   l = x Wr^T (or given); idx, w = top-k and softmax over it
//   h = silu(x Wg^T) * (x Wu^T);  out[t] = sum_j w[t][j] h[t, j] Wd^T
//
// All of it is a read of the chosen experts' weights, so both products are built
// as a stream of them: two blocks an SM, whose warps cut the contraction in slices of 64
// elements.  A warp's slices of 16 weight rows go from memory to the registers of
// warp-wide products (mma.sync: a few rows need a hundredth of the tensor cores'
// rate), two or three of them on their way; the rows that they multiply come along.  The
// block's share is a run of features, cut to a feature and not to a tile, so that all
// SMs end together, and the stream does not stop between tiles or experts.
//
// Slices through shared memory were slower (one token of the wide experts, 105 us at the
// copy rate): bulk copies of 1 KB by a warp of their own 223 us (their issue, a
// lane at a time), cp.async by each warp 164 (its 185 instructions a slice).
//
// The logits are read, and the tokens routed, by every block for itself: that takes
// about a microsecond and saves a launch and its results' way through memory.  The
// second product's blocks start as the first's end (programmatic launch): their first
// slices are there when the last h is written.
//
// h goes between the two in two numbers of the weights' type, hi + lo, as two
// rows of the second product: rounded to one it would cost the result as much again as its
// own rounding.  In fp16 lo is held times 2^11, which brings it to hi's range: as it is it
// would be a subnormal number, or nothing, beside an h below 0.1 (of an h of about 2e-6 the
// result was off by twenty times its rounding).
#include <algorithm>

#include "rows_dev.cuh"

namespace symmoe {
namespace few_tokens {

using namespace rows;

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int SLICE = 64;   // contraction elements of a warp's step
constexpr int W_ROWS = 16;  // weight rows of a tile
constexpr int MOST_TOKENS = 32, MOST_EXPERTS = 1024, MOST_PAIRS = 32 * MOST_TOKENS;
constexpr int BLOCKS = 2;   // an SM
// A product's rows of x: 8 NB (and of h 4 NB, hi and lo side by side); an expert's rows
// beyond those take its weights again, out of L2.  NB = 1 up to a row for each expert on
// average, else 2, with three and two slices on their way, what 128 registers hold.  NB 1 / 2
// in us (bytes at the copy rate): eight experts of 4096 x 14336, two a token, 1 token 114 / 124 (105), 4 tokens
// 324 / 291 (287), 8 tokens 422 / 388 (378), 32 tokens 741 / 541 (420); 256 experts of 7168 x 2048,
// eight a token, 1 token 124 / 132 (105), 8 tokens 802 / 832 (755), 32 tokens 2243 / 2310 (2143).
// (Two slices instead of three with NB = 1: 118, 366, 126, 765 and 2173.  One block of twice
// the slices: 130 and 2373; three blocks of two: 117, 351, 119, 780 and 2357.)

// h - hi is at most 2^-11 of hi, so that this many times of it is no larger; bf16 has fp32's range
template <typename T>
constexpr float LO_SCALE = std::is_same<T, __half>::value ? 2048.f : 1.f;

struct Args {
  const uint16_t *x, *wg, *wu, *wd, *wr;
  float *logits;
  int32_t *idx;
  float *w;
  uint16_t *out, *h;  // h: [2][T k][I], hi and lo
  int64_t ldx, ld_out, g_group, g_ld, u_group, u_ld, d_group, d_ld, r_ld;
  int T, H, I, E, k;
};

// ---------------------------------------------------------------------------
// The router's product: a block for each expert, its warps cut the contraction
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) router_kernel(const Args p) {
  pdl_launch_dependents();
  __shared__ float part[8][8];
  const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint16_t *w = p.wr + e * p.r_ld;
  for (int t0 = 0; t0 < p.T; t0 += 8) {
    float s[8] = {};
    for (int c = threadIdx.x * 8; c < p.H; c += 256 * 8) {
      float a[8], b[8];
      unpack<T, 8>(__ldg(reinterpret_cast<const uint4 *>(w + c)), a);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        unpack<T, 8>(__ldg(reinterpret_cast<const uint4 *>(p.x + min(t0 + t, p.T - 1) * p.ldx + c)), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[t] += a[i] * b[i];
      }
    }
    warp_sums<8>(s);
    if (lane == 0)
#pragma unroll
      for (int t = 0; t < 8; ++t) part[warp][t] = s[t];
    __syncthreads();
    if (threadIdx.x < 8 && t0 + threadIdx.x < p.T) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v += part[i][threadIdx.x];
      p.logits[(int64_t)(t0 + threadIdx.x) * p.E + e] = v;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Routing, by every block
// ---------------------------------------------------------------------------
// The chosen experts and their rows, in shared memory
struct Routes {
  uint32_t mask[MOST_EXPERTS];      // bit t: token t takes part in the expert
  float weight[MOST_PAIRS];         // of a row
  float pair_weight[MOST_PAIRS];    // of a pair t k + j; < 0: takes no part
  uint16_t expert[MOST_PAIRS];      // of a pair
  uint16_t slot[MOST_EXPERTS];      // the expert's place in `live`
  uint16_t live[MOST_EXPERTS];      // experts with rows, ascending
  uint16_t first[MOST_EXPERTS + 1]; // their rows
  uint8_t token[MOST_PAIRS];        // of a row
  int experts;                      // with rows
};
// A float's place in the order as an integer: equal numbers (-0 and 0) are equal,
// NaN is 1, below all others; 0 is left for "none".
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  if (v != v) return 1u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key == 1u) return NAN;
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// One token by one warp: k rounds of the largest key left, the lowest expert of those that have it
template <int PER_LANE>
__device__ __forceinline__ void route_token(const Args &p, Routes &r, int t, bool write) {
  const int lane = threadIdx.x & 31;
  const float *l = p.logits + (int64_t)t * p.E;
  uint32_t key[PER_LANE];
#pragma unroll
  for (int i = 0; i < PER_LANE; ++i) key[i] = lane + 32 * i < p.E ? key_of(__ldcg(l + lane + 32 * i)) : 0u;
  uint32_t mine = 0u;
  int my_expert = 0;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    uint32_t e = ~0u;
#pragma unroll
    for (int i = PER_LANE - 1; i >= 0; --i)
      if (key[i] == best) e = lane + 32 * i;
    e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i)
      if (e == lane + 32 * i) key[i] = 0u;
    if (lane == j) mine = best, my_expert = (int)e;
  }
  const float v = value_of(mine), top = __shfl_sync(0xffffffffu, v, 0);
  const bool part = lane < p.k && v != -INFINITY;
  float z[1] = {part ? expf(v - top) : 0.f};
  const float own = z[0];
  warp_sums<1>(z);
  if (lane < p.k) {
    const float w = part ? own / z[0] : 0.f;
    r.expert[t * p.k + lane] = my_expert;
    r.pair_weight[t * p.k + lane] = part ? w : -1.f;
    if (part) atomicOr(&r.mask[my_expert], 1u << t);
    if (write) {
      p.idx[t * p.k + lane] = my_expert;
      p.w[t * p.k + lane] = w;
    }
  }
}
__device__ inline void route(const Args &p, Routes &r, bool write) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += THREADS) r.mask[e] = 0u;
  __syncthreads();
  for (int t = warp; t < p.T; t += WARPS) {
    if (p.E <= 32) route_token<1>(p, r, t, write);
    else if (p.E <= 128) route_token<4>(p, r, t, write);
    else if (p.E <= 256) route_token<8>(p, r, t, write);
    else route_token<32>(p, r, t, write);
  }
  __syncthreads();
  if (warp == 0) {
    int experts = 0, rows = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane, n = e < p.E ? __popc(r.mask[e]) : 0;
      const uint32_t live = __ballot_sync(0xffffffffu, n > 0);
      int sum = n;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, s);
        if (lane >= s) sum += o;
      }
      if (n > 0) {
        const int at = experts + __popc(live & ((1u << lane) - 1u));
        r.slot[e] = at;
        r.live[at] = e;
        r.first[at] = rows + sum - n;
      }
      experts += __popc(live);
      rows += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      r.first[experts] = rows;
      r.experts = experts;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.k; i += THREADS) {
    const float w = r.pair_weight[i];
    if (w < 0.f) continue;  // (a NaN takes part)
    const int t = i / p.k, e = r.expert[i];
    const int row = r.first[r.slot[e]] + __popc(r.mask[e] & ((1u << t) - 1u));
    r.token[row] = t;
    r.weight[row] = w;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// A warp's stream of weight slices
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// weights: read once, past L1
__device__ __forceinline__ uint4 load_weights(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(reinterpret_cast<uint64_t>(p)));
  return v;
}

// Tiles of 16 weight rows in the order that a block walks them, with the rows they
// multiply; `Tiles` has live(), next(), weight(i): row i of the tile, row(i): row i of the
// 8 NB that it multiplies, and load_row.  The warp takes slices warp, warp + WARPS, ...
// of every tile's K elements.
//
// A product m16n8k16 wants pairs of contraction elements from each lane; which ones is
// free as long as both operands agree: lane 4g + t takes elements 8t .. 8t + 7 and 32 + 8t ..
// of a slice (16-byte loads; a row's are 128 bytes) of weight rows g and g + 8 and of
// row g of each eight others.
template <typename T, int NB, int DEPTH, typename Tiles>
struct Stream {
  struct Slice {
    uint4 w[4], x[2 * NB];
  };
  struct Place {  // of the next slice to load
    Tiles tile;
    const uint16_t *lo, *hi, *x[NB];
    int k;
    __device__ explicit Place(const Tiles &first) : tile(first) { open(); }
    __device__ __forceinline__ void open() {
      const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
      k = threadIdx.x / 32 * SLICE;
      if (!tile.live()) return;
      lo = tile.weight(g) + k + 8 * t, hi = tile.weight(g + 8) + k + 8 * t;
#pragma unroll
      for (int j = 0; j < NB; ++j) x[j] = tile.row(8 * j + g) + k + 8 * t;
    }
    __device__ __forceinline__ void next(int K) {
      k += WARPS * SLICE;
      if (k < K) {
        lo += WARPS * SLICE, hi += WARPS * SLICE;
#pragma unroll
        for (int j = 0; j < NB; ++j) x[j] += WARPS * SLICE;
      } else {
        tile.next();
        open();
      }
    }
  };
  Place at;
  int K;
  Slice s[DEPTH];
  __device__ Stream(const Tiles &first, int K_) : at(first), K(K_) {}
  static __device__ __forceinline__ uint4 zero() { return make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load_w(const Place &a, Slice &v) const {
    const int t = threadIdx.x & 3;
    if (a.k + SLICE <= K) {
      v.w[0] = load_weights(a.lo), v.w[1] = load_weights(a.hi);
      v.w[2] = load_weights(a.lo + 32), v.w[3] = load_weights(a.hi + 32);
    } else {  // the last elements: zeros past the end (of multiples of 8)
      const bool one = a.k + 8 * t < K, two = a.k + 32 + 8 * t < K;
      v.w[0] = one ? load_weights(a.lo) : zero(), v.w[1] = one ? load_weights(a.hi) : zero();
      v.w[2] = two ? load_weights(a.lo + 32) : zero(), v.w[3] = two ? load_weights(a.hi + 32) : zero();
    }
  }
  __device__ __forceinline__ void load_x(const Place &a, Slice &v) const {
    const int t = threadIdx.x & 3;
    const bool one = a.k + 8 * t < K, two = a.k + 32 + 8 * t < K;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (a.k + SLICE <= K) {
        v.x[2 * j] = Tiles::load_row(a.x[j]), v.x[2 * j + 1] = Tiles::load_row(a.x[j] + 32);
      } else {
        v.x[2 * j] = one ? Tiles::load_row(a.x[j]) : zero();
        v.x[2 * j + 1] = two ? Tiles::load_row(a.x[j] + 32) : zero();
      }
    }
  }
  // All tiles: finish(acc) at the end of each, with the warp's part of the sums.
  // The first slices' weights are loaded before ready(), which waits for the rows.
  template <typename Ready, typename Finish>
  __device__ __forceinline__ void run(Tiles &now, Ready ready, Finish finish) {
    float acc[NB][4];
    auto clear = [&]() {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    };
    clear();
    const int slices = ((K + SLICE - 1) / SLICE - (int)threadIdx.x / 32 + WARPS - 1) / WARPS;  // of a tile
    if (slices <= 0) {
      ready();
      for (; now.live(); now.next()) finish(acc);
      return;
    }
    Place rows = at;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (at.tile.live()) {
        load_w(at, s[d]);
        at.next(K);
      }
    ready();
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (rows.tile.live()) {
        load_x(rows, s[d]);
        rows.next(K);
      }
    for (int left = slices; now.live();) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (!now.live()) break;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const uint4 &l = s[d].w[2 * c], &h = s[d].w[2 * c + 1], &x = s[d].x[2 * j + c];
            mma16816<T>(acc[j], l.x, h.x, l.y, h.y, x.x, x.y);
            mma16816<T>(acc[j], l.z, h.z, l.w, h.w, x.z, x.w);
          }
        if (at.tile.live()) {
          load_w(at, s[d]);
          load_x(at, s[d]);
          at.next(K);
        }
        if (--left == 0) {
          left = slices;
          finish(acc);
          clear();
          now.next();
        }
      }
    }
  }
};
// (asm: the warps come to it from several places in the code)
__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 0;" ::: "memory"); }

// ---------------------------------------------------------------------------
// h = silu(x Wg^T) * (x Wu^T).  A tile is up to 8 features of an expert: their gate
// rows are the product's rows 0..7 and their up rows 8..15, so that a lane ends
// with both of a feature.
// ---------------------------------------------------------------------------
constexpr int UP_FEATURES = 8, DOWN_FEATURES = 16, MOST_CLUSTER = 8;

// This block's features of all live experts, counted through; `MOST` rows at a time
template <int MOST>
struct UpTiles {
  const Args &p;
  const Routes &r;
  int left, l, c, nf, first, n;  // features left, expert's slot, feature, features, first row, rows
  __device__ UpTiles(const Args &p_, const Routes &r_) : p(p_), r(r_) {
    const int64_t all = (int64_t)r.experts * p.I, at = all * blockIdx.x / gridDim.x;
    left = (int)(all * (blockIdx.x + 1) / gridDim.x - at);
    l = (int)(at / p.I), c = (int)(at - (int64_t)l * p.I);
    open();
  }
  __device__ __forceinline__ bool live() const { return left > 0; }
  __device__ __forceinline__ void open() {
    if (!live()) return;
    nf = min(min(UP_FEATURES, p.I - c), left);
    first = r.first[l];
    n = min(MOST, r.first[l + 1] - first);
  }
  __device__ __forceinline__ void next() {
    first += n;
    n = min(MOST, r.first[l + 1] - first);
    if (n > 0) return;
    left -= nf, c += nf;
    if (c == p.I) c = 0, ++l;
    open();
  }
  // (a row past the last is the last again: a row or column of the product of its own, not stored)
  __device__ __forceinline__ const uint16_t *weight(int i) const {
    const int e = r.live[l], f = c + min(i & 7, nf - 1);
    return i < 8 ? p.wg + e * p.g_group + f * p.g_ld : p.wu + e * p.u_group + f * p.u_ld;
  }
  __device__ __forceinline__ const uint16_t *row(int i) const { return p.x + r.token[first + min(i, n - 1)] * p.ldx; }
  static __device__ __forceinline__ uint4 load_row(const uint16_t *q) { return __ldg(reinterpret_cast<const uint4 *>(q)); }
};

template <typename T, int NB, int DEPTH>
__global__ void __launch_bounds__(THREADS, BLOCKS) up_kernel(const Args p) {
  __shared__ Routes r;
  __shared__ float part[2][8 * NB][WARPS][W_ROWS];  // the warps' sums, of two tiles in turn
  pdl_wait();               // the router's logits
  pdl_launch_dependents();  // the second product reads them too, before it waits for this kernel
  route(p, r, blockIdx.x == 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  using Tiles = UpTiles<8 * NB>;
  Tiles now(p, r);
  Stream<T, NB, DEPTH, Tiles> w(now, p.H);
  int turn = 0;
  w.run(now, [] {}, [&](const float(&acc)[NB][4]) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[turn][8 * j + 2 * t + (i & 1)][warp][g + 8 * (i >> 1)] = acc[j][i];
    block_sync();  // (this half was read before the barrier of the tile between)
    const int row = threadIdx.x / UP_FEATURES, c = threadIdx.x % UP_FEATURES;
    if (row < now.n && c < now.nf) {
      float gate = 0.f, up = 0.f;
#pragma unroll
      for (int v = 0; v < WARPS; ++v) {
        gate += part[turn][row][v][c];
        up += part[turn][row][v][UP_FEATURES + c];
      }
      const float h = gate / (1.f + expf(-gate)) * up;
      const T hi = Elem<T>::put(h);
      const float back = Elem<T>::get(hi);
      const T lo = Elem<T>::put(fabsf(back) <= 3.4028235e38f ? (h - back) * LO_SCALE<T> : 0.f);  // (beyond the type's range hi alone is infinite)
      uint16_t *to = p.h + (int64_t)(now.first + row) * p.I + now.c + c;
      to[0] = *reinterpret_cast<const uint16_t *>(&hi);
      to[(int64_t)p.T * p.k * p.I] = *reinterpret_cast<const uint16_t *>(&lo);
    }
    turn ^= 1;
  });
}

// ---------------------------------------------------------------------------
// out = sum of w h Wd^T.  A cluster of blocks takes a run of features, 16 at a time, and
// each of its blocks every size-th live expert; every warp adds its part of the
// contraction to sums of its own for each token, joined at the end in the warps' and
// the blocks' order (distributed shared memory).  One block a cluster where the features
// alone keep the SMs busy; with fewer of them a block's way through all experts
// bounds the call (7 tokens, 24 experts of 1032 x 520: the layer 32 us, 27 with four blocks a cluster).
// The product's columns are four rows of h's hi and the same four of lo, for each eight of NB.
// ---------------------------------------------------------------------------
template <int MOST>
struct DownTiles {
  const Args &p;
  const Routes &r;
  int begin, features, tiles, rank, size, i;
  int f, nf, l, first, n;  // feature, features, expert's slot, first row, rows
  __device__ DownTiles(const Args &p_, const Routes &r_, int rank_, int size_) : p(p_), r(r_), rank(rank_), size(size_), i(0), l(rank_) {
    const int cluster = blockIdx.x / size, clusters = gridDim.x / size;
    begin = (int)((int64_t)p.H * cluster / clusters);
    features = (int)((int64_t)p.H * (cluster + 1) / clusters) - begin;
    tiles = (features + DOWN_FEATURES - 1) / DOWN_FEATURES;
    open();
  }
  __device__ __forceinline__ bool live() const { return i < tiles && rank < r.experts; }
  __device__ __forceinline__ void cut() { f = begin + features * i / tiles, nf = begin + features * (i + 1) / tiles - f; }  // evenly
  __device__ __forceinline__ void open() {
    if (!live()) return;
    cut();
    first = r.first[l];
    n = min(MOST, r.first[l + 1] - first);
  }
  __device__ __forceinline__ bool last() const { return l + size >= r.experts && first + n == r.first[l + 1]; }  // of its features
  __device__ __forceinline__ void next() {
    first += n;
    n = min(MOST, r.first[l + 1] - first);
    if (n > 0) return;
    if ((l += size) >= r.experts) l = rank, ++i;
    open();
  }
  __device__ __forceinline__ const uint16_t *weight(int j) const {
    return p.wd + r.live[l] * p.d_group + (f + min(j, nf - 1)) * p.d_ld;
  }
  __device__ __forceinline__ const uint16_t *row(int j) const {
    const int pair = first + min(j / 8 * 4 + (j & 3), n - 1);
    return p.h + (int64_t)(j & 4 ? p.T * p.k + pair : pair) * p.I;
  }
  static __device__ __forceinline__ uint4 load_row(const uint16_t *q) { return __ldcg(reinterpret_cast<const uint4 *>(q)); }
};

template <typename T, int NB, int DEPTH>
__global__ void __launch_bounds__(THREADS, BLOCKS) down_kernel(const Args p) {
  __shared__ Routes r;
  extern __shared__ float sums[];  // [WARPS][T][16], and the block's [T][16]
  route(p, r, false);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const int warp_floats = p.T * DOWN_FEATURES;
  float *mine = sums + warp * warp_floats;
  for (int i = lane; i < warp_floats; i += 32) mine[i] = 0.f;
  __syncwarp();
  using Tiles = DownTiles<4 * NB>;
  const int rank = (int)cluster_rank(), size = (int)cluster_size();
  Tiles now(p, r, rank, size);
  float *block_sum = sums + WARPS * warp_floats;
  auto store = [&](int f, int nf) {
    auto put = [&](int i, float v) {
      const int to = i / DOWN_FEATURES, c = i % DOWN_FEATURES;
      const T o = Elem<T>::put(v);
      if (c < nf) p.out[to * p.ld_out + f + c] = *reinterpret_cast<const uint16_t *>(&o);
    };
    block_sync();
    for (int i = threadIdx.x; i < warp_floats; i += THREADS) {
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < WARPS; ++j) {
        v += sums[j * warp_floats + i];
        sums[j * warp_floats + i] = 0.f;
      }
      if (size == 1) put(i, v);
      else block_sum[i] = v;
    }
    if (size == 1) {
      block_sync();
      return;
    }
    cluster_barrier();
    for (int i = rank * THREADS + threadIdx.x; i < warp_floats; i += size * THREADS) {  // this block's share of the joining
      float v = 0.f;
      for (int q = 0; q < size; ++q) v += load_from(block_sum + i, q);
      put(i, v);
    }
    cluster_barrier();
  };
  Stream<T, NB, DEPTH, Tiles> w(now, p.I);
  w.run(now, [] { pdl_wait(); },  // for the first product's h (and out may be its x)
        [&](const float(&acc)[NB][4]) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = acc[j][i] + __shfl_xor_sync(0xffffffffu, acc[j][i], 2) * (1.f / LO_SCALE<T>);  // hi + lo: columns 4 apart (lanes t < 2 have hi)
              const int row = 4 * j + 2 * t + (i & 1);
              if (t < 2 && row < now.n) mine[r.token[now.first + row] * DOWN_FEATURES + g + 8 * (i >> 1)] += r.weight[now.first + row] * v;
            }
          __syncwarp();
          if (now.last()) store(now.f, now.nf);
        });
  if (rank >= r.experts)  // none for this block (every expert of every token may be masked): the others wait for it
    for (; now.i < now.tiles; ++now.i) {
      now.cut();
      store(now.f, now.nf);
    }
}

template <typename T, int NB, int DEPTH>
static cudaError_t products(const Args &p, int num_sms, cudaStream_t st) {
  cudaError_t err;
  if (p.wr) {
    err = launch_pdl(up_kernel<T, NB, DEPTH>, dim3(BLOCKS * num_sms), dim3(THREADS), 0, st, p);
  } else {
    up_kernel<T, NB, DEPTH><<<BLOCKS * num_sms, THREADS, 0, st>>>(p);
    err = cudaGetLastError();
  }
  if (err != cudaSuccess) return err;
  // blocks of a cluster: as many as leave each cluster 16 features, no more than experts may be live
  const int blocks = BLOCKS * num_sms, runs = (p.H + DOWN_FEATURES - 1) / DOWN_FEATURES;
  int size = 1;
  while (2 * size <= MOST_CLUSTER && 2 * size * runs <= blocks && 2 * size <= std::min(p.E, p.T * p.k)) size *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks / size * size);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (WARPS + 1) * p.T * DOWN_FEATURES * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, down_kernel<T, NB, DEPTH>, p);
}
template <typename T>
static cudaError_t run(const Args &p, int num_sms, cudaStream_t st) {
  if (p.wr) {
    router_kernel<T><<<p.E, 256, 0, st>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return p.T * p.k <= p.E ? products<T, 1, 3>(p, num_sms, st) : products<T, 2, 2>(p, num_sms, st);
}

}  // namespace few_tokens

size_t few_tokens_workspace(int tokens, int inter, int topk) { return (size_t)tokens * topk * inter * 4; }

cudaError_t launch_few_tokens(const sym_few_tokens &a, int num_sms, cudaStream_t st) {
  using namespace few_tokens;
  auto half = [](const void *p) { return reinterpret_cast<const uint16_t *>(p); };
  const Args p{half(a.x), half(a.w_gate), half(a.w_up), half(a.w_down), half(a.w_router), a.logits, a.idx, a.w,
               reinterpret_cast<uint16_t *>(a.out), reinterpret_cast<uint16_t *>(a.work), a.ld_x, a.ld_out, a.gate_group, a.gate_ld,
               a.up_group, a.up_ld, a.down_group, a.down_ld, a.router_ld, a.tokens, a.hidden, a.inter, a.num_experts, a.topk};
  return a.dtype == SYM_FP16 ? run<__half>(p, num_sms, st) : run<__nv_bfloat16>(p, num_sms, st);
}

}  // namespace symmoe
