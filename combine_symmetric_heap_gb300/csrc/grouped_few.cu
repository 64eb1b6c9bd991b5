// grouped_few.cu -- the grouped product for a few rows in all (single tokens
// being served): out[r] = W_e x[r] or x[r] W_e on the CUDA cores.
//
// With so few rows the product is a read of the live groups' weights.  The
// tensor-core kernel gives a 256-feature tile to a pair of SMs, which leaves most
// SMs idle when one or two groups are live; here every row is cut into small
// blocks of features.  Blocks are made per row, not per group, since the row
// counts are on the device: the block of a row that starts a run of NR rows of
// its group takes the run, blocks of the other rows leave.  Sums run in fp32 in
// a fixed order.
#include "rows_dev.cuh"

namespace symmoe {
namespace few {

using namespace rows;

constexpr int RUN = 4;  // rows of a group that share one read of the weights
// Rows in all up to which a product is taken here.  Measured against the
// tensor-core kernel (us, 2 of 8 groups with a row each, cold weights): w [F][C]
// 4096 -> 14336 36.4 / 50.5 (0.96 of the copy rate), 14336 -> 4096 38.7 / 67.7; w
// [C][F] 14336 -> 4096 41.3 / 67.9.  8 groups with a row: 38.2 / 47.4, but w
// [C][F] 46.7 / 44.1.  Where rows share a group the arithmetic counts: 4 rows of
// one group, 7168 -> 2048, take 25.2 (w [C][F] 49.8) against 15.0 (25.2) in warp-wide
// products (grouped_thin.cu), so a group has two rows (one) on average at most; 8
// groups with a row each, 51.9 / 62.1.
constexpr int64_t FEW_ROWS = 8, FEW_ROWS_TRANS = 4;
constexpr int MOST_COLS = 16384;  // of x: a run fits shared memory

struct Args {
  const int32_t *cnt, *off;
  int G;
  int32_t *status;
  const uint16_t *x, *w;
  uint16_t *out;
  int64_t ldx, w_group, w_ld, ld_out;
  int rows, F, C;
};

// The run of rows this block takes: (group, rows), rows 0 for none.  Block (0, 0)
// also flags the groups that do not lie in [0, rows).
__device__ __forceinline__ int2 find_run(const Args &p, int r) {
  __shared__ int found[2];
  if (threadIdx.x == 0) found[1] = 0;
  __syncthreads();
  for (int e = threadIdx.x; e < p.G; e += blockDim.x) {
    const int c = p.cnt[e], o = p.off[e];
    if (c < 0 || o < 0 || (int64_t)o + c > p.rows) {
      if (p.status && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, SYM_STATUS_OVERFLOW);
    } else if (o <= r && r < o + c && (r - o) % RUN == 0) {
      found[0] = e;
      found[1] = min(RUN, o + c - r);
    }
  }
  __syncthreads();
  return make_int2(found[0], found[1]);
}

template <typename T>
__device__ __forceinline__ float one(uint16_t v) {
  return Elem<T>::get(*reinterpret_cast<const T *>(&v));
}
template <typename T>
__device__ __forceinline__ uint16_t one(float v) {
  const T t = Elem<T>::put(v);
  return *reinterpret_cast<const uint16_t *>(&t);
}

// rows [r, r + NR) of x into shared memory, [NR][stride]
__device__ __forceinline__ void stage_x(const Args &p, int r, int nr, uint16_t *xs, int stride) {
  for (int i = 0; i < nr; ++i)
    for (int c = threadIdx.x * 8; c < p.C; c += blockDim.x * 8) {
      const uint16_t *from = p.x + (int64_t)(r + i) * p.ldx + c;
      if (c + 8 <= p.C) *reinterpret_cast<uint4 *>(xs + i * stride + c) = *reinterpret_cast<const uint4 *>(from);
      else for (int j = 0; c + j < p.C; ++j) xs[i * stride + c + j] = from[j];
    }
  __syncthreads();
}

// w [F][C]: a warp takes FW features, its lanes 8 columns of each at a time
template <typename T, int NR, int FW>
__device__ __forceinline__ void by_features(const Args &p, int r, int e, int nr) {
  const int lane = threadIdx.x & 31;
  const int f0 = (blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32) * FW;
  if (f0 >= p.F) return;
  const uint16_t *w = p.w + e * p.w_group;
  const uint16_t *x[NR];  // all warps of the block read them: out of L1
#pragma unroll
  for (int i = 0; i < NR; ++i) x[i] = p.x + (int64_t)(r + min(i, nr - 1)) * p.ldx;
  float acc[NR][FW];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < FW; ++j) acc[i][j] = 0.f;
  const int full = p.C / 8;
#pragma unroll(NR == 1 ? 4 : 2)
  for (int v = lane; v < full; v += 32) {
    uint4 q[FW];
#pragma unroll
    for (int j = 0; j < FW; ++j)
      q[j] = *reinterpret_cast<const uint4 *>(w + (int64_t)min(f0 + j, p.F - 1) * p.w_ld + v * 8);
    float xv[NR][8];
#pragma unroll
    for (int i = 0; i < NR; ++i) unpack<T, 8>(__ldg(reinterpret_cast<const uint4 *>(x[i] + v * 8)), xv[i]);
#pragma unroll
    for (int j = 0; j < FW; ++j) {
      float wv[8];
      unpack<T, 8>(q[j], wv);
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][j] += wv[k] * xv[i][k];
    }
  }
  if (const int c = full * 8 + lane; c < p.C)
#pragma unroll
    for (int j = 0; j < FW; ++j) {
      const float wv = one<T>(w[(int64_t)min(f0 + j, p.F - 1) * p.w_ld + c]);
#pragma unroll
      for (int i = 0; i < NR; ++i) acc[i][j] += wv * one<T>(x[i][c]);
    }
#pragma unroll
  for (int i = 0; i < NR; ++i) warp_sums<FW>(acc[i]);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int j = 0; j < FW; ++j)
        if (i < nr && f0 + j < p.F) p.out[(int64_t)(r + i) * p.ld_out + f0 + j] = one<T>(acc[i][j]);
}

// w [C][F]: a block takes 64 features, 8 lanes of 8 each; its other threads
// take every 64th contraction row, and their sums are added at the end
constexpr int T_THREADS = 512, T_FEATURES = 64;
template <typename T, int NR>
__device__ __forceinline__ void by_rows(const Args &p, int r, int e, int nr, uint16_t *xs) {
  __shared__ float part[T_THREADS / 32][NR][T_FEATURES];
  const int stride = (p.C + 7) & ~7, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  stage_x(p, r, nr, xs, stride);
  const int f = blockIdx.x * T_FEATURES + (threadIdx.x & 7) * 8;
  const uint16_t *w = p.w + e * p.w_group + f;
  float acc[NR][8];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;
  auto add = [&](int c, const float(&wv)[8]) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float xv = one<T>(xs[i * stride + c]);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[i][k] += wv[k] * xv;
    }
  };
  if (f + 8 <= p.F) {
#pragma unroll 8
    for (int c = threadIdx.x >> 3; c < p.C; c += T_THREADS / 8) {
      float wv[8];
      unpack<T, 8>(*reinterpret_cast<const uint4 *>(w + (int64_t)c * p.w_ld), wv);
      add(c, wv);
    }
  } else if (f < p.F) {
    for (int c = threadIdx.x >> 3; c < p.C; c += T_THREADS / 8) {
      float wv[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) wv[k] = f + k < p.F ? one<T>(w[(int64_t)c * p.w_ld + k]) : 0.f;
      add(c, wv);
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[i][k] += __shfl_xor_sync(0xffffffffu, acc[i][k], 8);
      acc[i][k] += __shfl_xor_sync(0xffffffffu, acc[i][k], 16);
      if (lane < 8) part[warp][i][lane * 8 + k] = acc[i][k];
    }
  __syncthreads();
  for (int t = threadIdx.x; t < NR * T_FEATURES; t += T_THREADS) {
    const int i = t / T_FEATURES, k = t % T_FEATURES, g = blockIdx.x * T_FEATURES + k;
    if (i >= nr || g >= p.F) continue;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < T_THREADS / 32; ++v) s += part[v][i][k];
    p.out[(int64_t)(r + i) * p.ld_out + g] = one<T>(s);
  }
}

// grid (feature blocks, rows)
template <typename T, int FW>
__global__ void __launch_bounds__(256) few_rows_kernel(const Args p) {
  const int2 run = find_run(p, blockIdx.y);
  const int r = blockIdx.y;
  if (run.y == 0) return;
  if (run.y == 1) by_features<T, 1, FW>(p, r, run.x, 1);
  else if (run.y == 2) by_features<T, 2, FW>(p, r, run.x, 2);
  else by_features<T, RUN, FW>(p, r, run.x, run.y);
}
template <typename T>
__global__ void __launch_bounds__(T_THREADS) few_rows_trans_kernel(const Args p) {
  extern __shared__ __align__(16) uint16_t xs[];
  const int2 run = find_run(p, blockIdx.y);
  const int r = blockIdx.y;
  if (run.y == 0) return;
  if (run.y == 1) by_rows<T, 1>(p, r, run.x, 1, xs);
  else if (run.y == 2) by_rows<T, 2>(p, r, run.x, 2, xs);
  else by_rows<T, RUN>(p, r, run.x, run.y, xs);
}

}  // namespace few

// Does the call go to these kernels?  One slot, so that the rows there are bound
// the live ones; a run of x fits shared memory.
bool few_rows_product(const sym_groups &g, const sym_rows &x, int trans) {
  return x.slots == 1 && x.rows <= (trans ? few::FEW_ROWS_TRANS : few::FEW_ROWS) &&
         x.rows <= (int64_t)(trans ? 1 : 2) * g.groups && x.cols <= few::MOST_COLS;
}

cudaError_t launch_few_rows(const sym_groups &g, int fp16, const sym_rows &x, const void *w, int64_t w_group,
                            int64_t w_ld, int trans, const sym_rows &out, int num_sms, cudaStream_t st) {
  using namespace few;
  const Args p{g.cnt, g.off, g.groups, g.status, reinterpret_cast<const uint16_t *>(x.ptr),
               reinterpret_cast<const uint16_t *>(w), reinterpret_cast<uint16_t *>(out.ptr), x.ld, w_group, w_ld, out.ld,
               (int)x.rows, out.cols, x.cols};
  // rows of x a block reads: 1, 2 or RUN (a run of three reads a fourth that is not stored)
  const size_t smem = trans ? (size_t)(x.rows <= 2 ? x.rows : RUN) * ((x.cols + 7) & ~7) * 2 : 0;
  auto go = [&](auto kern, int threads, int features) {
    const cudaError_t err = allow_smem(kern, trans ? RUN * MOST_COLS * 2 : 0);
    if (err != cudaSuccess) return err;
    kern<<<dim3((out.cols + features - 1) / features, (unsigned)x.rows), threads, smem, st>>>(p);
    return cudaGetLastError();
  };
  if (trans)
    return fp16 ? go(few_rows_trans_kernel<__half>, T_THREADS, T_FEATURES)
                : go(few_rows_trans_kernel<__nv_bfloat16>, T_THREADS, T_FEATURES);
  // four features a warp (more loads in flight) where that still gives every SM
  // two blocks a row
  if (out.cols >= 32 * 2 * num_sms)
    return fp16 ? go(few_rows_kernel<__half, 4>, 256, 32) : go(few_rows_kernel<__nv_bfloat16, 4>, 256, 32);
  return fp16 ? go(few_rows_kernel<__half, 2>, 256, 16) : go(few_rows_kernel<__nv_bfloat16, 2>, 256, 16);
}

}  // namespace symmoe
