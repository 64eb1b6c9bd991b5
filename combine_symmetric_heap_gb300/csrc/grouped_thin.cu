// grouped_thin.cu -- the grouped product for tens of rows in all: out[r] = W_e x[r]
// or x[r] W_e, bound by the read of the live groups' weights.
//
// The tensor-core kernel of long row tiles (grouped.cu) gives 256 features to a
// pair of SMs and walks the contraction there: with few groups of few features
// most SMs idle and the others are bound by their own loads.  Here a block takes
// 16, 32 or 64 features and its sixteen warps cut the contraction; weights go from
// memory to the registers of a warp-wide matrix product (mma.sync: these rows need
// a hundredth of the tensor cores' rate) without a stop in shared memory, and the
// warps' sums are added at the end in a fixed order, in fp32.
//
// A warp-wide product m16n8k16 wants pairs of contraction elements from each lane;
// which ones is free as long as both operands agree.  Lane 4g + t takes the eight
// at 8t of every 32 (a 16-byte load), as two products' four each.
#include <algorithm>

#include "rows_dev.cuh"

namespace symmoe {
namespace thin {

using namespace rows;

constexpr int WARPS = 16;
constexpr int K_STEP = 32;         // contraction elements of a warp's step
constexpr int T_FEATURES = 64;     // of a block, w [C][F]
constexpr int MOST_SMEM = 4 * WARPS * T_FEATURES * 16;  // the warps' sums, at most

struct Args {
  const int32_t *cnt, *off;
  int G;
  int32_t *status;
  const uint16_t *x, *w;
  uint16_t *out;
  int64_t ldx, w_group, w_ld, ld_out;
  int rows, F, C;
};

// This block's group: (first row, rows), rows 0 for none.  A group outside
// [0, rows) is empty, and flagged.
__device__ __forceinline__ int2 group_rows(const Args &p, int e) {
  const int c = p.cnt[e], o = p.off[e];
  if (c < 0 || o < 0 || (int64_t)o + c > p.rows) {
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, SYM_STATUS_OVERFLOW);
    return make_int2(0, 0);
  }
  return make_int2(o, c);
}

// elements [k, k + 8) of a row of n; those past the end are zeros
__device__ __forceinline__ uint4 eight(const uint16_t *row, int k, int n) {
  if (k + 8 <= n) return *reinterpret_cast<const uint4 *>(row + k);
  uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < n) v[i / 2] |= (uint32_t)row[k + i] << (16 * (i & 1));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

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

// The warps' sums part[warp][row][feature] added and stored: rows [r, r + n),
// features [f0, f0 + NF)
template <typename T, int ROWS, int NF>
__device__ __forceinline__ void join(const Args &p, const float *part, int r, int n, int f0) {
  __syncthreads();
  for (int i = threadIdx.x; i < n * NF; i += 32 * WARPS) {
    const int row = i / NF, f = i % NF;
    if (f0 + f >= p.F) continue;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < WARPS; ++v) s += part[(v * ROWS + row) * NF + f];
    const T t = Elem<T>::put(s);
    p.out[(int64_t)(r + row) * p.ld_out + f0 + f] = *reinterpret_cast<const uint16_t *>(&t);
  }
  __syncthreads();
}

// w [F][C], 16 MT features, rows [r, r + n) of up to 8 NB: features are the
// product's rows, rows of x its columns.  A row past the group's last is the last
// again (a column of the product of its own, not stored); a feature likewise.
template <typename T, int MT, int NB, int UNROLL>
__device__ __forceinline__ void by_features(const Args &p, int r, int n, int e, int f0, float *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const uint16_t *w[2 * MT], *x[NB];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) w[i] = p.w + e * p.w_group + (int64_t)min(f0 + 8 * i + g, p.F - 1) * p.w_ld;
#pragma unroll
  for (int i = 0; i < NB; ++i) x[i] = p.x + (int64_t)(r + min(8 * i + g, n - 1)) * p.ldx;
  float acc[MT][NB][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.f;
  auto products = [&](const uint4(&a)[2 * MT], const uint4(&b)[NB]) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        mma16816<T>(acc[i][j], a[2 * i].x, a[2 * i + 1].x, a[2 * i].y, a[2 * i + 1].y, b[j].x, b[j].y);
        mma16816<T>(acc[i][j], a[2 * i].z, a[2 * i + 1].z, a[2 * i].w, a[2 * i + 1].w, b[j].z, b[j].w);
      }
  };
  const int whole = p.C / K_STEP;
#pragma unroll UNROLL
  for (int s = warp; s < whole; s += WARPS) {
    const int k = s * K_STEP + 8 * t;
    uint4 a[2 * MT], b[NB];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) a[i] = *reinterpret_cast<const uint4 *>(w[i] + k);
#pragma unroll
    for (int j = 0; j < NB; ++j) b[j] = *reinterpret_cast<const uint4 *>(x[j] + k);
    products(a, b);
  }
  if (whole * K_STEP < p.C && warp == whole % WARPS) {
    const int k = whole * K_STEP + 8 * t;
    uint4 a[2 * MT], b[NB];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) a[i] = eight(w[i], k, p.C);
#pragma unroll
    for (int j = 0; j < NB; ++j) b[j] = eight(x[j], k, p.C);
    __syncwarp();
    products(a, b);
  }
  constexpr int NF = 16 * MT;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        part[(warp * 8 * NB + 8 * j + 2 * t + (k & 1)) * NF + 16 * i + 8 * (k >> 1) + g] = acc[i][j][k];
  join<T, 8 * NB, NF>(p, part, r, n, f0);
}

// grid (feature blocks, groups).  Two blocks an SM with two steps' loads in flight
// each, or (DEEP) one with four, for grids that leave an SM one block: 16 rows of
// four groups, 7168 -> 2048, 35.5 / 39.6 us; of one group 19.1 / 15.0.  (The
// two-block form's 64 registers spill: 52 bytes stored and 152 loaded a thread with
// 32 features, 28 and 68 with 16.)
template <typename T, int MT, bool DEEP>
__global__ void __launch_bounds__(32 * WARPS, DEEP ? 1 : 2) thin_kernel(const Args p) {
  extern __shared__ __align__(16) float part[];
  const int e = blockIdx.y, f0 = blockIdx.x * 16 * MT;
  const int2 rows = group_rows(p, e);
  // rows of a pass: with 32 features, 32 rows' sums would not fit 64 registers
  constexpr int PASS = MT == 2 ? 16 : 32, U = DEEP ? 2 : 1;
  for (int i = 0; i < rows.y; i += PASS) {
    const int r = rows.x + i, n = min(PASS, rows.y - i);
    if (n <= 8) by_features<T, MT, 1, 2 * U>(p, r, n, e, f0, part);
    else if (n <= 16) by_features<T, MT, 2, 2 * U / MT>(p, r, n, e, f0, part);
    else if constexpr (PASS == 32) by_features<T, MT, 4, U>(p, r, n, e, f0, part);
  }
}

// w [C][F], 64 features, rows [r, r + n) of up to 16: rows of x are the
// product's rows; its eight columns g are features 8g + j, one product for each
// j, so that a lane's features are a 16-byte load, and pairs of contraction rows
// are put together word by word.
template <typename T>
__device__ __forceinline__ void by_rows(const Args &p, int r, int n, int e, int f0, float *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const uint16_t *w = p.w + e * p.w_group;
  const int f = f0 + 8 * g;
  const uint16_t *x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = p.x + (int64_t)(r + min(8 * i + g, n - 1)) * p.ldx;
  float acc[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[j][k] = 0.f;
  auto products = [&](const uint4(&a)[2], const uint4(&b)[8]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t *q[4] = {&b[4 * s].x, &b[4 * s + 1].x, &b[4 * s + 2].x, &b[4 * s + 3].x};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(q[0][j / 2], q[1][j / 2], sel), b1 = __byte_perm(q[2][j / 2], q[3][j / 2], sel);
        if (s == 0) mma16816<T>(acc[j], a[0].x, a[1].x, a[0].y, a[1].y, b0, b1);
        else mma16816<T>(acc[j], a[0].z, a[1].z, a[0].w, a[1].w, b0, b1);
      }
    }
  };
  const int whole = f0 + T_FEATURES <= p.F ? p.C / K_STEP : 0;  // steps of whole vectors only
  for (int s = warp; s < whole; s += WARPS) {
    const int k = s * K_STEP + 8 * t;
    uint4 a[2], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = *reinterpret_cast<const uint4 *>(w + (int64_t)(k + i) * p.w_ld + f);
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = *reinterpret_cast<const uint4 *>(x[i] + k);
    products(a, b);
  }
  const int steps = (p.C + K_STEP - 1) / K_STEP;
  for (int s = whole + (warp + WARPS - whole % WARPS) % WARPS; s < steps; s += WARPS) {
    const int k = s * K_STEP + 8 * t;
    uint4 a[2], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = k + i < p.C ? eight(w + (int64_t)(k + i) * p.w_ld, f, p.F) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = eight(x[i], k, p.C);
    __syncwarp();
    products(a, b);
  }
  constexpr int NF = T_FEATURES;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) part[(warp * 16 + 8 * (k >> 1) + g) * NF + 8 * (2 * t + (k & 1)) + j] = acc[j][k];
  join<T, 16, NF>(p, part, r, n, f0);
}

template <typename T>
__global__ void __launch_bounds__(32 * WARPS) thin_trans_kernel(const Args p) {
  extern __shared__ __align__(16) float part[];
  const int e = blockIdx.y, f0 = blockIdx.x * T_FEATURES;
  const int2 rows = group_rows(p, e);
  for (int i = 0; i < rows.y; i += 16) by_rows<T>(p, rows.x + i, min(16, rows.y - i), e, f0, part);
}

}  // namespace thin
// Does the call go to these kernels?  One slot, so that the rows there are bound
// the live ones; up to 16 rows, or 32 of at least four groups (a group's weights
// are read again every 32 rows, every 16 with w [C][F]); so few tiles of the
// tensor-core kernel that they fill its pairs once, or twice with w [F][C].  Times
// of a single call on cold weights against that kernel's (us, some 8 of them the
// call's own; 16 rows):
//   groups, live   C -> F           w [F][C]      w [C][F]
//   1, 1         7168 -> 2048     15.0 /  41.6  25.2 /  41.6   taken
//   1, 1        14336 -> 4096     41.6 /  72.3  45.7 /  70.3   taken
//   4, 4         7168 -> 2048     35.5 /  47.7  33.4 /  45.7   taken
//   8, 2         7168 -> 2048     21.1 /  41.6  27.3 /  41.6   taken
//   8, 8         7168 -> 2048     56.0 /  60.2  56.0 /  57.0   taken
//   8, 8        14336 -> 4096    160.4 / 176.8 178.8 / 164.5   taken / not
//   32, 32       7168 -> 2048    189   / 183     (32 rows)     not
// 32 rows of one group: 31.4 / 41.6, but 14336 -> 4096 94.8 / 72.3.
bool thin_product(const sym_groups &g, const sym_rows &x, const sym_rows &out, int trans, int num_sms) {
  return x.slots == 1 && x.rows <= (g.groups >= 4 ? 32 : 16) &&
         (int64_t)g.groups * ((out.cols + 255) / 256) <= (trans ? num_sms / 2 : num_sms);
}

cudaError_t launch_thin_product(const sym_groups &g, int fp16, const sym_rows &x, const void *w, int64_t w_group,
                                int64_t w_ld, int trans, const sym_rows &out, int num_sms, cudaStream_t st) {
  using namespace thin;
  const Args p{g.cnt, g.off, g.groups, g.status, reinterpret_cast<const uint16_t *>(x.ptr),
               reinterpret_cast<const uint16_t *>(w), reinterpret_cast<uint16_t *>(out.ptr), x.ld, w_group, w_ld, out.ld,
               (int)x.rows, out.cols, x.cols};
  auto go = [&](auto kern, int features, int rows) {
    const size_t smem = sizeof(float) * WARPS * features * rows;
    const cudaError_t err = allow_smem(kern, MOST_SMEM);
    if (err != cudaSuccess) return err;
    kern<<<dim3((out.cols + features - 1) / features, (unsigned)g.groups), 32 * WARPS, smem, st>>>(p);
    return cudaGetLastError();
  };
  if (trans)
    return fp16 ? go(thin_trans_kernel<__half>, T_FEATURES, 16) : go(thin_trans_kernel<__nv_bfloat16>, T_FEATURES, 16);
  const int rows = x.rows <= 8 ? 8 : x.rows <= 16 ? 16 : 32;  // that a pass takes
  // 32 features a block (x is read half as often) where that still gives every SM one
  if (out.cols >= 32 * num_sms)
    return fp16 ? go(thin_kernel<__half, 2, false>, 32, std::min(rows, 16))
                : go(thin_kernel<__nv_bfloat16, 2, false>, 32, std::min(rows, 16));
  if ((int64_t)g.groups * ((out.cols + 15) / 16) <= num_sms)
    return fp16 ? go(thin_kernel<__half, 1, true>, 16, rows) : go(thin_kernel<__nv_bfloat16, 1, true>, 16, rows);
  return fp16 ? go(thin_kernel<__half, 1, false>, 16, rows) : go(thin_kernel<__nv_bfloat16, 1, false>, 16, rows);
}

}  // namespace symmoe
