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
//   - X is hi + lo, two fp16 numbers (22 bits): a X is taken of both, B X of hi;
//   - A and B are their diagonal in fp32 and the rest in fp16.  With D and O for
//     the two, A A = D D + D O + O D + O O: only O O is a product of matrices, the
//     rest belongs to one element each.  As X comes near to orthogonality the
//     diagonals come near to constants and the rests to zero, and so does what
//     their rounding leaves.
// All are held times a power of two that keeps them in fp16's range: X (entries at
// most its largest singular value; 1 / sqrt(m n) at first) times 2^13, A times 2^10, B
// times 2^8.
#include <algorithm>

#include "rows_dev.cuh"

namespace symmoe {
namespace orth {

using namespace rows;

constexpr float X_SCALE = 8192.f, A_SCALE = 1024.f, B_SCALE = 256.f;

// A matrix' part of the workspace
struct Layout {
  int64_t ld_x, ld_a;                      // rows of X, of A and B: multiples of 64 elements
  size_t x_bytes, a_bytes;                 // one copy of X's hi or lo, of A or B
  size_t hi, lo, a, b, diag_a, diag_b, sums, total;  // offsets; hi, lo: two copies each
};
constexpr int SUMS = 64;  // partial sums of squares
static Layout layout_of(int rows, int cols) {
  Layout l;
  const int m = std::min(rows, cols);
  auto up = [](size_t v, size_t to) { return (v + to - 1) / to * to; };
  l.ld_x = up(cols, 64), l.ld_a = up(m, 64);
  l.x_bytes = up((size_t)rows * l.ld_x * 2, 256), l.a_bytes = up((size_t)m * l.ld_a * 2, 256);
  l.hi = 0, l.lo = 2 * l.x_bytes, l.a = 4 * l.x_bytes, l.b = l.a + l.a_bytes;
  l.diag_a = l.b + l.a_bytes, l.diag_b = l.diag_a + up((size_t)m * 4, 256);
  l.sums = l.diag_b + up((size_t)m * 4, 256), l.total = l.sums + SUMS * 8;
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
// what a step reads and writes: copy `turn` of X to the other
struct State {
  __half *hi, *lo, *A, *B;
  float *da, *db;
};
__device__ __forceinline__ State state_of(const Call &p, int matrix, int copy) {
  char *w = p.work + matrix * p.l.total;
  return State{reinterpret_cast<__half *>(w + p.l.hi + copy * p.l.x_bytes), reinterpret_cast<__half *>(w + p.l.lo + copy * p.l.x_bytes),
               reinterpret_cast<__half *>(w + p.l.a), reinterpret_cast<__half *>(w + p.l.b),
               reinterpret_cast<float *>(w + p.l.diag_a), reinterpret_cast<float *>(w + p.l.diag_b)};
}

// Partial sums of squares, grid (SUMS, matrices), in 64 bits: any fp32 values
// can be squared in them.
template <typename T>
__global__ void __launch_bounds__(256) squares_kernel(const Call p) {
  __shared__ double part[8];
  const T *g = reinterpret_cast<const T *>(p.g) + blockIdx.y * p.g_stride;
  double s = 0;
  for (int r = blockIdx.x; r < p.rows; r += SUMS)
    for (int c = threadIdx.x; c < p.cols; c += 256) {
      const double v = Elem<T>::get(g[r * p.ldg + c]);
      s += v * v;
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
__device__ __forceinline__ void split(float v, __half *hi, __half *lo) {
  const __half h = __float2half_rn(v);
  *hi = h;
  *lo = __float2half_rn(v - __half2float(h));
}
// X_SCALE / (|g| + eps) as two factors, the first a power of two that brings the
// largest g into range
__device__ __forceinline__ float2 normaliser(const double *sums, float eps) {
  double s = 0;
  for (int i = 0; i < SUMS; ++i) s += sums[i];
  const double norm = sqrt(s) + (double)eps;
  if (norm == 0) return make_float2(1.f, 0.f);
  if (!(norm <= 1.7e308)) return make_float2(1.f, NAN);
  const int e = max(-126, min(126, -ilogb(norm)));
  return make_float2(ldexpf(1.f, e), (float)(X_SCALE / ldexp(norm, e)));
}
template <typename T>
__global__ void __launch_bounds__(256) start_kernel(const Call p) {
  __shared__ float2 f;
  const T *g = reinterpret_cast<const T *>(p.g) + blockIdx.y * p.g_stride;
  if (threadIdx.x == 0) f = normaliser(reinterpret_cast<const double *>(p.work + blockIdx.y * p.l.total + p.l.sums), p.eps);
  __syncthreads();
  const State s = state_of(p, blockIdx.y, 0);
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x)
    for (int c = threadIdx.x; c < p.cols; c += 256)
      split(Elem<T>::get(g[r * p.ldg + c]) * f.x * f.y, s.hi + r * p.l.ld_x + c, s.lo + r * p.l.ld_x + c);
}
template <typename T>
__global__ void __launch_bounds__(256) finish_kernel(const Call p, int copy) {
  T *out = reinterpret_cast<T *>(p.out) + blockIdx.y * p.out_stride;
  const State s = state_of(p, blockIdx.y, copy);
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x)
    for (int c = threadIdx.x; c < p.cols; c += 256) {
      const int64_t i = r * p.l.ld_x + c;
      out[r * p.ld_out + c] = Elem<T>::put((__half2float(s.hi[i]) + __half2float(s.lo[i])) * (p.scale / X_SCALE));
    }
}

enum Kind { GRAM, POLY, UPDATE };
// One 64 x 64 tile of a product, 16 x 16 threads of 4 x 4
template <int KIND>
__global__ void __launch_bounds__(256) product_kernel(const Call p, int copy) {
  __shared__ float as[16][65], bs[16][65];
  const State s = state_of(p, blockIdx.z, copy), to = state_of(p, blockIdx.z, copy ^ 1);
  const int64_t lx = p.l.ld_x, la = p.l.ld_a;
  const int M = KIND == UPDATE ? p.rows : p.m, N = KIND == UPDATE ? p.cols : p.m;
  const int K = KIND == GRAM ? (p.tall ? p.rows : p.cols) : p.m;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  auto left = [&](int i, int k) {
    if (KIND == GRAM) return p.tall ? s.hi[k * lx + i] : s.hi[i * lx + k];
    if (KIND == POLY) return s.A[i * la + k];
    return p.tall ? s.hi[i * lx + k] : s.B[i * la + k];
  };
  auto right = [&](int k, int j) {
    if (KIND == GRAM) return p.tall ? s.hi[k * lx + j] : s.hi[j * lx + k];
    if (KIND == POLY) return s.A[k * la + j];
    return p.tall ? s.B[k * la + j] : s.hi[k * lx + j];
  };
  float acc[4][4] = {};
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int e = threadIdx.x; e < 1024; e += 256) {
      const int k = e % 16, i = e / 16;
      as[k][i] = i0 + i < M && k0 + k < K ? __half2float(left(i0 + i, k0 + k)) : 0.f;
      bs[e / 64][e % 64] = j0 + e % 64 < N && k0 + e / 64 < K ? __half2float(right(k0 + e / 64, j0 + e % 64)) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += as[k][ty * 4 + i] * bs[k][tx * 4 + j];
    __syncthreads();
  }
  for (int u = 0; u < 4; ++u)
    for (int v = 0; v < 4; ++v) {
      const int i = i0 + ty * 4 + u, j = j0 + tx * 4 + v;
      if (i >= M || j >= N) continue;
      if (KIND == GRAM) {
        const float r = acc[u][v] / (X_SCALE * X_SCALE);
        if (i == j) s.da[i] = r;
        s.A[i * la + j] = __float2half_rn(i == j ? 0.f : r * A_SCALE);
      } else if (KIND == POLY) {
        const float oo = acc[u][v] / (A_SCALE * A_SCALE), o = __half2float(s.A[i * la + j]) / A_SCALE, di = s.da[i], dj = s.da[j];
        if (i == j) s.db[i] = p.b * di + p.c * (di * di + oo);
        s.B[i * la + j] = __float2half_rn(i == j ? 0.f : B_SCALE * ((p.b + p.c * (di + dj)) * o + p.c * oo));
      } else {
        const float x = __half2float(s.hi[i * lx + j]) + __half2float(s.lo[i * lx + j]);
        split((p.a + s.db[p.tall ? j : i]) * x + acc[u][v] / B_SCALE, to.hi + i * lx + j, to.lo + i * lx + j);
      }
    }
}

}  // namespace orth

// (bytes of one matrix, bytes that the call runs best with)
void orthogonalize_workspace(int count, int rows, int cols, int, size_t *least, size_t *best) {
  *least = orth::layout_of(rows, cols).total;
  *best = *least * std::max(count, 1);
}

cudaError_t launch_orthogonalize(const sym_orthogonalize &o, int, cudaStream_t st) {
  using namespace orth;
  Call p{};
  p.l = layout_of(o.rows, o.cols);
  p.g_stride = o.g_stride, p.ldg = o.ld_g, p.out_stride = o.out_stride, p.ld_out = o.ld_out;
  p.work = reinterpret_cast<char *>(o.work);
  p.rows = o.rows, p.cols = o.cols, p.m = std::min(o.rows, o.cols), p.tall = o.rows > o.cols;
  p.a = o.coeffs[0], p.b = o.coeffs[1], p.c = o.coeffs[2], p.eps = o.eps, p.scale = o.scale;
  const int each = (int)std::min<uint64_t>(o.work_bytes / p.l.total, o.count);
  const int64_t gs = o.g_dtype == SYM_FP32 ? 4 : 2;
  for (int at = 0; at < o.count; at += each) {
    const unsigned n = std::min(each, o.count - at);
    p.g = reinterpret_cast<const char *>(o.g) + at * o.g_stride * gs;
    p.out = reinterpret_cast<char *>(o.out) + at * o.out_stride * 2;
    const dim3 lines(std::min(o.rows, 1024), n);
    auto start = [&](auto t) {
      using T = decltype(t);
      squares_kernel<T><<<dim3(SUMS, n), 256, 0, st>>>(p);
      start_kernel<T><<<lines, 256, 0, st>>>(p);
    };
    if (o.g_dtype == SYM_BF16) start(__nv_bfloat16());
    else if (o.g_dtype == SYM_FP16) start(__half());
    else start(float());
    const unsigned tm = (p.m + 63) / 64, tr = (p.rows + 63) / 64, tc = (p.cols + 63) / 64;
    for (int i = 0; i < o.steps; ++i) {
      product_kernel<GRAM><<<dim3(tm, tm, n), 256, 0, st>>>(p, i & 1);
      product_kernel<POLY><<<dim3(tm, tm, n), 256, 0, st>>>(p, i & 1);
      product_kernel<UPDATE><<<dim3(tc, tr, n), 256, 0, st>>>(p, i & 1);
    }
    if (o.out_dtype == SYM_BF16) finish_kernel<__nv_bfloat16><<<lines, 256, 0, st>>>(p, o.steps & 1);
    else finish_kernel<__half><<<lines, 256, 0, st>>>(p, o.steps & 1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace symmoe
