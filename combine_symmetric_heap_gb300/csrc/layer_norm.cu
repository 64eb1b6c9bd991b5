// layer_norm.cu -- layer norm of rows with the residual sum in the same pass,
// and its gradient with the reductions of the weight's and the bias'.
//
//   s = x + add;  h = (s - mean) * rstd * w + b     rstd = (mean((s - mean)^2) + eps)^-1/2
//
// Backward, with n = (s - mean) * rstd and g = dh * w:
//   dx = dsum + rstd * (g - mean(g) - n * mean(g * n)),  dw = sum dh * n,  db = sum dh
// (means over a row's columns, sums over the rows).
//
// Both are bound by the tensors' bytes.  The variance is the mean of squared
// distances from the mean, a second walk of the row: the difference of the mean
// square and the squared mean would lose what a row far from zero has left.
#include <algorithm>
#include <initializer_list>

#include "rows_dev.cuh"

namespace symmoe {
namespace layer {

using namespace rows;

struct Fwd {
  const void *x, *add, *w, *b;
  void *sum, *h;
  float *mean, *rstd;
  int64_t ldx, ld_add, ld_sum, ldh;  // elements
  int rows, cols;
  float eps;
};
struct Bwd {
  const void *dh, *s, *dsum, *w;
  const float *mean, *rstd;
  void *dx, *dw, *db;
  float *ws;  // partial sums, [parts][2][cols]
  int64_t ld_dh, ld_s, ld_dsum, ld_dx;
  int rows, cols, parts;
};

template <typename T>
__device__ __forceinline__ const T *at(const void *p, int row, int64_t ld) {
  return reinterpret_cast<const T *>(p) + row * ld;
}
template <typename T>
__device__ __forceinline__ T *at(void *p, int row, int64_t ld) {
  return reinterpret_cast<T *>(p) + row * ld;
}

// A row's variance by its sum of squares v holds where v neither left the range of
// fp32 nor is so small that squares vanished from it.
__device__ __forceinline__ bool squares_hold(float v, float inv, float eps) {
  return v <= 3e38f && v * inv + eps >= 1e-30f;
}
// Otherwise the row is taken again times a power of two that brings its largest
// element to [1, 2): the exponent of it, from the group's largest.
__device__ __forceinline__ int row_exponent(float largest, float *buf, int warp, int warps, int &turn) {
  float m[1] = {largest};
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], s));
  if (warps > 1) {
    float *b = buf + turn * 32;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) b[warp] = m[0];
    __syncthreads();
    m[0] = (threadIdx.x & 31) < warps ? b[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], s));
  }
  return m[0] > 0.f && m[0] <= 3.4028235e38f ? ilogbf(m[0]) : 0;
}
// rstd of a row whose scaled squares sum to v
__device__ __forceinline__ float scaled_rstd(float v, int e, float inv, float eps) {
  return (float)(1.0 / sqrt(ldexp((double)v * inv, 2 * e) + (double)eps));
}

// Forward for rows of any length: walked for the mean, the variance and the result
// (out of L2 after the first time).
template <typename T, int V>
__global__ void __launch_bounds__(512) layer_norm_kernel(const Fwd p) {
  __shared__ float buf[2 * 32];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const float inv = 1.f / p.cols;
  int turn = 0;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T *x = at<T>(p.x, r, p.ldx), *add = p.add ? at<T>(p.add, r, p.ld_add) : nullptr;
    auto each = [&](auto &&f) {  // f(c, s) for this thread's vectors
      for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) {
        float s[V], t[V];
        load<T, V>(x + c, s);
        if (add) {
          load<T, V>(add + c, t);
#pragma unroll
          for (int i = 0; i < V; ++i) s[i] += t[i];
        }
        f(c, s);
      }
    };
    float m[1] = {0.f}, v[1] = {0.f};
    each([&](int, float(&s)[V]) {
#pragma unroll
      for (int i = 0; i < V; ++i) m[0] += s[i];
    });
    group_sums<1>(m, buf, warp, warps, turn);
    const float first = m[0] * inv;
    each([&](int, float(&s)[V]) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[0] += (s[i] - first) * (s[i] - first);
    });
    group_sums<1>(v, buf, warp, warps, turn);
    float mean = m[0] * inv, rstd = rsqrtf(v[0] * inv + p.eps);
    if (!squares_hold(v[0], inv, p.eps)) {
      float largest = 0.f;
      each([&](int, float(&s)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) largest = fmaxf(largest, fabsf(s[i]));
      });
      const int e = row_exponent(largest, buf, warp, warps, turn);
      m[0] = v[0] = 0.f;
      each([&](int, float(&s)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) m[0] += ldexpf(s[i], -e);
      });
      group_sums<1>(m, buf, warp, warps, turn);
      const float scaled = m[0] * inv;
      each([&](int, float(&s)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = ldexpf(s[i], -e) - scaled;
          v[0] += d * d;
        }
      });
      group_sums<1>(v, buf, warp, warps, turn);
      mean = ldexpf(scaled, e);
      rstd = scaled_rstd(v[0], e, inv, p.eps);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
    each([&](int c, float(&s)[V]) {  // each column is read before it is written: h or sum may be x or add
      if (p.sum) store<T, V>(at<T>(p.sum, r, p.ld_sum) + c, s);
      if (!p.h) return;
      float t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = (s[i] - mean) * rstd;
      if (p.w) {
        load<T, V>(reinterpret_cast<const T *>(p.w) + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= t[i];
      }
      if (p.b) {
        load<T, V>(reinterpret_cast<const T *>(p.b) + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] += t[i];
      }
      store<T, V>(at<T>(p.h, r, p.ldh) + c, s);
    });
  }
}

// Bytes [n, n + 16) of a and b behind one another; n even, up to 16
__device__ __forceinline__ uint4 turned(const uint4 &a, const uint4 &b, int n) {
  if (n & 16) return b;
  uint32_t t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) t[i] = n & 8 ? t[i + 2] : t[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) t[i] = n & 4 ? t[i + 1] : t[i];
  const int bits = n & 2 ? 16 : 0;
  return make_uint4(__funnelshift_r(t[0], t[1], bits), __funnelshift_r(t[1], t[2], bits),
                    __funnelshift_r(t[2], t[3], bits), __funnelshift_r(t[3], t[4], bits));
}

// Columns [c, c + V) of a row of any alignment, zeros outside [0, cols): two words on 16-byte
// boundaries where both are the row's own, else single elements
template <typename T, int V>
__device__ __forceinline__ uint4 load_turned(const T *row, int c, int cols) {
  const int bytes = (int)(reinterpret_cast<uintptr_t>(row + c) & 15), first = c - bytes / (int)sizeof(T);
  if (first >= 0 && first + 2 * V <= cols) {
    const uint4 *q = reinterpret_cast<const uint4 *>(row + first);
    return turned(q[0], q[1], bytes);
  }
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = c + i >= 0 && c + i < cols ? Elem<T>::get(row[c + i]) : 0.f;
  return pack<T, V>(f);
}

// Whether the 16 bytes from column c of row r on lie between a tensor's first and last
// element.  A row's first and last word may hold elements of the rows beside it, which
// another block may be writing: they are read and not used.
template <typename T>
__device__ __forceinline__ bool word_inside(const void *from, int64_t ld, int rows, int cols, int r, int c) {
  if (r >= 8 && r + 8 < rows) return true;  // (at least as many elements on both sides)
  const int64_t word = reinterpret_cast<int64_t>(at<T>(from, r, ld)) + c * (int64_t)sizeof(T);
  return word >= reinterpret_cast<int64_t>(from) && word + 16 <= reinterpret_cast<int64_t>(at<T>(from, rows - 1, ld) + cols);
}

// Forward for rows that fit the registers: a thread holds NV vectors of V columns, so the
// row is read once.  WARP: a warp has a row (four rows a block), else a block.
//
// SHIFT: the rows start off 16-byte boundaries, all tensors' by as much; the grid is a multiple
// of the rows after which that repeats, so that a block's (a warp's) rows start alike.  Vectors
// lie on the boundaries, the first and last of a row with elements that are not its own.  They
// are read all the same, but not past the first and last row, and all words of a row before the
// first is looked at: with a branch around each read a row's latencies add up (16384 x 4095 bf16
// with the sum 174 us, 60000 x 1001 195).  The weights are turned to the vectors once, into
// shared memory.  So 16384 x 4095 140 us, 414 with single elements; 8192 x 7167 110 and 392;
// 60000 x 1001 118 and 251; fp32 8192 x 4095 112 and 219, 4099 x 1001 18 and 19.  Whole vectors
// take 85 us; without the sum 16384 x 4095 96 us, 60000 x 1001 77, 16384 x 4096 52.  What is left is latency: 20 warps
// an SM, each of which reads, reduces twice and stores a row before it asks for the next (issue slots
// half used, DRAM 46% busy, 3.7 of the 9.8 cycles between a warp's instructions a wait for loads).  The
// threads are the most with little spilled; with 1024 and 64 registers 131, 109 and fp32 143 us, with 640 137, 132 and 101.
constexpr int SHIFT_THREADS = 768;
template <typename T, int V, int NV, bool WARP, bool SHIFT>
__global__ void __launch_bounds__(WARP ? 128 : SHIFT ? SHIFT_THREADS : 1024, WARP && SHIFT ? 4 : 1) layer_norm_held_kernel(const Fwd p) {
  __shared__ float buf[2 * 32];
  extern __shared__ __align__(16) uint4 weights_smem[];
  const int warps = WARP ? 1 : blockDim.x / 32, warp = WARP ? 0 : threadIdx.x / 32;
  const int thread = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
  const int each = WARP ? blockDim.x / 32 : 1;
  const float inv = 1.f / p.cols;
  int turn = 0;
  const int first = blockIdx.x * each + (WARP ? (int)threadIdx.x / 32 : 0);
  const int off = SHIFT ? (int)((reinterpret_cast<uintptr_t>(at<T>(p.x, first, p.ldx)) & 15) / sizeof(T)) : 0;
  auto column = [&](int j) { return (thread + j * threads) * V - off; };
  auto whole = [&](int c) { return !SHIFT || (c >= 0 && c + V <= p.cols); };
  auto own = [&](int c) { return c >= 0 && c < p.cols; };
  auto mine = [&](int k, int j) { return weights_smem + (k * NV + j) * (int)blockDim.x + threadIdx.x; };
  if (SHIFT) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (column(j) >= p.cols) continue;
      if (p.w) *mine(0, j) = load_turned<T, V>(reinterpret_cast<const T *>(p.w), column(j), p.cols);
      if (p.b) *mine(1, j) = load_turned<T, V>(reinterpret_cast<const T *>(p.b), column(j), p.cols);
    }
  }
  for (int r = first; r < p.rows; r += gridDim.x * each) {
    const T *x = at<T>(p.x, r, p.ldx), *add = p.add ? at<T>(p.add, r, p.ld_add) : nullptr;
    float s[NV][V], m[1] = {0.f}, v[1] = {0.f};
    auto weights = [&](int k, int j, float(&f)[V]) {
      if constexpr (SHIFT) unpack<T, V>(*mine(k, j), f);
      else load<T, V>(reinterpret_cast<const T *>(k ? p.b : p.w) + column(j), f);
    };
    auto put = [&](T *row, int c, const float(&f)[V]) {
      if (SHIFT) store_part<T, V>(row, c, p.cols, f);
      else store<T, V>(row + c, f);
    };
    if constexpr (SHIFT) {  // words first, all of them under way, then their elements
      uint4 raw[NV];
      auto fetch = [&](const T *row) {
        if (r >= 8 && r + 8 < p.rows) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            raw[j] = column(j) < p.cols ? *reinterpret_cast<const uint4 *>(row + column(j)) : make_uint4(0, 0, 0, 0);
        } else {  // (a word may reach past the tensor)
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            float f[V];
            load_part<T, V>(row, column(j), p.cols, f);
            raw[j] = pack<T, V>(f);
          }
        }
      };
      auto values = [&](int j, float(&f)[V]) {
        unpack<T, V>(raw[j], f);
        if (!whole(column(j)))
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = own(column(j) + i) ? f[i] : 0.f;
      };
      fetch(x);
#pragma unroll
      for (int j = 0; j < NV; ++j) values(j, s[j]);
      if (add) {
        fetch(add);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float t[V];
          values(j, t);
#pragma unroll
          for (int i = 0; i < V; ++i) s[j][i] += t[i];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (column(j) < p.cols) {
          load<T, V>(x + column(j), s[j]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) s[j][i] = 0.f;
        }
      }
      if (add) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (column(j) < p.cols) {
            float t[V];
            load<T, V>(add + column(j), t);
#pragma unroll
            for (int i = 0; i < V; ++i) s[j][i] += t[i];
          }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) m[0] += s[j][i];
    group_sums<1>(m, buf, warp, warps, turn);
    auto squares = [&](float mean, float scale) {  // of the distances, scaled
      v[0] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (column(j) < p.cols)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float d = s[j][i] * scale - mean;
            if (whole(column(j)) || own(column(j) + i)) v[0] += d * d;
          }
      group_sums<1>(v, buf, warp, warps, turn);
    };
    float mean = m[0] * inv;
    squares(mean, 1.f);
    float rstd = rsqrtf(v[0] * inv + p.eps);
    if (!squares_hold(v[0], inv, p.eps)) {
      float largest = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) largest = fmaxf(largest, fabsf(s[j][i]));
      const int e = max(-126, min(126, row_exponent(largest, buf, warp, warps, turn)));
      const float scale = ldexpf(1.f, -e);
      m[0] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) m[0] += s[j][i] * scale;
      group_sums<1>(m, buf, warp, warps, turn);
      squares(m[0] * inv, scale);
      mean = ldexpf(m[0] * inv, e);
      rstd = scaled_rstd(v[0], e, inv, p.eps);
    }
    if (thread == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = column(j);
      if (c >= p.cols) continue;
      if (p.sum) put(at<T>(p.sum, r, p.ld_sum), c, s[j]);
      if (!p.h) continue;
      float t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) s[j][i] = (s[j][i] - mean) * rstd;
      if (p.w) {
        weights(0, j, t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] *= t[i];
      }
      if (p.b) {
        weights(1, j, t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] += t[i];
      }
      put(at<T>(p.h, r, p.ldh), c, s[j]);
    }
  }
}

// Backward for rows of up to 8192 columns, everything in one pass: a block walks its rows, a
// thread has the same NV vectors of V columns of each and keeps their two column sums in
// registers.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(1024) layer_norm_bwd_kernel(const Bwd p) {
  __shared__ float buf[2 * 32 * 2];
  using Raw = typename std::conditional<V == 1, T, uint4>::type;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const float inv = 1.f / p.cols;
  int turn = 0;
  auto column = [&](int j) { return ((int)threadIdx.x + j * (int)blockDim.x) * V; };
  struct Row {
    Raw dh[NV], s[NV], dsum[NV];
    float mean, rstd;
  };
  auto fetch = [&](Row &row, int r) {
    row.mean = p.mean[r], row.rstd = p.rstd[r];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = column(j);
      if (c >= p.cols) continue;
      row.dh[j] = *reinterpret_cast<const Raw *>(at<T>(p.dh, r, p.ld_dh) + c);
      row.s[j] = *reinterpret_cast<const Raw *>(at<T>(p.s, r, p.ld_s) + c);
      if (p.dsum) row.dsum[j] = *reinterpret_cast<const Raw *>(at<T>(p.dsum, r, p.ld_dsum) + c);
    }
  };
  auto values = [&](const Raw &q, float(&f)[V]) {
    if constexpr (V == 1) f[0] = Elem<T>::get(q);
    else unpack<T, V>(q, f);
  };
  Raw w[NV];
  float sum_w[NV][V], sum_b[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (p.w && column(j) < p.cols) w[j] = *reinterpret_cast<const Raw *>(reinterpret_cast<const T *>(p.w) + column(j));
#pragma unroll
    for (int i = 0; i < V; ++i) sum_w[j][i] = sum_b[j][i] = 0.f;
  }
  Row now;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    fetch(now, r);
    float v[2] = {0.f, 0.f};
    auto g_and_n = [&](int j, float(&h)[V], float(&g)[V], float(&n)[V]) {
      values(now.dh[j], h);
      values(now.s[j], n);
      if (p.w) {
        values(w[j], g);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] *= h[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = h[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) n[i] = (n[i] - now.mean) * now.rstd;
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (column(j) >= p.cols) continue;
      float h[V], g[V], n[V];
      g_and_n(j, h, g, n);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[0] += g[i];
        v[1] += g[i] * n[i];
        sum_w[j][i] += h[i] * n[i];
        sum_b[j][i] += h[i];
      }
    }
    if (p.dx) {
      group_sums<2>(v, buf, warp, warps, turn);
      const float mg = v[0] * inv, mgn = v[1] * inv;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (column(j) >= p.cols) continue;
        float h[V], g[V], n[V];
        g_and_n(j, h, g, n);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = now.rstd * (g[i] - mg - n[i] * mgn);
        if (p.dsum) {
          values(now.dsum[j], h);
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] += h[i];
        }
        store<T, V>(at<T>(p.dx, r, p.ld_dx) + column(j), g);
      }
    }
  }
  if (!p.dw && !p.db) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (column(j) >= p.cols) continue;
    float *to = p.ws + (int64_t)blockIdx.x * 2 * p.cols + column(j);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      to[i] = sum_w[j][i];
      to[p.cols + i] = sum_b[j][i];
    }
  }
}

// The same with 16-byte vectors, for rows whose tensors fit shared memory four rows deep: two rows
// at a time, so that both take one block reduction, and the rows after them on their
// way (cp.async, each thread into its own shared memory: no barrier guards the copies).
// With one row at a time out of registers a row's chain (read, reduce, finish) bounds it:
// 8192 x 7168 114 us, 91 so.
// SHIFT: the rows start off 16-byte boundaries, all tensors' by as much; the grid is a
// multiple of the rows after which that repeats, so that a block's rows start alike and its
// threads keep their columns: vectors on the boundaries, the first and last of a row with
// elements that are not its own.  Those are copied all the same (a wait for single elements
// costs more than all the rest) and taken as zeros, but not past the first and last row.
// 16384 x 4095 bf16 130 us, 273 with single elements; 8192 x 7167 134 and 400; 60000 x 1001
// 177 and 215.  (At most 96 registers: 9 warps twice on an SM; with 101 it was 196 us.)
// CLUSTER: the blocks of a cluster share rows too long for one, each a run of columns; they
// read one another's four sums (buffers in turn: one barrier a pair).  4096 x 16383 bf16 187
// us, 414 with single elements read twice, 2048 x 16383 fp32 184 and 254; not for aligned rows,
// which are faster read twice (2048 x 16384 fp32 191 us so and 160, 8000 x 8400 bf16 188 and 146).
template <typename T, int NV, bool SHIFT, bool CLUSTER>
__global__ void __launch_bounds__(SHIFT ? 640 : 512) layer_norm_bwd_staged_kernel(const Bwd p, int pairs, int arrays) {
  constexpr int V = Elem<T>::VEC;
  extern __shared__ __align__(16) uint4 rows_smem[];
  __shared__ float buf[2 * 128], cross[2 * 4];
  const int ranks = CLUSTER ? (int)cluster_size() : 1, rank = CLUSTER ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / ranks, step = gridDim.x / ranks;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, threads = blockDim.x;
  const float inv = 1.f / p.cols;
  int turn = 0, cross_turn = 0;
  const int off = SHIFT ? (int)((reinterpret_cast<uintptr_t>(at<T>(p.dh, unit, p.ld_dh)) & 15) / sizeof(T)) : 0;
  auto column = [&](int j) { return ((int)threadIdx.x + (rank * NV + j) * threads) * V - off; };
  auto whole = [&](int c) { return !SHIFT || (c >= 0 && c + V <= p.cols); };
  // vector j of array a (dh, s, dsum) of row q of pair slot k
  auto place = [&](int k, int q, int a, int j) { return rows_smem + ((((k * 2 + q) * arrays + a) * NV + j) * threads + threadIdx.x); };
  auto copy = [&](uint4 *to, const void *from, int64_t ld, int r, int c) {
    const T *row = at<T>(from, r, ld);
    if (whole(c) || word_inside<T>(from, ld, p.rows, p.cols, r, c)) {
      cp_async16(to, row + c);
    } else {
      float f[V];
      load_part<T, V>(row, c, p.cols, f);
      *to = pack<T, V>(f);
    }
  };
  int ahead = unit, put = 0;
  auto fetch = [&]() {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = ahead + q * step;
      if (r >= p.rows) break;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column(j);
        if (c >= p.cols) continue;
        copy(place(put, q, 0, j), p.dh, p.ld_dh, r, c);
        copy(place(put, q, 1, j), p.s, p.ld_s, r, c);
        if (arrays > 2) copy(place(put, q, 2, j), p.dsum, p.ld_dsum, r, c);
      }
    }
    cp_async_commit();
    ahead += 2 * step;
    put = put + 1 == pairs ? 0 : put + 1;
  };
  uint4 w[NV];
  float sum_w[NV][V], sum_b[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (p.w && column(j) < p.cols) {
      const T *from = reinterpret_cast<const T *>(p.w);
      if (SHIFT) w[j] = load_turned<T, V>(from, column(j), p.cols);
      else w[j] = *reinterpret_cast<const uint4 *>(from + column(j));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sum_w[j][i] = sum_b[j][i] = 0.f;
  }
  float mean[2], rstd[2];  // of the next pair
  auto statistics = [&](int r) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (r + q * step < p.rows) mean[q] = p.mean[r + q * step], rstd[q] = p.rstd[r + q * step];
  };
  for (int k = 0; k + 1 < pairs; ++k) fetch();
  statistics(unit);
  int take = 0;
  for (int r = unit; r < p.rows; r += 2 * step) {
    fetch();
    if (pairs == 2) cp_async_wait<1>();
    else cp_async_wait<2>();
    if constexpr (SHIFT) {  // the other rows' elements to zeros (so is w beside its columns)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column(j);
        if (whole(c) || c >= p.cols) continue;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            T *word = reinterpret_cast<T *>(place(take, q, a, j));
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (c + i < 0 || c + i >= p.cols) word[i] = Elem<T>::put(0.f);
          }
      }
    }
    const bool two = r + step < p.rows;
    const float m[2] = {mean[0], mean[1]}, rs[2] = {rstd[0], rstd[1]};
    statistics(r + 2 * step);
    auto g_and_n = [&](int q, int j, float(&h)[V], float(&g)[V], float(&n)[V]) {
      unpack<T, V>(*place(take, q, 0, j), h);
      unpack<T, V>(*place(take, q, 1, j), n);
      if (p.w) {
        unpack<T, V>(w[j], g);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] *= h[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = h[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) n[i] = (n[i] - m[q]) * rs[q];
    };
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (q && !two) break;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (column(j) >= p.cols) continue;
        float h[V], g[V], n[V];
        g_and_n(q, j, h, g, n);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[2 * q] += g[i];
          v[2 * q + 1] += g[i] * n[i];
          sum_w[j][i] += h[i] * n[i];
          sum_b[j][i] += h[i];
        }
      }
    }
    if (p.dx) {
      block_sums4(v, buf, warp, warps, turn);
      if constexpr (CLUSTER) {
        const int lane = threadIdx.x & 31;
        float *mine = cross + cross_turn * 4;
        cross_turn ^= 1;
        if (threadIdx.x == 0)
#pragma unroll
          for (int k = 0; k < 4; ++k) mine[k] = v[k];
        cluster_barrier();
        float sum = lane < 4 * ranks ? load_from(mine + (lane & 3), lane >> 2) : 0.f;
#pragma unroll
        for (int d = 16; d > 2; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(~0u, sum, k);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q && !two) break;
        const float mg = v[2 * q] * inv, mgn = v[2 * q + 1] * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (column(j) >= p.cols) continue;
          float h[V], g[V], n[V];
          g_and_n(q, j, h, g, n);
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] = rs[q] * (g[i] - mg - n[i] * mgn);
          if (arrays > 2) {
            unpack<T, V>(*place(take, q, 2, j), h);
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] += h[i];
          }
          T *to = at<T>(p.dx, r + q * step, p.ld_dx);
          if (SHIFT) store_part<T, V>(to, column(j), p.cols, g);
          else store<T, V>(to + column(j), g);
        }
      }
    }
    take = take + 1 == pairs ? 0 : take + 1;
  }
  cp_async_wait<0>();
  if (CLUSTER) cluster_barrier();  // nobody leaves before its sums are read
  if (!p.dw && !p.db) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (column(j) >= p.cols) continue;
    float *to = p.ws + (int64_t)unit * 2 * p.cols + column(j);
    if constexpr (SHIFT) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (column(j) + i >= 0 && column(j) + i < p.cols) to[i] = sum_w[j][i], to[p.cols + i] = sum_b[j][i];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        *reinterpret_cast<float4 *>(to + i) = make_float4(sum_w[j][i], sum_w[j][i + 1], sum_w[j][i + 2], sum_w[j][i + 3]);
        *reinterpret_cast<float4 *>(to + p.cols + i) = make_float4(sum_b[j][i], sum_b[j][i + 1], sum_b[j][i + 2], sum_b[j][i + 3]);
      }
    }
  }
}

// dx for rows of any length
template <typename T, int V>
__global__ void __launch_bounds__(512) layer_norm_dx_kernel(const Bwd p) {
  __shared__ float buf[2 * 32 * 2];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const float inv = 1.f / p.cols;
  int turn = 0;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const float mean = p.mean[r], rstd = p.rstd[r];
    const T *dh = at<T>(p.dh, r, p.ld_dh), *sr = at<T>(p.s, r, p.ld_s);
    auto each = [&](auto &&f) {  // f(c, g, n)
      for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) {
        float g[V], n[V], t[V];
        load<T, V>(dh + c, g);
        load<T, V>(sr + c, n);
        if (p.w) {
          load<T, V>(reinterpret_cast<const T *>(p.w) + c, t);
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] *= t[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) n[i] = (n[i] - mean) * rstd;
        f(c, g, n);
      }
    };
    float v[2] = {0.f, 0.f};
    each([&](int, float(&g)[V], float(&n)[V]) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[0] += g[i];
        v[1] += g[i] * n[i];
      }
    });
    group_sums<2>(v, buf, warp, warps, turn);
    const float mg = v[0] * inv, mgn = v[1] * inv;
    each([&](int c, float(&g)[V], float(&n)[V]) {
      float t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = rstd * (g[i] - mg - n[i] * mgn);
      if (p.dsum) {
        load<T, V>(at<T>(p.dsum, r, p.ld_dsum) + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] += t[i];
      }
      store<T, V>(at<T>(p.dx, r, p.ld_dx) + c, g);
    });
  }
}

// Column sums of dh n and dh over a part of the rows: grid (column tiles, parts).
// A thread has a vector of columns, the block's 8 warps every eighth row.
constexpr int SUM_WARPS = 8;
template <typename T, int V>
__global__ void __launch_bounds__(32 * SUM_WARPS) layer_norm_columns_kernel(const Bwd p) {
  __shared__ float part[SUM_WARPS][2][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int c = (blockIdx.x * 32 + lane) * V;
  float a[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = b[i] = 0.f;
  if (c < p.cols)
    for (int r = blockIdx.y * SUM_WARPS + warp; r < p.rows; r += gridDim.y * SUM_WARPS) {
      const float mean = p.mean[r], rstd = p.rstd[r];
      float g[V], n[V];
      load<T, V>(at<T>(p.dh, r, p.ld_dh) + c, g);
      load<T, V>(at<T>(p.s, r, p.ld_s) + c, n);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] += g[i] * ((n[i] - mean) * rstd);
        b[i] += g[i];
      }
    }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    part[warp][0][lane * V + i] = a[i];
    part[warp][1][lane * V + i] = b[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * 32 * V; i += blockDim.x) {
    const int k = i / (32 * V), j = i % (32 * V), col = blockIdx.x * 32 * V + j;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < SUM_WARPS; ++v) s += part[v][k][j];
    if (col < p.cols) p.ws[((int64_t)blockIdx.y * 2 + k) * p.cols + col] = s;
  }
}
// The parts' sums added in order: grid (columns / 32, 2), every warp takes every 32nd part
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_join_kernel(const Bwd p) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane, k = blockIdx.y;
  T *to = reinterpret_cast<T *>(k ? p.db : p.dw);
  if (!to) return;
  pdl_wait();
  float s = 0.f;
  if (c < p.cols)
#pragma unroll 8
    for (int i = warp; i < p.parts; i += 32) s += p.ws[((int64_t)i * 2 + k) * p.cols + c];
  part[warp][lane] = s;
  __syncthreads();
  float v[1] = {part[lane][warp]};
  warp_sums<1>(v);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < p.cols) to[col] = Elem<T>::put(v[0]);
}

static bool vec_ok(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> lds, int cols, int64_t es) {
  for (const void *q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) % 16) return false;
  for (int64_t l : lds)
    if (l * es % 16) return false;
  return cols * es % 16 == 0;
}
static int threads_of(int cols, int v) { return std::min(512, std::max(32, (cols / v + 31) / 32 * 32)); }
// rows' parts of the column sums in the general kernels
static int parts_of(int64_t rows, int num_sms) { return (int)std::max<int64_t>(1, std::min<int64_t>((rows + 63) / 64, num_sms)); }

// The one-pass backward out of registers: columns a thread (8, or 4 single elements in rows of
// up to 4096: 4099 x 1001 in fp32 16 us instead of 24), threads, and blocks: what the SMs hold,
// with some rows each so that the partial sums stay few.
constexpr int FUSED_COLS = 8192, FOUR_COLS = 4096;
struct BwdShape {
  int threads, blocks;
};
static BwdShape bwd_shape(int64_t rows, int cols, int each, int num_sms) {
  const int threads = (cols + 32 * each - 1) / (32 * each) * 32, resident = 1024 / threads;
  return {threads, (int)std::max<int64_t>(1, std::min<int64_t>((rows + 3) / 4, (int64_t)num_sms * std::max(1, std::min(resident, 16))))};
}

// The staged form of it: 16 columns a thread, two or three pairs of rows in shared memory; rows
// off 16-byte boundaries that are longer than the register form's are shared by two to eight blocks.
// Aligned fp32 rows, of those with the stream's gradient: 8192 x 4608 93 us (floor 90), x 6144 165 (120), x 8192 196 (160).
constexpr int STAGED_SMEM = 220 * 1024;
struct StagedShape {
  int threads, ranks, blocks, pairs;  // blocks: times ranks; pairs 0: does not fit
  size_t smem;
};
static StagedShape staged_shape(int64_t rows, int cols, int size, int arrays, bool shift, int num_sms) {
  const int alike = shift ? 16 / size : 1;  // rows after which the starts repeat
  StagedShape s = {0, 1, 0, 0};
  size_t pair;
  for (;; s.ranks *= 2) {
    const int each = (cols + alike - 1 + s.ranks - 1) / s.ranks;
    s.threads = (each + 511) / 512 * 32;
    pair = (size_t)2 * arrays * s.threads * 16 * size;
    if (s.threads <= 512 && 2 * pair <= STAGED_SMEM) break;
    if (!shift || cols <= FUSED_COLS || s.ranks == 8) return s;
  }
  const int resident = std::max(1, std::min({(shift ? 576 : 512) / s.threads, 16, (int)(STAGED_SMEM / (2 * pair))}));
  s.pairs = STAGED_SMEM / resident >= 3 * pair + 2048 ? 3 : 2;
  s.smem = s.pairs * pair;
  s.blocks = (int)std::max<int64_t>(1, std::min<int64_t>((rows + 7) / 8, (int64_t)num_sms * resident / s.ranks));
  s.blocks = std::max(alike, s.blocks / alike * alike);
  return s;
}

constexpr int HELD_COLS = 32768;  // of a row in a block's registers, 32 a thread
// ... and off 16-byte boundaries, whose turned weights take 64 elements a thread of shared memory
static int shifted_cols(int size) { return std::min(SHIFT_THREADS, STAGED_SMEM / (64 * size) / 32 * 32) * 32 - (16 / size - 1); }
template <typename T, int V, bool SHIFT>
static cudaError_t fwd(const Fwd &p, int num_sms, cudaStream_t st) {
  constexpr int NV = V == 8 ? 4 : V == 4 ? 8 : 32, EACH = NV * V;
  static_assert(1024 * EACH == HELD_COLS, "columns of a block");
  const int cols = SHIFT ? p.cols + V - 1 : p.cols;  // with what may lie before a row
  const bool warp = cols <= 32 * EACH;
  if (!SHIFT && cols > HELD_COLS) {
    layer_norm_kernel<T, V><<<std::min(p.rows, num_sms * 8), threads_of(p.cols, V), 0, st>>>(p);
    return cudaGetLastError();
  }
  const int threads = warp ? 128 : (cols + 32 * EACH - 1) / (32 * EACH) * 32;
  int blocks = warp ? (p.rows + 3) / 4 : p.rows;
  size_t smem = 0;
  auto launch = [&](auto kern) {
    if (SHIFT) {
      smem = (size_t)2 * NV * threads * 16;
      const cudaError_t err = allow_smem(kern, STAGED_SMEM);
      if (err != cudaSuccess) return err;
      const int resident = std::max(1, std::min({(warp ? 1024 : SHIFT_THREADS) / threads, 16, (int)(STAGED_SMEM / smem)}));
      blocks = std::min(blocks, std::max(8, num_sms * resident / 8 * 8));  // (starts repeat after 8 rows or fewer)
    }
    kern<<<blocks, threads, smem, st>>>(p);
    return cudaGetLastError();
  };
  return warp ? launch(layer_norm_held_kernel<T, V, NV, true, SHIFT>) : launch(layer_norm_held_kernel<T, V, NV, false, SHIFT>);
}
template <typename T, int V, bool SHIFT>
static cudaError_t bwd(Bwd p, int num_sms, cudaStream_t st) {
  const bool sums = p.dw || p.db;
  auto join = [&]() { return launch_pdl(layer_norm_join_kernel<T>, dim3((p.cols + 31) / 32, 2), dim3(1024), 0, st, p); };
  if constexpr (V > 1 || SHIFT) {
    const int arrays = p.dsum ? 3 : 2;
    const StagedShape s = staged_shape(p.rows, p.cols, sizeof(T), arrays, SHIFT, num_sms);
    if (s.pairs) {
      p.parts = s.blocks;
      auto launch = [&](auto kern) {
        cudaError_t err = allow_smem(kern, STAGED_SMEM);
        if (err != cudaSuccess) return err;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(s.blocks * s.ranks);
        cfg.blockDim = dim3(s.threads);
        cfg.dynamicSmemBytes = s.smem;
        cfg.stream = st;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = s.ranks, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = s.ranks > 1;
        return cudaLaunchKernelEx(&cfg, kern, p, (int)s.pairs, (int)arrays);
      };
      cudaError_t err = cudaSuccess;
      if constexpr (SHIFT)
        if (s.ranks > 1) err = launch(layer_norm_bwd_staged_kernel<T, 16 / Elem<T>::VEC, true, true>);
      if constexpr (!SHIFT || sizeof(T) == 2)
        if (s.ranks == 1) err = launch(layer_norm_bwd_staged_kernel<T, 16 / Elem<T>::VEC, SHIFT, false>);
      return err != cudaSuccess || !sums ? err : join();
    }
  }
  if (p.cols <= FUSED_COLS) {
    const bool four = V == 1 && p.cols <= FOUR_COLS;
    const BwdShape s = bwd_shape(p.rows, p.cols, four ? 4 : 8, num_sms);
    p.parts = s.blocks;
    if constexpr (V != 8) {  // (16-bit vectors of so many columns fit shared memory)
      if (four) layer_norm_bwd_kernel<T, V, V == 1 ? 4 : 2><<<s.blocks, s.threads, 0, st>>>(p);
      else layer_norm_bwd_kernel<T, V, V == 1 ? 8 : 2><<<s.blocks, s.threads, 0, st>>>(p);
    }
    const cudaError_t err = cudaGetLastError();
    return err != cudaSuccess || !sums ? err : join();
  }
  // (the column sums first: dx may be dh or s)
  if (sums) {
    p.parts = parts_of(p.rows, num_sms);
    layer_norm_columns_kernel<T, V><<<dim3((p.cols + 32 * V - 1) / (32 * V), p.parts), 32 * SUM_WARPS, 0, st>>>(p);
    cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess) err = join();
    if (err != cudaSuccess) return err;
  }
  if (!p.dx) return cudaSuccess;
  layer_norm_dx_kernel<T, V><<<std::min(p.rows, num_sms * 8), threads_of(p.cols, V), 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace layer

size_t layer_norm_workspace(int64_t rows, int cols, int num_sms) {
  using namespace layer;
  int parts = parts_of(rows, num_sms);
  for (int size : {2, 4})
    for (int arrays : {2, 3})
      for (bool shift : {false, true}) parts = std::max(parts, staged_shape(rows, cols, size, arrays, shift, num_sms).blocks);
  if (cols <= FUSED_COLS) 
    for (int each : {4, 8})
      if (each > 4 || cols <= FOUR_COLS) parts = std::max(parts, bwd_shape(rows, cols, each, num_sms).blocks);
  return (size_t)parts * 2 * cols * sizeof(float);
}

cudaError_t launch_layer_norm(const sym_layer_norm &a, int num_sms, cudaStream_t st) {
  using namespace layer;
  const Fwd p{a.x, a.add, a.w, a.b, a.sum, a.h, a.mean, a.rstd, a.ld_x, a.ld_add, a.ld_sum, a.ld_h, (int)a.rows, a.cols, a.eps};
  const int64_t es = a.dtype == SYM_FP32 ? 4 : 2;
  const bool one = a.rows <= 1;  // (a single row has no stride)
  const bool vec = vec_ok({p.x, p.add, p.w, p.b, p.sum, p.h},
                          {one ? 0 : p.ldx, p.add && !one ? p.ld_add : 0, p.sum && !one ? p.ld_sum : 0, p.h && !one ? p.ldh : 0},
                          p.cols, es);
  // every row of all tensors as far off a boundary as x's
  auto like_x = [&](const void *q, int64_t ld) {
    return !q || ((reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p.x)) % 16 == 0 && (one || (ld - p.ldx) * es % 16 == 0));
  };
  const bool shift = !vec && p.cols <= shifted_cols((int)es) && like_x(p.add, p.ld_add) && like_x(p.sum, p.ld_sum) && like_x(p.h, p.ldh);
  auto go = [&](auto t) {
    using T = decltype(t);
    constexpr int V = Elem<T>::VEC;
    return vec ? fwd<T, V, false>(p, num_sms, st) : shift ? fwd<T, V, true>(p, num_sms, st) : fwd<T, 1, false>(p, num_sms, st);
  };
  return a.dtype == SYM_BF16 ? go(__nv_bfloat16()) : a.dtype == SYM_FP16 ? go(__half()) : go(float());
}

cudaError_t launch_layer_norm_bwd(const sym_layer_norm_grad &a, int num_sms, cudaStream_t st) {
  using namespace layer;
  const Bwd p{a.dh, a.s, a.dsum, a.w, a.mean, a.rstd, a.dx, a.dw, a.db, reinterpret_cast<float *>(a.work), a.ld_dh, a.ld_s,
              a.ld_dsum, a.ld_dx, (int)a.rows, a.cols, 0};
  const int64_t es = a.dtype == SYM_FP32 ? 4 : 2;
  const bool one = a.rows <= 1;
  const bool vec = vec_ok({p.dh, p.s, p.dsum, p.w, p.dx, p.dw, p.db},
                          {one ? 0 : p.ld_dh, one ? 0 : p.ld_s, p.dsum && !one ? p.ld_dsum : 0, p.dx && !one ? p.ld_dx : 0},
                          p.cols, es);
  // every row of all tensors as far off a boundary as dh's (in 32 bits of long rows alone: of others single
  // elements do as well: 8192 x 4095 151 us so and 155, 4099 x 1001 29 and 22)
  auto like_dh = [&](const void *q, int64_t ld) {
    return !q || ((reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p.dh)) % 16 == 0 && (one || (ld - p.ld_dh) * es % 16 == 0));
  };
  const bool shift = !vec && (es == 2 || p.cols > FUSED_COLS) && like_dh(p.s, p.ld_s) && like_dh(p.dsum, p.ld_dsum) && like_dh(p.dx, p.ld_dx);
  auto go = [&](auto t) {
    using T = decltype(t);
    return vec ? bwd<T, Elem<T>::VEC, false>(p, num_sms, st) : shift ? bwd<T, 1, true>(p, num_sms, st) : bwd<T, 1, false>(p, num_sms, st);
  };
  return a.dtype == SYM_BF16 ? go(__nv_bfloat16()) : a.dtype == SYM_FP16 ? go(__half()) : go(float());
}

}  // namespace symmoe
