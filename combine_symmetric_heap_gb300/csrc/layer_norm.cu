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

// Forward for rows that fit the registers: a thread holds NV vectors of V columns, so the
// row is read once.  WARP: a warp has a row (four rows a block), else a block.
template <typename T, int V, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) layer_norm_held_kernel(const Fwd p) {
  __shared__ float buf[2 * 32];
  const int warps = WARP ? 1 : blockDim.x / 32, warp = WARP ? 0 : threadIdx.x / 32;
  const int thread = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
  const int each = WARP ? blockDim.x / 32 : 1;
  const float inv = 1.f / p.cols;
  int turn = 0;
  for (int r = blockIdx.x * each + (WARP ? (int)threadIdx.x / 32 : 0); r < p.rows; r += gridDim.x * each) {
    const T *x = at<T>(p.x, r, p.ldx), *add = p.add ? at<T>(p.add, r, p.ld_add) : nullptr;
    float s[NV][V], m[1] = {0.f}, v[1] = {0.f};
    auto column = [&](int j) { return (thread + j * threads) * V; };
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
            v[0] += d * d;
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
      if (p.sum) store<T, V>(at<T>(p.sum, r, p.ld_sum) + c, s[j]);
      if (!p.h) continue;
      float t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) s[j][i] = (s[j][i] - mean) * rstd;
      if (p.w) {
        load<T, V>(reinterpret_cast<const T *>(p.w) + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] *= t[i];
      }
      if (p.b) {
        load<T, V>(reinterpret_cast<const T *>(p.b) + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] += t[i];
      }
      store<T, V>(at<T>(p.h, r, p.ldh) + c, s[j]);
    }
  }
}

// Backward for rows of up to 8192 columns, everything in one pass: a block walks its rows, a
// thread has the same NV vectors of V columns of each and keeps their two column sums in
// registers.  AHEAD: the next row's vectors are loaded before this row's sums.
template <typename T, int V, int NV, bool AHEAD>
__global__ void __launch_bounds__(AHEAD ? 512 : 1024) layer_norm_bwd_kernel(const Bwd p) {
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
  if (AHEAD && (int)blockIdx.x < p.rows) fetch(now, blockIdx.x);
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    Row next;
    if (!AHEAD) fetch(now, r);
    else if (r + (int)gridDim.x < p.rows) fetch(next, r + gridDim.x);
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
    if (AHEAD) now = next;
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

// The same for rows in 16-byte vectors whose tensors fit shared memory four rows deep: two rows
// at a time, so that both take one block reduction, and the rows after them on their
// way (cp.async, each thread into its own shared memory: no barrier guards the copies).
// With one row at a time out of registers a row's chain (read, reduce, finish) bounds it:
// 8192 x 7168 114 us, 91 so.
template <typename T, int NV>
__global__ void __launch_bounds__(512) layer_norm_bwd_staged_kernel(const Bwd p, int pairs, int arrays) {
  constexpr int V = Elem<T>::VEC;
  extern __shared__ __align__(16) uint4 rows_smem[];
  __shared__ float buf[2 * 128];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, threads = blockDim.x;
  const float inv = 1.f / p.cols;
  int turn = 0;
  auto column = [&](int j) { return ((int)threadIdx.x + j * threads) * V; };
  // vector j of array a (dh, s, dsum) of row q of pair slot k
  auto place = [&](int k, int q, int a, int j) { return rows_smem + ((((k * 2 + q) * arrays + a) * NV + j) * threads + threadIdx.x); };
  int ahead = blockIdx.x, put = 0;
  const int step = gridDim.x;
  auto fetch = [&]() {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = ahead + q * step;
      if (r >= p.rows) break;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column(j);
        if (c >= p.cols) continue;
        cp_async16(place(put, q, 0, j), at<T>(p.dh, r, p.ld_dh) + c);
        cp_async16(place(put, q, 1, j), at<T>(p.s, r, p.ld_s) + c);
        if (arrays > 2) cp_async16(place(put, q, 2, j), at<T>(p.dsum, r, p.ld_dsum) + c);
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
    if (p.w && column(j) < p.cols) w[j] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(p.w) + column(j));
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
  statistics(blockIdx.x);
  int take = 0;
  for (int r = blockIdx.x; r < p.rows; r += 2 * step) {
    fetch();
    if (pairs == 2) cp_async_wait<1>();
    else cp_async_wait<2>();
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
          store<T, V>(at<T>(p.dx, r + q * step, p.ld_dx) + column(j), g);
        }
      }
    }
    take = take + 1 == pairs ? 0 : take + 1;
  }
  cp_async_wait<0>();
  if (!p.dw && !p.db) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (column(j) >= p.cols) continue;
    float *to = p.ws + (int64_t)blockIdx.x * 2 * p.cols + column(j);
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      *reinterpret_cast<float4 *>(to + i) = make_float4(sum_w[j][i], sum_w[j][i + 1], sum_w[j][i + 2], sum_w[j][i + 3]);
      *reinterpret_cast<float4 *>(to + p.cols + i) = make_float4(sum_b[j][i], sum_b[j][i + 1], sum_b[j][i + 2], sum_b[j][i + 3]);
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

// The one-pass backward out of registers: columns a thread (16 in vectors of 16-bit types, whose
// raw rows take few registers; 8 in fp32 vectors; single elements 8, or 4 in rows of up to
// 4096: 4099 x 1001 in fp32 16 us instead of 24), threads, and blocks: what the SMs hold, with
// some rows each so that the partial sums stay few.
constexpr int FUSED_COLS = 8192, FOUR_COLS = 4096;
struct BwdShape {
  int threads, blocks;
};
static BwdShape bwd_shape(int64_t rows, int cols, int each, int num_sms) {
  const int threads = (cols + 32 * each - 1) / (32 * each) * 32, resident = (each == 16 ? 512 : 1024) / threads;
  return {threads, (int)std::max<int64_t>(1, std::min<int64_t>((rows + 3) / 4, (int64_t)num_sms * std::max(1, std::min(resident, 16))))};
}

// The staged form of it: 16 columns a thread, two or three pairs of rows in shared memory
constexpr int STAGED_SMEM = 220 * 1024;
struct StagedShape {
  int threads, blocks, pairs;  // pairs 0: does not fit
  size_t smem;
};
static StagedShape staged_shape(int64_t rows, int cols, int size, int arrays, int num_sms) {
  StagedShape s = {(cols + 511) / 512 * 32, 0, 0, 0};
  const size_t pair = (size_t)2 * arrays * s.threads * 16 * size;
  if (s.threads > 512 || 2 * pair > STAGED_SMEM) return s;
  const int resident = std::max(1, std::min({512 / s.threads, 16, (int)(STAGED_SMEM / (2 * pair))}));
  s.pairs = STAGED_SMEM / resident >= 3 * pair + 2048 ? 3 : 2;
  s.smem = s.pairs * pair;
  s.blocks = (int)std::max<int64_t>(1, std::min<int64_t>((rows + 7) / 8, (int64_t)num_sms * resident));
  return s;
}

template <typename T, int V>
static cudaError_t fwd(const Fwd &p, int num_sms, cudaStream_t st) {
  constexpr int NV = V == 8 ? 4 : V == 4 ? 8 : 32, EACH = NV * V;  // 32 columns a thread
  if (p.cols <= 32 * EACH) {
    const int blocks = (p.rows + 3) / 4;
    layer_norm_held_kernel<T, V, NV, true><<<blocks, 128, 0, st>>>(p);
  } else if (p.cols <= 1024 * EACH) {
    layer_norm_held_kernel<T, V, NV, false><<<p.rows, (p.cols + 32 * EACH - 1) / (32 * EACH) * 32, 0, st>>>(p);
  } else {
    layer_norm_kernel<T, V><<<std::min(p.rows, num_sms * 8), threads_of(p.cols, V), 0, st>>>(p);
  }
  return cudaGetLastError();
}
template <typename T, int V>
static cudaError_t bwd(Bwd p, int num_sms, cudaStream_t st) {
  const bool sums = p.dw || p.db;
  auto join = [&]() { return launch_pdl(layer_norm_join_kernel<T>, dim3((p.cols + 31) / 32, 2), dim3(1024), 0, st, p); };
  if constexpr (V > 1) {
    const int arrays = p.dsum ? 3 : 2;
    const StagedShape s = staged_shape(p.rows, p.cols, sizeof(T), arrays, num_sms);
    if (s.pairs) {
      auto kern = layer_norm_bwd_staged_kernel<T, 16 / V>;
      cudaError_t err = allow_smem(kern, STAGED_SMEM);
      if (err != cudaSuccess) return err;
      p.parts = s.blocks;
      kern<<<s.blocks, s.threads, s.smem, st>>>(p, s.pairs, arrays);
      err = cudaGetLastError();
      return err != cudaSuccess || !sums ? err : join();
    }
  }
  if (p.cols <= FUSED_COLS) {
    const bool four = V == 1 && p.cols <= FOUR_COLS;
    const BwdShape s = bwd_shape(p.rows, p.cols, V == 8 ? 16 : four ? 4 : 8, num_sms);
    p.parts = s.blocks;
    if (four) layer_norm_bwd_kernel<T, V, V == 1 ? 4 : 2, V == 8><<<s.blocks, s.threads, 0, st>>>(p);
    else layer_norm_bwd_kernel<T, V, V == 1 ? 8 : 2, V == 8><<<s.blocks, s.threads, 0, st>>>(p);
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
    for (int arrays : {2, 3}) parts = std::max(parts, staged_shape(rows, cols, size, arrays, num_sms).blocks);
  if (cols <= FUSED_COLS) 
    for (int each : {4, 8, 16})
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
  if (a.dtype == SYM_BF16) return vec ? fwd<__nv_bfloat16, 8>(p, num_sms, st) : fwd<__nv_bfloat16, 1>(p, num_sms, st);
  if (a.dtype == SYM_FP16) return vec ? fwd<__half, 8>(p, num_sms, st) : fwd<__half, 1>(p, num_sms, st);
  return vec ? fwd<float, 4>(p, num_sms, st) : fwd<float, 1>(p, num_sms, st);
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
  if (a.dtype == SYM_BF16) return vec ? bwd<__nv_bfloat16, 8>(p, num_sms, st) : bwd<__nv_bfloat16, 1>(p, num_sms, st);
  if (a.dtype == SYM_FP16) return vec ? bwd<__half, 8>(p, num_sms, st) : bwd<__half, 1>(p, num_sms, st);
  return vec ? bwd<float, 4>(p, num_sms, st) : bwd<float, 1>(p, num_sms, st);
}

}  // namespace symmoe
